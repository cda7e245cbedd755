"""What the objects of layer.py refuse (on the host: no kernel runs)."""
import copy

import pytest

torch = pytest.importorskip("torch")
import dynamic_sparsity_approximate_amd as E  # noqa: E402
from test_decoder_host import DIM, parts  # noqa: E402


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_what_calls_have_the_address_of_cannot_be_replaced():
    b = E.KVBatch(ints(2, 3), ints(2), ints(3))
    c = E.KVCache(4, 2, 64, page_tokens=16, device="cpu")
    for obj, names in ((b, ("page_table", "kv_lens", "q_starts")), (c, ("k", "v", "k_scale", "v_scale"))):
        for name in names:
            was = getattr(obj, name)
            with pytest.raises(AttributeError, match=name):
                setattr(obj, name, was + 1)
            with pytest.raises(AttributeError, match=name):
                setattr(obj, name, was.clone())
            with pytest.raises(AttributeError, match=name):
                delattr(obj, name)
            assert getattr(obj, name) is was and was.data_ptr() in (
                b._ptrs[1:] if obj is b else (c.desc.k, c.desc.v, c.desc.k_scale, c.desc.v_scale))
    for name, value in (("format", E.EFFORT_KV_I8), ("page_tokens", 32), ("pages", 5), ("kv_heads", 1), ("head_dim", 128)):
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, value)


def test_writing_in_place_is_allowed():
    b = E.KVBatch(ints(2, 3), ints(2), ints(3))
    was = b.kv_lens
    b.kv_lens += 1
    b.kv_lens.add_(1)
    b.page_table[0, 1] = 7
    assert b.kv_lens is was and was.tolist() == [2, 2]
    b.note = "a program's own"
    b.note = "another"


def test_copies_have_their_own_addresses():
    b = E.KVBatch(ints(2, 3), ints(2), ints(3))
    b.desc(5)
    d = copy.deepcopy(b)
    assert d._ptrs == (3, d.page_table.data_ptr(), d.kv_lens.data_ptr(), d.q_starts.data_ptr())
    assert d.kv_lens.data_ptr() != b.kv_lens.data_ptr() and d.desc(5).kv_lens == d.kv_lens.data_ptr()
    c = E.KVCache(4, 2, 64, page_tokens=16, format=E.EFFORT_KV_I8, device="cpu")
    e = copy.deepcopy(c)
    assert e.desc.format == E.EFFORT_KV_I8 and e.desc.k == e.k.data_ptr() != c.k.data_ptr()
    assert copy.copy(c).desc.v == c.v.data_ptr() and copy.copy(b).kv_lens is b.kv_lens


@pytest.mark.parametrize("big", [1 << 31, 1 << 32, (1 << 32) + 64, -(1 << 31) - 1])
def test_numbers_beyond_32_bits(big):
    """A window of 2^32 must not be taken for 0, nor 2^32 + 64 for 64."""
    c = E.KVCache(4, 2, 64, page_tokens=16, device="cpu")
    b = E.KVBatch(ints(2, 3), ints(2), ints(3))
    with pytest.raises(ValueError, match="window"):
        c.attend(b, torch.zeros(2, 4, 64), window=big)
    with pytest.raises(ValueError, match="rot_dim"):
        E.rope_table(1e4, 1, big, "cpu")


def on_meta():
    """Parts of a step with one of them on another device."""
    one, far = torch.ones(DIM), torch.ones(DIM, device="meta")
    cache = E.KVCache(4, 2, 64, page_tokens=16, device="cpu")
    yield dict(x=torch.zeros(2, DIM, device="meta"))  # the matrices, among others
    yield dict(caches=[cache, E.KVCache(4, 2, 64, page_tokens=16, device="meta")])
    yield dict(batch=E.KVBatch(*(torch.zeros(s, dtype=torch.int32, device="meta") for s in ((2, 2), (2,), (3,)))))
    yield dict(norms=[(one, one), (one, far)])
    yield dict(head_norm=far)


@pytest.mark.parametrize("change", list(on_meta()))
def test_a_step_on_two_devices(change):
    with pytest.raises(ValueError, match="device"):
        E.DecoderStep(**dict(parts(), **change))


@pytest.mark.parametrize("bad", [torch.ones(DIM - 1), torch.ones(1, DIM), torch.ones(DIM).half(), torch.ones(2 * DIM)[::2]])
def test_norm_weights_that_do_not_fit_a_step(bad):
    one = torch.ones(DIM)
    for change in (dict(norms=[(one, one), (bad, one)]), dict(norms=[(one, bad)] * 2), dict(head_norm=bad)):
        with pytest.raises(ValueError, match="norm weights"):
            E.DecoderStep(**dict(parts(), **change))
