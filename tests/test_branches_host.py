"""Refusals of the operators for several continuations of a sequence, and what
their plain definitions say of themselves: no GPU (the addresses are never read)."""
import ctypes
import math
import pickle

import numpy as np
import pytest

import _branches as R
import _layer as L
import dynamic_sparsity_approximate_amd as E
from dynamic_sparsity_approximate_amd import binding as B
from test_layer_host import A, APPEND, ATTEND, BAD_BATCH, BAD_CACHE, batch, cache, call, refused

EX = dict(cache=None, batch=None, parents=A, dtype=E.EFFORT_F32, rope=A, rope_rows=256, rot_dim=128, interleaved=0,
          q_norm=A, q_norm_stride=0, k_norm=A, k_norm_stride=128, eps=1e-5, q=A, q_stride=4096, q_heads=32, q_out=2 * A,
          q_out_stride=4096, k=A, k_stride=1024, v=A, v_stride=1024)
TREE = dict(cache=None, batch=None, parents=A, **{k: v for k, v in ATTEND.items() if k not in ("cache", "batch")})
SELECT = dict(dtype=E.EFFORT_F32, logits=A, stride=100, scores=A, ended=None, end_token=0, items=2, beams=3, vocab=100,
              keep=4, out_scores=A, out_parents=A, out_tokens=A, ws=A, ws_bytes=1 << 40)


def book(**kw):
    d = dict(seqs=2, max_pages=4, page_tokens=64, reserved=0, pages=10, table_stride=4, page_table=A, kv_lens=A, refs=A,
             info=A)
    d.update(kw)
    return E.effort_kv_book(**d)


def einval(fn, *args, code=B.EFFORT_EINVAL):
    with pytest.raises(E.EffortError) as e:
        fn(*args, stream=0)
    assert e.value.code == code, e.value


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_bad_caches(bad):
    refused(B.EFFORT_EINVAL, E.effort_kv_append_ex, EX, c=cache(**bad))
    refused(B.EFFORT_EINVAL, E.effort_kv_attention_tree, TREE, c=cache(**bad))
    c = B.kv_caches([cache(), cache(**bad)])
    einval(E.effort_kv_grow, book(), c, 2, None, 1, A, 1 << 40)
    einval(E.effort_kv_copy_pages, c, 2, A, A, 3)
    einval(E.effort_kv_accept, c, 2, batch(), A, A, A, A, 1 << 40)


@pytest.mark.parametrize("bad", BAD_BATCH)
def test_bad_batches(bad):
    refused(B.EFFORT_EINVAL, E.effort_kv_append_ex, EX, b=batch(**bad))
    refused(B.EFFORT_EINVAL, E.effort_kv_attention_tree, TREE, b=batch(**bad))
    einval(E.effort_kv_accept, B.kv_caches([cache()]), 1, batch(**bad), A, A, A, A, 1 << 40)


@pytest.mark.parametrize("bad", [dict(parents=A + 2), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf),
                                 dict(q_norm_stride=127), dict(k_norm_stride=-128), dict(q_norm=A + 2), dict(k_norm=A + 1),
                                 dict(dtype=3), dict(rot_dim=12), dict(rope_rows=255), dict(q_stride=4095),
                                 dict(q_heads=33), dict(k=None), dict(v_stride=1023)])
def test_append_ex_refuses(bad):
    refused(B.EFFORT_EINVAL, E.effort_kv_append_ex, EX, **bad)


@pytest.mark.parametrize("bad", [dict(parents=None), dict(parents=A + 2), dict(scale=math.nan), dict(window=-1),
                                 dict(q_heads=12), dict(out=A), dict(ws=A + 64), dict(ws=None)])
def test_tree_attention_refuses(bad):
    refused(B.EFFORT_EINVAL, E.effort_kv_attention_tree, TREE, **bad)


def test_workspaces():
    for args in ((2, 3, 32), (1, 64, 32), (8, 600, 64)):
        n = E.effort_kv_tree_workspace_bytes(cache(), *args)
        assert n > 0 and n % 4 == 0
    refused(B.EFFORT_ENOSPACE, E.effort_kv_attention_tree, TREE,
            ws_bytes=E.effort_kv_tree_workspace_bytes(cache(), 2, 3, 32) - 1)
    assert E.effort_kv_tree_workspace_bytes(cache(), 0, 0, 32) == 0
    n = E.effort_kv_grow_workspace_bytes(book())
    einval(E.effort_kv_grow, book(), B.kv_caches([cache()]), 1, None, 1, A, n - 1, code=B.EFFORT_ENOSPACE)
    n = E.effort_kv_accept_workspace_bytes(2)
    einval(E.effort_kv_accept, B.kv_caches([cache()]), 1, batch(), A, A, A, A, n - 1, code=B.EFFORT_ENOSPACE)
    n = E.effort_beam_workspace_bytes(2, 3, 100)
    with pytest.raises(E.EffortError) as e:
        E.effort_beam_select(**dict(SELECT, ws_bytes=n - 1), stream=0)
    assert e.value.code == B.EFFORT_ENOSPACE
    for bad in ((-1, 3, 100), (2, 0, 100), (2, 65, 100), (2, 3, 0), (2, 3, (1 << 20) + 1), (1 << 24, 2, 5)):
        with pytest.raises(E.EffortError):
            E.effort_beam_workspace_bytes(*bad)
    for bad in (-1, E.EFFORT_KV_MAX_SEQS + 1):
        with pytest.raises(E.EffortError):
            E.effort_kv_accept_workspace_bytes(bad)


@pytest.mark.parametrize("bad", [dict(seqs=-1), dict(seqs=1025), dict(max_pages=0), dict(page_tokens=48), dict(reserved=1),
                                 dict(pages=0), dict(pages=1 << 31), dict(table_stride=3), dict(page_table=None),
                                 dict(kv_lens=A + 1), dict(refs=None), dict(info=A + 2),
                                 dict(max_pages=1 << 25, table_stride=1 << 25)])
def test_bad_books(bad):
    einval(E.effort_kv_fork, book(**bad), A, None)
    einval(E.effort_kv_grow, book(**bad), B.kv_caches([cache()]), 1, None, 1, A, 1 << 40)


def test_pages_refuse():
    one = B.kv_caches([cache()])
    einval(E.effort_kv_fork, book(), None, None)
    einval(E.effort_kv_fork, book(), A + 2, None)
    einval(E.effort_kv_fork, book(), A, A + 2)
    einval(E.effort_kv_grow, book(pages=11), one, 1, None, 1, A, 1 << 40)  # the caches have other pages
    einval(E.effort_kv_grow, book(page_tokens=32), one, 1, None, 1, A, 1 << 40)
    einval(E.effort_kv_grow, book(), one, -1, None, 1, A, 1 << 40)
    einval(E.effort_kv_grow, book(), None, 1, None, 1, A, 1 << 40)
    einval(E.effort_kv_grow, book(), one, 1, A + 2, 1, A, 1 << 40)
    einval(E.effort_kv_grow, book(), one, 1, None, 1, A + 128, 1 << 40)
    einval(E.effort_kv_copy_pages, B.kv_caches([cache(), cache(pages=11)]), 2, A, A, 1)
    einval(E.effort_kv_copy_pages, one, 1, None, A, 1)
    einval(E.effort_kv_copy_pages, one, 1, A, A + 2, 1)
    einval(E.effort_kv_copy_pages, one, 1, A, A, -1)
    einval(E.effort_kv_accept, one, 0, batch(), A, A, A, A, 1 << 40)
    for bad in (dict(parents=A + 2), dict(leaf=None), dict(lens_out=A + 1), dict(ws=A + 8)):
        d = dict(parents=A, leaf=A, lens_out=A, ws=A)
        d.update(bad)
        einval(E.effort_kv_accept, one, 1, batch(), *d.values(), 1 << 40)


@pytest.mark.parametrize("bad", [dict(dtype=7), dict(logits=None), dict(logits=A + 2), dict(stride=99), dict(scores=None),
                                 dict(scores=A + 2), dict(items=-1), dict(beams=0), dict(beams=65), dict(vocab=0),
                                 dict(vocab=(1 << 20) + 1, stride=1 << 21), dict(keep=0), dict(keep=129),
                                 dict(out_scores=None), dict(out_parents=A + 2), dict(out_tokens=None), dict(ws=A + 32),
                                 dict(ws=None)])
def test_beam_selection_refuses(bad):
    with pytest.raises(E.EffortError) as e:
        E.effort_beam_select(**dict(SELECT, **bad), stream=0)
    assert e.value.code == B.EFFORT_EINVAL


def test_nothing_to_do_needs_no_device():
    for b in (batch(seqs=0, page_table=None, kv_lens=None, q_starts=None), batch(tokens=0)):
        call(E.effort_kv_append_ex, EX, b=b)
        call(E.effort_kv_attention_tree, TREE, b=b)
    none = book(seqs=0, page_table=None, kv_lens=None, refs=None, info=None)
    E.effort_kv_fork(none, None, None, stream=0)
    E.effort_kv_grow(none, B.kv_caches([cache()]), 1, None, 1, None, 0, stream=0)
    E.effort_kv_copy_pages(B.kv_caches([cache()]), 1, None, None, 0, stream=0)
    E.effort_kv_copy_pages(None, 0, A, A, 5, stream=0)
    E.effort_kv_accept(B.kv_caches([cache()]), 1, batch(seqs=0), None, None, None, None, 0, stream=0)
    E.effort_beam_select(**dict(SELECT, items=0, logits=None, scores=None), stream=0)


def test_struct_size_matches_the_header():
    assert ctypes.sizeof(E.effort_kv_book) == 4 * 4 + 2 * 8 + 4 * 8


def test_python_refuses():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    k, s = z(4, 2, 16, 64, dtype=torch.uint8), z(4, 2)
    one = E.KVCache.wrap(k, k.clone(), s, s.clone())
    for bad in (z(3), z(2, 2, **i32), z(8, **i32)[::2]):
        with pytest.raises(ValueError):
            E.KVBatch(z(3, 5, **i32), z(3, **i32), z(4, **i32), parents=bad)
    b = E.KVBatch(z(3, 5, **i32), z(3, **i32), z(4, **i32), parents=z(6, **i32))
    with pytest.raises(AttributeError):
        b.parents = z(6, **i32)
    assert torch.equal(pickle.loads(pickle.dumps(b)).parents, b.parents)
    with pytest.raises(ValueError, match="parents"):
        b.desc(7)
    kv, q = z(2, 2, 64), z(2, 4, 64)
    for bad in (dict(k_norm=z(63)), dict(k_norm=z(3, 64)), dict(k_norm=z(64).half()), dict(q_norm=z(64)),
                dict(q=q, q_norm=z(2, 64)), dict(q=q, q_norm=z(128)[::2])):
        with pytest.raises(ValueError):
            one.append(b, kv, kv, **bad)
    with pytest.raises(ValueError):  # everything is right but the device
        one.append(b, kv, kv, q=q, q_norm=z(4, 64), k_norm=z(64))
    other = E.KVCache.wrap(z(5, 2, 16, 64, dtype=torch.uint8), z(5, 2, 16, 64, dtype=torch.uint8), z(5, 2), z(5, 2))
    for bad in ([], [one, other]):
        with pytest.raises(ValueError):
            E.cache_set(bad)
    good = E.KVPages([one, one], torch.tensor([[0, 1], [0, -1], [3, 9]], **i32), z(3, **i32))
    assert good.refs.tolist() == [2, 1, 0, 1]
    with pytest.raises(AttributeError):
        good.refs = z(4, **i32)
    with pytest.raises(ValueError):
        pickle.loads(pickle.dumps(good)).fork(z(2, **i32))
    for bad in (dict(page_table=z(3, 2)), dict(page_table=z(2, 3, **i32).t()), dict(kv_lens=z(2, **i32)),
                dict(refs=z(5, **i32))):
        d = dict(page_table=z(3, 2, **i32), kv_lens=z(3, **i32), refs=None)
        d.update(bad)
        with pytest.raises(ValueError):
            E.KVPages([one], **d)
    for bad in (z(2, **i32), z(3), z(3, 1, **i32)):
        with pytest.raises(ValueError):
            good.fork(bad)
        with pytest.raises(ValueError):
            good.fork(z(3, **i32), lens=bad)
        with pytest.raises(ValueError):
            good.grow(bad)
        with pytest.raises(ValueError):
            E.kv_accept([one], b, bad)
        with pytest.raises(ValueError):
            E.kv_accept([one], b, z(3, **i32), lens_out=bad)
    with pytest.raises(ValueError):
        good.grow(1 << 31)
    for bad in ((z(2, **i32), z(3, **i32)), (z(2), z(2)), (z(2, 1, **i32), z(2, 1, **i32))):
        with pytest.raises(ValueError):
            E.kv_copy_pages([one], *bad)
    sc = z(2, 3)
    for bad in (z(5, 10), z(2, 4, 10), z(3, 2, 10), z(2, 3, 20)[..., ::2], z(2, 6, 10)[:, :3]):
        with pytest.raises(ValueError):
            E.beam_select(bad, sc)
    for bad in (dict(ended=z(2, 3)), dict(ended=z(3, 2, dtype=torch.bool)), dict(keep=1 << 40), dict(end_token=1 << 31)):
        with pytest.raises(ValueError):
            E.beam_select(z(6, 10), sc, **bad)
    for bad in (z(2, 3, dtype=torch.float64), z(6), z(3, 2).t()):
        with pytest.raises((ValueError, TypeError)):
            E.beam_select(z(6, 10), bad)
    with pytest.raises(TypeError):
        E.beam_select(z(6, 10, dtype=torch.float64), sc)


# ---------------------------------------------------------------- the definitions themselves

def test_a_chain_is_no_tree_to_the_definitions():
    rng = np.random.default_rng(1)
    shape = (6, 2, 16, 64)
    c = {"k": L.encode(rng.integers(-100, 100, shape).astype(float), "i8"), "v": L.encode(rng.integers(-9, 9, shape).astype(float), "i8"),
         "ks": np.full(shape[:2], 0.01, np.float32), "vs": np.ones(shape[:2], np.float32)}
    table, lens, starts = np.array([[0, 1], [3, 2]]), [20, 30], [0, 4, 9]
    q = rng.standard_normal((9, 4, 64))
    chain = [-1, 0, 1, 2, -1, 0, 1, 2, 3]
    for window in (0, 6):
        a, b = R.attend(c, table, lens, starts, q, 0.1, window, "i8", "f32", chain)
        x, y = L.attend(c, table, lens, starts, q, 0.1, window, "i8", "f32")
        assert np.allclose(a, x, rtol=1e-12, atol=0) and (b >= y).all()
    assert R.line([-1, 0, 1, 1, 7], 4) == [4] and R.line([-1, 0, 1, 1], 3) == [0, 1, 3]
    d = {k: v.copy() for k, v in c.items()}
    assert R.accept([d], "i8", table, lens, starts, 9, chain, [2, -1]) == [19, 25]
    assert all(np.array_equal(d[k], c[k]) for k in c)


def test_shared_pages_of_the_definition():
    b = R.Book([[0, 1, -1], [0, 1, -1], [0, 1, -1]], [20, 20, 20], 6, 16, [])
    assert b.grow([1, 1, 0]) == 0  # the third still holds page 1: both others copy it
    assert b.table.tolist() == [[0, 2, -1], [0, 3, -1], [0, 1, -1]] and b.refs().tolist() == [3, 1, 1, 1, 0, 0]
    b.fork([1, 1, 1], [40, 16, 3])
    assert b.table.tolist() == [[0, 3, -1], [0, -1, -1], [0, -1, -1]] and b.lens == [21, 16, 3]
    assert b.grow([1, 1, 1]) == 0 and b.table.tolist() == [[0, 3, -1], [0, 1, -1], [2, -1, -1]]


def test_beam_definition_against_all_pairs():
    rng = np.random.default_rng(2)
    x, s = rng.standard_normal((1, 3, 11)), rng.standard_normal((1, 3))
    y = s[0][:, None] + x[0] - np.log(np.exp(x[0]).sum(-1, keepdims=True))
    order = np.argsort(-y.ravel(), kind="stable")[:7]
    got = R.beams(x, s, 7)
    assert got[1][0] == (order // 11).tolist() and got[2][0] == (order % 11).tolist()
    assert np.allclose(got[0][0], y.ravel()[order])


def test_beam_step_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    z, i32 = torch.zeros, dict(dtype=torch.int32)
    k, s = z(4, 2, 16, 64, dtype=torch.uint8), z(4, 2)
    one, other = (E.KVCache.wrap(k.clone(), k.clone(), s.clone(), s.clone()) for _ in range(2))
    table, lens = z(6, 3, **i32), z(6, **i32)
    pages = E.KVPages([one], table, lens)

    def step(rows=6, batch=None, caches=(one,)):
        return SimpleNamespace(x=z(rows, 8), batch=batch or E.KVBatch(table, lens, z(7, **i32)), caches=list(caches))

    beam = E.BeamStep(step(), pages, 3)
    assert beam.scores.tolist() == [[0.0, -math.inf, -math.inf]] * 2 and not beam.ended.any()
    tree = E.KVBatch(table, lens, z(7, **i32), parents=z(6, **i32))
    wide = E.KVBatch(table[:5], lens[:5], z(6, **i32))
    for bad in (dict(beams=4), dict(beams=0), dict(step=step(caches=[one, other])), dict(step=step(batch=tree)),
                dict(step=step(batch=wide)), dict(step=step(rows=12)),
                dict(step=step(batch=E.KVBatch(table.clone(), lens, z(7, **i32)))),
                dict(step=step(batch=E.KVBatch(table, lens.clone(), z(7, **i32))))):
        d = dict(step=step(), pages=pages, beams=3)
        d.update(bad)
        with pytest.raises(ValueError):
            E.BeamStep(**d)


def test_decoder_step_refuses_head_norms_and_trees_that_do_not_fit():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    z, i32 = torch.zeros, dict(dtype=torch.int32)
    mat = lambda m, n: SimpleNamespace(in_dim=m, out_dim=n, batch=4, layout=z(1, dtype=torch.uint8))  # noqa: E731
    layer = {"wq": mat(32, 128), "wk": mat(32, 64), "wv": mat(32, 64), "wo": mat(128, 32), "w1": mat(32, 48),
             "w3": mat(32, 48), "w2": mat(48, 32)}
    k, s = z(4, 1, 16, 64, dtype=torch.uint8), z(4, 1)
    cache = E.KVCache.wrap(k, k.clone(), s, s.clone())
    mk = lambda qk_norms=None, parents=None: E.DecoderStep(  # noqa: E731
        [layer], mat(32, 10), z(3, 32), [cache], E.KVBatch(z(1, 2, **i32), z(1, **i32), z(2, **i32), parents=parents),
        [(z(32), z(32))], z(32), qk_norms=qk_norms)
    mk()
    mk(qk_norms=[(z(64), z(1, 64))], parents=z(3, **i32))
    mk(qk_norms=[(z(2, 64), None)])
    for bad in (dict(qk_norms=[]), dict(qk_norms=[(z(63), None)]), dict(qk_norms=[(None, z(2, 64))]),
                dict(qk_norms=[(z(64).half(), None)]), dict(qk_norms=[(z(128)[::2], None)]), dict(parents=z(2, **i32))):
        with pytest.raises(ValueError):
            mk(**bad)
