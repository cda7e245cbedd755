"""What a step of whole decoder layers refuses when it is put together (on the
host: no kernel runs)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import dynamic_sparsity_approximate_amd as E  # noqa: E402
import synth  # noqa: E402

DIM, QD, KD, HID, VOCAB = 128, 256, 128, 192, 160
SHAPES = {"wq": (DIM, QD), "wk": (DIM, KD), "wv": (DIM, KD), "wo": (QD, DIM), "w1": (DIM, HID), "w3": (DIM, HID),
          "w2": (HID, DIM)}
MATS = {}


def mat(m, n, batch):
    if (m, n, batch) not in MATS:
        MATS[m, n, batch] = E.EffortMatrix(synth.matrix("decoder", m, n), P=16, device="cpu", batch=batch)
    return MATS[m, n, batch]


def parts(batch=2, tokens=2, **shapes):
    layers = [{r: mat(*shapes.get(r, SHAPES[r]), batch) for r in E.LAYER_ROLES} for _ in range(2)]
    one = torch.ones(DIM)
    return dict(layers=layers, head=mat(*shapes.get("head", (DIM, VOCAB)), batch), x=torch.zeros(tokens, DIM),
                caches=[E.KVCache(4, 2, 64, page_tokens=16, device="cpu") for _ in range(2)],
                batch=E.KVBatch(*(torch.zeros(s, dtype=torch.int32) for s in ((2, 2), (2,), (3,)))),
                norms=[(one, one)] * 2, head_norm=one)


def test_fits():
    step = E.DecoderStep(**parts())
    assert step.logits.shape == (2, VOCAB) and len(step.out) == 2 and step.groups is None


@pytest.mark.parametrize("shapes", [dict(wq=(DIM, 192)), dict(wk=(DIM, 256)), dict(wv=(DIM, 192)), dict(wo=(DIM, DIM)),
                                    dict(w3=(DIM, 128)), dict(w2=(DIM, DIM)), dict(w2=(HID, QD)), dict(head=(QD, VOCAB)),
                                    dict(w1=(QD, HID))])
def test_matrices_that_do_not_fit(shapes):
    with pytest.raises(ValueError):
        E.DecoderStep(**parts(**shapes))


@pytest.mark.parametrize("change", [dict(x=torch.zeros(DIM)), dict(x=torch.zeros(0, DIM)),
                                    dict(x=torch.zeros(2, DIM, dtype=torch.float16)),
                                    dict(x=torch.zeros(2, 2 * DIM)[:, ::2]), dict(x=torch.zeros(3, DIM)),
                                    dict(x=torch.zeros(2, QD)), dict(caches=[]), dict(norms=[])])
def test_inputs_that_do_not_fit(change):
    with pytest.raises(ValueError):
        E.DecoderStep(**dict(parts(), **change))


def test_a_batch_cannot_be_recorded():
    with pytest.raises(ValueError, match="recorded"):
        E.DecoderStep(**parts()).enqueue(0.5, record=object())
