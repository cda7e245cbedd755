"""A step of whole decoder layers (DecoderStep): every link is compared with its
plain definition on the input that the GPU used, so that no error hides behind
the next link: matvecs with the oracle, the rest with tests/_layer.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
import oracle  # noqa: E402
import synth  # noqa: E402
from _parity import REL_L2_TOL, check, rel_l2  # noqa: E402

DIM, QH, KH, HD, HID, VOCAB, T = 512, 8, 2, 64, 1024, 640, 16
SHAPES = {"wq": (DIM, QH * HD), "wk": (DIM, KH * HD), "wv": (DIM, KH * HD), "wo": (QH * HD, DIM), "w1": (DIM, HID),
          "w3": (DIM, HID), "w2": (HID, DIM)}
LAYERS, CAP = 2, 4


class Stack:
    def __init__(self, lens, new, rows, seed, fmt="e4m3", window=0, inter=False):
        if not torch.cuda.is_available():
            pytest.skip("no GPU")
        self.rng = rng = np.random.default_rng(seed)
        self.fmt, self.window, self.inter = fmt, window, inter
        self.W = [{r: synth.matrix("decoder", *SHAPES[r], layer=l, w=r) for r in E.LAYER_ROLES} for l in range(LAYERS)]
        self.Wh = synth.matrix("decoder", DIM, VOCAB, w="head")
        self.probes = {id(w): oracle.probes(w, 16) for w in [self.Wh] + [x for d in self.W for x in d.values()]}
        mat = lambda w: E.EffortMatrix(w, P=16, batch=rows)  # noqa: E731
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.lens, self.starts = np.array(lens), [0] + list(np.cumsum(new))
        self.table = rng.permutation(len(lens) * CAP + 1)[:len(lens) * CAP].reshape(len(lens), CAP)
        caches = [E.KVCache(len(lens) * CAP + 1, KH, HD, T, format=E.EFFORT_KV_I8 if fmt == "i8" else E.EFFORT_KV_E4M3)
                  for _ in range(LAYERS)]
        shape = caches[0].k.shape
        self.np = [{"k": np.zeros(shape, np.uint8), "v": np.zeros(shape, np.uint8), "ks": np.zeros(shape[:2], np.float32),
                    "vs": np.zeros(shape[:2], np.float32)} for _ in range(LAYERS)]
        i32 = lambda a: to(np.array(a, np.int32))  # noqa: E731
        self.batch = E.KVBatch(i32(self.table), i32(self.lens), i32(self.starts))
        self.norms = [[(rng.random(DIM) + 0.5).astype(np.float32) for _ in range(2)] for _ in range(LAYERS)]
        self.head_norm = (rng.random(DIM) + 0.5).astype(np.float32)
        self.rope = L.rope_rows(10000.0, CAP * T, HD)
        self.x = torch.zeros(rows, DIM, device="cuda")
        self.step = E.DecoderStep([{r: mat(w) for r, w in d.items()} for d in self.W], mat(self.Wh), self.x, caches,
                                  self.batch, [tuple(map(to, n)) for n in self.norms], to(self.head_norm),
                                  rope=to(self.rope), interleaved=inter, window=window)

    def next_x(self):
        self.x.copy_(torch.from_numpy(self.rng.standard_normal(self.x.shape).astype(np.float32)))

    def advance(self, by):
        self.lens = self.lens + np.asarray(by)
        self.batch.kv_lens.copy_(torch.from_numpy(self.lens.astype(np.int32)))

    def matvecs(self, key, w, x, effort, y, res):
        for i in range(len(x)):
            ref = oracle.run(w, self.probes[id(w)], np.ascontiguousarray(x[i]), effort)
            if res is not None:
                check(res[key], ref, where=key, y=y[i])
            else:
                assert rel_l2(y[i], ref["y"]) <= REL_L2_TOL, key

    def check(self, effort, record=None):
        """Every link of the step that has just run; `record` as given to it."""
        torch.cuda.synchronize()
        res = record.results() if record is not None else None
        e = effort if callable(effort) else (lambda l, r: effort)
        get = lambda t: t.cpu().numpy()  # noqa: E731
        rows = len(self.x)
        pos = L.positions(self.lens, self.starts, rows)
        r = get(self.x).astype(np.float64)
        step = 2.0 ** -24

        def norm(r, w, got, err):
            # `err` is how far off the stream that the norm read may be; the mean of 512 squares and
            # its root, and two products, are within 2^-20 of their values
            _, ref, _ = L.norm(r, None, None, None, 1.0, w.astype(np.float64), 1e-5)
            rms = np.sqrt((r * r).mean(-1, keepdims=True))
            slack = (err + np.sqrt((err * err).mean(-1, keepdims=True)) * np.abs(r) / rms) / rms * w
            assert (np.abs(got - ref) <= 2.0 ** -20 * np.abs(ref) + slack).all()

        for l in range(LAYERS):
            o = {k: get(t) for k, t in self.step.out[l].items()}
            norm(r, self.norms[l][0], o["hq"], step * np.abs(r))
            for k in ("wq", "wk", "wv"):
                self.matvecs((l, k), self.W[l][k], o["hq"], e(l, k), o[k], res)
            heads = lambda a: a.reshape(rows, -1, HD)  # noqa: E731
            q = heads(o["q"]).astype(np.float64)
            for row, s, p in pos:
                x = heads(o["wq"])[row].astype(np.float64)
                d = np.abs(q[row] - L.rotate(x, self.rope[p], self.inter))
                assert (d <= 4 * step * np.abs(x).max()).all()
            c, cache = self.np[l], self.step.caches[l]
            L.append(c, self.table, self.lens, self.starts, heads(o["wk"]), heads(o["wv"]), self.rope, self.inter, self.fmt)
            for name, scale, codes in (("k", cache.k_scale, cache.k), ("v", cache.v_scale, cache.v)):
                assert np.array_equal(get(scale), c[name + "s"]) and L.same_codes(get(codes), c[name], self.fmt)
            ref, tol = L.attend(c, self.table, self.lens, self.starts, q, HD ** -0.5, self.window, self.fmt, "f32")
            for row, s, p in pos:
                assert (np.abs(heads(o["a"])[row] - ref[row]) <= tol[row]).all()
            self.matvecs((l, "wo"), self.W[l]["wo"], o["a"], e(l, "wo"), o["wo"], res)
            mid = r + o["wo"]
            # r itself was rounded to fp32 before, and the sum is now
            assert (np.abs(o["r"] - mid) <= step * (np.abs(r) + np.abs(mid))).all()
            norm(o["r"].astype(np.float64), self.norms[l][1], o["hf"], 0.0 * mid)
            for k in ("w1", "w3"):
                self.matvecs((l, k), self.W[l][k], o["hf"], e(l, k), o[k], res)
            assert rel_l2(o["g"], oracle.silu_mul(o["w1"], o["w3"])) <= 1e-6
            self.matvecs((l, "w2"), self.W[l]["w2"], o["g"], e(l, "w2"), o["w2"], res)
            r = o["r"].astype(np.float64) + o["w2"]
        assert (np.abs(get(self.step.r) - r) <= step * np.abs(r)).all()
        norm(r, self.head_norm, get(self.step.h), step * np.abs(r))
        self.matvecs((None, "head"), self.Wh, get(self.step.h), e(None, "head"), get(self.step.logits), res)


def test_one_sequence_recorded():
    s = Stack([1], [1], 1, seed=1)
    effort = E.EffortSchedule(0.3, {(None, "w2"): 0.2, (1, None): 0.5, (None, "head"): 0.7})
    for t in range(3):
        s.next_x()
        rec = E.Recorder(s.x.device)
        s.step.enqueue(effort, record=rec)
        s.check(effort, rec)
        s.advance(1)


@pytest.mark.parametrize("fmt,window,inter", [("e4m3", 0, False), ("i8", 5, True)])
def test_prompt_then_tokens(fmt, window, inter):
    """Two sequences' prompts (17 tokens would not fit the 16 vectors of a call),
    then their tokens one by one on the same caches, then none for one of them."""
    s = Stack([9, 4], [9, 4], 13, seed=2, fmt=fmt, window=window, inter=inter)
    s.next_x()
    s.step.enqueue(0.4)
    s.check(0.4)
    for new in ([1, 1], [2, 1], [0, 1]):
        s.starts = [0] + list(np.cumsum(new))
        s.batch.q_starts.copy_(torch.tensor(s.starts, dtype=torch.int32))
        s.advance(torch.tensor(new, dtype=torch.int32))
        s.next_x()  # the rows behind the last sequence hold values, too
        s.step.enqueue(0.4)
        s.check(0.4)


@pytest.mark.parametrize("rows", [1, 3])
def test_captured_step(rows):
    """One capture serves every step: the lengths advance on the device."""
    s = Stack([3, 15, 30][:rows], [1] * rows, rows, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.next_x()
    s.step.enqueue(0.25, stream=side)  # loads the kernels, and is itself a step
    torch.cuda.current_stream().wait_stream(side)
    s.check(0.25)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step.enqueue(0.25)
    for _ in range(5):
        s.advance(1)
        s.next_x()
        s.step.logits.fill_(float("nan"))
        g.replay()
        s.check(0.25)
