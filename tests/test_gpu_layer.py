"""The operators between a decoder layer's matvecs against their 64-bit
definitions (tests/_layer.py): codes and scales of the cache exactly, attention
and norms within bounds that count their roundings."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMT = {"e4m3": E.EFFORT_KV_E4M3, "i8": E.EFFORT_KV_I8}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(new):
    return [0] + list(np.cumsum(new))


class Case:
    """A cache with random pages, page tables of sequences of `lens` tokens in a
    shuffled pool, and the numpy copy the definitions run on."""

    def __init__(self, seed, lens, new, heads=2, group=2, dim=128, page=32, fmt="e4m3", dtype="f32", room=0,
                 garbage=True, spread=0):
        dev()
        self.rng = rng = np.random.default_rng(seed)
        self.heads, self.group, self.dim, self.page, self.fmt, self.dtype = heads, group, dim, page, fmt, dtype
        self.lens, self.new = list(lens), list(new)
        self.starts = starts_of(new)
        counts = [-(-(t + room) // page) for t in lens]
        self.pages = sum(counts) + 2
        order = rng.permutation(self.pages)
        cols = max(counts + [1])
        self.table = np.full((len(lens), cols), -7, np.int64)
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = order[at:at + c]
            at += c
        shape = (self.pages, heads, page, dim)
        if fmt == "i8":
            mk = lambda: rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)  # noqa: E731
        else:
            mk = lambda: L.encode(np.clip(rng.standard_normal(shape) * 90, -448, 448), fmt)  # noqa: E731
        sc = lambda: 2.0 ** (-6 + rng.integers(-spread, spread + 1, shape[:2])).astype(np.float64)  # noqa: E731
        self.np = {"k": mk(), "v": mk(), "ks": sc().astype(np.float32), "vs": sc().astype(np.float32)}
        if garbage:  # behind every end, and in pages of nobody: codes and scales that are NaN
            live = np.zeros((self.pages, page), bool)
            for s, t in enumerate(lens):
                for p in range(max(t, 0)):
                    live[self.table[s, p // page], p % page] = True
            for name in "kv":
                self.np[name][np.broadcast_to(~live[:, None, :, None], shape)] = 0x7F if fmt == "e4m3" else 0x80
                self.np[name + "s"][~live.any(1)] = np.nan
        to = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.cache = E.KVCache.wrap(to(self.np["k"]), to(self.np["v"]), to(self.np["ks"]), to(self.np["vs"]),
                                    FMT[fmt])
        self.batch = E.KVBatch(torch.from_numpy(self.table.astype(np.int32)).cuda(), ints(self.lens),
                               ints(self.starts))

    def rand(self, heads, scale=1.0, rows=None):
        n = self.starts[-1] if rows is None else rows
        x = self.rng.standard_normal((n, heads, self.dim)) * scale
        return torch.from_numpy(x).to(DT[self.dtype]).cuda()

    def check_cache(self):
        torch.cuda.synchronize()
        for name in "kv":
            got = getattr(self.cache, name + "_scale").cpu().numpy()
            assert np.array_equal(got, self.np[name + "s"], equal_nan=True), name
            assert L.same_codes(getattr(self.cache, name).cpu().numpy(), self.np[name], self.fmt), name

    def check_attend(self, q, window=0, scale=None, out=None, got=None):
        sc = self.dim ** -0.5 if scale is None else scale
        if got is None:
            got = self.cache.attend(self.batch, q, window=window, scale=scale, out=out)
        torch.cuda.synchronize()
        ref, tol = L.attend(self.np, self.table, self.lens, self.starts, f64(q), sc, window, self.fmt, self.dtype)
        g = f64(got)
        rows = [r for r, _, _ in L.positions(self.lens, self.starts, len(q))]
        assert np.array_equal(np.isnan(g[rows]), np.isnan(ref[rows]))
        d = np.abs(g[rows] - ref[rows])
        ok = ~np.isnan(ref[rows])
        worst = float((d[ok] / (tol[rows][ok] + 1e-300)).max()) if ok.any() else 0.0
        assert (d[ok] <= tol[rows][ok]).all(), worst
        return got, worst


# ---------------------------------------------------------------- table

def test_rope_table():
    d = dev()
    for base, rows, rot in ((10000.0, 300, 128), (500000.0, 70000, 64), (2.0, 5, 8)):
        got = E.rope_table(base, rows, rot, d).cpu().numpy()
        ref = L.rope_rows(base, rows, rot)
        # the angle is off by its own rounding in double, the result by one rounding
        assert np.abs(got.astype(np.float64) - ref).max() <= 2.0 ** -23


# ---------------------------------------------------------------- append

APPEND = [
    # fmt, dtype, dim, page, rot, interleaved
    ("e4m3", "f32", 128, 64, 128, False), ("e4m3", "f32", 128, 32, 64, True), ("e4m3", "bf16", 64, 16, 64, False),
    ("e4m3", "f16", 64, 128, 24, True), ("i8", "f32", 128, 16, 128, True), ("i8", "f16", 64, 32, 8, False),
    ("i8", "bf16", 128, 128, 128, False), ("e4m3", "bf16", 128, 64, 0, False),
]


@pytest.mark.parametrize("fmt,dtype,dim,page,rot,inter", APPEND)
def test_append_exact(fmt, dtype, dim, page, rot, inter):
    # none, one, a page's end, several pages, one that starts in a page's middle
    lens, new = [40, 1, page, 3 * page + 5, 2 * page + 7, 0], [0, 1, 1, 2 * page + 9, 3, 0]
    c = Case(3, lens, new, dim=dim, page=page, fmt=fmt, dtype=dtype)
    k, v, q = c.rand(2, 3.0), c.rand(2), c.rand(4)
    rope = L.rope_rows(10000.0, c.table.shape[1] * page, rot) if rot else None
    got = c.cache.append(c.batch, k, v, q=q, rope=None if rope is None else torch.from_numpy(rope).cuda(),
                         interleaved=inter)
    L.append(c.np, c.table, lens, c.starts, f64(k), f64(v), rope, inter, fmt)
    c.check_cache()
    ref, size = f64(q), np.abs(f64(q))
    for row, s, p in L.positions(lens, c.starts, len(k)):
        if rope is not None:
            ref[row] = L.rotate(ref[row], rope[p], inter)
            size[row] = np.abs(size[row]) + np.abs(L.rotate(size[row], np.abs(rope[p]) * [1, -1], inter))
    # two fp32 roundings of the terms, one of the result
    assert (np.abs(f64(got) - ref) <= 2.0 ** -23 * size + L.HALF_STEP[dtype] * np.abs(ref) + 2.0 ** -25).all()


def test_append_many_steps_grow_scales():
    """One token a call: scales that grow within a page re-express its older
    tokens; over 70 steps the cache follows the definition exactly."""
    for fmt in ("e4m3", "i8"):
        c = Case(5, [1, 30], [1, 1], fmt=fmt, room=80, garbage=False)
        rope = L.rope_rows(10000.0, c.table.shape[1] * c.page, 128)
        rt = torch.from_numpy(rope).cuda()
        for step in range(70):
            mag = 2.0 ** (step % 11 - 5)
            k, v = c.rand(2, mag), c.rand(2, 1.0 / mag)
            c.cache.append(c.batch, k, v, rope=rt)
            L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), rope, False, fmt)
            c.check_cache()
            c.lens = [t + 1 for t in c.lens]
            c.batch.kv_lens.add_(1)


def test_append_ties_zeros_extremes():
    """Values on ties between codes, all zeros, tiny and huge magnitudes."""
    for fmt in ("e4m3", "i8"):
        c = Case(6, [5, 5, 5, 5, 5], [5] * 5, fmt=fmt)
        k = torch.zeros(25, 2, 128, device="cuda")
        grid = torch.arange(-127.0, 127.5, 0.5) if fmt == "i8" else torch.from_numpy(
            np.concatenate([(L.E4M3_POS[1:] + L.E4M3_POS[:-1]) / 2, -L.E4M3_POS])).float()
        k[0:5].view(-1)[:len(grid)] = grid.cuda()
        k[0, :, 0] = L.QMAX[fmt]
        k[5:10] = 1e-30 * torch.randn(5, 2, 128, device="cuda")
        k[10:15] = 3e38 * torch.rand(5, 2, 128, device="cuda")
        k[15:20] = 1e-42 * torch.randn(5, 2, 128, device="cuda")
        v = k.flip(0).contiguous()
        c.cache.append(c.batch, k, v)
        L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), None, False, fmt)
        c.check_cache()


def test_append_to_scales_of_another_program():
    """Pages whose scales are no powers of two keep them while they suffice."""
    for fmt in ("e4m3", "i8"):
        for inter in (False, True):
            c = Case(61, [20, 40, 33], [3, 5, 1], fmt=fmt)
            c.np["ks"] = (0.03 + 0.05 * c.rng.random(c.np["ks"].shape)).astype(np.float32)
            c.np["vs"] = (0.03 + 0.05 * c.rng.random(c.np["vs"].shape)).astype(np.float32)
            c.cache.k_scale.copy_(torch.from_numpy(c.np["ks"]))
            c.cache.v_scale.copy_(torch.from_numpy(c.np["vs"]))
            k, v = c.rand(2), c.rand(2, 40.0)
            rope = L.rope_rows(10000.0, c.table.shape[1] * c.page, 128)
            c.cache.append(c.batch, k, v, rope=torch.from_numpy(rope).cuda(), interleaved=inter)
            L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), rope, inter, fmt)
            c.check_cache()


def test_append_to_negative_scales():
    """They are poisoned: the page becomes NaN unless it is begun anew."""
    c = Case(64, [20, 40, 32], [3, 5, 32], page=32)
    for name in ("ks", "vs"):
        c.np[name][c.table[:, 0]] = [-2.0, -0.0]
        c.np[name][c.table[1, 1]] = [0.5, -1.0]
        getattr(c.cache, name[0] + "_scale").copy_(torch.from_numpy(c.np[name]))
    k, v = c.rand(2), c.rand(2)
    c.cache.append(c.batch, k, v)
    L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), None, False, "e4m3")
    assert np.isnan(c.np["ks"][c.table[0, 0]]).all() and np.isfinite(c.np["ks"][c.table[2, 0]]).all()
    c.check_cache()


def test_nothing_to_do():
    """No rows, no sequences."""
    d = dev()
    r, out = E.norm_residual(torch.empty(0, 64, device=d), torch.empty(0, 64, device=d))
    assert r.shape == out.shape == (0, 64)
    c = Case(65, [40], [0], page=32)
    none = torch.empty(0, 2, 128, device=d)
    q = c.cache.append(c.batch, none, none, q=torch.empty(0, 4, 128, device=d))
    assert q.shape == (0, 4, 128) and c.cache.attend(c.batch, q).shape == (0, 4, 128)
    nobody = E.KVBatch(torch.empty(0, 3, dtype=torch.int32, device=d), ints([]), ints([0]))
    x = c.rand(2, rows=3)
    out = torch.full((3, 2, 128), 7.0, device=d)
    assert c.cache.append(nobody, x, x, q=x, q_out=out) is out and (out == 7).all()
    assert c.cache.attend(nobody, x, out=out) is out and (out == 7).all()
    c.check_cache()


def test_append_rows_of_nobody_and_bad_pages():
    """Padded rows, a negative position, a length behind the table, page ids out
    of range: nothing of them is stored and their q rows stay."""
    page = 16
    lens, new = [20, 2, 90, 33, -4, 0], [2, 5, 4, 20, 3, 2]
    c = Case(7, [20, 2, 64, 33, 0, 0], new, page=page)
    c.lens = lens
    c.batch.kv_lens.copy_(ints(lens))
    c.table[3, 1] = c.pages
    c.table[0, 1] = -1
    c.batch.page_table.copy_(torch.from_numpy(c.table.astype(np.int32)))
    n = c.starts[-1] + 7  # 7 rows behind the last sequence
    k, v, q = c.rand(2, rows=n), c.rand(2, rows=n), c.rand(4, rows=n)
    rope = L.rope_rows(10000.0, c.table.shape[1] * page, 128)
    q_out = torch.full_like(q, 77.0)
    c.cache.append(c.batch, k, v, q=q, rope=torch.from_numpy(rope).cuda(), q_out=q_out)
    L.append(c.np, c.table, lens, c.starts, f64(k), f64(v), rope, False, "e4m3")
    c.check_cache()
    cap = c.table.shape[1] * page
    written = {r for r, _, p in L.positions(lens, c.starts, n) if 0 <= p < cap}
    for r in range(n):
        assert bool((q_out[r] == 77.0).all()) == (r not in written), r


def test_append_poison_and_fresh_start():
    page = 16
    c = Case(8, [20, 20], [2, 2], page=page)
    k, v = c.rand(2), c.rand(2)
    k[0, 0, 3], v[2, 1, 7] = float("nan"), float("inf")
    c.cache.append(c.batch, k, v)
    L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), None, False, "e4m3")
    assert np.isnan(c.np["ks"]).any() and np.isnan(c.np["vs"]).any()
    c.check_cache()
    q = c.rand(4)
    got, _ = c.check_attend(q)  # the poisoned heads are NaN, the others are not
    assert torch.isnan(got[0:2, 0:2]).all() and not torch.isnan(got[0:2, 2:]).any()
    assert torch.isnan(got[2:4, 2:]).all() and not torch.isnan(got[2:4, :2]).any()
    # the page's next user starts at its slot 0 and is clean
    c.lens, c.new = [16 + 3, 16 + 3], [3, 3]
    c.starts = starts_of(c.new)
    c.batch = E.KVBatch(c.batch.page_table, ints(c.lens), ints(c.starts))
    k, v = c.rand(2), c.rand(2)
    c.cache.append(c.batch, k, v)
    L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), None, False, "e4m3")
    c.check_cache()
    c.check_attend(c.rand(4))


def test_append_strided_unaligned_in_place():
    for dtype in ("f32", "bf16"):
        c = Case(9, [70, 9], [40, 9], dtype=dtype)
        fused = c.rand(4 + 2 + 2)
        flat = torch.zeros(49 * (8 * 128 + 3) + 5, dtype=DT[dtype], device="cuda")
        rows = flat[5:].view(49, 8 * 128 + 3)[:, :8 * 128]  # odd stride, not 16-byte aligned
        rows.copy_(fused.view(49, -1))
        rope = L.rope_rows(10000.0, c.table.shape[1] * c.page, 128)
        rt = torch.from_numpy(rope).cuda()
        view = rows.unflatten(1, (8, 128))
        a = c.cache.append(c.batch, view[:, 4:6], view[:, 6:], q=view[:, :4], rope=rt)
        L.append(c.np, c.table, c.lens, c.starts, f64(fused[:, 4:6]), f64(fused[:, 6:]), rope, False, "e4m3")
        c.check_cache()
        q = fused[:, :4].contiguous()
        b = c.cache.append(c.batch, fused[:, 4:6], fused[:, 6:], q=q, rope=rt, q_out=q)
        assert b is q and torch.equal(a, q)
        c.check_cache()  # appended again over itself: the same


# ---------------------------------------------------------------- attention

ATTEND = [
    # fmt, dtype, dim, page, group, window
    ("e4m3", "f32", 128, 64, 4, 0), ("e4m3", "bf16", 128, 16, 4, 0), ("e4m3", "f16", 64, 32, 3, 0),
    ("i8", "f32", 64, 128, 1, 0), ("i8", "bf16", 128, 32, 8, 0), ("i8", "f16", 128, 16, 2, 50),
    ("e4m3", "f32", 128, 32, 5, 1), ("e4m3", "bf16", 64, 64, 16, 33), ("e4m3", "f32", 64, 16, 20, 7),
]


@pytest.mark.parametrize("fmt,dtype,dim,page,group,window", ATTEND)
@pytest.mark.parametrize("kind", ["one", "few", "prompt", "one in a long table", "few in a long table"])
def test_attend(fmt, dtype, dim, page, group, window, kind):
    room = 3000 if "long" in kind else 0
    if kind == "one in a long table":
        lens = [1, 15, 31, 32, 33, 127, 128, 129, 0, 300]
        new = [1] * len(lens)
    elif kind == "one":
        lens = [1, 15, 16, 17, 0, 31, 32, 33, 127, 128, 129, 700, 1403]
        new = [1] * len(lens)
    elif kind.startswith("few"):
        lens, new = [7, 1, 40, 0, 333, 5, 64, 200], [7, 1, 3, 2, 5, 0, 4, 8]
    else:
        lens, new = [130, 65, 64, 300, 33, 1, 257], [130, 65, 17, 41, 33, 1, 128]
    c = Case(11, lens, new, group=group, dim=dim, page=page, fmt=fmt, dtype=dtype, room=room)
    _, worst = c.check_attend(c.rand(2 * group, 1.5), window=window)
    say("attend %s %s %s D %d page %d group %d window %d: %.3f of the bound" % (
        kind, fmt, dtype, dim, page, group, window, worst))


def test_attend_scales_far_apart():
    """Page scales from 2^-46 to 2^34: each row is right relative to its own
    largest weighted value."""
    for dtype in ("f32", "bf16"):
        for new in ([1, 1, 1], [40, 130, 1]):
            c = Case(12, [300, 130, 64], new, page=16, spread=40, dtype=dtype)
            c.np["ks"] = np.full_like(c.np["ks"], 2.0 ** -6)
            c.cache.k_scale.copy_(torch.from_numpy(c.np["ks"]))
            c.check_attend(c.rand(4, 1.5))


def test_attend_any_scale():
    """A cache that another program wrote: scales that are no powers of two, and zeros."""
    c = Case(13, [300, 77], [1, 30], page=16, garbage=False)
    for name in ("ks", "vs"):
        c.np[name] = (c.rng.random(c.np[name].shape) * 0.05).astype(np.float32)
        c.np[name][c.table[0, 2]] = 0.0
    c.cache.k_scale.copy_(torch.from_numpy(c.np["ks"]))
    c.cache.v_scale.copy_(torch.from_numpy(c.np["vs"]))
    c.check_attend(c.rand(4, 1.5))


def test_attend_rows_of_nobody_and_bad_pages():
    page = 16
    for new in ([2, 5, 4, 20, 3, 2, 1], [1, 1, 1, 1, 1, 1, 1]):
        c = Case(14, [20, 2, 64, 33, 0, 0, 40], new, page=page, garbage=False)
        c.lens = [20, 2, 90, 33, -4, 0, 40]
        c.batch.kv_lens.copy_(ints(c.lens))
        c.table[3, 1] = c.pages
        c.table[0, 1] = -1
        c.table[6, :] = -1  # no page at all: rows that see nothing
        c.batch.page_table.copy_(torch.from_numpy(c.table.astype(np.int32)))
        n = c.starts[-1] + 3
        q = c.rand(4, rows=n)
        out = torch.full_like(q, 77.0)
        c.check_attend(q, out=out)
        assert bool((out[-3:] == 77.0).all()) and bool((out[c.starts[6]:c.starts[7]] == 0.0).all())


@pytest.mark.parametrize("fmt,dtype,dim,page", [("e4m3", "bf16", 128, 64), ("i8", "f16", 64, 16),
                                                ("e4m3", "f32", 128, 32)])
def test_attend_chunk_behind_a_long_prefix(fmt, dtype, dim, page):
    """Few blocks of 128 rows whose tokens are shared out and joined."""
    c = Case(51, [1450, 1171], [263, 259], heads=1, group=4, dim=dim, page=page, fmt=fmt, dtype=dtype)
    c.check_attend(c.rand(4, 2.0))
    c.check_attend(c.rand(4, 2.0), window=700)


@pytest.mark.parametrize("window", [1, 300, 895, 896, 897, 2000])
@pytest.mark.parametrize("dtype,page,new", [("f32", 64, [1, 1, 1]), ("bf16", 16, [8, 5, 1])])
def test_attend_window_of_a_long_table(dtype, page, new, window):
    c = Case(53, [5000, 2777, 40], new, group=4, page=page, dtype=dtype)
    c.check_attend(c.rand(8, 2.0), window=window)


def test_attend_more_blocks_of_rows_than_65535():
    """131100 tokens of 64 query heads: rows here and there against the definition."""
    c = Case(52, [131100], [131100], heads=1, group=64, dim=64, page=128, dtype="f16", garbage=False)
    q = torch.randn(131100, 64, 64, device="cuda", dtype=torch.float16)
    got = c.cache.attend(c.batch, q, window=16)
    torch.cuda.synchronize()
    for i in (0, 1, 63, 65534, 65535, 100001, 131070, 131099):
        ref, tol = L.attend(c.np, c.table, [i + 1], [0, 1], f64(q[i:i + 1]), 64 ** -0.5, 16, "e4m3", "f16")
        assert (np.abs(f64(got[i:i + 1]) - ref) <= tol).all(), i


@pytest.mark.parametrize("new", [[1], [5], [40], [1, 1], [3, 60]])
@pytest.mark.parametrize("room", [0, 3000])
def test_rows_before_the_first_sequence(new, room):
    """q_starts[0] > 0: the rows before it are nobody's."""
    lens = [n + 50 for n in new]
    c = Case(62, lens, new, page=16, room=room)
    c.starts = [x + 37 for x in c.starts]
    c.batch = E.KVBatch(c.batch.page_table, ints(lens), ints(c.starts))
    n = c.starts[-1] + 2
    q, k, v = c.rand(4, rows=n), c.rand(2, rows=n), c.rand(2, rows=n)
    q_out, out = torch.full_like(q, 77.0), torch.full_like(q, 77.0)
    c.cache.append(c.batch, k, v, q=q, q_out=q_out)
    L.append(c.np, c.table, lens, c.starts, f64(k), f64(v), None, False, "e4m3")
    c.check_cache()
    c.check_attend(q, out=out)
    for t in (q_out, out):
        assert bool((t[:37] == 77.0).all()) and bool((t[-2:] == 77.0).all())
    assert torch.equal(q_out[37:-2], q[37:-2])


def test_attend_poisoned_page_reaches_only_who_sees_it():
    page = 16
    for name in ("ks", "vs"):
        c = Case(15, [100, 200], [60, 30], page=page)
        c.np[name][c.table[0, 4], 1] = np.inf  # positions 64 .. 79 of sequence 0, head 1
        c.np[name][c.table[1, 2], 0] = np.nan
        getattr(c.cache, name[0] + "_scale").copy_(torch.from_numpy(c.np[name]))
        q = c.rand(4)
        c.np = dict(c.np)
        got = c.cache.attend(c.batch, q)
        torch.cuda.synchronize()
        nan = torch.isnan(got).all(-1).cpu().numpy()
        assert np.array_equal(nan, torch.isnan(got).any(-1).cpu().numpy())
        want = np.zeros_like(nan)
        want[100 - 60 - 40 + 24:60, 2:] = True  # position 40 + i >= 64
        want[60:, :2] = True
        assert np.array_equal(nan, want)
        c.check_attend(q, got=got)


def test_attend_large_scores_and_uniform():
    c = Case(16, [500, 129], [1, 129], dtype="f32")
    c.check_attend(c.rand(4, 300.0))       # one key takes all
    c.check_attend(c.rand(4, 1e-20))       # all keys alike
    q = c.rand(4)
    c.check_attend(q, scale=0.0)
    c.check_attend(q, scale=-0.3)
    q[0, 0] = 0.0
    q[5, 3, 7] = float("inf")
    q[6, 2] = float("nan")
    got = c.cache.attend(c.batch, q)
    torch.cuda.synchronize()
    nan = torch.isnan(got)
    assert nan[5, 3].all() and nan[6, 2].all()
    nan[5, 3] = nan[6, 2] = False
    assert not nan.any()


def test_attend_strided():
    for dtype in ("f32", "bf16"):
        for new in ([1, 1], [40, 30]):
            c = Case(17, [100, 45], new, dtype=dtype)
            n = c.starts[-1]
            flat = torch.zeros(n * (5 * 128 + 1) + 1, dtype=DT[dtype], device="cuda")
            q = flat[1:].view(n, 5 * 128 + 1)[:, :512].unflatten(1, (4, 128))
            q.copy_(c.rand(4))
            out = torch.full((n, 6, 128), 77.0, dtype=DT[dtype], device="cuda")
            c.check_attend(q, out=out[:, 1:5])
            assert bool((out[:, 0] == 77.0).all()) and bool((out[:, 5] == 77.0).all())
            flat_out = torch.zeros_like(flat)
            c.check_attend(q, out=flat_out[1:].view(n, 5 * 128 + 1)[:, :512].unflatten(1, (4, 128)))


def test_attend_many_sequences():
    rng = np.random.default_rng(18)
    lens = [int(x) for x in rng.integers(0, 60, 700)]
    new = [min(t, int(x)) for t, x in zip(lens, rng.integers(0, 3, 700))]
    c = Case(18, lens, new, heads=1, group=2, dim=64, page=16, dtype="f16")
    c.check_attend(c.rand(2))


def test_attend_far_pages():
    """Pages whose codes lie behind 2^31 and 2^32 bytes."""
    d = dev()
    heads, page, dim, pages = 8, 128, 128, 33000
    k = torch.empty((pages, heads, page, dim), dtype=torch.uint8, device=d)
    v = torch.empty_like(k)
    ks = torch.full((pages, heads), 2.0 ** -6, device=d)
    vs = ks.clone()
    cache = E.KVCache.wrap(k, v, ks, vs)
    table = np.array([[32999, 16384, 5, 20000]])
    batch = E.KVBatch(torch.from_numpy(table.astype(np.int32)).cuda(), ints([400]), ints([0, 400]))
    rng = np.random.default_rng(19)
    rand = lambda h: torch.from_numpy(rng.standard_normal((400, h, dim))).float().cuda()  # noqa: E731
    kk, vv, q = rand(heads), rand(heads), rand(heads)
    cache.append(batch, kk, vv)
    small = {n: t[table[0]].cpu().numpy() for n, t in (("k", k), ("v", v), ("ks", ks), ("vs", vs))}
    want = {"k": np.zeros_like(small["k"]), "v": np.zeros_like(small["v"]), "ks": np.ones((4, heads), np.float32),
            "vs": np.ones((4, heads), np.float32)}
    order = np.array([[0, 1, 2, 3]])
    L.append(want, order, [400], [0, 400], f64(kk), f64(vv), None, False, "e4m3")
    for n in ("ks", "vs"):
        assert np.array_equal(small[n], want[n])
    for n in "kv":
        small[n][3, :, 16:] = 0
        assert L.same_codes(small[n], want[n], "e4m3")
    for new in (400, 1):
        batch = E.KVBatch(batch.page_table, ints([400]), ints([0, new]))
        got = cache.attend(batch, q[-new:])
        torch.cuda.synchronize()
        ref, tol = L.attend(small, order, [400], [0, new], f64(q[-new:]), dim ** -0.5, 0, "e4m3", "f32")
        assert (np.abs(f64(got) - ref) <= tol).all()


# ---------------------------------------------------------------- norm

NORM = [
    # rows, n, dtype, resid type, post, gate, pre, resid
    (1, 4096, "f32", "f32", False, None, True, True), (3, 1, "f32", "f32", True, "row", True, True),
    (5, 127, "bf16", "bf16", True, "channel", True, True), (2, 5000, "f16", "f32", True, "row", False, True),
    (300, 512, "bf16", "f32", False, "channel", True, True), (4, 14336, "f16", "f16", True, None, True, True),
    (2, 40001, "f32", "f32", True, "channel", True, True), (7, 8192, "bf16", "bf16", True, "row", True, False),
    (1, 20000, "bf16", "f32", True, "row", True, True), (17, 1000, "f32", "f32", False, None, True, False),
]


def norm_inputs(rows, n, dtype, rdt, post, gate, pre, resid, seed=21):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    to = lambda t, d: t.to(DT[d]).cuda()  # noqa: E731
    return dict(x=to(rand(rows, n) * 2, dtype), resid=to(rand(rows, n) * 3, rdt) if resid else None,
                post_w=to(1 + 0.3 * rand(n), dtype) if post else None,
                gate=None if gate is None else to(rand(n) if gate == "channel" else rand(rows, n), dtype),
                pre_w=to(1 + 0.3 * rand(n), dtype) if pre else None)


def norm_check(a, r, out, dtype, rdt, scale, eps):
    h = {k: None if t is None else f64(t) for k, t in a.items()}
    ref_r, ref_out, size = L.norm(h["x"], h["resid"], h["post_w"], h["gate"], scale, h["pre_w"], eps)
    # sums of n squares over at least 256 threads, then a few roundings of each term
    n = a["x"].shape[-1]
    e = (n / 256 + 24) * 2.0 ** -24
    small = 2.0 ** -25 if "f16" in (dtype, rdt) else 0.0
    if r is not None:
        assert (np.abs(f64(r) - ref_r) <= e * size + L.HALF_STEP[rdt] * np.abs(ref_r) + small).all()
    if out is not None:
        unit = np.abs(ref_out) / np.maximum(np.abs(ref_r), 1e-300)
        tol = 3 * e * np.maximum(size * unit, np.abs(ref_out)) + L.HALF_STEP[dtype] * np.abs(ref_out) + small
        assert (np.abs(f64(out) - ref_out) <= tol).all()


@pytest.mark.parametrize("rows,n,dtype,rdt,post,gate,pre,resid", NORM)
def test_norm(rows, n, dtype, rdt, post, gate, pre, resid):
    dev()
    a = norm_inputs(rows, n, dtype, rdt, post, gate, pre, resid)
    ro = None if resid else torch.empty(rows, n, dtype=DT[rdt], device="cuda")
    r, out = E.norm_residual(**a, scale=0.7, eps=1e-5, resid_out=ro)
    norm_check(a, r, out, dtype, rdt, 0.7, 1e-5)
    r2, none = E.norm_residual(**a, scale=0.7, eps=1e-5, with_norm=False, resid_out=ro)
    assert none is None and torch.equal(r, r2)
    none, out2 = E.norm_residual(**a, scale=0.7, eps=1e-5, with_sum=False)
    if resid or rdt == dtype:
        assert none is None and torch.equal(out, out2)


@pytest.mark.parametrize("n", [2, 9, 1030, 8190, 8193, 16386, 30001, 32766, 32769])
@pytest.mark.parametrize("dtype,rdt", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_norm_odd_widths(n, dtype, rdt):
    dev()
    a = norm_inputs(3, n, dtype, rdt, True, "row", True, True, seed=23)
    r, out = E.norm_residual(**a, scale=0.7, eps=1e-5)
    norm_check(a, r, out, dtype, rdt, 0.7, 1e-5)


def test_norm_in_place_strided_unaligned():
    dev()
    for dtype in ("f32", "bf16"):
        for n in (1024, 777, 30000):
            a = norm_inputs(6, n, dtype, dtype, True, "row", True, True, seed=22)
            want = E.norm_residual(**a, scale=-1.5)
            wide = {}
            for k in ("x", "resid", "gate"):
                flat = torch.zeros(6 * (n + 5) + 3, dtype=DT[dtype], device="cuda")
                wide[k] = flat[3:].view(6, n + 5)[:, :n]
                wide[k].copy_(a[k])
            r, out = E.norm_residual(wide["x"], wide["resid"], a["post_w"], wide["gate"], -1.5, a["pre_w"],
                                     resid_out=wide["resid"], out=wide["x"])
            norm_check(a, r, out, dtype, dtype, -1.5, 1e-5)
            r, out = E.norm_residual(a["x"], a["resid"], a["post_w"], a["gate"], -1.5, a["pre_w"],
                                     resid_out=a["resid"], out=a["x"])
            assert torch.equal(r, want[0]) and torch.equal(out, want[1])
    x = torch.randn(5000, device="cuda")
    r, out = E.norm_residual(x, pre_w=torch.ones_like(x))  # one row, no residual
    assert torch.equal(r, x) and math.isclose(float(out.square().mean()), 1.0, rel_tol=1e-4)
    r, out = E.norm_residual(torch.zeros(3, 64, device="cuda"), eps=1e-6)
    assert not out.any() and not r.any()


def test_norm_nan_stays_in_its_row():
    dev()
    a = norm_inputs(4, 600, "f32", "f32", True, None, True, True)
    a["x"][1, 5], a["resid"][2, 9] = float("nan"), float("inf")
    r, out = E.norm_residual(**a)
    assert torch.isnan(out[1]).all() and torch.isnan(r[1]).all()
    assert torch.isnan(out[2, 9]) and torch.isfinite(r[[0, 3]]).all() and torch.isfinite(out[[0, 3]]).all()


# ---------------------------------------------------------------- together

def test_steps_captured_and_replayed():
    """Decode steps of a padded batch, captured once: the graph follows the
    lengths, the page table and the inputs that the program changes between
    replays, with other work in between."""
    d = dev()
    c = Case(31, [5, 63, 64, 0], [1, 1, 1, 1], heads=2, group=4, dim=128, page=32, room=40, garbage=False)
    rope = L.rope_rows(10000.0, c.table.shape[1] * c.page, 128)
    rt = torch.from_numpy(rope).cuda()
    q, k, v, res = c.rand(8), c.rand(2), c.rand(2), torch.randn(4, 8 * 128, device=d)
    w = torch.rand(8 * 128, device=d) + 0.5

    def step():
        qr = c.cache.append(c.batch, k, v, q=q, rope=rt)
        o = c.cache.attend(c.batch, qr)
        return (qr, o) + E.norm_residual(o.view(4, -1), res, post_w=w, pre_w=w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # loads the kernels; appends at the same positions that the first replay uses
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), rope, False, "e4m3")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(6):
        for t, h in ((q, 8), (k, 2), (v, 2)):
            t.copy_(c.rand(h, 2.0 ** (rep % 3)))
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), rope, False, "e4m3")
        c.check_cache()
        live = [0, 1, 2] + ([3] if c.lens[3] > 0 else [])
        c.check_attend(torch.nan_to_num(outs[0]), got=outs[1])
        r, out, _ = L.norm(f64(outs[1]).reshape(4, -1), f64(res), f64(w), None, 1.0, f64(w), 1e-5)
        assert np.abs(f64(outs[2]) - r).max() <= 1e-4 and np.abs(f64(outs[3]) - out).max() <= 1e-4
        eager = c.cache.attend(c.batch, torch.nan_to_num(outs[0]))
        assert torch.equal(eager[live], outs[1][live])
        c.lens = [t + 1 for t in c.lens[:3]] + [0 if rep < 3 else c.lens[3] + 1]
        c.batch.kv_lens.copy_(ints(c.lens))


def test_two_streams_at_once():
    """Two caches on two streams, calls overlapping, results as alone."""
    dev()
    cs = [Case(40 + i, [900 + 50 * i, 300], [1, 1], heads=4, page=64) for i in range(2)]
    qs = [c.rand(8) for c in cs]
    alone = [c.cache.attend(c.batch, q) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [c.cache.attend(c.batch, q, stream=s) for c, q, s in zip(cs, qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
