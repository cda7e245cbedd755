"""Edges of the operators between a decoder layer's matvecs: what a call's
documentation allows beside the usual (test_gpu_layer.py), against the same
64-bit definitions."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
from dynamic_sparsity_approximate_amd import binding as B  # noqa: E402
from _parity import REL_L2_TOL, rel_l2  # noqa: E402
from test_gpu_decoder import Stack  # noqa: E402
from test_gpu_layer import DT, Case, dev, f64, ints, say  # noqa: E402


# ---------------------------------------------------------------- attention: values

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("lens,new,page,room", [([5, 70], [1, 1], 16, 0), ([5, 70], [1, 1], 64, 3000),
                                                ([40, 9], [5, 4], 32, 3000), ([130, 65], [130, 65], 32, 0),
                                                ([130, 65], [130, 65], 64, 0), ([1400], [130], 64, 0)])
def test_attend_infinite_queries(dtype, lens, new, page, room):
    """A row of q with an infinity is NaN whatever sign it gives the scores,
    also where every score would be -inf; its neighbours are as ever."""
    c = Case(71, lens, new, group=4, page=page, dtype=dtype, room=room)
    c.np["k"][..., 0] = L.encode(96.0, "e4m3")  # with a key of this sign, q[0] = -inf makes every score -inf
    c.cache.k.copy_(torch.from_numpy(c.np["k"]))
    q = c.rand(8, 1.5)
    n = len(q)
    hit = {(0, 0): [(0, -np.inf)], (0, 3): [(0, np.inf)], (n - 1, 5): [(0, -np.inf), (9, -np.inf)],
           (n // 2, 6): [(0, np.nan)], (n // 2, 7): [(0, -np.inf), (64, np.nan)]}
    for (row, h), at in hit.items():
        for i, x in at:
            q[row, h, i] = x
    with np.errstate(invalid="ignore"):
        got, _ = c.check_attend(q)
    for row, h in hit:
        assert torch.isnan(got[row, h]).all(), (row, h)
    assert int(torch.isnan(got).any(-1).sum()) == len(hit)


@pytest.mark.parametrize("lens,new,page,window,within", [
    ([200], [1], 16, 50, 1), ([3000], [1], 16, 1500, 1), ([3000, 1510], [5, 3], 16, 1500, 1),
    ([700, 333], [60, 41], 16, 100, 1), ([700, 353], [60, 41], 32, 90, 1), ([4000], [64], 32, 90, 0),
    ([4000], [64], 32, 60, 1)])
@pytest.mark.parametrize("dtype,fmt", [("f32", "e4m3"), ("bf16", "i8")])
def test_attend_scales_in_front_of_the_window(lens, new, page, window, within, dtype, fmt):
    """Pages that the window has left hold anything: here finite scales of 1e30
    and codes that are NaN."""
    c = Case(72, lens, new, group=4, page=page, fmt=fmt, dtype=dtype)
    inside = 0  # pages that nobody sees in a step of 32 or 64 tokens that somebody does
    for s, (t, n) in enumerate(zip(lens, new)):
        first = max(0, t - n + 1 - window)
        old = c.table[s, :first // page]
        inside += first // page > (first & ~(31 if n * 4 <= 32 else 63)) // page
        for name in "kv":
            c.np[name + "s"][old] = 1e30
            c.np[name][old] = 0x7F if fmt == "e4m3" else 0x80
            getattr(c.cache, name).copy_(torch.from_numpy(c.np[name]))
            getattr(c.cache, name + "_scale").copy_(torch.from_numpy(c.np[name + "s"]))
    assert bool(inside) == bool(within)
    got, _ = c.check_attend(c.rand(8, 1.5), window=window)
    assert bool((got != 0).any(-1).all())


# ---------------------------------------------------------------- sizes of one launch and more

def test_norm_of_more_rows_than_one_launch_has():
    """2^26 + 5 narrow rows, which one launch (2^32 threads) could not have:
    strided rows, a gate of its own for each, the first and last rows and those
    around every border of a launch's rows against the definition, all of them
    against torch in 32 bits."""
    dev()
    rows, n = (1 << 26) + 5, 4
    g = torch.Generator(device="cuda").manual_seed(91)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    x, resid, gate = rand(rows, n + 2)[:, :n], rand(rows, n), rand(rows, n + 1)[:, :n]
    post, pre = 1 + 0.25 * rand(n), 1 + 0.25 * rand(n)
    out = torch.full((rows, n + 2), 7.0, dtype=torch.float16, device="cuda")
    r, h = E.norm_residual(x, resid.float(), post_w=post, gate=gate, scale=0.5, pre_w=pre, out=out[:, :n])
    torch.cuda.synchronize()
    assert bool((out[:, n:] == 7.0).all())
    step = ((1 << 32) - 1) // 1024
    at = torch.tensor(sorted({i + d for i in range(0, rows, step) for d in (-1, 0) if i + d >= 0} | {rows - 1}), device="cuda")
    ref_r, ref, size = L.norm(f64(x[at]), f64(resid[at]), f64(post), f64(gate[at]), 0.5, f64(pre), 1e-5)
    # a sum of 4 squares, a mean, a root, a quotient and three products: within 2^-20 of their values
    err = 2.0 ** -20 * size
    assert (np.abs(f64(r[at]) - ref_r) <= err).all()
    rms = np.sqrt((ref_r * ref_r).mean(-1, keepdims=True) + 1e-5)
    slack = (err + np.sqrt((err * err).mean(-1, keepdims=True)) * np.abs(ref_r) / rms) / rms * f64(pre)
    assert (np.abs(f64(h[at]) - ref) <= slack + (2.0 ** -20 + 2.0 ** -11) * np.abs(ref) + 2.0 ** -25).all()
    for i in range(0, rows, 1 << 23):
        j = slice(i, i + (1 << 23))
        t = x[j].float()
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-5) * post.float()
        t = resid[j].float() + 0.5 * gate[j].float() * t
        # both sides round each of at most three terms of magnitude up to 2^5 a few times
        assert float((r[j] - t).abs().max()) <= 2.0 ** -14
    torch.cuda.empty_cache()


def test_append_of_more_pages_than_one_launch_has():
    """2^24 tokens of 8 heads in pages of 16: (pages, heads, keys or values) and
    the queries behind them need more blocks than one launch (2^32 threads) has.
    Pages and queries here and there against the definition, every scale against torch."""
    d = dev()
    T, H, D, rot = 16, 8, 64, 8
    tokens, pages = 1 << 24, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(92)
    part = torch.randn(1 << 20, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.empty(tokens, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for i in range(16):
        k[i << 20:(i + 1) << 20] = part * (1.0 + 0.25 * i)
        v[i << 20:(i + 1) << 20] = part.flip(0) * 2.0 ** i
    del part
    q = k.clone()
    cache = E.KVCache(pages, H, D, page_tokens=T)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    batch = E.KVBatch(table, torch.tensor([tokens], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    rope = E.rope_table(10000.0, tokens, rot, d)
    got = cache.append(batch, k, v, q=q, rope=rope, q_out=q)
    torch.cuda.synchronize()
    assert got is q
    # the scales of values, which are not rotated: least powers of two (of bf16 sizes, exact in fp32)
    for i in range(0, pages, 1 << 16):
        top = v[i * T:(i + (1 << 16)) * T].view(1 << 16, T, H, D).abs().amax((1, 3)).float()
        e = torch.frexp(top / 448.0)[1]
        e = torch.where(top <= 448.0 * torch.ldexp(torch.ones_like(top), e - 1), e - 1, e)
        want = torch.ldexp(torch.ones_like(top), e)
        assert torch.equal(cache.v_scale.flip(0)[i:i + (1 << 16)], want)
    for pg in (0, 1, 77777, pages // 2 - 1, pages // 2, pages - 2, pages - 1):
        at = slice(pg * T, (pg + 1) * T)
        cs = rope[at].cpu().numpy()
        want = {n: np.zeros((1, H, T, D), np.uint8) for n in "kv"}
        want.update({n: np.zeros((1, H), np.float32) for n in ("ks", "vs")})
        rows = [(r, 0, r) for r in range(T)]
        L.append(want, np.array([[0]]), [T], [0, T], f64(k[at]), f64(v[at]), cs, False, "e4m3")
        mine = pages - 1 - pg
        for name, t, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
            assert np.array_equal(s[mine].cpu().numpy(), want[name + "s"][0]), (pg, name)
            assert L.same_codes(t[mine].cpu().numpy(), want[name][0], "e4m3"), (pg, name)
        for r, _, p in rows:
            x = f64(k[pg * T + r])
            ref = L.rotate(x, cs[p], False)
            assert (np.abs(f64(got[pg * T + r]) - ref) <= 2.0 ** -22 * np.abs(x).max() + 2.0 ** -8 * np.abs(ref)).all()
    del k, v, q, got, cache, rope
    torch.cuda.empty_cache()


def test_rope_table_of_more_entries_than_one_launch_has():
    """2^26 + 9 rows of 64 pairs: rows at the borders of a launch's 2^31 entries."""
    d = dev()
    rows, rot = (1 << 26) + 9, 128
    table = torch.full((rows, rot // 2, 2), 7.0, device=d)
    E.effort_rope_table(1e6, rows, rot, table, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert not any(bool((table[i:i + (1 << 22)] == 7.0).any()) for i in range(0, rows, 1 << 22))
    at = np.array([0, 1, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, (1 << 26) - 1, 1 << 26, rows - 1])
    ang = at[:, None].astype(np.float64) * 1e6 ** (-np.arange(0, rot, 2) / rot)
    got = f64(table[torch.from_numpy(at).to(d)])
    # the angle, up to 2^26, is off by three roundings in double, the result by one in fp32
    bound = 3 * 2.0 ** -53 * 2.0 ** 26 + 2.0 ** -24
    assert np.abs(got - np.stack([np.cos(ang), np.sin(ang)], -1)).max() <= bound
    del table
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype,inter,rot", [("f32", False, 128), ("f32", True, 64), ("bf16", False, 24)])
def test_append_keys_that_grow_beyond_fp32(fmt, dtype, inter, rot):
    """Rotation makes an element up to 2^0.5 times larger: beyond the largest
    fp32 number its code is still the nearest one."""
    c = Case(75, [40, 33], [40, 9], fmt=fmt, dtype=dtype)
    k, v = c.rand(2), c.rand(2)
    big = torch.finfo(DT[dtype]).max
    k[:20] = big * torch.sign(k[:20])
    k[20:40] *= 5e37
    k[41:44] = big * torch.sign(k[41:44])
    k[44:] *= 1e-42  # their scale is a far larger one's, or their codes 0
    rope = L.rope_rows(10000.0, c.table.shape[1] * c.page, rot)
    c.cache.append(c.batch, k, v, rope=torch.from_numpy(rope).cuda(), interleaved=inter)
    L.append(c.np, c.table, c.lens, c.starts, f64(k), f64(v), rope, inter, fmt)
    assert np.isfinite(c.np["ks"][c.table[:, 0]]).all()
    c.check_cache()


def test_append_with_a_table_above_one():
    """Cosines and sines of another program, times 3: keys that end beyond what
    any scale takes have the largest code, none is a NaN."""
    c = Case(76, [40], [40])
    k, v = c.rand(2), c.rand(2)
    k[3] = 3.4e38 * torch.sign(k[3])
    rope = 3 * L.rope_rows(10000.0, c.table.shape[1] * c.page, 128)
    c.cache.append(c.batch, k, v, rope=torch.from_numpy(rope).cuda())
    pg = c.table[0, 0]
    assert bool((c.cache.k_scale[pg] == 2.0 ** 120).all())
    codes = c.cache.k[pg].cpu().numpy()
    y = np.stack([L.rotate(f64(k[t]), rope[t], False) for t in range(32)])
    want = L.encode(np.clip(y.transpose(1, 0, 2) / 2.0 ** 120, -448, 448), "e4m3")
    assert L.same_codes(codes, want, "e4m3") and int((L.decode(codes, "e4m3") == 448).sum()) > 0


# ---------------------------------------------------------------- attention: shared out and joined

def parts_of(c, window, rt):
    """The (block, slot) that the split must leave parts in: blocks take the
    items' 128-token chunks evenly, in order of sequence, head, row tile."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    items, cap = [], c.table.shape[1] * c.page
    for s, t in enumerate(c.lens):
        n = c.starts[s + 1] - c.starts[s]
        first, end = max(0, t - n + 1 - window) if window else 0, min(t, cap)
        if n > 0 and end > first:
            items += [-(-(end - first // 32 * 32) // 128)] * (c.heads * -(-n * c.group // (16 * rt)))
    total = sum(items)
    assert total > blocks, "every block must have several chunks"
    edges = [total * b // blocks for b in range(blocks + 1)]
    want, b, at = set(), 0, 0
    whole = 0
    for n in items:
        while edges[b + 1] <= at:
            b += 1
        i = b
        whole += edges[i + 1] >= at + n
        while edges[i + 1] < at + n or edges[i] > at:
            want.add((i, 1 if edges[i] <= at else 0))
            if edges[i + 1] >= at + n:
                break
            i += 1
        at += n
    return want, whole, blocks


def split_call(c, q, window):
    """attend with a workspace of the test's own: (out, (block, slot) of the
    parts found in it, row tiles)."""
    need = E.effort_kv_workspace_bytes(c.cache.desc, len(c.lens), len(q), c.heads * c.group)
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    tile = blocks * 2 * 16 * (c.dim + 2) * 4
    assert need in (tile, 2 * tile), "not a call that is split over blocks"
    ws = torch.full((need // 4,), 0x7FC0BEEF, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    stride = q.shape[1] * c.dim
    E.effort_kv_attention(c.cache.desc, c.batch.desc(len(q)), {"f32": 0, "f16": 1, "bf16": 2}[c.dtype], q, stride,
                          q.shape[1], c.dim ** -0.5, window, out, stride, ws, need,
                          stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    first = ws.view(blocks, 2, -1)[:, :, 0].cpu().numpy()
    return out, {(int(b), int(s)) for b, s in zip(*np.nonzero(first != 0x7FC0BEEF))}, need // tile


def wide(c, tokens):
    """The same batch in a page table with room for `tokens`."""
    more = -(-tokens // c.page) - c.table.shape[1]
    if more > 0:
        c.table = np.concatenate([c.table, np.full((len(c.lens), more), -7)], 1)
        c.batch = E.KVBatch(torch.from_numpy(c.table.astype(np.int32)).cuda(), ints(c.lens), ints(c.starts))
    return c


LONG = [8192, 1000, 0, 7001, 129, 4097, 6000, 1, 2500, 3333, 5120, 1537, 7777, 640, 4500, 2999]
SPLIT = [
    # lens, new, heads, group, dim, page, fmt, dtype, window, four rows a joining block
    (LONG, [1] * 16, 4, 4, 64, 64, "i8", "f32", 0, True),
    (LONG, [1] * 16, 4, 8, 128, 128, "i8", "bf16", 0, True),
    (LONG, [1] * 16, 8, 2, 64, 16, "e4m3", "f16", 1500, True),
    (LONG, [7, 5, 0, 8, 8, 1, 3, 1, 6, 8, 2, 8, 0, 8, 5, 8], 4, 4, 64, 32, "i8", "bf16", 0, True),
    (LONG, [7, 5, 0, 8, 8, 1, 3, 1, 6, 8, 2, 8, 0, 8, 5, 8], 4, 4, 128, 16, "i8", "f32", 2000, True),
    ([40000], [1], 3, 4, 64, 64, "i8", "f32", 0, False),
    ([9000, 31000], [7, 5], 2, 4, 128, 128, "i8", "f16", 0, False),
    ([9000, 31000, 2000, 4000], [60, 1, 1, 2], 2, 1, 64, 64, "i8", "f32", 0, False),
]


@pytest.mark.parametrize("lens,new,heads,group,dim,page,fmt,dtype,window,four", SPLIT)
def test_attend_several_chunks_a_block(lens, new, heads, group, dim, page, fmt, dtype, window, four):
    """More chunks than blocks: blocks that go on from one item, and one
    sequence, to the next, that have items whole, that leave both of their parts."""
    c = Case(73, lens, new, heads=heads, group=group, dim=dim, page=page, fmt=fmt, dtype=dtype)
    q = c.rand(heads * group, 1.5)
    out, parts, rt = split_call(c, q, window)
    want, whole, blocks = parts_of(c, window, rt)
    assert parts == want
    both = any((b, 1) in parts for b, s in parts if s == 0)
    assert four == (16 * len(lens) * heads > blocks) and (not four or (both and whole))
    _, worst = c.check_attend(q, window=window, got=out)
    say("%d parts, %d items whole: %.3f of the bound" % (len(parts), whole, worst))
    assert torch.equal(out, c.cache.attend(c.batch, q, window=window))


def test_attend_many_sequences_in_a_wide_table():
    """700 and 1024 sequences share out their chunks: entries of the plan hold
    three and four of them, many without tokens."""
    for seqs, window, dtype in ((700, 0, "f16"), (1024, 1400, "f32")):
        rng = np.random.default_rng(seqs)
        lens = [int(x) for x in rng.integers(0, 60, seqs)]
        for s in (0, 255, 300, seqs - 1):
            lens[s] = 2000 + s
        new = [min(t, int(x)) for t, x in zip(lens, rng.integers(0, 3, seqs))]
        new[300] = 5
        c = wide(Case(seqs, lens, new, heads=2, group=2, dim=64, page=16, fmt="i8", dtype=dtype), 4000)
        q = c.rand(4)
        out, parts, rt = split_call(c, q, window)
        assert parts == parts_of(c, window, rt)[0] and rt == 1
        c.check_attend(q, window=window, got=out)


@pytest.mark.parametrize("lens,new,page,dtype,window", [
    ([3000, 2500, 1, 700], [512, 1, 1, 1], 64, "bf16", 0), ([3000, 2500, 1, 700], [512, 1, 1, 1], 16, "f32", 0),
    ([900] + [1200 + 37 * i for i in range(15)], [150] + [1] * 15, 32, "f16", 0),
    ([3000, 2500, 1, 700], [512, 1, 1, 3], 32, "f32", 600)])
def test_attend_a_prompt_beside_single_tokens(lens, new, page, dtype, window):
    c = Case(74, lens, new, group=4, dim=64, page=page, fmt="i8", dtype=dtype)
    c.check_attend(c.rand(8, 1.5), window=window)


@pytest.mark.parametrize("lens,new,heads", [([30000], [1], 3), ([9000, 7000, 8000], [2, 1, 4], 4)])
def test_attend_holes_and_poison_among_the_parts(lens, new, heads):
    """Parts that see nothing (absent pages), and parts that are NaN, are joined
    with others: only the poisoned heads of rows that see the page are NaN."""
    for name in ("ks", "vs"):
        c = Case(77, lens, new, heads=heads, group=4, dim=64, page=32, fmt="i8")
        c.table[0, 60:150] = -1
        c.table[-1, 3:9] = c.pages
        c.np[name][c.table[0, 200], 1] = np.inf
        c.np[name][c.table[-1, 1], 0] = np.nan
        getattr(c.cache, name[0] + "_scale").copy_(torch.from_numpy(c.np[name]))
        c.batch.page_table.copy_(torch.from_numpy(c.table.astype(np.int32)))
        q = c.rand(4 * heads, 1.5)
        out, parts, rt = split_call(c, q, 0)
        assert parts == parts_of(c, 0, rt)[0]
        c.check_attend(q, got=out)
        nan = torch.isnan(out).any(-1)
        assert nan[:new[0], 4:8].all() and nan[-new[-1]:, :4].all() and int(nan.sum()) == 4 * (new[0] + new[-1])


# ---------------------------------------------------------------- attention: streams and graphs

def overlapping():
    """Two calls that leave parts in their workspaces, split and prompt, with their results alone."""
    cs = [Case(80, LONG, [1] * 16, heads=4, group=4, dim=64, page=64, fmt="i8"),
          Case(81, LONG[::-1], [1] * 16, heads=4, group=4, dim=64, page=64, fmt="i8"),
          Case(82, [3000], [100], heads=2, group=4, dim=64, page=64, fmt="i8"),
          Case(83, [2900], [100], heads=2, group=4, dim=64, page=64, fmt="i8")]
    qs = [c.rand(c.heads * c.group) for c in cs]
    for c, q in zip(cs, qs):
        assert E.effort_kv_workspace_bytes(c.cache.desc, len(c.lens), len(q), c.heads * c.group) > 0
    alone = [c.check_attend(q)[0] for c, q in zip(cs, qs)]
    return [[(c, q, a) for c, q, a in zip(cs[i:i + 2], qs[i:i + 2], alone[i:i + 2])] for i in (0, 2)]


def test_workspaces_of_two_streams():
    for pair in overlapping():
        streams = [torch.cuda.Stream() for _ in pair]
        outs = []
        for _ in range(20):
            outs += [(c.cache.attend(c.batch, q, stream=s), a) for (c, q, a), s in zip(pair, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, a) for o, a in outs)


def test_workspaces_of_two_graphs():
    for pair in overlapping():
        graphs = []
        for c, q, a in pair:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = [c.cache.attend(c.batch, q) for _ in range(5)]
            graphs.append((g, outs, a))
        streams = [torch.cuda.Stream() for _ in pair]
        for _ in range(4):
            for _, outs, _ in graphs:
                for o in outs:
                    o.fill_(float("nan"))
            torch.cuda.synchronize()
            for (g, _, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for _, outs, a in graphs:
                assert all(torch.equal(o, a) for o in outs)


@pytest.mark.parametrize("new,window,heads", [([1] * 4, 0, 3), ([1] * 4, 2500, 8), ([8] * 4, 0, 3), ([20] * 4, 0, 2)])
def test_replays_follow_the_lengths(new, window, heads):
    """One captured call of a wide table, split and joined, or a prompt's: its
    chunks are fewer than the blocks, then more, then fewer."""
    c = Case(84, [8192] * 4, new, heads=heads, group=4, dim=64, page=64, fmt="i8", garbage=False)
    q = c.rand(4 * heads)
    g = torch.cuda.CUDAGraph()
    c.cache.attend(c.batch, q, window=window)  # loads the kernels
    with torch.cuda.graph(g):
        out = c.cache.attend(c.batch, q, window=window)
    for lens in ([40, 100, 0, 700], [8192, 8100, 7000, 5000], [1, 8192, 8192, 8192], [300, 41, 8000, 2], [8192] * 4):
        c.lens = lens
        c.batch.kv_lens.copy_(ints(lens))
        q.copy_(c.rand(4 * heads, 1.5))
        out.fill_(float("nan"))
        g.replay()
        c.check_attend(q, window=window, got=out)
        assert torch.equal(out, c.cache.attend(c.batch, q, window=window))


# ---------------------------------------------------------------- whole layers

@pytest.mark.parametrize("rows", [3, 9])
def test_rows_of_nobody_stay_out_of_a_step(rows):
    """What the rows behind the last sequence hold, NaN and infinities included,
    changes nothing of the others and of the caches."""
    runs = []
    for fill in (0.0, float("nan"), float("inf")):
        s = Stack([3, 7], [1, 1], rows, seed=5)
        for _ in range(2):
            s.next_x()
            s.x[2:] = fill
            s.step.enqueue(0.4)
            s.advance(1)
        torch.cuda.synchronize()
        stored = [(L.decode(t.cpu().numpy(), "e4m3"), f64(scale)) for c in s.step.caches
                  for t, scale in ((c.k, c.k_scale), (c.v, c.v_scale))]
        runs.append((f64(s.step.logits[:2]), stored))
    for logits, stored in runs[1:]:
        assert rel_l2(logits, runs[0][0]) <= REL_L2_TOL
        for (codes, scale), (codes0, scale0) in zip(stored, runs[0][1]):
            assert np.array_equal(scale == 0, scale0 == 0)
            # sums in another order may move a value by a step of its code, 2^-3 of it
            x, x0 = (c * s[:, :, None, None] for c, s in ((codes, scale), (codes0, scale0)))
            assert rel_l2(x, x0) <= 2.0 ** -3


# ---------------------------------------------------------------- attention: what 16-bit rows keep

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new,page,room", [([333, 1000, 17], [1, 1, 1], 64, 0), ([333, 1000, 17], [1, 1, 1], 16, 3000),
                                                ([500, 77], [5, 8], 32, 0), ([9000, 4000], [5, 8], 32, 0)])
def test_attend_keeps_the_weights_of_16_bit_rows(dtype, lens, new, page, room):
    """Up to 32 rows a sequence: what fp32 rows are held to, and one rounding of
    the output (small scores, which add little to that)."""
    c = Case(78, lens, new, group=4, page=page, dtype=dtype, room=room)
    q = c.rand(8, 0.01)
    got = f64(c.cache.attend(c.batch, q))
    ref, tol = L.attend(c.np, c.table, c.lens, c.starts, f64(q), c.dim ** -0.5, 0, "e4m3", "f32")
    # rounding moves a result by half a step of what is rounded, itself within tol of ref
    tol = tol + L.HALF_STEP[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
    worst = float((np.abs(got - ref) / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("rows", [1, 3])
def test_a_step_on_another_device_than_the_current_one(rows, monkeypatch):
    """With one device at hand: when torch says that another one is current, every
    call of the step is made with the tensors' own device made current."""
    s = Stack([3, 15, 30][:rows], [1] * rows, rows, seed=6)
    s.next_x()
    current = [1]

    class Device(torch.cuda.device):
        def __enter__(self):
            self.was, current[0] = current[0], self.idx
            return super().__enter__()

        def __exit__(self, *a):
            current[0] = self.was
            return super().__exit__(*a)

    calls = []
    for name in ("effort_matvec", "effort_matvec_multi", "effort_matvec_batched", "effort_silu_mul", "effort_kv_append",
                 "effort_kv_attention", "effort_norm_residual"):
        def call(*a, of=getattr(B, name), name=name, **kw):
            calls.append((name, current[0] == s.x.device.index))
            return of(*a, **kw)
        monkeypatch.setattr(B, name, call)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    s.step.enqueue(0.25)
    monkeypatch.undo()
    # two layers and the head; q k v, and w1 w3, are one call each for a single row
    assert len(calls) == (2 * 9 + 2 if rows == 1 else 2 * 12 + 2)
    assert all(ok for _, ok in calls), [n for n, ok in calls if not ok]
    s.check(0.25)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [-97, 105])
@pytest.mark.parametrize("new,page,room", [([1, 1], 16, 0), ([1, 3], 64, 3000), ([90, 40], 16, 0), ([90, 40], 64, 0)])
def test_attend_tiny_and_huge_value_scales(dtype, exponent, new, page, room):
    """Scales of 2^-100 to 2^-94, and of 2^102 to 2^108."""
    c = Case(79, [300, 77], new, group=4, page=page, dtype=dtype, room=room, garbage=False, spread=3)
    c.np["ks"][:] = 2.0 ** -6
    c.np["vs"] = (c.np["vs"].astype(np.float64) * 2.0 ** (6 + exponent)).astype(np.float32)
    c.cache.k_scale.copy_(torch.from_numpy(c.np["ks"]))
    c.cache.v_scale.copy_(torch.from_numpy(c.np["vs"]))
    c.check_attend(c.rand(8, 1.5))
