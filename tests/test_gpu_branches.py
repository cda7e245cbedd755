"""Several continuations of a sequence over the paged cache, against their 64-bit
definitions (tests/_branches.py): norms of heads, trees of new tokens, pages that
sequences share, accepted paths, beam search's selection."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _branches as R  # noqa: E402
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
from test_gpu_layer import DT, FMT, Case, dev, f64, ints, say  # noqa: E402


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Tree(Case):
    """A Case whose new tokens are trees (parents: a list for all rows, or None)."""

    def __init__(self, seed, lens, new, parents="random", **kw):
        super().__init__(seed, lens, new, **kw)
        if parents == "random":
            parents = [p for n in new for p in R.random_tree(self.rng, n)]
        self.parents = parents
        if parents is not None:
            self.batch = E.KVBatch(self.batch.page_table, self.batch.kv_lens, self.batch.q_starts, parents=ints(parents))

    def check_tree(self, q, window=0, scale=None):
        sc = self.dim ** -0.5 if scale is None else scale
        got = self.cache.attend(self.batch, q, window=window, scale=scale)
        torch.cuda.synchronize()
        ref, tol = R.attend(self.np, self.table, self.lens, self.starts, f64(q), sc, window, self.fmt, self.dtype,
                            self.parents)
        g = f64(got)
        rows = [r[0] for r in R.rows_of(self.lens, self.starts, len(q), self.parents)]
        assert np.array_equal(np.isnan(g[rows]), np.isnan(ref[rows]))
        ok = ~np.isnan(ref[rows])
        d = np.abs(g[rows] - ref[rows])
        worst = float((d[ok] / (tol[rows][ok] + 1e-300)).max()) if ok.any() else 0.0
        say("worst", worst)
        assert (d[ok] <= tol[rows][ok]).all(), worst
        return got


# ---------------------------------------------------------------- append

APPEND = [
    # fmt, dtype, dim, page, rot, interleaved, norms, tree
    ("e4m3", "f32", 128, 64, 128, False, "qk", True), ("e4m3", "f32", 128, 32, 64, True, "q", False),
    ("e4m3", "bf16", 64, 16, 64, False, "k", True), ("e4m3", "f16", 64, 128, 24, True, "heads", False),
    ("i8", "f32", 128, 16, 128, True, "heads", True), ("i8", "f16", 64, 32, 8, False, "qk", True),
    ("i8", "bf16", 128, 128, 128, False, "", True), ("e4m3", "bf16", 128, 64, 0, False, "qk", True),
    ("e4m3", "f32", 64, 64, 0, False, "qk", False), ("i8", "bf16", 64, 16, 64, True, "k", False),
]


@pytest.mark.parametrize("fmt,dtype,dim,page,rot,inter,norms,tree", APPEND)
def test_append_with_norms_and_trees(fmt, dtype, dim, page, rot, inter, norms, tree):
    # none, one, a page's end, several pages, one that starts in a page's middle, all of a sequence
    lens = [40, 1, page, 3 * page + 5, 2 * page + 7, 0, 21]
    new = [0, 1, 1, 2 * page + 9, 3, 0, 21]
    c = Tree(3, lens, new, dim=dim, page=page, fmt=fmt, dtype=dtype, parents="random" if tree else None)
    k, v, q = c.rand(2, 3.0), c.rand(2), c.rand(4, 40.0)
    weights = lambda n: (cuda(c.rng.random((n, dim) if norms == "heads" else dim) + 0.5)).to(DT[dtype])  # noqa: E731
    qn = weights(4) if norms in ("q", "qk", "heads") else None
    kn = weights(2) if norms in ("k", "qk", "heads") else None
    rope = L.rope_rows(10000.0, c.table.shape[1] * page, rot) if rot else None
    got = c.cache.append(c.batch, k, v, q=q, rope=None if rope is None else cuda(rope), interleaved=inter, q_norm=qn,
                         k_norm=kn, eps=1e-6)
    f = lambda t: None if t is None else f64(t)  # noqa: E731
    ref, size = R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), rope, inter, fmt, c.parents, f(qn), f(kn),
                         1e-6)
    c.check_cache()
    # a normed element is rounded once (half of 2^-23 of it, in either term), a product and the sum are; then the result
    assert (np.abs(f64(got) - ref) <= 2.0 ** -22 * size + L.HALF_STEP[dtype] * np.abs(ref) + 2.0 ** -25).all()


def test_append_ex_strided_rows_and_q_alone_or_absent():
    lens, new = [77, 30], [13, 30]
    c = Tree(5, lens, new, page=16, dtype="bf16")
    n, h = sum(new), 2
    fused = c.rand(9, rows=n)  # rows of q, k, v and one head of nobody
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:8]
    w = cuda(c.rng.random(128) + 0.5).bfloat16()
    rope = L.rope_rows(10000.0, c.table.shape[1] * 16, 128)
    out = torch.full((n, 5, 128), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:]
    got = c.cache.append(c.batch, k, v, q=q, rope=cuda(rope), q_norm=w, k_norm=w, q_out=out)
    assert got.data_ptr() == out.data_ptr()
    ref, size = R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), rope, False, "e4m3", c.parents, f64(w),
                         f64(w), 1e-5)
    c.check_cache()
    assert (np.abs(f64(got) - ref) <= 2.0 ** -22 * size + 2.0 ** -8 * np.abs(ref)).all()
    # misaligned elements, keys alone: the same tokens once more
    base = torch.empty(n * 2 * h * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:]
    kv = base.view(n, 2 * h, 128)
    kv.copy_(fused[:, 4:8])
    assert c.cache.append(c.batch, kv[:, :h], kv[:, h:], rope=cuda(rope), k_norm=w) is None
    R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), rope, False, "e4m3", c.parents, f64(w), f64(w), 1e-5)
    c.check_cache()


def test_head_norms_of_unusual_rows():
    """The largest and smallest numbers have norms; a NaN, an infinity, or zeros without eps poison their page and head."""
    lens, new = [6, 3, 3, 3], [6, 3, 3, 3]
    c = Tree(6, lens, new, page=16, parents=None, group=1)
    k, v, q = c.rand(2), c.rand(2), c.rand(2)
    k[0] = 3e38
    k[1] = -1e-38
    k[2, 0, 1:] = 0.0
    q[0], q[1] = 3e38, 1e-38
    k[6, 0, 5] = math.nan
    k[9, 1, 5] = math.inf
    k[12, 0] = 0.0
    q[6, 1, 0] = math.inf
    q[9, 1] = 0.0
    w = cuda(c.rng.random(128).astype(np.float32) + 0.5)
    rope = L.rope_rows(10000.0, c.table.shape[1] * 16, 128)
    got = c.cache.append(c.batch, k, v, q=q, rope=cuda(rope), q_norm=w, k_norm=w, eps=0.0)
    ref, size = R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), rope, False, "e4m3", None, f64(w), f64(w),
                         0.0)
    c.check_cache()
    bad = np.isnan(c.np["ks"])
    page = lambda s: c.table[s, 0]  # noqa: E731
    assert bad[page(1), 0] and bad[page(2), 1] and bad[page(3), 0] and not bad[page(0)].any() and not bad[page(1), 1]
    g = f64(got)
    assert np.isnan(g[6, 1]).sum() == 2 and np.isnan(g[9, 1]).all()  # inf / inf, and its partner of the rotation
    ok = ~np.isnan(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    assert (np.abs(g - ref)[ok] <= 2.0 ** -22 * size[ok] + 2.0 ** -24 * np.abs(ref)[ok]).all()


def test_what_is_no_tree_is_left_alone():
    """More tokens than a tree has, or than the sequence; parents that are none; pages that are absent."""
    lens, new = [600, 5, 40, 50], [513, 9, 8, 20]
    wild = [7, -5, 0, 2 ** 31 - 1, 4, -2 ** 31, 2, 9]
    par = [i - 1 for i in range(513)] + [i - 1 for i in range(9)] + wild + [i - 1 for i in range(20)]
    c = Tree(7, lens, new, page=16, parents=par, dim=64)
    c.table[3, 2] = c.pages  # of tokens 32 .. 47
    c.batch.page_table.copy_(ints(c.table.tolist()))
    k, v, q = c.rand(2), c.rand(2), c.rand(4)
    rope = L.rope_rows(10000.0, c.table.shape[1] * 16, 64)
    out = torch.full_like(q, 5.0)
    got = c.cache.append(c.batch, k, v, q=q, rope=cuda(rope), q_out=out)
    ref, _ = R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), rope, False, "e4m3", par)
    c.check_cache()
    g = f64(got)
    assert (g[:522] == 5.0).all() and np.isnan(ref[:522]).all() and not np.isnan(ref[522:]).any()
    assert np.abs(g[522:] - ref[522:]).max() <= 2.0 ** -20
    a = c.check_tree(got)
    assert (f64(a)[:522] == 0.0).all()
    far = Tree(7, lens, new, page=16, parents=par, dim=64, room=1100, group=4)
    assert (f64(far.check_tree(far.rand(8)))[:522] == 0.0).all()


# ---------------------------------------------------------------- attention of trees

TREES = [
    # heads, group, dim, page, fmt, dtype, lens, new, window: rows of up to 16, 32, 64, 128 and more
    (2, 2, 128, 16, "e4m3", "f32", [5, 70, 300], [5, 6, 7], 0),
    (2, 4, 64, 32, "i8", "bf16", [9, 200, 64], [8, 8, 8], 0),
    (1, 1, 128, 64, "e4m3", "f16", [130], [15], 20),
    (2, 4, 128, 64, "e4m3", "f32", [410, 64, 15], [15, 15, 15], 0),
    (2, 4, 128, 16, "i8", "f32", [333, 90], [16, 13], 50),
    (2, 3, 64, 16, "e4m3", "f16", [500, 26, 129, 64], [25, 25, 20, 1], 100),
    (1, 8, 128, 128, "e4m3", "bf16", [1000, 64], [64, 64], 0),
    (2, 4, 128, 64, "i8", "bf16", [700, 33], [32, 33], 0),
    (1, 4, 64, 64, "i8", "f16", [640, 512], [300, 512], 0),
    (1, 2, 128, 32, "e4m3", "bf16", [900], [130], 64),
]


@pytest.mark.parametrize("room", [0, 1100])  # tables of more than 1024 tokens are shared out in another way
@pytest.mark.parametrize("heads,group,dim,page,fmt,dtype,lens,new,window", TREES)
def test_tree_attention(heads, group, dim, page, fmt, dtype, lens, new, window, room):
    c = Tree(11, lens, new, heads=heads, group=group, dim=dim, page=page, fmt=fmt, dtype=dtype, spread=3, room=room)
    c.check_tree(c.rand(heads * group, 1.5), window=window)


@pytest.mark.parametrize("room", [0, 1100])
@pytest.mark.parametrize("new,group,dtype", [(12, 1, "f32"), (20, 3, "bf16"), (40, 4, "f16")])
def test_chains_forests_and_lines(new, group, dtype, room):
    """A chain is causal attention; tokens of no parent see themselves alone of the new ones."""
    lens = [new + 100, new, new + 3]
    chain = Tree(12, lens, [new] * 3, group=group, dtype=dtype, parents=[i - 1 for i in range(new)] * 3,
                 room=room)
    q = chain.rand(2 * group)
    chain.check_attend(q, got=chain.check_tree(q))
    Tree(12, lens, [new] * 3, group=group, dtype=dtype, parents=[-1] * 3 * new, room=room).check_tree(q)
    comb = [(i - 2 if i % 2 == 0 else i - 1) if i else -1 for i in range(new)]
    Tree(12, lens, [new] * 3, group=group, dtype=dtype, parents=comb * 3, room=room).check_tree(q, window=5)
    Tree(12, lens, [new] * 3, group=group, dtype=dtype, parents=comb * 3, room=room).check_tree(q, window=1000)


@pytest.mark.parametrize("room", [0, 1100])
@pytest.mark.parametrize("new,group", [(5, 2), (20, 4), (40, 4)])
def test_poison_reaches_only_rows_that_see_it(new, group, room):
    """Of a page of drafted tokens, and of a committed one behind a window."""
    lens = [64 + new, 200]
    c = Tree(13, lens, [new, new], group=group, page=16, room=room)
    for page, head in ((c.table[0, (64 + new - 1) // 16], 0), (c.table[1, (200 - new - 30) // 16], 1)):
        c.np["ks"][page, head] = np.nan
        c.cache.k_scale[int(page), head] = math.nan
    q = c.rand(2 * group)
    got = f64(c.check_tree(q))
    assert np.isnan(got).any() and not np.isnan(got[:, group:][:new]).any()
    c.check_tree(q, window=25)


def test_many_sequences_and_blocks_of_several_items():
    """More sequences than the plan has entries; blocks that take parts of several items; lengths of all kinds."""
    rng = np.random.default_rng(14)
    for seqs, new, group, page, room in ((300, 3, 2, 16, 0), (300, 12, 4, 16, 1100), (40, 17, 4, 64, 1100),
                                         (70, 20, 3, 16, 1100), (70, 20, 3, 16, 0)):
        lens = [int(n + rng.integers(0, 300)) for n in [new] * seqs]
        lens[3] = 0
        count = [new] * seqs
        count[3], count[5] = 0, 1
        c = Tree(14, lens, count, heads=1, group=group, page=page, dtype="bf16", room=room)
        c.check_tree(c.rand(group))


@pytest.mark.parametrize("room", [0, 1100])
def test_rows_behind_the_last_sequence_stay_and_scales_are_signed(room):
    c = Tree(15, [90, 50], [20, 20], group=4, room=room, parents=R.random_tree(np.random.default_rng(1), 20) * 2 + [0] * 9)
    q = c.rand(8, rows=49)
    out = torch.full_like(q, 3.0)
    c.cache.attend(c.batch, q, out=out)
    assert (out[40:] == 3.0).all() and not (out[:40] == 3.0).any()
    c.check_tree(q[:40], scale=-0.3)
    c.check_tree(q[:40], scale=0.0)


@pytest.mark.parametrize("lens,new,cols", [([1300, 1200, 40], [20, 20, 20], 70), ([1130, 1119], [30, 12], 70),
                                           ([1300, 1200], [20, 40], 65), ([500, 130], [20, 40], 8)])
def test_lengths_beyond_the_table(lens, new, cols):
    """Tokens behind the last page of the table are not seen, new ones nor committed ones."""
    c = Tree(16, lens, new, group=4, page=16, dtype="bf16")
    c.table = np.ascontiguousarray(c.table[:, :cols])
    c.batch = E.KVBatch(ints(c.table.tolist()), c.batch.kv_lens, c.batch.q_starts, parents=c.batch.parents)
    q = c.rand(8)
    c.check_tree(q)
    c.check_tree(q, window=300)


# ---------------------------------------------------------------- pages

class Pool:
    """Some layers' caches with random codes, tables of sequences, and the model of them."""

    def __init__(self, seed, table, lens, pages, T=16, heads=2, dim=64, layers=2, fmt="e4m3"):
        dev()
        self.rng = rng = np.random.default_rng(seed)
        self.fmt = fmt
        shape = (pages, heads, T, dim)
        self.caches, model = [], []
        for _ in range(layers):
            np_ = {}
            for n in "kv":
                x = rng.standard_normal(shape) * 60
                np_[n] = L.encode(np.clip(x, -127, 127), fmt)
                np_[n + "s"] = (2.0 ** rng.integers(-8, -3, shape[:2])).astype(np.float32)
            model.append(np_)
            self.caches.append(E.KVCache.wrap(cuda(np_["k"].copy()), cuda(np_["v"].copy()), cuda(np_["ks"].copy()),
                                              cuda(np_["vs"].copy()), FMT[fmt]))
        self.model = R.Book(table, lens, pages, T, model)
        self.pages = E.KVPages(self.caches, ints(np.array(table).tolist()), ints(lens))

    def check(self):
        torch.cuda.synchronize()
        m = self.model
        assert self.pages.page_table.cpu().numpy().tolist() == m.table.tolist()
        assert self.pages.kv_lens.tolist() == m.lens
        assert self.pages.refs.cpu().numpy().tolist() == m.refs().tolist()
        for c, x in zip(self.caches, m.caches):
            for n in "kv":
                assert np.array_equal(getattr(c, n).cpu().numpy(), x[n]), n
                assert np.array_equal(getattr(c, n + "_scale").cpu().numpy(), x[n + "s"], equal_nan=True)


@pytest.mark.parametrize("seqs,cols,pages,T,seed", [(4, 12, 40, 16, 0), (9, 70, 200, 32, 1), (1, 3, 3, 128, 2),
                                                     (300, 5, 700, 16, 3), (1024, 4, 3000, 16, 4), (16, 300, 900, 16, 5)])
def test_fork_and_grow_follow_their_definitions(seqs, cols, pages, T, seed):
    """Steps of a search, and of a serving loop: beams follow parents, some end, some are cut, all grow, some by much."""
    p = Pool(seed, np.full((seqs, cols), -1), [0] * seqs, pages, T=T, layers=1 if seqs > 100 else 2)
    rng, m = p.rng, p.model
    missing = []
    for step in range(14):
        say(seqs, cols, "step", step)
        more = [int(rng.integers(-1, 3)) for _ in range(seqs)]
        if step % 5 == 0:
            more[int(rng.integers(seqs))] = int(rng.integers(1, 3 * T))
        if step % 7 == 6:
            more = [1] * seqs
        got = int(p.pages.grow(ints(more) if step % 2 else (ints(more) if len(set(more)) > 1 else more[0])))
        missing.append(m.grow(more))
        assert got == missing[-1]
        p.check()
        source = [int(rng.integers(-1, seqs + 1)) if rng.random() < 0.5 else s for s in range(seqs)]
        keep = [int(rng.integers(-2, 40 * T)) for _ in range(seqs)] if step % 3 == 2 else None
        p.pages.fork(ints(source), lens=None if keep is None else ints(keep))
        m.fork(source, keep)
        p.check()
    p.pages.fork(ints([-1] * seqs))
    assert not p.pages.refs.any() and not p.pages.kv_lens.any() and (p.pages.page_table == -1).all()


def test_grow_reports_what_is_missing_and_changes_nothing():
    table = [[0, 1, -1], [0, 1, -1], [0, 1, 2]]
    p = Pool(3, table, [20, 20, 33], 4)
    for more, missing in (([16, 16, 1], 3), ([0, 0, 16], 1), ([100, 0, 0], 6)):  # (5 columns that the table has not, 2 pages where one is free)
        assert int(p.pages.grow(ints(more))) == missing == p.model.grow(more)
        p.check()
    assert int(p.pages.grow(ints([0, 1, 1]))) == 0 == p.model.grow([0, 1, 1])  # the one free page
    p.check()
    assert p.pages.page_table[1, 1] == 3


def test_grow_leaves_absent_pages_and_pages_of_other_tables():
    """An absent page that should hold older tokens, ids outside the caches, and holders in a table of another call."""
    table = [[0, -3, 1], [5, 99, -1], [2, 3, -1], [2, 3, -1]]
    p = Pool(4, table, [20, 16, 20, 20], 9)
    other = E.KVPages(p.caches, ints([[3]]), ints([4]), refs=p.pages.refs)
    p.pages.refs[3] += 1
    assert int(p.pages.grow(ints([1, 1, 1, 1]))) == 0
    torch.cuda.synchronize()
    # lowest free pages in order: 4, 6, 7; both sequences copy page 3, which `other` holds
    assert p.pages.page_table.tolist() == [[0, -3, 1], [5, 4, -1], [2, 6, -1], [2, 7, -1]]
    assert p.pages.refs.tolist() == [1, 1, 2, 1, 1, 1, 1, 1, 0]
    for c in p.caches:
        assert torch.equal(c.k[6, :, :4], c.k[3, :, :4]) and torch.equal(c.v[7, :, :4], c.v[3, :, :4])
        assert torch.equal(c.k_scale[6], c.k_scale[3])
    assert int(other.grow(1)) == 0 and other.page_table.tolist() == [[3]]


def test_copy_pages():
    p = Pool(5, [[0]], [1], 12, layers=3, dim=128, T=128)
    src, dst = [1, 2, 3, -1, 4, 40, 5], [7, 8, 9, 10, -2, 11, 5]
    E.kv_copy_pages(p.caches, ints(src), ints(dst))
    for x in p.model.caches:
        for a, b in zip(src[:3], dst[:3]):
            for n in ("k", "v", "ks", "vs"):
                x[n][b] = x[n][a]
    p.check()
    some = E.cache_set(p.caches)
    E.kv_copy_pages(some, ints([]), ints([]))
    E.kv_copy_pages(some, ints([6]), ints([0]))
    for x in p.model.caches:
        for n in ("k", "v", "ks", "vs"):
            x[n][0] = x[n][6]
    p.check()


ACCEPT = [("e4m3", 64, 16, 0), ("i8", 128, 16, 1), ("e4m3", 128, 32, 2), ("i8", 64, 64, 3)]


@pytest.mark.parametrize("fmt,dim,T,seed", ACCEPT)
def test_accept(fmt, dim, T, seed):
    """Paths within a page and over several, none, all of a chain, scales that are no powers of two, poisoned pages."""
    rng = np.random.default_rng(seed)
    new = [1, 9, 30, 64, 0, 17, 40, 5, 100, 600, 8]
    lens = [n + int(rng.integers(0, 3 * T)) for n in new]
    lens[10] = 3  # fewer than its new tokens
    cols = max(-(-t // T) for t in lens)
    order = rng.permutation(len(new) * cols)
    table = order.reshape(len(new), cols)
    table[7, :] = table[7, :] if lens[7] < T else np.where(np.arange(cols) == lens[7] // T, -1, table[7])
    trees = [[int(rng.integers(max(-1, i - 4), i)) for i in range(n)] for n in new]
    p = Pool(seed, table, lens, len(order), T=T, dim=dim, layers=3, fmt=fmt)
    for x, c in zip(p.model.caches[1:], p.caches[1:]):  # any scales in the second, far apart ones in the third
        for n in "kv":
            s = rng.random(x[n + "s"].shape) * (1 if x is p.model.caches[1] else 2.0 ** rng.integers(-20, 4, x[n + "s"].shape))
            x[n + "s"][:] = s.astype(np.float32) + 1e-9
            getattr(c, n + "_scale").copy_(cuda(x[n + "s"]))
    for s in (2, 8):  # poisoned pages among a path's
        page = table[s, (lens[s] - 1) // T]
        p.model.caches[0]["ks"][page, 0] = np.nan
        p.caches[0].k_scale[int(page), 0] = math.nan
    starts = [0] + list(np.cumsum(new))
    flat = [x for t in trees for x in t]
    batch = E.KVBatch(p.pages.page_table, p.pages.kv_lens, ints(starts), parents=ints(flat))
    deep = lambda t: max(range(len(t)), key=lambda i: len(R.line(t, i)))  # noqa: E731
    for leaf in ([0, 8, deep(trees[2]), deep(trees[3]), 0, -1, 39, 2, deep(trees[8]), 5, 3],
                 [1, 3, 29, 20, -1, 16, 40, 4, 60, -1, 0]):
        out = torch.zeros(len(new), dtype=torch.int32, device="cuda")
        assert E.kv_accept(p.caches, batch, ints(leaf), lens_out=out) is out
        torch.cuda.synchronize()
        ref = R.accept(p.model.caches, fmt, p.model.table, lens, starts, len(flat), flat, leaf)
        assert out.tolist() == ref
        for c, x in zip(p.caches, p.model.caches):
            for n in "kv":
                assert np.array_equal(getattr(c, n + "_scale").cpu().numpy(), x[n + "s"], equal_nan=True), n
                assert L.same_codes(getattr(c, n).cpu().numpy(), x[n], fmt), n
    # a chain only cuts the lengths, in place
    chain = E.KVBatch(p.pages.page_table, p.pages.kv_lens, ints(starts))
    leaf = [0, 3, -1, 70, 0, 2, 3, 4, 50, 200, 1]
    assert E.kv_accept(p.caches, chain, ints(leaf)) is chain.kv_lens
    assert chain.kv_lens.tolist() == R.accept(p.model.caches, fmt, p.model.table, lens, starts, len(flat), None, leaf)


# ---------------------------------------------------------------- beams

def check_beams(logits, scores, keep=None, ended=None, end_token=0, **kw):
    got = E.beam_select(logits, scores, keep=keep, ended=ended, end_token=end_token, **kw)
    torch.cuda.synchronize()
    items, nb = scores.shape
    x = f64(logits).reshape(items, nb, -1)
    ref = R.beams(x, f64(scores), nb if keep is None else keep, None if ended is None else ended.cpu().numpy(), end_token)
    assert got[1].tolist() == ref[1] and got[2].tolist() == ref[2]
    a, b = f64(got[0]), np.array(ref[0])
    assert np.array_equal(np.isinf(a), np.isinf(b))
    ok = ~np.isinf(b)
    # the sum's error in front of the logarithm, and the result's own rounding
    assert (np.abs(a - b)[ok] <= 2.0 ** -22 + 2.0 ** -24 * np.abs(b[ok])).all()
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("items,nb,vocab,keep", [(1, 1, 1, 1), (1, 4, 32000, 4), (3, 5, 1000, 10), (2, 64, 777, 128),
                                                 (2, 1, 40, 64), (1, 3, 2049, 128), (5, 2, 70001, 3), (9, 8, 513, 1)])
def test_beams(dtype, items, nb, vocab, keep):
    dev()
    rng = np.random.default_rng(vocab)
    x = cuda(rng.standard_normal((items, nb, vocab)) * 3).to(DT[dtype])
    s = cuda((rng.standard_normal((items, nb)) * 2 - 10).astype(np.float32))
    check_beams(x, s, keep=keep)
    ended = cuda(rng.random((items, nb)) < 0.3)
    check_beams(x.flatten(0, 1), s, keep=keep, ended=ended, end_token=5)


def test_beams_ties_go_to_the_lower_beam_and_token():
    dev()
    for nb, vocab, keep in ((3, 5000, 20), (1, 100, 128), (4, 300000, 100), (64, 40, 128)):
        flat = torch.full((nb, vocab), -2.5, device="cuda")
        s, p, t = check_beams(flat, torch.zeros(1, nb, device="cuda"), keep=keep)
        n = min(keep, nb * vocab)
        assert t[0, :n].tolist() == [i % vocab for i in range(n)] and p[0, :n].tolist() == [i // vocab for i in range(n)]
    # zeros of both signs are equal; equal rows at other places; few values
    x = torch.zeros(2, 70, device="cuda")
    x[:, ::2] = -0.0
    check_beams(x, torch.zeros(1, 2, device="cuda"), keep=9)
    rng = np.random.default_rng(2)
    row = rng.integers(0, 3, 4001).astype(np.float32)
    check_beams(cuda(np.stack([row] * 4)).bfloat16(), torch.zeros(1, 4, device="cuda"), keep=50)
    up = torch.arange(200000, device="cuda", dtype=torch.float32).view(2, -1) * 1e-4
    check_beams(up, torch.zeros(1, 2, device="cuda"), keep=128)


def test_beams_that_continue_nothing():
    dev()
    rng = np.random.default_rng(3)
    nb = 9
    x = cuda(rng.standard_normal((2, nb, 600)).astype(np.float32))
    x[0, 1, 7] = math.nan
    x[0, 2, 8] = math.inf
    x[0, 3] = -math.inf
    x[0, 4, :598] = -math.inf
    x[0, 5] = 3e38
    x[0, 6, 3] = -3e38
    x[1] = -math.inf
    s = torch.zeros(2, nb, device="cuda")
    s[0, 0], s[0, 7], s[0, 8] = -math.inf, math.nan, math.inf
    _, p, t = check_beams(x, s, keep=12)
    assert (p[1] == -1).all() and (t[1] == -1).all()
    # only ended beams, more than are kept, in the order of their scores
    e = torch.ones(2, nb, dtype=torch.bool, device="cuda")
    s = torch.arange(2 * nb, device="cuda", dtype=torch.float32).view(2, nb)
    _, p, t = check_beams(x, s, keep=4, ended=e, end_token=-3)
    assert p.tolist() == [[8, 7, 6, 5], [17, 16, 15, 14]] and (t == -3).all()


def test_beams_rows_apart_unaligned_and_in_place():
    dev()
    rng = np.random.default_rng(4)
    for dtype in ("f32", "bf16"):
        wide = cuda(rng.standard_normal((6, 1111)) * 2).to(DT[dtype])
        x = wide[:, 3:1002]
        s = cuda(-rng.random((2, 3)).astype(np.float32))
        want = check_beams(x, s)
        out = (s, torch.empty(2, 3, dtype=torch.int32, device="cuda"), torch.empty(2, 3, dtype=torch.int32, device="cuda"))
        got = E.beam_select(x, s, out=out)
        assert got[0] is s and all(torch.equal(a, b) for a, b in zip(got, want))


def test_beams_far_apart_scores():
    """The first bound must hold whatever the scores' sizes: logits near 2^20 in one beam, small ones in another."""
    dev()
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 6, 3000)).astype(np.float32)
    x[0, 1] = 1e6 + rng.integers(0, 3000, 3000) * 0.0625
    x[0, 2] = -1e6 - rng.integers(0, 3000, 3000) * 0.0625
    s = np.array([[0, 1e-3, 2e-3, -1e6, 1e6, -3e38]], np.float32)
    check_beams(cuda(x), cuda(s), keep=100)
    check_beams(cuda(x[:, :4]), cuda(s[:, :4]), keep=100)
    check_beams(cuda(x[:, :3]), cuda(s[:, :3]), keep=128)


def test_beams_of_more_items_than_a_launch_has_blocks():
    dev()
    n = (1 << 21) + 3
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(n, 2, generator=g, device="cuda")
    s, p, t = E.beam_select(x, torch.zeros(n, 1, device="cuda"))
    assert torch.equal(p[:, 0], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(t[:, 0], (x[:, 1] > x[:, 0]).int())
    want = -torch.log1p(torch.exp(-(x[:, 0] - x[:, 1]).abs().double()))
    assert float((s[:, 0].double() - want).abs().max()) <= 2.0 ** -22 + 2.0 ** -24


def test_caches_beyond_32_bits_do_what_small_ones_do():
    """Codes behind 4 GiB: the same pages under low and high numbers."""
    dev()
    high, T, heads, dim = 33000, 128, 8, 128
    rng = np.random.default_rng(7)
    big = E.KVCache(high + 6, heads, dim, T)
    small = E.KVCache(8, heads, dim, T)
    for c in ("k", "v"):
        getattr(small, c).copy_(cuda(L.encode(rng.standard_normal((8, heads, T, dim)) * 60, "e4m3")))
        getattr(small, c + "_scale").copy_(cuda((2.0 ** rng.integers(-8, -3, (8, heads))).astype(np.float32)))
        getattr(big, c)[high - 2:].copy_(getattr(small, c))
        getattr(big, c + "_scale")[high - 2:].copy_(getattr(small, c + "_scale"))
    new, lens = 20, [T * 2 + 5, T + 30]
    par = ints(R.random_tree(rng, new) + R.random_tree(rng, new))
    k, v, q = (cuda(rng.standard_normal((2 * new, h, dim)).astype(np.float32)) for h in (heads, heads, 2 * heads))
    rope = E.rope_table(10000.0, 4 * T, dim)
    got = []
    for c, at in ((small, 0), (big, high - 2)):
        table = [[at + 3, at + 1, at + 6, -1], [at + 2, at + 5, -1, -1]]
        pages = E.KVPages([c], ints(table), ints([lens[0] - new, lens[1] - new]))
        pages.refs[:max(at, 0)] = 1  # nothing free below
        pages.fork(ints([0, 0]))
        assert int(pages.grow(1)) == 0  # one copies the last page, which both hold
        copy = c.k[int(pages.page_table[0, 1])].clone()
        assert pages.page_table[0, 1] == at and pages.page_table[1, 1] == at + 1
        pages.page_table.copy_(ints(table))
        pages.kv_lens.copy_(ints(lens))
        batch = E.KVBatch(pages.page_table, pages.kv_lens, ints([0, new, 2 * new]), parents=par)
        a = c.append(batch, k, v, q=q, rope=rope, q_norm=torch.ones(dim, device="cuda"))
        o = c.attend(batch, a)
        n = E.kv_accept([c], batch, ints([new - 1, new - 2]), lens_out=ints([0, 0]))
        E.kv_copy_pages([c], ints([at + 6]), ints([at + 7]))
        torch.cuda.synchronize()
        got.append([copy, a, o, n] + [t[at:at + 8].clone() for t in (c.k, c.v, c.k_scale, c.v_scale)])
    for x, y in zip(*got):
        assert torch.equal(x, y)
