"""Edges of the operators for several continuations of a sequence: what 16-bit rows of trees
keep of their weights, trees of very many rows, beams whose
logits are large, searches without room."""
import math
from types import SimpleNamespace

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _branches as R  # noqa: E402
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
from test_gpu_branches import Tree, cuda  # noqa: E402
from test_gpu_layer import DT, dev, f64, ints, say  # noqa: E402


# ---------------------------------------------------------------- trees: what 16-bit rows keep

@pytest.mark.parametrize("room", [0, 1100])  # tables of more than 1024 tokens are shared out in another way
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,group,dim,page,fmt,lens,new,window", [
    (2, 4, 128, 64, "e4m3", [700, 33], [32, 33], 0), (1, 8, 128, 16, "i8", [300, 90], [40, 30], 0),
    (2, 3, 64, 16, "e4m3", [500, 26, 129, 64], [25, 25, 20, 13], 100), (1, 4, 64, 64, "i8", [640, 212], [100, 212], 0),
    (2, 4, 128, 128, "e4m3", [410, 64, 15], [15, 14, 15], 0), (2, 2, 128, 16, "i8", [70, 300], [6, 7], 0)])
def test_trees_keep_the_weights_of_16_bit_rows(heads, group, dim, page, fmt, lens, new, window, dtype, room):
    """What fp32 rows are held to, and one rounding of the output (small scores, which add little to that),
    however wide the page table is."""
    c = Tree(51, lens, new, heads=heads, group=group, dim=dim, page=page, fmt=fmt, dtype=dtype, room=room)
    q = c.rand(heads * group, 0.01)
    got = f64(c.cache.attend(c.batch, q, window=window))
    ref, tol = R.attend(c.np, c.table, c.lens, c.starts, f64(q), dim ** -0.5, window, fmt, "f32", c.parents)
    # rounding moves a result by half a step of what is rounded, itself within tol of ref
    tol = tol + L.HALF_STEP[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
    worst = float((np.abs(got - ref) / (tol + 1e-300)).max())
    say("worst", worst)
    assert worst <= 1.0, worst


def test_trees_of_more_rows_than_a_launch_has_blocks():
    """2^27 rows of a sequence that is no tree become 0, those of a tree behind them what they are alone."""
    dev()
    big, new, group, dim = 1 << 21, 40, 64, 64
    c = Tree(52, [2000], [new], heads=1, group=group, dim=dim, page=64, dtype="bf16")
    q = c.rand(group)
    want = c.check_tree(q)
    batch = E.KVBatch(c.batch.page_table.repeat(2, 1), ints([7, 2000]), ints([0, big, big + new]),
                      parents=torch.cat([ints([-1]).repeat(big), c.batch.parents]))
    rows = torch.zeros(big + new, group, dim, dtype=torch.bfloat16, device="cuda")
    rows[big:] = q
    out = torch.full_like(rows, 3.0)
    c.cache.attend(batch, rows, out=out)
    assert not bool(out[:big].any())
    # another split of the sums: both are within the bound of the 64-bit result
    ref, tol = R.attend(c.np, c.table, c.lens, c.starts, f64(q), dim ** -0.5, 0, "e4m3", "bf16", c.parents)
    assert (np.abs(f64(out[big:]) - ref) <= tol).all() and want.shape == q.shape


# ---------------------------------------------------------------- beams: large logits

def check_large(x, s, keep, **kw):
    """beam_select against its definition, whatever the logits' size."""
    got = E.beam_select(x, s, keep=keep, **kw)
    torch.cuda.synchronize()
    rows, scores = f64(x), f64(s)
    ref = R.beams(rows, scores, keep)
    a, b = f64(got[0]), np.array(ref[0])
    assert got[1].tolist() == ref[1] and got[2].tolist() == ref[2]
    assert np.array_equal(np.isinf(a), np.isinf(b))
    # the sum's error in front of the logarithm and the result's own rounding; both sides round the log sum of a
    # row to a double, 2^-53 of it each, and the difference to it is within those roundings of itself again
    top = np.abs(np.where(np.isfinite(rows), rows, 0.0)).max(-1)
    near = np.where(top < 2.0 ** 60, top, 0.0)  # beyond, no log sum reaches half a step
    own = np.take_along_axis(near, np.maximum(np.array(ref[1]) - np.arange(len(rows))[:, None] * rows.shape[1], 0), 1)
    ok = ~np.isinf(b)
    d = np.abs(np.where(ok, a, 0.0) - np.where(ok, b, 0.0))
    assert (d <= 2.0 ** -22 + 2.0 ** -24 * np.abs(np.where(ok, b, 0.0)) + 2.0 ** -51 * own).all(), d.max()
    return got


PLACES = {"top": lambda v: slice(v // 3, v // 3 + 1), "all": lambda v: slice(0, v), "first 512": lambda v: slice(0, 512),
          "a wave's 2048": lambda v: slice(2048, 4096), "the last part": lambda v: slice(v // 2048 * 2048, v)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [4500, 45077])  # waves of 512 logits, and of 2048
@pytest.mark.parametrize("place", list(PLACES))
def test_beams_of_large_finite_logits(dtype, vocab, place):
    """One logit, a row, or a part that one wave reads, far from the others: forbidden tokens, or sure ones."""
    dev()
    rng = np.random.default_rng(61)
    sizes = [1e6, 2.0 ** 24, 1e8, 1e9, 5e9, 1e10, 1e12, 1e15, 1e20, 1e30, 2.0 ** 120, 3e38]
    at = [z * sign for z in sizes for sign in (1.0, -1.0)]
    items, nb = len(at) // 2 * 2, 4  # in beam 0 and 2: the large ones; 1 and 3: ordinary
    x = rng.standard_normal((items, nb, vocab)) * 3
    for i in range(items):
        x[i, 0, PLACES[place](vocab)] = at[i]
        x[i, 2, PLACES[place](vocab)] = at[(i + 5) % items]
    s = rng.standard_normal((items, nb)).astype(np.float32) - 12
    check_large(cuda(x.astype(np.float32)).to(DT[dtype]), cuda(s), 6)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("keep", [3, 64])
def test_beams_of_rows_of_the_lowest_number_keep_their_scores(dtype, keep):
    """A mask of the type's lowest number that forbids every token of a beam, next to beams that continue."""
    dev()
    rng = np.random.default_rng(62)
    low = torch.finfo(DT[dtype]).min
    x = cuda(rng.standard_normal((4, 3, 3001)).astype(np.float32)).to(DT[dtype])
    s = cuda(np.array([[-12, -11, -3], [-1, -12.5, -14], [-40, -41, -30], [-7, -8, -9]], np.float32))
    x[0, 0] = low
    x[1, 2] = low
    x[2, 1] = low
    x[3] = low
    check_large(x, s, keep)


def test_beams_of_the_largest_scores_and_logits():
    """The first bound must hold where a score and a log sum of the largest size meet."""
    dev()
    rng = np.random.default_rng(63)
    x = rng.standard_normal((3, 4, 2600)).astype(np.float32)
    x[0, 0] = 3.4e38
    x[1, 1] = -3.4e38
    x[1, 2, 7] = 3.4e38
    x[2, 0], x[2, 1] = -3.4e38, 3.4e38
    s = np.array([[-3.4e38, -5, -1e30, -6], [-2, 3.4e38, -3.4e38, 1e30], [3.4e38, -3.4e38, 3e38, -3e38]], np.float32)
    for keep in (5, 128):
        check_large(cuda(x), cuda(s), keep)


# ---------------------------------------------------------------- searches

class Search:
    """A BeamStep over a step of given logits that appends a key and a value for each row."""

    def __init__(self, prompt, items, beams, pages, cols, end=-1, T=16, vocab=50, seed=71):
        dev()
        rng = np.random.default_rng(seed)
        rows = items * beams
        self.cache = E.KVCache(pages, 2, 64, T)
        self.pages = E.KVPages([self.cache], ints([[-1] * cols] * rows), ints([0] * rows))
        batch = E.KVBatch(self.pages.page_table, self.pages.kv_lens, ints(list(range(rows + 1))))
        self.logits = torch.zeros(rows, vocab, device="cuda")
        self.kv = cuda(rng.standard_normal((rows, 2, 64)).astype(np.float32))

        def enqueue(effort, stream=None):
            self.cache.append(batch, self.kv, self.kv, stream=stream)
            return self.logits

        # every item's prompt in its first beam, then in all
        assert int(self.pages.grow(ints([prompt if b % beams == 0 else 0 for b in range(rows)]))) == 0
        first = E.KVBatch(self.pages.page_table, self.pages.kv_lens,
                          ints([prompt * (-(-b // beams)) for b in range(rows + 1)]))
        x = cuda(rng.standard_normal((prompt * items, 2, 64)).astype(np.float32))
        self.cache.append(first, x, x)
        self.pages.fork(ints([b // beams * beams for b in range(rows)]))
        assert int(self.pages.grow(1)) == 0
        step = SimpleNamespace(x=torch.zeros(rows, 8, device="cuda"), batch=batch, caches=[self.cache], enqueue=enqueue)
        self.search = E.BeamStep(step, self.pages, beams, end_token=end)

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)]


@pytest.mark.parametrize("captured", [False, True])
def test_a_search_without_room_writes_nothing_more(captured):
    """Beams that share their last page when the pages run out: later steps leave the cache as it is."""
    s = Search(20, 1, 4, pages=6, cols=8)  # the prompt's full page, a copy of the other for each beam, one free
    rng = np.random.default_rng(72)
    run = lambda: s.search.enqueue(1.0)  # noqa: E731
    if captured:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            s.search.enqueue(1.0, side)
        run = graph.replay
    steps = 0
    while int(s.search.short) == 0:
        s.logits.copy_(torch.from_numpy(rng.standard_normal(s.logits.shape) * 5))
        run()
        steps += 1
        assert steps < 20
    before = s.state()
    for _ in range(3):
        s.kv.copy_(torch.from_numpy(rng.standard_normal(s.kv.shape) * 3))
        run()
        (torch.ones(1000, device="cuda") * 2).sum().item()
        assert all(torch.equal(a, b) for a, b in zip(before, s.state()))
        assert int(s.search.short) > 0 and not s.pages.kv_lens.any()
    held = s.pages.page_table[(s.pages.page_table >= 0)].long().cpu()
    assert s.pages.refs.tolist() == torch.bincount(held, minlength=6).tolist()


@pytest.mark.parametrize("prompt", [14, 15, 20])  # end tokens inside a page, at its end, at its beginning
def test_ended_beams_keep_their_length_and_room(prompt):
    """Beams that end early stay as they are, however many steps follow; the others go on."""
    s = Search(prompt, 2, 2, pages=20, cols=3, end=9)
    rng = np.random.default_rng(73)
    length, held = [prompt + 1] * 4, None
    for step in range(40):
        x = rng.standard_normal(s.logits.shape) * 0.1
        x[:, 9] = -50.0
        if step == 1:
            x[2:, 9] = 50.0  # the second item's beams end
        if step == 5:
            x[:2, 9] = 50.0  # the first's
        s.logits.copy_(torch.from_numpy(x))
        was = s.search.ended.view(-1).tolist()
        s.search.enqueue(1.0)
        torch.cuda.synchronize()
        parents = s.search.parents.view(-1).tolist()
        length = [length[p] + (0 if was[p] else 1) for p in parents]
        assert s.pages.kv_lens.tolist() == length
        assert s.search.ended.view(-1).tolist() == [step >= 5, step >= 5, step >= 1, step >= 1]
        assert int(s.search.short) == 0
        table = s.pages.page_table[s.pages.page_table >= 0].long().cpu()
        assert s.pages.refs.tolist() == torch.bincount(table, minlength=20).tolist()
        if step >= 7:  # nothing changes any more: not the tables but for a last page, not what they stand for
            now = []
            for b in range(4):
                pos = torch.arange(length[b] - 1)
                at = s.pages.page_table[b].cpu()[pos // 16].long()
                now.append(s.cache.k.cpu()[at, :, pos % 16].clone())
            assert held is None or all(torch.equal(a, b) for a, b in zip(held, now))
            held = now
    assert length == [prompt + 7, prompt + 7, prompt + 3, prompt + 3]


def test_a_search_on_a_streams_handle():
    """`stream` as everywhere else: None, a stream, or its handle."""
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream):
        s = Search(20, 1, 3, pages=20, cols=8)
        s.logits.copy_(torch.from_numpy(np.random.default_rng(74).standard_normal(s.logits.shape)))
        torch.cuda.synchronize()
        for _ in range(3):
            s.search.enqueue(1.0, stream)
        got.append([s.search.scores, s.search.tokens, s.pages.kv_lens, s.pages.page_table] + s.state())
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# ---------------------------------------------------------------- pages: wide tables

@pytest.mark.parametrize("seqs,cols", [(3, (1 << 22) + 77), (513, 1 << 26)])
def test_fork_of_tables_with_very_many_columns(seqs, cols):
    """More columns than a launch has blocks for; of the widest tables, more than it has threads for."""
    dev()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * seqs * cols + (8 << 30):
        pytest.skip("the table needs %d GB" % (4 * seqs * cols >> 30))
    cache = E.KVCache(40, 1, 64, 16)
    table = torch.full((seqs, cols), -1, dtype=torch.int32, device="cuda")
    table[0, :7] = ints([5, 6, 7, 8, 9, 10, 11])
    at = [0, 64, 1 << 20, (1 << 22) - 1, 1 << 22, cols - 1]  # entries of others, near and far
    for i, c in enumerate(at):
        table[1 + i % 2, c] = 20 + i
    refs = torch.zeros(40, dtype=torch.int32, device="cuda")
    refs[5:12] = 1
    refs[20:20 + len(at)] = 1
    pages = E.KVPages([cache], table, ints([100] + [16 * cols] * 2 + [0] * (seqs - 3)), refs=refs)
    pages.fork(ints([0, 0, 2] + [0] * (seqs - 3)))
    want = torch.full((seqs, 8), -1, dtype=torch.int32)
    want[:, :7] = torch.arange(5, 12)
    want[2] = -1
    assert torch.equal(table[:, :8].cpu(), want)
    assert not (table[1, 8:] >= 0).any()  # the second follows the first, the third itself
    assert [int(table[2, c]) for c in at] == [20 + i if i % 2 else -1 for i in range(len(at))]
    held = [0] * 40
    held[5:12] = [seqs - 1] * 7
    for i in range(1, len(at), 2):
        held[20 + i] = 1
    assert refs.tolist() == held
    assert pages.kv_lens.tolist() == [100, 100, 16 * cols] + [100] * (seqs - 3)
    del table, pages
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- paths: more parents than rows

def test_accept_with_more_parents_than_a_call_has_rows():
    """`parents` may be longer than the rows, by any number: a buffer for the largest batch."""
    c = Tree(55, [70, 40], [9, 12], page=16, parents=R.random_tree(np.random.default_rng(2), 9) * 2 + [0, 1, 2])
    long = torch.full(((1 << 24) + 5,), -1, dtype=torch.int32, device="cuda")
    long[:21] = c.batch.parents
    batch = E.KVBatch(c.batch.page_table, c.batch.kv_lens, c.batch.q_starts, parents=long)
    got = E.kv_accept([c.cache], batch, ints([8, 11]), lens_out=ints([0, 0]))
    assert got.tolist() == R.accept([c.np], "e4m3", c.table, c.lens, c.starts, 21, c.parents, [8, 11])
    c.check_cache()


# ---------------------------------------------------------------- head norms: weights of any size

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [False, True])  # weights of each head, or shared
@pytest.mark.parametrize("size,weight", [(2.0 ** 58, 1e-25), (2.0 ** -58, 1e30), (1.0, 1e-37), (1.0, 1e36),
                                         (2.0 ** 55, 1e-36), (2.0 ** -50, 1e37), (1.0, 0.0)])
def test_head_norms_with_weights_of_any_size(size, weight, heads, dtype):
    """The weight's product with 1 / rms may leave fp32 where the normed element does not."""
    lens, new = [40, 7], [21, 7]
    c = Tree(56, lens, new, page=16, dtype=dtype, parents=None, garbage=False)
    k, v, q = c.rand(2), c.rand(2), c.rand(4, size)
    w = c.rng.random((4, 128) if heads else 128) + 0.5
    w[..., ::3] *= weight
    w = cuda(w.astype(np.float32)).to(DT[dtype])
    got = c.cache.append(c.batch, k, v, q=q, q_norm=w, eps=0.0)
    ref, qsize = R.append(c.np, c.table, lens, c.starts, f64(q), f64(k), f64(v), None, False, "e4m3", None, f64(w), None,
                          0.0)
    # 1 / rms, its product with the weight, that with the element, and the result: four roundings to fp32 at most
    # (2^-22 in all), and one to the result's type; the least numbers are 2^-149 apart in fp32, 2^-133 in bf16, and
    # a rounding among them is off by half of that: the element's in fp32 and the result's
    least = 2.0 ** -149 if dtype == "f32" else 2.0 ** -150 + 2.0 ** -134
    off = np.abs(f64(got) - ref) / (2.0 ** -22 * qsize + L.HALF_STEP[dtype] * np.abs(ref) + least)
    worst = float(np.where(np.isnan(off), np.inf, off).max())
    assert worst <= 1.0, worst
