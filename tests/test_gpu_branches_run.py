"""Several continuations of a sequence, used together: beam search and trees of
drafted tokens over whole decoder layers, captured and replayed, on other streams."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _branches as R  # noqa: E402
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
import synth  # noqa: E402
from _parity import rel_l2  # noqa: E402
from test_gpu_branches import Pool, Tree, cuda  # noqa: E402
from test_gpu_layer import dev, f64, ints, say  # noqa: E402

DIM, QH, KH, HD, HID, VOCAB, T = 256, 4, 2, 64, 512, 320, 16
SHAPES = {"wq": (DIM, QH * HD), "wk": (DIM, KH * HD), "wv": (DIM, KH * HD), "wo": (QH * HD, DIM), "w1": (DIM, HID),
          "w3": (DIM, HID), "w2": (HID, DIM)}


class Model:
    """Decoder layers and an embedding; `step` runs some rows over the model's caches."""

    def __init__(self, seed, layers, pages, rows):
        dev()
        rng = np.random.default_rng(seed)
        self.mats = [{r: E.EffortMatrix(synth.matrix("branches", *SHAPES[r], layer=l, w=r), P=16, batch=rows)
                      for r in E.LAYER_ROLES} for l in range(layers)]
        self.head = E.EffortMatrix(synth.matrix("branches", DIM, VOCAB, w="head"), P=16, batch=rows)
        self.embed = cuda(rng.standard_normal((VOCAB, DIM)).astype(np.float32))
        one = lambda n: cuda((rng.random(n) + 0.5).astype(np.float32))  # noqa: E731
        self.norms, self.head_norm = [(one(DIM), one(DIM)) for _ in range(layers)], one(DIM)
        self.qk = [(one(HD), one(HD)) for _ in range(layers)]
        self.rope = E.rope_table(10000.0, 1024, HD)
        self.layers, self.pages = layers, pages

    def caches(self):
        return [E.KVCache(self.pages, KH, HD, T) for _ in range(self.layers)]

    def step(self, caches, batch, rows):
        x = torch.zeros(rows, DIM, device="cuda")
        return E.DecoderStep(self.mats, self.head, x, caches, batch, self.norms, self.head_norm, rope=self.rope,
                             qk_norms=self.qk)

    def alone(self, tokens, at_once=1):
        """Logits behind each token of one sequence, decoded one by one (in a cache of its own)."""
        caches, out = self.caches(), []
        lens = ints([0])
        batch = E.KVBatch(ints([list(range(self.pages))]), lens, ints([0, 1]))
        step = self.step(caches, batch, 1)
        for t in tokens:
            lens.add_(1)
            step.x.copy_(self.embed[t][None])
            out.append(f64(step.enqueue(1.0))[0].copy())
        return out


def log_softmax(x):
    return x - x.max() - math.log(np.exp(x - x.max()).sum())


@pytest.mark.parametrize("captured", [False, True])
def test_beam_search_over_decoder_layers(captured):
    """Two prompts, three beams each: every step's beams are what the plain selection makes of the step's own
    logits; at the end each beam's score is that of its tokens, decoded alone."""
    m = Model(1, 2, 60, 6)
    prompts = [[5, 17, 200, 31, 8] * 4, [9, 300, 12]]
    items, beams, cols, end = 2, 3, 5, 7
    table = np.full((6, cols), -1)
    caches = m.caches()
    pages = E.KVPages(caches, ints(table.tolist()), ints([0] * 6))
    # the prompts, one token after the other, in the first beam of each item
    one = m.step(caches, E.KVBatch(pages.page_table, pages.kv_lens, ints([0, 1, 1, 1, 2, 2, 2])), 2)
    short = E.KVBatch(pages.page_table, pages.kv_lens, ints([0, 1, 1, 1, 1, 1, 1]))
    only = m.step(caches, short, 1)
    for i in range(len(prompts[0]) - 1):
        both = i < len(prompts[1]) - 1
        assert int(pages.grow(ints([1, 0, 0, 1 if both else 0, 0, 0]))) == 0
        step, toks = (one, [prompts[0][i], prompts[1][i]]) if both else (only, [prompts[0][i]])
        step.x.copy_(m.embed[toks])
        step.enqueue(1.0)
    pages.fork(ints([0, 0, 0, 3, 3, 3]))
    assert int(pages.grow(1)) == 0
    step = m.step(caches, E.KVBatch(pages.page_table, pages.kv_lens, ints(list(range(7)))), 6)
    search = E.BeamStep(step, pages, beams, end_token=end)
    step.x.copy_(m.embed[[prompts[0][-1]] * 3 + [prompts[1][-1]] * 3])
    history = [list(prompts[b // 3]) for b in range(6)]
    graph = None
    if captured:
        side = torch.cuda.Stream()
        keep = [t.clone() for t in (search.scores, search.ended, pages.page_table, pages.kv_lens, pages.refs)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # the first call of everything is not captured
            search.enqueue(1.0, side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for t, k in zip((search.scores, search.ended, pages.page_table, pages.kv_lens, pages.refs), keep):
            t.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            search.enqueue(1.0, side)
    ended = np.zeros((items, beams), bool)
    for n in range(14):
        say("step", n)
        before = f64(search.scores)
        if graph is None:
            search.enqueue(1.0)
        else:
            graph.replay()
        torch.cuda.synchronize()
        logits = f64(step.logits).reshape(items, beams, VOCAB)
        sc, par, tok = R.beams(logits, before, beams, ended, end)
        assert search.parents.tolist() == par and search.tokens.tolist() == tok
        history = [history[p] + [t] for p, t in zip(sum(par, []), sum(tok, []))]
        ended = np.array(tok) == end
        assert search.ended.tolist() == ended.tolist()
        step.x.copy_(m.embed[search.tokens.view(-1).long()])
        refs = np.bincount(pages.page_table.cpu().numpy()[pages.page_table.cpu().numpy() >= 0], minlength=60)
        assert pages.refs.tolist() == refs.tolist()
    assert int(search.short) == 0
    # shared pages and copies hold what each line's own cache holds: the score of the last step's line
    for b in (0, 2, 4):
        if end in history[b]:
            continue
        own = m.alone(history[b][:-1])
        start = len(prompts[b // 3]) - 1
        score = sum(log_softmax(own[i])[history[b][i + 1]] for i in range(start, len(own)))
        # 14 log probabilities of logits whose fp32 sums differ in order (an 8-bit code may fall to the other side)
        assert abs(score - float(search.scores.view(-1)[b])) <= 14 * 0.02


def test_drafted_trees_over_a_decoder_layer():
    """The logits behind each drafted token are those of its line decoded alone; after a path is accepted,
    decoding goes on as if only it had been there."""
    m = Model(2, 1, 12, 16)
    rng = np.random.default_rng(3)
    prompts = [list(rng.integers(0, VOCAB, 21)), list(rng.integers(0, VOCAB, 30))]
    drafts = [list(rng.integers(0, VOCAB, 9)), list(rng.integers(0, VOCAB, 7))]
    trees = [[-1, 0, 0, 1, 1, 2, -1, 6, 3], [-1, 0, 1, -1, 3, 4, 4]]
    caches = m.caches()
    table = ints(rng.permutation(12)[:10].reshape(2, 5).tolist())
    lens = ints([0, 0])
    feed = m.step(caches, E.KVBatch(table, lens, ints([0, 1, 2])), 2)
    for i in range(30):
        lens.add_(ints([1 if i < 21 else 0, 1]))
        feed_ = feed if i < 21 else m.step(caches, E.KVBatch(table, lens, ints([0, 0, 1])), 1)
        feed_.x.copy_(m.embed[[p[i] for p in prompts if i < len(p)]])
        feed_.enqueue(1.0)
    batch = E.KVBatch(table, lens, ints([0, 9, 16]), parents=ints(trees[0] + trees[1]))
    step = m.step(caches, batch, 16)
    lens.add_(ints([9, 7]))
    step.x.copy_(m.embed[drafts[0] + drafts[1]])
    got = f64(step.enqueue(1.0))
    for s, at in ((0, 0), (1, 9)):
        for i in range(len(trees[s])):
            line = R.line(trees[s], i)
            want = m.alone(prompts[s] + [drafts[s][j] for j in line])[-1]
            # codes are alike; scores and weights differ by their fp32 sums' order (2^-20), which the layer's norm
            # and three products carry on
            assert rel_l2(got[at + i], want) <= 1e-4, (s, i)
    E.kv_accept(caches, batch, ints([8, 6]))
    torch.cuda.synchronize()
    lines = [R.line(trees[0], 8), R.line(trees[1], 6)]
    assert lens.tolist() == [21 + len(lines[0]), 30 + len(lines[1])]
    after = [11, 13]
    lens.add_(1)
    feed.x.copy_(m.embed[after])
    got = f64(feed.enqueue(1.0))
    for s in range(2):
        want = m.alone(prompts[s] + [drafts[s][j] for j in lines[s]] + [after[s]])[-1]
        # a page's scale may have been set by a token that is not on the path: codes differ by half a step of
        # 2^-4 here and there, of some of the tokens
        assert rel_l2(got[s], want) <= 2e-2, s


def test_captured_trees_and_paths_follow_what_changes_between_replays():
    """Attention, append and accept of trees in one graph; parents, lengths, leaves and queries change."""
    rng = np.random.default_rng(4)
    new, cols = [12, 30], 12
    c = Tree(20, [60, 100], new, group=2, page=16, dtype="bf16", room=60, garbage=False)
    w = cuda(rng.random(128) + 0.5).bfloat16()
    rope_np = L.rope_rows(10000.0, c.table.shape[1] * 16, 128)
    rope, n = cuda(rope_np), sum(new)
    k, v, q = c.rand(2), c.rand(2), c.rand(4)
    leaf, out = ints([3, 20]), ints([0, 0])
    hold = {}

    def run():
        hold["q"] = c.cache.append(c.batch, k, v, q=q, rope=rope, q_norm=w, k_norm=w)
        hold["a"] = c.cache.attend(c.batch, hold["q"], window=40)
        E.kv_accept([c.cache], c.batch, leaf, lens_out=out)

    side = torch.cuda.Stream()
    saved = [t.clone() for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for t, x in zip((c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale), saved):
        t.copy_(x)
    for i in range(4):
        say("replay", i)
        c.parents = [p for m in new for p in R.random_tree(rng, m)]
        c.batch.parents.copy_(ints(c.parents))
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape)))
        leaf.copy_(ints([int(rng.integers(12)), int(rng.integers(30))]))
        # behind everything of the last round: fresh pages, so that codes of the model and the cache agree
        base = [48 + 16 * i, 70 + 16 * i]
        c.lens = [base[0] + 12, base[1] + 30]
        c.batch.kv_lens.copy_(ints(c.lens))
        graph.replay()
        (torch.ones(1000, device="cuda") * 2).sum().item()  # the program's own work between replays
        torch.cuda.synchronize()
        f = lambda t: f64(t)  # noqa: E731
        ref, size = R.append(c.np, c.table, c.lens, c.starts, f(q), f(k), f(v), rope_np, False, "e4m3", c.parents, f(w),
                             f(w), 1e-5)
        assert (np.abs(f(hold["q"]) - ref) <= 2.0 ** -22 * size + 2.0 ** -8 * np.abs(ref)).all()
        want, tol = R.attend(c.np, c.table, c.lens, c.starts, f(hold["q"]), 128 ** -0.5, 40, "e4m3", "bf16", c.parents)
        assert (np.abs(f(hold["a"]) - want) <= tol).all()
        assert out.tolist() == R.accept([c.np], "e4m3", c.table, c.lens, c.starts, n, c.parents, leaf.tolist())
        c.check_cache()


def test_two_streams_and_two_graphs_have_their_own_workspaces():
    """Selections, growths and tree attention on two streams at once, and two graphs of them replayed together."""
    rng = np.random.default_rng(5)
    logits = [cuda(rng.standard_normal((8, 50000)).astype(np.float32)) for _ in range(2)]
    scores = [cuda(-rng.random((2, 4)).astype(np.float32)) for _ in range(2)]
    trees = [Tree(30 + i, [300, 200], [20, 20], group=4, page=16, room=900 * (2 - i)) for i in range(2)]
    qs = [t.rand(8) for t in trees]
    pools = [Pool(6 + i, [[0, 1, -1], [0, 1, -1], [0, 1, 2]], [20, 20, 33], 30) for i in range(2)]
    work = lambda i: (*E.beam_select(logits[i], scores[i], keep=8), trees[i].cache.attend(trees[i].batch, qs[i]))  # noqa: E731
    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append((*E.beam_select(logits[i], scores[i], keep=8, stream=s),
                        trees[i].cache.attend(trees[i].batch, qs[i], stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, held, source = [], [], ints([1, 0, 2])
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held.append(work(i))
            pools[i].pages.fork(source)
            pools[i].pages.grow(1)
        graphs.append(g)
    for n in range(3):
        for i, (g, s) in enumerate(zip(graphs, streams)):
            with torch.cuda.stream(s):
                g.replay()
            pools[i].model.fork([1, 0, 2])
            assert pools[i].model.grow([1, 1, 1]) == 0
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        for p in pools:
            p.check()
