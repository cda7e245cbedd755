"""Measured cases of the operators that let a sequence have several continuations over the paged 8-bit cache.

  append  q and k normed for each head, rotated by their positions (in a tree: by their depth), and
          k and v appended to the cache
  tree    attention of a tree of drafted tokens over the cache: each sees what is committed and its ancestors
  beam    beam search's selection over beams and vocabulary
  fork    beams follow their parents: page tables, counts of holders, and room for the next tokens, with
          copies of the pages that would be written by two, in every layer's cache
  accept  the accepted path of a tree moves to consecutive slots, in every layer's cache

`run` computes them with elementary torch operations, or, where `own` is set, through the
package's entry points.  `exact` computes the same results in 64 bits, sequence by sequence.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"e4m3": 448.0, "i8": 127.0}
MIN_EXP = -64  # the least exponent of a scale
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of one sequence, norms of queries and keys: batch-1 decode, a matter of latency
        dict(name="append_one", op="append", seqs=1, new=1, tree=False, length=700, spread=1, heads=8, group=4, dim=128,
             page=64, rot=128, inter=False, dtype="f32", fmt="e4m3", mix=1),
        # 12 sequences' trees of up to 16 drafted tokens, narrow heads, half of each rotated
        dict(name="append_trees", op="append", seqs=12, new=16, tree=True, length=3001, spread=6, heads=4, group=3,
             dim=64, page=32, rot=32, inter=True, dtype="f16", fmt="i8", mix=2),
        # prompts of different lengths behind some cached tokens, q, k and v in one fused row
        dict(name="append_prompts", op="append", seqs=7, new=1500, tree=False, length=2500, spread=3, heads=8, group=4,
             dim=128, page=64, rot=128, inter=False, dtype="bf16", fmt="e4m3", mix=3),
        # a tree of 15 drafted tokens early in a conversation
        dict(name="tree_one_short", op="tree", seqs=1, new=15, length=410, spread=1, heads=8, group=4, dim=128,
             page=64, window=0, dtype="f32", fmt="e4m3", mix=4),
        # a serving batch of 8, 32 drafted tokens each
        dict(name="tree_batch8", op="tree", seqs=8, new=32, length=8192, spread=6, heads=8, group=4, dim=128,
             page=64, window=0, dtype="bf16", fmt="e4m3", mix=5),
        # a wide tree of 64 against a long document
        dict(name="tree_long_i8", op="tree", seqs=1, new=64, length=100003, spread=1, heads=8, group=4, dim=128,
             page=128, window=0, dtype="bf16", fmt="i8", mix=6),
        # many sequences with a sliding window, odd trees, narrow heads, small pages
        dict(name="tree_window_odd", op="tree", seqs=24, new=25, length=6001, spread=5, heads=4, group=3, dim=64,
             page=16, window=1000, dtype="f16", fmt="e4m3", mix=7),
        # one prompt with four beams
        dict(name="beam_one", op="beam", items=1, beams=4, keep=4, vocab=32000, ended=0.0, masked=0.0, dtype="f32"),
        # 32 prompts with eight beams each, twice as many candidates kept, some beams ended, a large odd vocabulary
        dict(name="beam_batch32", op="beam", items=32, beams=8, keep=16, vocab=100003, ended=0.1, masked=0.01,
             dtype="bf16"),
        # four beams of one prompt, one layer's cache: a matter of latency
        dict(name="fork_small", op="fork", items=1, beams=4, layers=1, length=333, own=60, more=1, heads=8, dim=128,
             page=64, fmt="e4m3", mix=8),
        # two prompts with eight beams each, the caches of 32 layers
        dict(name="fork_layers", op="fork", items=2, beams=8, layers=32, length=1000, own=150, more=1, heads=8, dim=128,
             page=64, fmt="e4m3", mix=9),
        # the accepted paths of eight trees, the caches of 32 layers
        dict(name="accept_layers", op="accept", seqs=8, new=16, layers=32, length=900, spread=3, heads=8, dim=128, page=64,
             fmt="e4m3", mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "beam", "beam", "fork", "accept"])
    mix = rng.randrange(1 << 30)
    fmt, dtype = rng.choice(["e4m3", "e4m3", "i8"]), rng.choice(["f32", "f16", "bf16"])
    if op == "beam":
        beams, vocab = _log(rng, 1, 32), _log(rng, 100, 130000)
        size = 2 if dtype == "f32" else 1
        items = _log(rng, 1, max(1, min(64, 25000000 // (beams * vocab * size))))
        return dict(op=op, items=items, beams=beams, keep=rng.choice([beams, 2 * beams, _log(rng, 1, 64)]), vocab=vocab,
                    ended=rng.choice([0.0, 0.2]), masked=rng.choice([0.0, 0.02]), dtype=dtype)
    heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "fork":
        items, layers = _log(rng, 1, 4), _log(rng, 1, 32)
        beams = rng.randint(1, min(8, 16 // items))
        return dict(op=op, items=items, beams=beams, layers=layers, length=_log(rng, 1, 2000), own=_log(rng, 1, 200),
                    more=rng.choice([1, 1, 1, rng.randint(2, 40)]), heads=heads, dim=dim, page=page,
                    fmt=fmt, mix=mix)
    if op == "accept":
        new = _log(rng, 2, 64)
        return dict(op=op, seqs=_log(rng, 1, 16), new=new, layers=_log(rng, 1, 16), length=new + _log(rng, 1, 900),
                    spread=rng.randint(1, 4), heads=heads, dim=dim, page=page, fmt=fmt, mix=mix)
    group = rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        tree = rng.random() < 0.4
        new = _log(rng, 2, 64) if tree else 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        seqs = _log(rng, 1, max(1, min(64, 3000 // new)))
        return dict(op=op, seqs=seqs, new=new, tree=tree, length=new + _log(rng, 1, 4096), spread=rng.randint(1, 8),
                    heads=heads, group=min(group, 4), dim=dim, page=page, rot=rng.choice([dim, dim, dim // 2, 0]),
                    inter=rng.random() < 0.4, dtype=dtype, fmt=fmt, mix=mix)
    new = _log(rng, 2, 64)
    length = new + _log(rng, 1, 32768)
    seqs = _log(rng, 1, max(1, min(32, 2000000 // (length * new))))
    return dict(op=op, seqs=seqs, new=new, length=length, spread=rng.randint(1, 8), heads=heads, group=group, dim=dim,
                page=page, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype=dtype, fmt=fmt, mix=mix)


def _shape(case):
    """Per sequence: its new tokens and its length with them.  The first sequence has the case's own
    numbers; the others have lengths down to 1 / spread of them, and new tokens down to a half or alike."""
    r = random.Random(case["mix"])
    new, lens = [], []
    for s in range(case["seqs"]):
        f = 1.0 if s == 0 else r.uniform(1.0 / case["spread"], 1.0)
        n = case["new"] if s == 0 or case["new"] == 1 else max(1, int(case["new"] * (max(0.5, f) if case["new"] <= 64 else f)))
        new.append(n)
        lens.append(max(n, int(case["length"] * f)))
    return new, lens


def _parents(case, new):
    """Trees of drafted tokens: several first tokens, then some two continuations of each."""
    r = random.Random(case["mix"] + 1)
    trees = []
    for n in new:
        roots = max(1, min(n, r.randint(1, 4)))
        trees.append([-1 if i < roots else max(0, min(i - 1, (i - roots) // 2 + r.randint(-1, 1))) for i in range(n)])
    return trees


def _line(tree, i):
    """Token i's ancestors and itself, the first one first."""
    line = []
    while i >= 0:
        line.append(i)
        i = tree[i]
    return line[::-1]


def _leaves(case, trees):
    """The last accepted token of every tree: one of some depth, or none."""
    r = random.Random(case["mix"] + 2)
    return [max((r.randrange(len(t)) for _ in range(4)), key=lambda i: len(_line(t, i))) if r.random() > 0.1 else -1
            for t in trees]


def _seen(tree, length, window):
    """Visible (token, key) pairs of a tree's tokens, and the keys that any of them sees."""
    base = length - len(tree)
    pairs = 0
    for i in range(len(tree)):
        d = len(_line(tree, i))
        pairs += min(base + d, window) if window else base + d
    return pairs, len(tree) + (min(base, window - 1) if window else base)


def _sources(case):
    """Which beam each beam continues; a beam that is continued at all continues itself, too."""
    r = random.Random(case["mix"])
    source = []
    for i in range(case["items"]):
        stay = sorted(r.sample(range(case["beams"]), max(1, round(case["beams"] * 0.4))))
        source += [i * case["beams"] + (b if b in stay else r.choice(stay)) for b in range(case["beams"])]
    return source


def work(case):
    op = case["op"]
    if op == "beam":
        n = case["items"] * case["beams"] * case["vocab"]
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + 12 * case["items"] * case["keep"], "flops": 4 * n}
    row = case["heads"] * case["dim"]
    if op == "fork":
        seqs = case["items"] * case["beams"]
        part = (case["length"] + case["own"]) % case["page"]
        copies = seqs - len(set(_sources(case))) if part else 0
        return {"bytes": 4 * copies * part * row * case["layers"] + 8 * seqs * (_columns(case) + 2), "flops": 0}
    new, lens = _shape(case)
    if op == "accept":
        trees = _parents(case, new)
        moved = sum(sum(a != i for i, a in enumerate(_line(t, f))) for t, f in zip(trees, _leaves(case, trees)))
        return {"bytes": 4 * moved * row * case["layers"] + 12 * sum(new), "flops": 0}
    size = DTYPES[case["dtype"]].itemsize
    if op == "append":
        n = sum(new)
        b = n * (2 * row * case["group"] * size + 2 * row * (size + 1) + 4 * case["rot"])
        return {"bytes": b, "flops": 7 * n * (case["group"] + 1) * row + 2 * n * row}
    seen = [_seen(t, n, case["window"]) for t, n in zip(_parents(case, new), lens)]
    b = sum(k for _, k in seen) * 2 * row + sum(new) * 2 * row * case["group"] * size
    return {"bytes": b, "flops": 4 * sum(p for p, _ in seen) * row * case["group"]}


# ------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e in 64 bits, exactly, for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rne(x, fmt):
    """x in 64 bits -> the nearest value of the 8-bit format, ties to even; |x| is within its range."""
    if fmt == "i8":
        return torch.round(x)
    e = torch.frexp(x)[1].clamp(min=-5) - 4  # e4m3: 3 fraction bits, the least exponent of 2 is -6
    return torch.round(x * _pow2(-e)) * _pow2(e)


def _encode(x, fmt):
    """Codes of the nearest values of the format."""
    x = _rne(x, fmt)
    return x.to(torch.int8).view(torch.uint8) if fmt == "i8" else x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return codes.view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn).float()


def _scale_of(amax, fmt):
    """The least power of two 2^e, e >= MIN_EXP, with amax <= QMAX * 2^e (amax in 64 bits)."""
    e = torch.frexp(amax / QMAX[fmt])[1]
    e = torch.where(amax <= QMAX[fmt] * _pow2(e - 1), e - 1, e)
    return _pow2(torch.where(amax == 0, MIN_EXP, e).clamp(min=MIN_EXP))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(case, lens, g, spare=3):
    """Pages of every sequence, in a shuffled pool with some pages to spare."""
    counts = [-(-t // case["page"]) for t in lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c]
        at += c
    return pages, table


def _columns(case):
    return -(-(case["length"] + case["own"] + case["more"]) // case["page"]) + 1


def _shared_pages(case, g):
    """Beams of some prompts: the prompts' full pages shared by their beams, the others a beam's own."""
    seqs, T = case["items"] * case["beams"], case["page"]
    both = case["length"] // T
    mine = -(-(case["length"] + case["own"]) // T) - both
    pages = case["items"] * both + seqs * (mine + 1 + -(-case["more"] // T)) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((seqs, _columns(case)), -1, dtype=torch.int32, device="cuda")
    table[:, :both] = order[:case["items"] * both].view(case["items"], both).repeat_interleave(case["beams"], 0)
    table[:, both:both + mine] = order[case["items"] * both:case["items"] * both + seqs * mine].view(seqs, mine)
    return pages, table


def _random_codes(shape, fmt, g):
    """Codes as uniform as they can be for the format, no NaN among them."""
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    return torch.where(c & 127 == 127, 3, c) if fmt == "e4m3" else torch.where(c == 128, 3, c)


def _cache(case, g, pages, fmt):
    """Codes and scales of pages of normal values, keys with some strong channels."""
    shape = (pages, case["heads"], case["page"], case["dim"])
    chan = torch.where(torch.rand(case["heads"], 1, case["dim"], generator=g, device="cuda") < 0.05, 5.0, 1.0)
    out = []
    for spread in (chan, 0.5):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty(shape[:2], dtype=torch.float32, device="cuda")
        step = max(1, (1 << 25) // (shape[1] * shape[2] * shape[3]))
        for p in range(0, pages, step):
            x = torch.randn((min(step, pages - p),) + shape[1:], generator=g, device="cuda") * spread
            scale = _scale_of(x.abs().amax((2, 3)).double(), fmt).float()
            y = x / scale[:, :, None, None]
            codes[p:p + step] = torch.round(y).to(torch.int8).view(torch.uint8) if fmt == "i8" else \
                y.to(torch.float8_e4m3fn).view(torch.uint8)
            scales[p:p + step] = scale
        out += [codes, scales]
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    s, op = dict(case=case), case["op"]
    if op == "beam":
        n, b, v = case["items"], case["beams"], case["vocab"]
        x = rand(n * b, v) * 2.5
        if case["masked"]:  # tokens that are forbidden
            x.masked_fill_(torch.rand(v, generator=g, device="cuda") < case["masked"], -math.inf)
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["scores"] = -12.0 + 1.5 * rand(n, b)
        s["ended"] = torch.rand(n, b, generator=g, device="cuda") < case["ended"]
        return s
    dt = DTYPES.get(case.get("dtype"))
    fmt, h, d = case["fmt"], case["heads"], case["dim"]
    if op == "fork":
        n = case["items"] * case["beams"]
        pages, s["table"] = _shared_pages(case, g)
        s["lens"] = _ints([case["length"] + case["own"]] * n)
        s["keep"], s["source"] = s["lens"].clone(), _ints(_sources(case))
        s["refs"] = torch.bincount(s["table"].flatten() + 1, minlength=pages + 1)[1:].to(torch.int32)
    else:
        new, lens = _shape(case)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        pages, s["table"] = _pages(case, lens, g)
        s["lens"], s["starts"], s["max_new"] = _ints(lens), _ints(starts), max(new)
        s["parents"] = None
        if case.get("tree", True):
            s["parents"] = _ints([p for t in _parents(case, new) for p in t])
    if op in ("fork", "accept"):
        for c in "kv":
            s[c] = _random_codes((case["layers"], pages, h, case["page"], d), fmt, g)
            e = torch.randint(-8, -3, (case["layers"], pages, h), generator=g, device="cuda")
            s[c + "s"] = _pow2(e).float()
        if op == "accept":
            s["leaf"] = _ints(_leaves(case, _parents(case, new)))
            s["now"] = torch.zeros_like(s["lens"])
    else:
        s["k"], s["ks"], s["v"], s["vs"] = _cache(case, g, pages, fmt)
    n = starts[-1] if op != "fork" else 0
    if op == "append":
        # one fused row a token: the query heads, the key heads, the value heads
        s["qkv"] = (rand(n, h * case["group"] + 2 * h, d) * (1.0 + rand(n, 1, 1).abs())).to(dt)
        s["q_norm"], s["k_norm"] = (1.0 + 0.2 * rand(d)).to(dt), (1.0 + 0.2 * rand(d)).to(dt)
        rows, rot = s["table"].shape[1] * case["page"], case["rot"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    elif op == "tree":
        s["q"] = (rand(n, h * case["group"], d) * 1.5).to(dt)
    if own:
        import dynamic_sparsity_approximate_amd as E
        f = E.EFFORT_KV_I8 if fmt == "i8" else E.EFFORT_KV_E4M3
        if op in ("fork", "accept"):
            s["caches"] = [E.KVCache.wrap(s["k"][i], s["v"][i], s["ks"][i], s["vs"][i], f) for i in range(case["layers"])]
        else:
            s["cache"] = E.KVCache.wrap(s["k"], s["v"], s["ks"], s["vs"], f)
        if op == "fork":
            s["pages"] = E.KVPages(s["caches"], s["table"], s["lens"], refs=s["refs"])
        else:
            s["batch"] = E.KVBatch(s["table"], s["lens"], s["starts"], parents=s["parents"])
    return s


# ------------------------------------------------------------------ one pass

def _lines(s):
    """[seqs][new][new]: whether token j is token i or its ancestor, and every token's depth."""
    n, starts = s["max_new"], s["starts"].long()
    i = torch.arange(n, device="cuda")
    rows = starts[:-1, None] + i
    one = torch.eye(n, device="cuda")
    at = s["parents"].long()[rows.clamp(max=len(s["parents"]) - 1)]
    up = ((at[..., None] == i) & (rows < starts[1:, None])[..., None]).float()  # to the parent
    # one + up + up^2 + ...: a tree of 64 tokens is at most 64 deep
    up2 = up @ up
    up4 = up2 @ up2
    up8 = up4 @ up4
    up16 = up8 @ up8
    lines = (one + up) @ (one + up2) @ (one + up4) @ (one + up8) @ (one + up16) @ (one + up16 @ up16)
    return lines > 0.5, lines.sum(-1).long() - 1


def _where(s, tokens):
    """Sequence of every new token, its number in it, and the position of the sequence's first one."""
    starts = s["starts"].long()
    tok = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(starts[1:], tok, right=True)
    return seq, tok - starts[:-1][seq], (s["lens"].long() - starts[1:] + starts[:-1])[seq]


def _normed(x, w):
    """Each head of x [tokens][heads][dim] normed, in 64 bits."""
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()


def _rotate(x, pos, table, inter):
    """x in 64 bits, [tokens][heads][dim]: its leading dimensions rotated."""
    half = table.shape[1]
    c, sn = table[pos].double()[:, None].unbind(-1)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    y = (a * c - b * sn, b * c + a * sn)
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _store(codes, scales, x, s, page, slot, fmt):
    """Appends x (64 bits, [tokens][heads][dim]) to codes and scales in place."""
    T = codes.shape[2]
    zero = torch.zeros(scales.shape, dtype=torch.float64, device="cuda")
    amax = zero.scatter_reduce(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill(0, page, True)
    fresh = torch.zeros_like(touched).index_put((page,), slot == 0, accumulate=True)
    old = scales.double()
    new = _scale_of(amax, fmt)
    new = torch.where(fresh[:, None], new, torch.maximum(new, old))
    new = torch.where(touched[:, None], new, old)
    # only the page of a sequence's first new token holds older rows
    head = s["starts"][:-1].long()
    part, keep = page[head], torch.arange(T, device="cuda")[None, None, :, None] < slot[head][:, None, None, None]
    was = codes[part]
    ratio = (old[part] / new[part])[:, :, None, None]
    codes[part] = torch.where(keep, _encode(_decode(was, fmt).double() * ratio, fmt), was)
    codes[page, :, slot] = _encode(x / new[page][..., None], fmt)
    scales.copy_(new)


def _stored(s):
    """The caches' codes as the values that they stand for, and their scales."""
    t = torch.int8 if s["case"]["fmt"] == "i8" else torch.float8_e4m3fn
    return {"k": s["k"].view(t), "v": s["v"].view(t), "k_scale": s["ks"], "v_scale": s["vs"]}


def _append(s):
    case = s["case"]
    h, fmt = case["heads"], case["fmt"]
    q, k, v = s["qkv"].split([h * case["group"], h, h], 1)
    if own:
        q = s["cache"].append(s["batch"], k, v, q=q, rope=s["rope"] if case["rot"] else None, interleaved=case["inter"],
                              q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    else:
        seq, i, base = _where(s, len(q))
        at = base + (i if s["parents"] is None else _lines(s)[1][seq, i])
        slot = base + i
        page, slot = s["table"][seq, slot // case["page"]].long(), slot % case["page"]
        k = _rotate(_normed(k, s["k_norm"]), at, s["rope"], case["inter"])
        q = _rotate(_normed(q, s["q_norm"]), at, s["rope"], case["inter"]).to(q.dtype)
        _store(s["k"], s["ks"], k, s, page, slot, fmt)
        _store(s["v"], s["vs"], v.double(), s, page, slot, fmt)
    return dict(_stored(s), q=q)


def _read(codes, scales, s, live):
    """Every sequence's tokens of the cache in 32 bits, [seqs][heads][tokens][dim], 0 behind its end."""
    table = s["table"].long()
    x = _decode(codes[table], s["case"]["fmt"]) * scales[table][..., None, None]
    x = x.transpose(1, 2).flatten(2, 3)
    return torch.where(live[:, None, :, None], x, 0.0)


def _tree(s):
    case, q = s["case"], s["q"]
    if own:
        return s["cache"].attend(s["batch"], q, window=case["window"])
    h, g, d, n = case["heads"], case["group"], case["dim"], s["max_new"]
    lens, starts = s["lens"].long(), s["starts"].long()
    t = torch.arange(s["table"].shape[1] * case["page"], device="cuda")
    live = t < lens[:, None]
    keys, vals = _read(s["k"], s["ks"], s, live), _read(s["v"], s["vs"], s, live)
    rows = (starts[:-1, None] + torch.arange(n, device="cuda")).clamp(max=len(q) - 1)
    x = q[rows].float().unflatten(2, (h, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs][heads][group * n][dim]
    lines, depth = _lines(s)
    base = (lens - starts[1:] + starts[:-1])[:, None]
    j = t - base  # the new token that each cached one is
    seen = lines.gather(2, j.clamp(0, n - 1)[:, None].expand(-1, n, -1)) & (j >= 0)[:, None] | (j < 0)[:, None]
    if case["window"]:
        # by depth: a committed token's is its distance in front of the new ones
        at = torch.where(j < 0, j, depth.gather(1, j.clamp(0, n - 1)))
        seen = seen & (at[:, None] > depth[..., None] - case["window"])
    seen = seen & live[:, None]
    score = (x @ keys.transpose(2, 3) / math.sqrt(d)).unflatten(2, (g, n))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3.0e38)
    score = score.sub_(top).exp_()
    out = (score.flatten(2, 3) @ vals).unflatten(2, (g, n)) / score.sum(-1, keepdim=True).clamp(min=1e-38)
    seq, i, _ = _where(s, len(q))
    return out.permute(0, 3, 1, 2, 4)[seq, i].flatten(1, 2).to(q.dtype)


def _beam(s):
    case, x, scores = s["case"], s["logits"], s["scores"]
    if own:
        import dynamic_sparsity_approximate_amd as E
        scores, parents, tokens = E.beam_select(x, scores, keep=case["keep"], ended=s["ended"], end_token=2)
        return {"scores": scores, "parents": parents, "tokens": tokens}
    n, b, v, keep = case["items"], case["beams"], case["vocab"], case["keep"]
    # a row's best: its logits in order as whole numbers, above the order of its tokens
    bits = (x.float() + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32 | (0xFFFFFFFF - torch.arange(v, device="cuda"))
    few = min(keep, v)
    tok = 0xFFFFFFFF - (key.topk(few, -1)[0] & 0xFFFFFFFF)
    y = x.double()
    top = y.amax(-1, keepdim=True)
    y = y.gather(1, tok) - ((y - top).exp().sum(-1, keepdim=True).log() + top)
    y = y.view(n, b, few) + scores.double()[..., None]
    tok = tok.view(n, b, few)
    # an ended beam is its own only continuation
    first = torch.arange(few, device="cuda") == 0
    stay = torch.where(first, scores.double()[..., None], -math.inf)
    y = torch.where(s["ended"][..., None], stay, y)
    tok = torch.where(s["ended"][..., None], 2, tok)
    y, at = torch.nn.functional.pad(y.flatten(1), (0, max(0, keep - b * few)), value=-math.inf).sort(
        dim=-1, descending=True, stable=True)
    y, at = y[:, :keep], at[:, :keep].clamp(max=b * few - 1)
    there = y > -math.inf
    parents = torch.where(there, at // few + b * torch.arange(n, device="cuda")[:, None], -1)
    tokens = torch.where(there, tok.flatten(1).gather(1, at), -1)
    return {"scores": y.float(), "parents": parents.int(), "tokens": tokens.int()}


def _holders(table, pages):
    """How many of the table's entries hold each page."""
    t = (table + 1).flatten()
    return torch.zeros(pages + 1, dtype=torch.long, device="cuda").scatter_add(0, t, torch.ones_like(t))[1:]


def _fork(s):
    case, T, pages = s["case"], s["case"]["page"], s["k"].shape[1]
    if own:
        s["pages"].fork(s["source"], lens=s["keep"])
        s["pages"].grow(case["more"])
    else:
        source = s["source"].long()
        lens = torch.minimum(s["keep"], s["lens"][source]).long()
        col, n = torch.arange(s["table"].shape[1], device="cuda"), len(source)
        table = torch.where(col < ((lens + T - 1) // T)[:, None], s["table"].long()[source], -1)
        refs = _holders(table, pages)
        # the pages that receive the next tokens; the first of them may hold older ones
        first, last, part = lens // T, (lens + case["more"] - 1) // T, lens % T
        page = torch.where(part > 0, table.gather(1, first[:, None])[:, 0], -1)
        same = (page[:, None] == page) & (page >= 0)
        held = torch.where(page >= 0, refs[page.clamp(min=0)], 0)
        i = torch.arange(n, device="cuda")
        keeps = (same.sum(1) == held) & ~(same & (i > i[:, None])).any(1)  # the last of them writes the page itself
        copy = (held > 1) & ~keeps
        needs = (col >= first[:, None]) & (col <= last[:, None]) & (table < 0) | copy[:, None] & (col == first[:, None])
        free = torch.sort((refs > 0).int(), stable=True)[1]
        table = torch.where(needs, free[(needs.flatten().cumsum(0) - 1).clamp(min=0)].view_as(table), table)
        to = table.gather(1, first[:, None])[:, 0]
        # those that copy nothing do what the first that copies does
        j = torch.where(copy, i, copy.int().argmax())
        src, dst = torch.where(copy, page, to)[j], to[j]
        old = (torch.arange(T, device="cuda") < part[j, None])[None, :, None, :, None]
        for c in "kv":
            s[c][:, dst] = torch.where(old, s[c][:, src], s[c][:, dst])
            s[c + "s"][:, dst] = s[c + "s"][:, src]
        s["table"].copy_(table)
        s["lens"].copy_(lens + case["more"])
        s["refs"].copy_(_holders(table, pages))
    return dict(_stored(s), table=s["table"], lens=s["lens"], refs=s["refs"])


def _accept(s):
    case, fmt = s["case"], s["case"]["fmt"]
    if own:
        import dynamic_sparsity_approximate_amd as E
        E.kv_accept(s["caches"], s["batch"], s["leaf"], lens_out=s["now"])
        return dict(_stored(s), lens=s["now"])
    T, n = case["page"], s["max_new"]
    leaf, starts = s["leaf"].long(), s["starts"].long()
    base = s["lens"].long() - starts[1:] + starts[:-1]
    lines = _lines(s)[0]
    i = torch.arange(n, device="cuda")
    on = lines.gather(1, leaf.clamp(min=0)[:, None, None].expand(-1, 1, n))[:, 0] & (leaf >= 0)[:, None]  # [seqs][n]
    count = on.sum(1)
    # those that are not on the path do what its first token does, or nothing at the first slot
    j = torch.where(on, i, on.int().argmax(1)[:, None])
    k = torch.where(on, on.cumsum(1) - 1, 0)
    seq = torch.arange(len(leaf), device="cuda")[:, None]
    table = s["table"].long()
    src, dst = (base[:, None] + j).flatten(), (base[:, None] + k).flatten()
    seq = seq.expand(-1, n).flatten()
    p0, s0, p1, s1 = table[seq, src // T], src % T, table[seq, dst // T], dst % T
    part, slot = table[seq[::n], base // T], base % T
    keep = (torch.arange(T, device="cuda") < slot[:, None])[None, :, None, :, None]
    for c in "kv":
        codes, scales = s[c], s[c + "s"]
        old = scales.double()
        x = _decode(codes[:, p0, :, s0], fmt).double().transpose(0, 1) * old[:, p0][..., None]  # [layers][tokens][heads][dim]
        amax = torch.where((p0 != p1)[:, None], x.abs().amax(-1), 0.0)
        amax = torch.zeros_like(old).scatter_reduce(1, p1[:, None].expand(len(old), -1, old.shape[2]), amax, "amax")
        now = torch.where(amax > 0, torch.maximum(old, _scale_of(amax, fmt)), old)
        was = codes[:, part]
        ratio = (old[:, part] / now[:, part])[..., None, None]
        codes[:, part] = torch.where(keep, _encode(_decode(was, fmt).double() * ratio, fmt), was)
        codes[:, p1, :, s1] = _encode(x / now[:, p1][..., None], fmt).transpose(0, 1)
        scales.copy_(now)
    s["now"].copy_(base + count)
    return dict(_stored(s), lens=s["now"])


def run(state):
    return {"append": _append, "tree": _tree, "beam": _beam, "fork": _fork, "accept": _accept}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

_E4M3 = None


def _grid():
    """The non-negative e4m3 values in order, from the format's definition."""
    global _E4M3
    if _E4M3 is None:
        v = [m * 2.0 ** -9 for m in range(8)]
        v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
        _E4M3 = torch.tensor(v[:127], dtype=torch.float64, device="cuda")
    return _E4M3


def _nearest(x, fmt):
    """The nearest value of the format; a tie goes to the even code."""
    if fmt == "i8":
        low = torch.floor(x)
        up = (x - low > 0.5) | ((x - low == 0.5) & (low % 2 != 0))
        return low + up.double()
    grid = _grid()
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(up == 0, hi, pick)
    return torch.copysign(grid[pick], x)


def _values(codes, fmt):
    c = codes.long()
    if fmt == "i8":
        return ((c + 128) % 256 - 128).double()
    side = torch.cat([_grid(), _grid().new_full((1,), math.nan)])
    return torch.where(c >= 128, -1.0, 1.0).double() * side[c & 127]


def _need(top, fmt):
    """The least power of two, at least 2^MIN_EXP, that takes `top`; on the host, where powers are exact."""
    need = (2.0 ** torch.ceil(torch.log2(top.cpu() / QMAX[fmt])).clamp(min=MIN_EXP)).to(top.device)
    need = torch.where(top > QMAX[fmt] * need, 2 * need, need)
    return torch.where((need > 2.0 ** MIN_EXP) & (top <= QMAX[fmt] * need / 2), need / 2, need)


def _exact_append(s):
    case = s["case"]
    h, T, fmt, rope = case["heads"], case["page"], case["fmt"], s["rope"].double()
    new, lens = _shape(case)
    trees = _parents(case, new) if case["tree"] else None
    out, vals, q_out, at = {}, {}, [], 0
    for name in "kv":
        vals[name] = _values(s[name], fmt)
        out[name + "_scale"] = s[name + "s"].double()
    half = rope.shape[1]
    first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)
    for i, (n, t) in enumerate(zip(new, lens)):
        x = s["qkv"][at:at + n].double()
        at += n
        for part, w in ((slice(0, h * case["group"]), s["q_norm"]), (slice(h * case["group"], -h), s["k_norm"])):
            y = x[:, part]
            x[:, part] = y * w.double() / torch.sqrt((y ** 2).sum(-1, keepdim=True) / case["dim"] + EPS)
        pos = [t - n + (len(_line(trees[i], j)) - 1 if trees else j) for j in range(n)]
        c, sn = rope[pos][:, None, :, 0], rope[pos][:, None, :, 1]
        y = x.clone()
        y[..., first] = x[..., first] * c - x[..., second] * sn
        y[..., second] = x[..., second] * c + x[..., first] * sn
        q_out.append(y[:, :-2 * h])
        for name, rows in (("k", y[:, -2 * h:-h]), ("v", x[:, -h:])):
            p = t - n
            while p < t:
                page, slot = int(s["table"][i, p // T]), p % T
                m = min(T - slot, t - p)
                part = rows[p - (t - n):p - (t - n) + m].transpose(0, 1)  # [heads][m][dim]
                need = _need(part.abs().amax((1, 2)), fmt)
                was = out[name + "_scale"][page].clone()
                now = need if slot == 0 else torch.maximum(need, was)
                if slot:
                    vals[name][page, :, :slot] = _nearest(vals[name][page, :, :slot] * (was / now)[:, None, None], fmt)
                vals[name][page, :, slot:slot + m] = _nearest(part / now[:, None, None], fmt)
                out[name + "_scale"][page] = now
                p += m
    out["q"] = torch.cat(q_out)
    return dict(out, **_whole(vals, fmt))


def _whole(vals, fmt):
    """Integers as such, e4m3 numbers in 64 bits."""
    return {c: v.to(torch.int8) if fmt == "i8" else v for c, v in vals.items()}


def _exact_tree(s):
    case, q = s["case"], s["q"].double()
    h, g, d, T = case["heads"], case["group"], case["dim"], case["page"]
    new, lens = _shape(case)
    out, at = [], 0
    for i, (tree, t) in enumerate(zip(_parents(case, new), lens)):
        n = len(tree)
        pages = s["table"][i, :-(-t // T)].long()
        kv = []
        for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = _values(codes[pages], case["fmt"]) * scales[pages].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(h, -1, d)[:, :t])
        rows = q[at:at + n].reshape(n, h, g, d)
        at += n
        hide = torch.ones(n, t, dtype=torch.bool)
        for j in range(n):
            line = _line(tree, j)
            see = list(range(t - n)) + [t - n + a for a in line]
            hide[j, see[-case["window"]:] if case["window"] else see] = False
        hide = hide.to(q.device)
        y = torch.empty_like(rows)
        for head in range(h):
            score = rows[:, head].transpose(0, 1) @ kv[0][head].t().contiguous() * d ** -0.5  # [group][n][tokens]
            y[:, head] = (torch.softmax(score.masked_fill(hide, -math.inf), -1) @ kv[1][head]).transpose(0, 1)
        out.append(y.reshape(n, h * g, d))
    return torch.cat(out)


def _exact_beam(s):
    case = s["case"]
    out = {"scores": [], "parents": [], "tokens": []}
    for i in range(case["items"]):
        found = []
        for b in range(case["beams"]):
            r = i * case["beams"] + b
            score = float(s["scores"][i, b])
            if bool(s["ended"][i, b]):
                found.append((-score, b, 0.0, 2, r))
                continue
            x = s["logits"][r].double()
            least = x.sort(descending=True)[0][min(case["keep"], len(x)) - 1]
            lse = float(torch.logsumexp(x, 0))
            for t in (x >= least).nonzero()[:, 0].tolist():
                y = float(x[t])
                if y > -math.inf:
                    found.append((-(score + (y - lse)), b, -y, t, r))
        found = sorted(found)[:case["keep"]]
        found += [(math.inf, 0, 0.0, -1, -1)] * (case["keep"] - len(found))
        out["scores"].append([-f[0] for f in found])
        out["parents"].append([f[4] for f in found])
        out["tokens"].append([f[3] for f in found])
    return {"scores": torch.tensor(out["scores"], dtype=torch.float64), "parents": torch.tensor(out["parents"], dtype=torch.int32),
            "tokens": torch.tensor(out["tokens"], dtype=torch.int32)}


def _exact_fork(s):
    case, T = s["case"], s["case"]["page"]
    old, had = s["table"].tolist(), s["lens"].tolist()
    pages, width = s["k"].shape[1], len(old[0])
    table, lens = [], []
    for src, most in zip(s["source"].tolist(), s["keep"].tolist()):
        lens.append(min(most, had[src]))
        table.append([p if c * T < lens[-1] else -1 for c, p in enumerate(old[src])])
    refs = [0] * pages
    for p in (p for row in table for p in row if p >= 0):
        refs[p] += 1
    vals = {c: _values(s[c], case["fmt"]) for c in "kv"}
    scales = {c: s[c + "s"].double() for c in "kv"}
    free = iter([p for p in range(pages) if refs[p] == 0])
    for i, t in enumerate(lens):
        for c in range(t // T, -(-(t + case["more"]) // T)):
            p = table[i][c]
            if p < 0:
                table[i][c] = next(free)
            elif refs[p] > 1:
                table[i][c] = q = next(free)
                refs[p] -= 1
                for x in "kv":
                    vals[x][:, q, :, :t % T] = vals[x][:, p, :, :t % T]
                    scales[x][:, q] = scales[x][:, p]
        lens[i] = t + case["more"]
    refs = [0] * pages
    for p in (p for row in table for p in row if p >= 0):
        refs[p] += 1
    ints = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(_whole(vals, case["fmt"]), k_scale=scales["k"], v_scale=scales["v"], table=ints(table).view(-1, width),
                lens=ints(lens), refs=ints(refs))


def _exact_accept(s):
    case, T, fmt = s["case"], s["case"]["page"], s["case"]["fmt"]
    new, lens = _shape(case)
    trees = _parents(case, new)
    vals = {c: _values(s[c], fmt) for c in "kv"}
    scales = {c: s[c + "s"].double() for c in "kv"}
    now = []
    for i, (tree, t, leaf) in enumerate(zip(trees, lens, _leaves(case, trees))):
        base, line = t - len(tree), _line(tree, leaf)
        now.append(base + len(line))
        at = lambda x: (int(s["table"][i, x // T]), x % T)  # noqa: B023,E731
        for c in "kv":
            v, sc = vals[c], scales[c]
            was = [v[:, p, :, k] * sc[:, p, :, None] for p, k in (at(base + a) for a in line)]
            had = sc.clone()
            for k, a in enumerate(line):
                p = at(base + k)[0]
                if at(base + a)[0] != p:
                    top = was[k].abs().amax(-1)
                    sc[:, p] = torch.where(top > 0, torch.maximum(sc[:, p], _need(top, fmt)), sc[:, p])
            p, slot = at(base)
            if slot and line:
                v[:, p, :, :slot] = _nearest(v[:, p, :, :slot] * (had[:, p] / sc[:, p])[..., None, None], fmt)
            for k, x in enumerate(was):
                p, slot = at(base + k)
                v[:, p, :, slot] = _nearest(x / sc[:, p, :, None], fmt)
    return dict(_whole(vals, fmt), k_scale=scales["k"], v_scale=scales["v"], lens=torch.tensor(now, dtype=torch.int32))


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "beam": _exact_beam, "fork": _exact_fork,
            "accept": _exact_accept}[case["op"]](s)
