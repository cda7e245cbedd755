"""Chains of approximate matvecs on one stream.

The Effort method is applied per weight matrix with a per-call effort (Show HN
thread "Speeding up LLM inference 2x times (possibly)": effort is a real-time
knob; the author runs Mistral and Mixtral through it).  These classes only
sequence calls into libeffort and own the intermediate buffers; every step of
the arithmetic, the glue included (silu(h1) * h3, the gated expert sum), runs
in the library's kernels.  A caller that repeats a chain captures `enqueue`
into a HIP graph.  DecodeStep takes the attention's results from outside;
DecoderStep runs whole layers over a paged cache, BeamStep a beam search of them.
"""
from __future__ import annotations

import math

from . import binding as B

LAYER_ROLES = ("wq", "wk", "wv", "wo", "w1", "w3", "w2")


class EffortSchedule:
    """An effort for every matrix of a chain instead of one for all: the
    author's reply in the HN thread likens effort to an equalizer with a
    setting per layer, token and matrix rather than one knob; the reply to
    uhlo counts roughly 32 * 6 separate knobs per decode step.

    Keys are (layer, role) in a decode step (the head is (None, "head")) and
    (expert, role) in an expert block.  Lookup order: (unit, role), then
    (None, role) (a role's effort in every unit), then (unit, None) (a unit's
    effort for every role), then `default`.  Every effort must lie in (0, 1].
    """

    def __init__(self, default: float, table=None):
        self.default = float(default)
        self.table = {k: float(e) for k, e in dict(table or {}).items()}
        for k, e in [("default", self.default)] + list(self.table.items()):
            if not (0.0 < e <= 1.0):
                raise ValueError("effort %r for %r is outside (0, 1]" % (e, k))

    def __call__(self, unit, role) -> float:
        t = self.table
        for k in ((unit, role), (None, role), (unit, None)):
            if k in t:
                return t[k]
        return self.default

    @classmethod
    def from_array(cls, efforts, roles=LAYER_ROLES, head=None, default=None):
        """efforts[l][k] is the effort of roles[k] in layer l; `head` the output
        head's (default: the mean of the table)."""
        table = {}
        flat = []
        for l, row in enumerate(efforts):
            if len(row) != len(roles):
                raise ValueError("layer %d: %d efforts for %d roles" % (l, len(row), len(roles)))
            for r, e in zip(roles, row):
                table[(l, r)] = float(e)
                flat.append(float(e))
        mean = sum(flat) / len(flat) if flat else 1.0
        table[(None, "head")] = float(head) if head is not None else mean
        return cls(default if default is not None else mean, table)


def _effort_of(effort, unit, role) -> float:
    return float(effort(unit, role)) if callable(effort) else float(effort)


class DecodeStep:
    """All matvecs of one decode step of a decoder stack.

    `layers` is a list of dicts role -> EffortMatrix with the roles of
    LAYER_ROLES; `head` is the output projection.  Per layer l: wq, wk, wv, w1
    and w3 multiply the layer input x[l]; wo multiplies a[l] (attention, which
    produces wo's input, is outside this path); w2 multiplies silu(h1) * h3,
    formed from the approximate outputs h1 = x W1 and h3 = x W3.  The head
    multiplies `head_in`.  Inputs are device fp32 vectors supplied by the caller.
    With `grouped`, the matrices of a layer that share x go through one
    multi-matrix call each: (wq, wk, wv) and (w1, w3).
    """

    def __init__(self, layers, head, x, a, head_in, grouped: bool = False):
        import torch

        from .device import EffortGroup

        if len(layers) != len(x) or len(layers) != len(a):
            raise ValueError("one x and one a vector per layer")
        self.layers, self.head = layers, head
        self.x, self.a, self.head_in = x, a, head_in
        dev = head_in.device
        self.out = []
        for L in layers:
            o = {r: torch.empty(L[r].out_dim, dtype=torch.float32, device=dev) for r in LAYER_ROLES}
            o["g"] = torch.empty(L["w1"].out_dim, dtype=torch.float32, device=dev)
            self.out.append(o)
        self.logits = torch.empty(head.out_dim, dtype=torch.float32, device=dev)
        self.calls = 7 * len(layers) + 1
        self.groups = ([(EffortGroup([L["wq"], L["wk"], L["wv"]]), EffortGroup([L["w1"], L["w3"]]))
                        for L in layers] if grouped else None)

    def inputs_of(self, l: int) -> dict:
        """role -> the device vector that role's matvec multiplies in layer l."""
        o = self.out[l]
        return {"wq": self.x[l], "wk": self.x[l], "wv": self.x[l], "wo": self.a[l], "w1": self.x[l],
                "w3": self.x[l], "w2": o["g"]}

    def enqueue(self, effort, stream=None, side_streams=None, record=None):
        """Issue every call on `stream` (None: torch's current stream).
        `effort` is one effort for every matrix or an EffortSchedule (per
        layer and role; the head is (None, "head")).  With `side_streams`
        (torch streams), the six matvecs of a layer that do not depend on each
        other run on separate streams (parallel branches when captured into a
        graph); w2 and the next layer wait for them.  With `record` (a
        Recorder), every matvec records its parity outputs under (layer,
        role), the head under (None, "head")."""
        import torch

        main = stream if stream is not None else torch.cuda.current_stream()
        rk = (lambda key: None) if record is None else (lambda key: (record, key))  # noqa: E731
        for l, L in enumerate(self.layers):
            o, ins = self.out[l], self.inputs_of(l)
            roles = ("wq", "wk", "wv", "wo", "w1", "w3")
            e = {r: _effort_of(effort, l, r) for r in LAYER_ROLES}
            if self.groups:
                qkv, gu = self.groups[l]
                side = list(side_streams[:2]) if side_streams else []
                s_qkv = side[0] if side else main
                s_o = side[-1] if side else main
                for ss in side:
                    ss.wait_stream(main)
                qkv.matvec(self.x[l], [e["wq"], e["wk"], e["wv"]], [o["wq"], o["wk"], o["wv"]], s_qkv,
                           record=None if record is None else
                           (record, [(l, "wq"), (l, "wk"), (l, "wv")]))
                L["wo"].matvec(ins["wo"], e["wo"], o["wo"], s_o, record=rk((l, "wo")))
                gu.matvec(self.x[l], [e["w1"], e["w3"]], [o["w1"], o["w3"]], main,
                          record=None if record is None else (record, [(l, "w1"), (l, "w3")]))
                for ss in side:
                    main.wait_stream(ss)
            elif side_streams:
                for k, r in enumerate(roles):
                    ss = side_streams[k % len(side_streams)]
                    ss.wait_stream(main)
                    L[r].matvec(ins[r], e[r], o[r], ss, record=rk((l, r)))
                for ss in side_streams[:len(roles)]:
                    main.wait_stream(ss)
            else:
                for r in roles:
                    L[r].matvec(ins[r], e[r], o[r], main, record=rk((l, r)))
            B.effort_silu_mul(o["w1"], o["w3"], L["w1"].out_dim, o["g"], main)
            L["w2"].matvec(o["g"], e["w2"], o["w2"], main, record=rk((l, "w2")))
        self.head.matvec(self.head_in, _effort_of(effort, None, "head"), self.logits, main,
                         record=rk((None, "head")))


class DecoderStep:
    """One step of whole decoder layers for the new tokens of a batch of
    sequences (a KVBatch): attention over the paged 8-bit cache included, so
    that nothing but the embeddings comes from outside.

    `layers` is a list of dicts role -> EffortMatrix with the roles of
    LAYER_ROLES, `head` the output projection, `caches` one KVCache per layer,
    `norms` one (before attention, before the feed-forward block) pair of norm
    weights per layer and `head_norm` the one before the head.  `x` [tokens][dim]
    holds the embeddings of the new tokens in the order of the batch, `rope` is a
    table of rope_table (None: no rotation), `qk_norms` one pair of weights per
    layer (each [head_dim], one row per head, or None) with which every head of q
    and k is normed before its rotation.  Per layer, with the residual stream r
    (r = x at first):
      h = norm(r); q, k, v = h Wq, h Wk, h Wv; k and v appended, q and k rotated
      r += attend(q) Wo; h = norm(r); r += (silu(h W1) * h W3) W2
    and logits = norm(r) Whead.  `out[l]` keeps what layer l computed.  A matrix
    needs `batch` >= tokens; a single row goes through the multi-matrix calls.

    A batch with parents takes trees of drafted tokens: row by row the logits
    behind each token's own line.  BeamStep makes a beam search of the step.

    The kernels read x, the page table, the lengths and the starts at every
    step: a captured step is replayed after the caller has updated them in
    place.  Rows that no sequence has do not touch the cache or other rows;
    their logits mean nothing.
    """

    def __init__(self, layers, head, x, caches, batch, norms, head_norm, rope=None, interleaved: bool = False,
                 window: int = 0, eps: float = 1e-5, qk_norms=None):
        import torch

        from .device import EffortGroup

        if qk_norms is None:
            qk_norms = [(None, None)] * len(layers)
        if len(qk_norms) != len(layers):
            raise ValueError("one pair of weights of the heads' norms per layer")
        if len(layers) != len(caches) or len(layers) != len(norms):
            raise ValueError("one cache and one pair of norm weights per layer")
        if x.dim() != 2 or x.dtype != torch.float32 or not x.is_contiguous() or x.shape[0] < 1:
            raise ValueError("x must be a contiguous float32 tensor [tokens][dim]")
        tokens, dim = x.shape
        for L, c in zip(layers, caches):
            qd, kd, hid, hd = L["wq"].out_dim, c.kv_heads * c.head_dim, L["w1"].out_dim, c.head_dim
            if qd % kd or any((L[r].in_dim, L[r].out_dim) != io for r, io in (
                    ("wq", (dim, qd)), ("wk", (dim, kd)), ("wv", (dim, kd)), ("wo", (qd, dim)), ("w1", (dim, hid)),
                    ("w3", (dim, hid)), ("w2", (hid, dim)))):
                raise ValueError("a layer's matrices do not fit x, its cache or each other")
        if head.in_dim != dim:
            raise ValueError("the head does not fit x")
        for L, c, pair in zip(layers, caches, qk_norms):
            for w, r in zip(pair, ("wq", "wk")):
                if w is not None and (w.shape not in ((c.head_dim,), (L[r].out_dim // c.head_dim, c.head_dim)) or
                                      w.dtype != torch.float32 or not w.is_contiguous() or w.device != x.device):
                    raise ValueError("weights of the heads' norms must be contiguous float32 tensors [head_dim] or "
                                     "[heads][head_dim] on %s" % x.device)
        if batch.parents is not None and batch.parents.shape[0] < tokens:
            raise ValueError("%d parents for %d rows" % (batch.parents.shape[0], tokens))
        weights = [w for pair in norms for w in pair] + [head_norm]
        if any(w.shape != (dim,) or w.dtype != torch.float32 or not w.is_contiguous() for w in weights):
            raise ValueError("norm weights must be contiguous float32 tensors [dim]")
        mats = [head] + [L[r] for L in layers for r in LAYER_ROLES]
        if any(t.device != x.device for t in [m.layout for m in mats] + [*caches, batch] + weights):
            raise ValueError("matrices, caches, batch and norm weights must be on x's device, %s" % x.device)
        short = [m.batch for m in mats if m.batch < tokens]
        if short:
            raise ValueError("a matrix was made for %d vectors a call, the step has %d rows" % (short[0], tokens))
        self.layers, self.head, self.x = layers, head, x
        self.caches, self.batch, self.norms, self.head_norm = caches, batch, norms, head_norm
        self.rope, self.interleaved, self.window, self.eps = rope, interleaved, window, eps
        self.qk_norms = qk_norms
        # zeros: rows of no sequence are never written by the attention
        mk = lambda n: torch.zeros((tokens, n), dtype=torch.float32, device=x.device)  # noqa: E731
        self.out = []
        for L in layers:
            o = {r: mk(L[r].out_dim) for r in LAYER_ROLES}
            o.update(hq=mk(dim), q=mk(L["wq"].out_dim), a=mk(L["wq"].out_dim), r=mk(dim), hf=mk(dim),
                     g=mk(L["w1"].out_dim))
            self.out.append(o)
        self.r, self.h = mk(dim), mk(dim)  # after the last layer: the stream, and its norm
        self.logits = mk(head.out_dim)
        self.groups = ([(EffortGroup([L["wq"], L["wk"], L["wv"]]), EffortGroup([L["w1"], L["w3"]]))
                        for L in layers] if tokens == 1 else None)

    def enqueue(self, effort, stream=None, record=None):
        """Issue the step on `stream` (None: torch's current stream).  `effort`
        as in DecodeStep.  With `record` (a Recorder; one row only), every matvec
        records its parity outputs under (layer, role), the head under (None,
        "head")."""
        import torch

        if record is not None and self.x.shape[0] != 1:
            raise ValueError("a step of %d rows cannot be recorded" % self.x.shape[0])
        if self.x.device.type != "cuda" or self.x.device.index == torch._C._cuda_getDevice():
            return self._enqueue(effort, stream, record)
        with torch.cuda.device(self.x.device):  # the matvecs launch on the current device
            return self._enqueue(effort, stream, record)

    def _enqueue(self, effort, stream, record):
        import torch

        from .layer import norm_residual

        tokens = self.x.shape[0]
        main = stream if stream is not None else torch.cuda.current_stream(self.x.device)  # (for the matvecs)

        def times(l, roles, x, ys, group=None):
            mats = [self.layers[l][r] if l is not None else self.head for r in roles]
            keys = [(l, r) for r in roles]
            es = [_effort_of(effort, *k) for k in keys]
            if tokens > 1:
                for m, e, y in zip(mats, es, ys):
                    m.matvec_batched(x, e, y, main)
            elif group is not None:
                group.matvec(x[0], es, [y[0] for y in ys], main, record=None if record is None else (record, keys))
            else:
                mats[0].matvec(x[0], es[0], ys[0][0], main, record=None if record is None else (record, keys[0]))

        r, add = None, self.x
        for l, (c, (before_attn, before_ffn), (qn, kn)) in enumerate(zip(self.caches, self.norms, self.qk_norms)):
            o, (qkv, gu) = self.out[l], self.groups[l] if self.groups else (None, None)
            heads = lambda t: t.view(tokens, -1, c.head_dim)  # noqa: B023,E731
            norm_residual(add, r, pre_w=before_attn, eps=self.eps, resid_out=self.r, out=o["hq"], stream=stream)
            times(l, ("wq", "wk", "wv"), o["hq"], [o["wq"], o["wk"], o["wv"]], qkv)
            c.append(self.batch, heads(o["wk"]), heads(o["wv"]), q=heads(o["wq"]), rope=self.rope,
                     interleaved=self.interleaved, q_out=heads(o["q"]), stream=stream, q_norm=qn, k_norm=kn,
                     eps=self.eps)
            c.attend(self.batch, heads(o["q"]), window=self.window, out=heads(o["a"]), stream=stream)
            times(l, ("wo",), o["a"], [o["wo"]])
            norm_residual(o["wo"], self.r, pre_w=before_ffn, eps=self.eps, resid_out=o["r"], out=o["hf"], stream=stream)
            times(l, ("w1", "w3"), o["hf"], [o["w1"], o["w3"]], gu)
            B.effort_silu_mul(o["w1"], o["w3"], o["g"].numel(), o["g"], main)
            times(l, ("w2",), o["g"], [o["w2"]])
            r, add = o["r"], o["w2"]
        norm_residual(add, r, pre_w=self.head_norm, eps=self.eps, resid_out=self.r, out=self.h, stream=stream)
        times(None, ("head",), self.h, [self.logits])
        return self.logits


class BeamStep:
    """One step of beam search: a DecoderStep whose rows are the beams of some
    prompts, one new token each, item after item; then the selection, the beams'
    reordering (KVPages.fork), and room for their next tokens (KVPages.grow).

    `pages` is a KVPages over the step's caches, page table and lengths.  Before
    the first step the caller has put the prompts into the caches, every beam's
    sequence holds its prompt (KVPages.fork shares it) and has room for its first
    token, and `scores` [items][beams] are 0 for one beam of an item and -inf for
    the others (as they are at first).  After each step `tokens`, `parents` (rows)
    and `scores` [items][beams] say what the beams are now, `ended` which of them
    have taken `end_token`: those stay as they are, end_token the last of their
    kv_lens tokens, which they append again in each step.  The caller writes the
    tokens' embeddings to the step's x.  `short` counts the pages that were missing, at
    most, in any step: once there are any, the results mean nothing, and the
    sequences stay empty, so that no page is written that somebody else may hold.
    The step may be captured once and replayed."""

    def __init__(self, step, pages, beams: int, end_token: int = -1):
        import torch

        rows, b = step.x.shape[0], step.batch
        if beams < 1 or rows % beams:
            raise ValueError("%d rows are not some items of %d beams" % (rows, beams))
        if b.parents is not None or b.seqs != rows:
            raise ValueError("a beam search's batch has one sequence per row, and no trees")
        if pages.page_table is not b.page_table or pages.kv_lens is not b.kv_lens:
            raise ValueError("pages must be over the batch's own page table and lengths")
        mine = {(c.k.data_ptr(), c.v.data_ptr()) for c in pages.caches.caches}
        if any((c.k.data_ptr(), c.v.data_ptr()) not in mine for c in step.caches):
            raise ValueError("pages must be over all the step's caches")
        self.step, self.pages, self.end_token = step, pages, end_token
        mk = lambda v, t: torch.full((rows // beams, beams), v, dtype=t, device=step.x.device)  # noqa: E731
        self.scores, self.parents, self.tokens = mk(-math.inf, torch.float32), mk(-1, torch.int32), mk(-1, torch.int32)
        self.scores[:, 0] = 0.0
        self.ended = mk(False, torch.bool)
        self.short = torch.zeros(1, dtype=torch.int32, device=step.x.device)

    def enqueue(self, effort, stream=None):
        """Issue the step on `stream` (None: torch's current stream); returns tokens."""
        import torch

        from .pages import beam_select

        dev = self.step.x.device
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        with torch.cuda.device(dev), torch.cuda.stream(stream):  # (None changes nothing)
            logits = self.step.enqueue(effort, stream)
            beam_select(logits, self.scores, ended=self.ended, end_token=self.end_token,
                        out=(self.scores, self.parents, self.tokens), stream=stream)
            # a beam that had ended before takes its last token's room again instead of more
            self.pages.kv_lens.sub_(self.ended.view(torch.uint8).view(-1))
            torch.eq(self.tokens, self.end_token, out=self.ended)
            self.pages.fork(self.parents.view(-1), stream=stream)
            torch.maximum(self.short, self.pages.grow(1, stream=stream), out=self.short)
            # without room the next tokens would fall on the last ones, in pages that beams share
            self.pages.kv_lens.mul_(self.short == 0)
        return self.tokens


class DenseDecodeStep:
    """The same chain with the dense fp16 GEMV (weights as device fp16 [in][out])."""

    def __init__(self, layers, head, x, a, head_in):
        import torch

        self.layers, self.head = layers, head
        self.x, self.a, self.head_in = x, a, head_in
        dev = head_in.device
        self.out = []
        for L in layers:
            o = {r: torch.empty(L[r].shape[1], dtype=torch.float32, device=dev) for r in LAYER_ROLES}
            o["g"] = torch.empty(L["w1"].shape[1], dtype=torch.float32, device=dev)
            self.out.append(o)
        self.logits = torch.empty(head.shape[1], dtype=torch.float32, device=dev)

    def enqueue(self, stream=None, side_streams=None):
        import torch

        main = stream if stream is not None else torch.cuda.current_stream()
        roles = ("wq", "wk", "wv", "wo", "w1", "w3")
        for l, L in enumerate(self.layers):
            o = self.out[l]
            ins = {"wq": self.x[l], "wk": self.x[l], "wv": self.x[l], "wo": self.a[l],
                   "w1": self.x[l], "w3": self.x[l]}
            for k, r in enumerate(roles):
                ss = side_streams[k % len(side_streams)] if side_streams else main
                if ss is not main:
                    ss.wait_stream(main)
                m, n = L[r].shape
                B.dense_gemv(L[r], ins[r], m, n, o[r], ss)
            if side_streams:
                for ss in side_streams[:len(roles)]:
                    main.wait_stream(ss)
            B.effort_silu_mul(o["w1"], o["w3"], L["w1"].shape[1], o["g"], main)
            m, n = L["w2"].shape
            B.dense_gemv(L["w2"], o["g"], m, n, o["w2"], main)
        m, n = self.head.shape
        B.dense_gemv(self.head, self.head_in, m, n, self.logits, main)


def route_top2(logits):
    """Top-2 experts of a router's logits (ties go to the lower index) and their
    gates, the softmax over the two chosen logits (computed in double, returned
    as fp32 values)."""
    vals = [float(x) for x in logits]
    order = sorted(range(len(vals)), key=lambda e: (-vals[e], e))
    e0, e1 = order[0], order[1]
    z = math.exp(vals[e1] - vals[e0])
    g0 = 1.0 / (1.0 + z)
    g1 = z / (1.0 + z)
    return e0, e1, float(g0), float(g1)


class MoEFFN:
    """A mixture-of-experts feed-forward block: expert e is (w1, w3, w2) as
    EffortMatrix, y = g0 * FFN_e0(x) + g1 * FFN_e1(x) with FFN(x) =
    (silu(x W1) * x W3) W2.  Only the two routed experts' layouts are read.
    With `grouped`, the four matrices that multiply x (w1 and w3 of both
    routed experts) go through one multi-matrix call, one gate call covers
    both experts and the two w2 go through another multi-matrix call (side
    streams are then not used)."""

    def __init__(self, experts, device, grouped: bool = False):
        import torch

        self.experts = experts  # entries that are never routed to may be None
        first = next(e for e in experts if e is not None)
        d_in, d_hid = first[0].in_dim, first[0].out_dim
        self.d_in, self.d_hid = d_in, d_hid
        mk = lambda n: torch.empty(n, dtype=torch.float32, device=device)  # noqa: E731
        # both experts' hidden vectors side by side, so that one gate call
        # covers the pair
        self.h1_all, self.h3_all, self.g_all = mk(2 * d_hid), mk(2 * d_hid), mk(2 * d_hid)
        self.h1 = [self.h1_all[:d_hid], self.h1_all[d_hid:]]
        self.h3 = [self.h3_all[:d_hid], self.h3_all[d_hid:]]
        self.g = [self.g_all[:d_hid], self.g_all[d_hid:]]
        self.o = [mk(d_in), mk(d_in)]
        self.y = mk(d_in)
        self.grouped = grouped
        if grouped:  # one workspace serves every pair of experts (they share shapes)
            d4 = [first[0].desc, first[1].desc] * 2
            self.ws_bytes = B.effort_workspace_bytes_multi(d4)
            self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)
            d2 = [first[2].desc] * 2
            self.ws2_bytes = B.effort_workspace_bytes_multi(d2)
            self.ws2 = torch.zeros(self.ws2_bytes, dtype=torch.uint8, device=device)

    def enqueue(self, x, route, effort, stream=None, side_streams=None, record=None):
        """`effort` is one effort for all six matvecs or an EffortSchedule keyed
        by (expert, role), role in ("w1", "w3", "w2").  With `side_streams` (at
        least two torch streams), the two experts run on separate streams, and
        w1 / w3 of an expert on separate streams when there are four.  With
        `record` (a Recorder), every matvec records its parity outputs under
        (expert, role)."""
        import torch

        main = stream if stream is not None else torch.cuda.current_stream()
        e0, e1, g0, g1 = route
        ns = len(side_streams) if side_streams else 0
        ef = lambda e, r: _effort_of(effort, e, r)  # noqa: E731
        if self.grouped:
            mats = [self.experts[e0][0], self.experts[e0][1], self.experts[e1][0], self.experts[e1][1]]
            keys = [(e0, "w1"), (e0, "w3"), (e1, "w1"), (e1, "w3")]
            args = ([M.desc for M in mats], [M.layout for M in mats], x, [ef(*k) for k in keys],
                    [self.h1[0], self.h3[0], self.h1[1], self.h3[1]], self.ws, self.ws_bytes)
            if record is None:
                B.effort_matvec_multi(*args, stream=main)
            else:
                cutoff, K, rks, fp = record.multi(keys, [M.in_dim for M in mats])
                B.effort_matvec_multi_debug(*args, cutoff, K, rks, fp, stream=main)
            B.effort_silu_mul(self.h1_all, self.h3_all, 2 * self.d_hid, self.g_all, main)
            w2s = [self.experts[e0][2], self.experts[e1][2]]
            keys2 = [(e0, "w2"), (e1, "w2")]
            args2 = ([M.desc for M in w2s], [M.layout for M in w2s], self.g, [ef(*k) for k in keys2],
                     self.o, self.ws2, self.ws2_bytes)
            if record is None:
                B.effort_matvec_multi(*args2, stream=main)
            else:
                cutoff, K, rks, fp = record.multi(keys2, [M.in_dim for M in w2s])
                B.effort_matvec_multi_debug(*args2, cutoff, K, rks, fp, stream=main)
            B.effort_axpby(self.o[0], g0, self.o[1], g1, self.d_in, self.y, main)
            return self.y
        rk = (lambda key: None) if record is None else (lambda key: (record, key))  # noqa: E731
        for k, e in enumerate((e0, e1)):
            w1, w3, w2 = self.experts[e]
            s1 = side_streams[k % ns] if ns >= 2 else main
            s3 = side_streams[2 + k] if ns >= 4 else s1
            for ss in {s1, s3}:
                if ss is not main:
                    ss.wait_stream(main)
            w1.matvec(x, ef(e, "w1"), self.h1[k], s1, record=rk((e, "w1")))
            w3.matvec(x, ef(e, "w3"), self.h3[k], s3, record=rk((e, "w3")))
            if s3 is not s1:
                s1.wait_stream(s3)
            B.effort_silu_mul(self.h1[k], self.h3[k], self.d_hid, self.g[k], s1)
            w2.matvec(self.g[k], ef(e, "w2"), self.o[k], s1, record=rk((e, "w2")))
        if ns >= 2:
            for ss in side_streams[:2]:
                main.wait_stream(ss)
        B.effort_axpby(self.o[0], g0, self.o[1], g1, self.d_in, self.y, main)
        return self.y
