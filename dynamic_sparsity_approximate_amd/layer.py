"""What a decoder layer needs between its matvecs: the paged 8-bit key/value
cache, the attention over it, and the residual sum with its norms (torch owns
the memory, libeffort does the arithmetic)."""
from __future__ import annotations

from . import binding as B

try:
    import torch

    _DTYPES = {torch.float32: B.EFFORT_F32, torch.float16: B.EFFORT_F16, torch.bfloat16: B.EFFORT_BF16}
except ImportError:  # the C binding alone works without torch
    _DTYPES = {}


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError("%s: %s is not one of float32, float16, bfloat16" % (name, t.dtype))
    return d


class _On:
    """Runs a call on the tensors' own device: `with _On(device, stream) as s`
    makes that device and `stream` (None: the device's current stream) current,
    so that what the call allocates belongs to that stream, and gives the
    stream's handle."""

    __slots__ = ("device", "stream", "_dev", "_ctx")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("the tensors must be on a GPU")
        self.device, self.stream, self._dev, self._ctx = device, stream, None, None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self._dev = torch.cuda.device(self.device)
            self._dev.__enter__()
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        s = self.stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=self.device)
        self._ctx = torch.cuda.stream(s)
        self._ctx.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        if self._dev is not None:
            self._dev.__exit__(*exc)


def _heads(t, name, tokens, dim, like):
    """(token stride, heads) of [tokens][heads][dim] rows of `like`'s type and device."""
    if t.dim() != 3 or t.shape[2] != dim or (tokens is not None and t.shape[0] != tokens):
        raise ValueError("%s: shape %s, wanted [%s, heads, %d]" % (
            name, tuple(t.shape), "tokens" if tokens is None else tokens, dim))
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s: %s on %s, wanted %s on %s" % (name, t.dtype, t.device, like.dtype, like.device))
    s0, s1, s2 = t.stride()
    h = t.shape[1]
    if s2 != 1 or (h > 1 and s1 != dim):
        raise ValueError("%s: a token's heads must be contiguous (strides %s)" % (name, (s0, s1, s2)))
    return (s0 if t.shape[0] > 1 else h * dim), h


class KVBatch:
    """The new tokens of a call and where they belong: int32 tensors on one
    device, page_table [seqs][max_pages], kv_lens [seqs] (lengths with the new
    tokens), q_starts [seqs + 1] (rows of q, k, v of each sequence).  Their
    contents are read by the kernels at every call, so a program (or a
    captured graph) may update them in place between calls."""

    def __init__(self, page_table, kv_lens, q_starts):
        for t, n in ((page_table, "page_table"), (kv_lens, "kv_lens"), (q_starts, "q_starts")):
            if t.dtype != torch.int32 or t.device != page_table.device:
                raise ValueError("%s must be an int32 tensor on page_table's device" % n)
        seqs = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
        if page_table.dim() != 2 or page_table.shape[0] != seqs or q_starts.shape != (seqs + 1,):
            raise ValueError("page_table [seqs][max_pages], kv_lens [seqs], q_starts [seqs + 1]: got %s, %s, %s" % (
                tuple(page_table.shape), tuple(kv_lens.shape), tuple(q_starts.shape)))
        if (page_table.shape[1] > 1 and page_table.stride(1) != 1) or not (
                kv_lens.is_contiguous() and q_starts.is_contiguous()):
            raise ValueError("page_table's rows, kv_lens and q_starts must be contiguous")
        self.page_table, self.kv_lens, self.q_starts = page_table, kv_lens, q_starts
        self.device = page_table.device
        stride = page_table.stride(0) if seqs > 1 else page_table.shape[1]
        self.desc = B.effort_kv_batch(seqs, page_table.shape[1], 0, stride, page_table.data_ptr(),
                                      kv_lens.data_ptr(), q_starts.data_ptr())

    def with_tokens(self, n: int):
        """The C descriptor for a call with n rows."""
        if self.desc.tokens != n:
            self.desc.tokens = n
        return self.desc


class KVCache:
    """A paged cache of keys and values held in 8 bits, with one scale per
    (page, head): codes k, v uint8 [pages][kv_heads][page_tokens][head_dim],
    k_scale, v_scale float32 [pages][kv_heads].  `append` writes new tokens,
    `attend` reads."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64,
                 format: int = B.EFFORT_KV_E4M3, device="cuda"):
        shape = (pages, kv_heads, page_tokens, head_dim)
        self._set(torch.zeros(shape, dtype=torch.uint8, device=device),
                  torch.zeros(shape, dtype=torch.uint8, device=device),
                  torch.zeros(shape[:2], dtype=torch.float32, device=device),
                  torch.zeros(shape[:2], dtype=torch.float32, device=device), format)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, format: int = B.EFFORT_KV_E4M3):
        """A cache over existing tensors (shared, not copied)."""
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale, format)
        return self

    def _set(self, k, v, k_scale, v_scale, format):
        if k.dim() != 4 or v.shape != k.shape or k.dtype != torch.uint8 or v.dtype != torch.uint8:
            raise ValueError("k and v must be uint8 [pages][kv_heads][page_tokens][head_dim]")
        if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2] or \
                k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise ValueError("k_scale and v_scale must be float32 [pages][kv_heads]")
        if any(t.device != k.device or not t.is_contiguous() for t in (k, v, k_scale, v_scale)):
            raise ValueError("the cache's tensors must be contiguous and on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.format = k, v, k_scale, v_scale, format
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = k.shape
        self.device = k.device
        self.desc = B.effort_kv_cache(format, self.kv_heads, self.head_dim, self.page_tokens, self.pages,
                                      k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())

    def _place(self, batch):
        if batch.device != self.device:
            raise ValueError("the batch is on %s, the cache on %s" % (batch.device, self.device))

    def append(self, batch: KVBatch, k, v, q=None, rope=None, interleaved: bool = False, q_out=None,
               stream=None):
        """Rotates k (and q) by their positions and appends k and v.  k, v
        [tokens][kv_heads][head_dim], q [tokens][q_heads][head_dim]; `rope` is a
        table of rope_table (None: no rotation).  Returns the rotated q (None
        without q); `q_out` may be q."""
        self._place(batch)
        tokens = k.shape[0]
        dt = _dtype(k, "k")
        ks, kh = _heads(k, "k", None, self.head_dim, k)
        vs, vh = _heads(v, "v", tokens, self.head_dim, k)
        if kh != self.kv_heads or vh != kh or k.device != self.device:
            raise ValueError("k and v must have the cache's %d heads and be on %s" % (self.kv_heads, self.device))
        rows = rot = 0
        if rope is not None:
            if rope.dim() != 3 or rope.shape[2] != 2 or rope.dtype != torch.float32 or \
                    not rope.is_contiguous() or rope.device != self.device:
                raise ValueError("rope must be a contiguous float32 table [rows][rot_dim / 2][2] on %s" % self.device)
            rows, rot = rope.shape[0], 2 * rope.shape[1]
        with _On(self.device, stream) as s:
            qs = qh = os = 0
            if q is not None:
                qs, qh = _heads(q, "q", tokens, self.head_dim, k)
                if q_out is None:
                    q_out = torch.empty((tokens, qh, self.head_dim), dtype=q.dtype, device=q.device)
                os, oh = _heads(q_out, "q_out", tokens, self.head_dim, k)
                if oh != qh:
                    raise ValueError("q_out must have q's heads")
            else:
                q_out = None
            B.effort_kv_append(self.desc, batch.with_tokens(tokens), dt, rope, rows, rot, int(interleaved), q, qs,
                               qh, q_out, os, k, ks, v, vs, s)
        return q_out

    def attend(self, batch: KVBatch, q, window: int = 0, scale=None, out=None, stream=None):
        """Causal attention of the new tokens' (rotated) queries over the cache,
        `append`ed tokens included.  q [tokens][q_heads][head_dim]; scale
        defaults to 1 / sqrt(head_dim); window 0: unlimited.  Returns out, of
        q's shape and type."""
        self._place(batch)
        tokens = q.shape[0]
        dt = _dtype(q, "q")
        qs, qh = _heads(q, "q", None, self.head_dim, q)
        if q.device != self.device:
            raise ValueError("q is on %s, the cache on %s" % (q.device, self.device))
        if scale is None:
            scale = self.head_dim ** -0.5
        with _On(self.device, stream) as s:
            if out is None:
                out = torch.empty((tokens, qh, self.head_dim), dtype=q.dtype, device=q.device)
            os, oh = _heads(out, "out", tokens, self.head_dim, q)
            if oh != qh:
                raise ValueError("out must have q's heads")
            n = B.effort_kv_workspace_bytes(self.desc, batch.desc.seqs, tokens, qh)
            # of this call alone: calls on other streams and other captured graphs have their own
            ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
            B.effort_kv_attention(self.desc, batch.with_tokens(tokens), dt, q, qs, qh, scale, window, out, os, ws,
                                  n, s)
        return out


def rope_table(base: float, rows: int, rot_dim: int, device="cuda", stream=None):
    """float32 [rows][rot_dim / 2][2]: (cos, sin) of row * base^(-2 pair / rot_dim)."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with _On(device, stream) as s:
        table = torch.empty((rows, rot_dim // 2, 2), dtype=torch.float32, device=device)
        B.effort_rope_table(base, rows, rot_dim, table, s)
    return table


def _rows(t, name, shape, dtype, device):
    """Row stride of a tensor [rows][n] (or [n])."""
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device:
        raise ValueError("%s: %s %s on %s, wanted %s %s on %s" % (
            name, t.dtype, tuple(t.shape), t.device, dtype, shape, device))
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s: its rows must be contiguous" % name)
    return t.stride(0) if len(shape) == 2 and shape[0] > 1 else shape[-1]


def norm_residual(x, resid=None, post_w=None, gate=None, scale: float = 1.0, pre_w=None, eps: float = 1e-5,
                  resid_out=None, out=None, with_sum: bool = True, with_norm: bool = True, stream=None):
    """The end of one block and the start of the next: t = x / rms(x) * post_w
    (post_w None: x), r = resid + scale * gate * t, out = r / rms(r) * pre_w.
    x [rows][n] or [n]; resid alike, of x's type or float32; gate [n] or
    [rows][n].  Returns (r, out); `with_sum` / `with_norm` False leave out one
    of them (None is returned for it).  resid_out may be resid, out may be x."""
    if x.dim() not in (1, 2):
        raise ValueError("x must be [rows][n] or [n]")
    dt, dev, shape = _dtype(x, "x"), x.device, tuple(x.shape)
    rows, n = (shape[0] if len(shape) == 2 else 1), shape[-1]
    xs = _rows(x, "x", shape, x.dtype, dev)
    rdt = resid.dtype if resid is not None else resid_out.dtype if resid_out is not None else x.dtype
    if rdt not in (x.dtype, torch.float32):
        raise TypeError("resid must be of x's type or float32")
    rs = _rows(resid, "resid", shape, rdt, dev) if resid is not None else 0
    for w, name in ((post_w, "post_w"), (pre_w, "pre_w")):
        if w is not None:
            _rows(w, name, (n,), x.dtype, dev)
    gs = 0
    if gate is not None:
        gs = _rows(gate, "gate", (n,) if gate.dim() == 1 else (rows, n), x.dtype, dev)
        gs = 0 if gate.dim() == 1 else gs
    with _On(dev, stream) as s:
        ros = os = 0
        if with_sum:
            if resid_out is None:
                resid_out = torch.empty(shape, dtype=rdt, device=dev)
            ros = _rows(resid_out, "resid_out", shape, rdt, dev)
        else:
            resid_out = None
        if with_norm:
            if out is None:
                out = torch.empty(shape, dtype=x.dtype, device=dev)
            os = _rows(out, "out", shape, x.dtype, dev)
        else:
            out = None
        B.effort_norm_residual(dt, rows, n, x, xs, _DTYPES[rdt], resid, rs, post_w, gate, gs, scale, pre_w, eps,
                               resid_out, ros, out, os, s)
    return resid_out, out
