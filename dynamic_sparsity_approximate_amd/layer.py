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


def _i32(x, name):
    """ctypes would pass on the low 32 bits of a larger number."""
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError("%s: %d does not fit 32 bits" % (name, x))


def _run(device, stream, call):
    """call(handle) on the tensors' own device with `stream` (None: that
    device's current stream), both made current, so that what the call
    allocates belongs to that stream.  The usual case, the current device and
    its current stream, costs a microsecond of host time; the contexts cost ten."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a GPU")
    if stream is None and device.index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _heads(t, name, tokens, dim, like):
    """(token stride, heads) of [tokens][heads][dim] rows of `like`'s type and device."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (tokens is not None and shape[0] != tokens):
        raise ValueError("%s: shape %s, wanted [%s, heads, %d]" % (
            name, tuple(shape), "tokens" if tokens is None else tokens, dim))
    if t is not like and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError("%s: %s on %s, wanted %s on %s" % (name, t.dtype, t.device, like.dtype, like.device))
    strides, h = t.stride(), shape[1]
    if strides[2] != 1 or (h > 1 and strides[1] != dim):
        raise ValueError("%s: a token's heads must be contiguous (strides %s)" % (name, strides))
    return (strides[0] if shape[0] > 1 else h * dim), h


class _Kept:
    """An object whose calls use the addresses and sizes that it was made with:
    the attributes of `_kept` cannot be replaced, or a tensor's memory could be
    freed while calls still use it."""

    _kept = frozenset()

    def __setattr__(self, name, value):
        # the same object may be assigned again: that is how `x.t += 1`, in place, ends
        if name in self._kept and self.__dict__.get(name, value) is not value:
            raise AttributeError("%s cannot be replaced, only written in place" % name)
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._kept:
            raise AttributeError("%s cannot be taken away" % name)
        object.__delattr__(self, name)


class KVBatch(_Kept):
    """The new tokens of a call and where they belong: int32 tensors on one
    device, page_table [seqs][max_pages], kv_lens [seqs] (lengths with the new
    tokens), q_starts [seqs + 1] (rows of q, k, v of each sequence).  Their
    contents are read by the kernels at every call, so a program (or a
    captured graph) may update them in place between calls; other tensors need
    another KVBatch."""

    _kept = frozenset(("page_table", "kv_lens", "q_starts", "device", "seqs"))

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
        self.seqs = seqs
        self._args = (seqs, page_table.shape[1])
        self._ptrs = (stride, page_table.data_ptr(), kv_lens.data_ptr(), q_starts.data_ptr())
        self._descs = {}

    def __reduce__(self):  # copies of the tensors have other addresses
        return KVBatch, (self.page_table, self.kv_lens, self.q_starts)

    def desc(self, tokens: int):
        """The C descriptor for a call with that many rows."""
        d = self._descs.get(tokens)
        if d is None:
            if len(self._descs) >= 64:
                self._descs.clear()
            d = self._descs[tokens] = B.effort_kv_batch(*self._args, tokens, *self._ptrs)
        return d


class KVCache(_Kept):
    """A paged cache of keys and values held in 8 bits, with one scale per
    (page, head): codes k, v uint8 [pages][kv_heads][page_tokens][head_dim],
    k_scale, v_scale float32 [pages][kv_heads].  `append` writes new tokens,
    `attend` reads.  The tensors may be written in place, not replaced."""

    _kept = frozenset(("k", "v", "k_scale", "v_scale", "format", "pages", "kv_heads", "page_tokens", "head_dim",
                       "device", "desc"))

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
        self._ws_bytes = {}

    def __reduce__(self):
        return KVCache.wrap, (self.k, self.v, self.k_scale, self.v_scale, self.format)

    def _place(self, batch):
        if batch.device != self.device:
            raise ValueError("the batch is on %s, the cache on %s" % (batch.device, self.device))

    def append(self, batch: KVBatch, k, v, q=None, rope=None, interleaved: bool = False, q_out=None,
               stream=None):
        """Rotates k (and q) by their positions and appends k and v.  k, v
        [tokens][kv_heads][head_dim], q [tokens][q_heads][head_dim]; `rope` is a
        table of rope_table (None: no rotation).  Returns the rotated q (None
        without q); `q_out` may be q.  Rows that no sequence has are not written:
        in a new tensor they hold anything."""
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
        qs, qh = _heads(q, "q", tokens, self.head_dim, k) if q is not None else (0, 0)

        def call(handle):
            out, os = None, 0
            if q is not None:
                if q_out is None:
                    out, os = q.new_empty((tokens, qh, self.head_dim)), qh * self.head_dim
                else:
                    out, (os, oh) = q_out, _heads(q_out, "q_out", tokens, self.head_dim, k)
                    if oh != qh:
                        raise ValueError("q_out must have q's heads")
            B.effort_kv_append(self.desc, batch.desc(tokens), dt, rope, rows, rot, int(interleaved), q, qs, qh, out,
                               os, k, ks, v, vs, handle)
            return out

        return _run(self.device, stream, call)

    def attend(self, batch: KVBatch, q, window: int = 0, scale=None, out=None, stream=None):
        """Causal attention of the new tokens' (rotated) queries over the cache,
        `append`ed tokens included.  q [tokens][q_heads][head_dim]; scale
        defaults to 1 / sqrt(head_dim); window 0: unlimited.  Returns out, of
        q's shape and type.  Rows that no sequence has are not written: in a new
        tensor they hold anything."""
        self._place(batch)
        tokens = q.shape[0]
        dt = _dtype(q, "q")
        qs, qh = _heads(q, "q", None, self.head_dim, q)
        if q.device != self.device:
            raise ValueError("q is on %s, the cache on %s" % (q.device, self.device))
        _i32(window, "window")
        if scale is None:
            scale = self.head_dim ** -0.5

        def call(handle):
            if out is None:
                o, os = q.new_empty((tokens, qh, self.head_dim)), qh * self.head_dim
            else:
                o, (os, oh) = out, _heads(out, "out", tokens, self.head_dim, q)
                if oh != qh:
                    raise ValueError("out must have q's heads")
            key = (batch.seqs, tokens, qh)
            n = self._ws_bytes.get(key)
            if n is None:
                n = B.effort_kv_workspace_bytes(self.desc, *key)
                if len(self._ws_bytes) >= 256:
                    self._ws_bytes.clear()
                self._ws_bytes[key] = n
            # of this call alone: calls on other streams and other captured graphs have their own
            ws = q.new_empty(n, dtype=torch.uint8) if n else None
            B.effort_kv_attention(self.desc, batch.desc(tokens), dt, q, qs, qh, scale, window, o, os, ws, n, handle)
            return o

        return _run(self.device, stream, call)


def rope_table(base: float, rows: int, rot_dim: int, device="cuda", stream=None):
    """float32 [rows][rot_dim / 2][2]: (cos, sin) of row * base^(-2 pair / rot_dim)."""
    _i32(rot_dim, "rot_dim")
    device = torch.device(device)
    if device.type == "cuda":
        current = torch.cuda.current_device()  # (initialises the device)
        device = torch.device("cuda", current if device.index is None else device.index)

    def call(handle):
        table = torch.empty((rows, rot_dim // 2, 2), dtype=torch.float32, device=device)
        B.effort_rope_table(base, rows, rot_dim, table, handle)
        return table

    return _run(device, stream, call)


def _rows(t, name, shape, dtype, device):
    """Row stride of a tensor [rows][n] (or [n])."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError("%s: %s %s on %s, wanted %s %s on %s" % (
            name, t.dtype, tuple(t.shape), t.device, dtype, tuple(shape), device))
    strides, n = t.stride(), shape[-1]
    if strides[-1] != 1 and n > 1:
        raise ValueError("%s: its rows must be contiguous" % name)
    return strides[0] if len(strides) == 2 and shape[0] > 1 else n


def norm_residual(x, resid=None, post_w=None, gate=None, scale: float = 1.0, pre_w=None, eps: float = 1e-5,
                  resid_out=None, out=None, with_sum: bool = True, with_norm: bool = True, stream=None):
    """The end of one block and the start of the next: t = x / rms(x) * post_w
    (post_w None: x), r = resid + scale * gate * t, out = r / rms(r) * pre_w.
    x [rows][n] or [n]; resid alike, of x's type or float32; gate [n] or
    [rows][n].  Returns (r, out); `with_sum` / `with_norm` False leave out one
    of them (None is returned for it).  resid_out may be resid, out may be x."""
    shape, dev, xdt = x.shape, x.device, x.dtype
    if len(shape) not in (1, 2):
        raise ValueError("x must be [rows][n] or [n]")
    dt = _dtype(x, "x")
    rows, n = (shape[0] if len(shape) == 2 else 1), shape[-1]
    xs = _rows(x, "x", shape, xdt, dev)
    rdt = resid.dtype if resid is not None else resid_out.dtype if resid_out is not None else xdt
    if rdt is not xdt and rdt is not torch.float32:
        raise TypeError("resid must be of x's type or float32")
    rs = _rows(resid, "resid", shape, rdt, dev) if resid is not None else 0
    if post_w is not None:
        _rows(post_w, "post_w", (n,), xdt, dev)
    if pre_w is not None:
        _rows(pre_w, "pre_w", (n,), xdt, dev)
    gs = 0
    if gate is not None:
        if gate.dim() == 1:
            _rows(gate, "gate", (n,), xdt, dev)
        else:
            gs = _rows(gate, "gate", (rows, n), xdt, dev)

    def call(handle):
        r = o = None
        ros = os = 0
        if with_sum:
            if resid_out is None:
                r, ros = x.new_empty(shape, dtype=rdt), n
            else:
                r, ros = resid_out, _rows(resid_out, "resid_out", shape, rdt, dev)
        if with_norm:
            if out is None:
                o, os = x.new_empty(shape), n
            else:
                o, os = out, _rows(out, "out", shape, xdt, dev)
        B.effort_norm_residual(dt, rows, n, x, xs, _DTYPES[rdt], resid, rs, post_w, gate, gs, scale, pre_w, eps, r,
                               ros, o, os, handle)
        return r, o

    return _run(dev, stream, call)
