"""Several continuations of a sequence over the paged 8-bit cache: which pages
they share (KVPages), the accepted path of a tree of drafted tokens, copies of
pages, and beam search's selection (torch owns the memory, libeffort does the
work)."""
from __future__ import annotations

from . import binding as B
from .layer import _DTYPES, KVBatch, _dtype, _i32, _Kept, _run

try:
    import torch
except ImportError:  # the C binding alone works without torch
    pass


_sizes = {}  # workspace bytes by a call's sizes


def _bytes(need, *sizes):
    n = _sizes.get((need, sizes))
    if n is None:
        if len(_sizes) >= 1024:
            _sizes.clear()
        n = _sizes[(need, sizes)] = need(*sizes)
    return n


def _vector(t, name, n, device):
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous int32 tensor [%d] on %s" % (name, n, device))
    return t


class _Set:
    """The caches of a model's layers: one page id stands for that page in each."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("no cache")
        c = self.caches[0]
        alike = c._alike
        if [o for o in self.caches if o._alike != alike]:
            raise ValueError("the caches must have the same pages and page_tokens and be on one device")
        self.pages, self.page_tokens, self.device = c.pages, c.page_tokens, c.device
        self.count = len(self.caches)
        self.descs = (B.effort_kv_cache * self.count).from_buffer_copy(b"".join([o._packed for o in self.caches]))


def _set(caches):
    return caches if isinstance(caches, _Set) else _Set(caches)


def cache_set(caches):
    """The caches of a model's layers as `KVPages`, `kv_accept` and
    `kv_copy_pages` take them, put together once instead of at every call."""
    return _Set(caches)


class KVPages(_Kept):
    """Who holds the pages of a set of caches: `page_table` int32
    [seqs][max_pages] (an entry outside [0, pages) holds nothing), `kv_lens` int32
    [seqs], and `refs` int32 [pages], how many entries hold each page (counted
    from the table if not given; tables that share the caches share one refs).
    A KVBatch over the same page_table and kv_lens sees every change.  Calls on
    one KVPages, or on several with one refs, must be ordered."""

    _kept = frozenset(("caches", "page_table", "kv_lens", "refs", "info", "_missing", "_ws", "device", "seqs"))

    def __init__(self, caches, page_table, kv_lens, refs=None):
        s = self.caches = _set(caches)
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != s.device or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 [seqs][max_pages], its rows contiguous, on %s" % s.device)
        self.seqs, cols = page_table.shape
        _vector(kv_lens, "kv_lens", self.seqs, s.device)
        if refs is None:
            held = page_table[(page_table >= 0) & (page_table < s.pages)]
            refs = torch.bincount(held, minlength=s.pages).to(torch.int32)
        self.page_table, self.kv_lens, self.refs = page_table, kv_lens, _vector(refs, "refs", s.pages, s.device)
        self.info = torch.zeros(4, dtype=torch.int32, device=s.device)
        self._missing = self.info[:1]
        self.device = s.device
        stride = page_table.stride(0) if self.seqs > 1 else cols
        self._book = B.effort_kv_book(self.seqs, cols, s.page_tokens, 0, s.pages, stride, page_table.data_ptr(),
                                      kv_lens.data_ptr(), refs.data_ptr(), self.info.data_ptr())
        # calls are ordered, because of refs, so that one workspace serves them all
        self._ws = self.info.new_empty(B.effort_kv_grow_workspace_bytes(self._book), dtype=torch.uint8)

    def __reduce__(self):  # copies of the tensors have other addresses
        return KVPages, (self.caches.caches, self.page_table, self.kv_lens, self.refs)

    def fork(self, source, lens=None, stream=None):
        """Sequence s becomes a copy of sequence source[s] as it was, cut to its
        first lens[s] tokens (None: uncut): its length, and the pages that hold
        these tokens, shared.  A source outside [0, seqs) empties the sequence.
        Pages that nobody holds any more are free."""
        _vector(source, "source", self.seqs, self.device)
        if lens is not None:
            _vector(lens, "lens", self.seqs, self.device)
        _run(self.device, stream, lambda handle: B.effort_kv_fork(self._book, source, lens, handle))

    def grow(self, more, stream=None):
        """Room for `more` new tokens of each sequence (an int, or int32 [seqs]):
        kv_lens grow, and every page that will receive new tokens is the
        sequence's own, a free one or a copy where others hold it.  Returns an
        int32 tensor [1] that the next call overwrites: the pages that were
        missing.  If there are any, nothing has changed, and the new tokens must
        not be appended."""
        each = None
        if isinstance(more, int):
            _i32(more, "more")
        else:
            each, more = _vector(more, "more", self.seqs, self.device), 0

        s = self.caches
        _run(self.device, stream, lambda handle: B.effort_kv_grow(
            self._book, s.descs, s.count, each, more, self._ws, self._ws.shape[0], handle))
        return self._missing


def kv_copy_pages(caches, src, dst, stream=None):
    """Copies pages src[i] to dst[i] (int32 tensors), codes and scales, in each of
    the caches (a list, or a cache_set).  Ids outside [0, pages) are passed over;
    no page may be written twice, nor be written and read."""
    s = _set(caches)
    n = src.shape[0] if src.dim() == 1 else -1
    _vector(src, "src", n, s.device)
    _vector(dst, "dst", n, s.device)
    _run(s.device, stream, lambda handle: B.effort_kv_copy_pages(s.descs, s.count, src, dst, n, handle))


def kv_accept(caches, batch: KVBatch, leaf, lens_out=None, stream=None):
    """Keeps a path of each sequence's new tokens (the batch's trees; without
    parents a chain): the new token leaf[s] and its ancestors move to the slots
    behind the committed tokens, in each of the caches (a list, or a cache_set),
    and the new length, all others forgotten, goes to lens_out (None:
    batch.kv_lens itself).  A leaf outside the new tokens (-1, say) keeps none.
    Returns lens_out."""
    s = _set(caches)
    if batch.device != s.device:
        raise ValueError("the batch is on %s, the caches on %s" % (batch.device, s.device))
    _vector(leaf, "leaf", batch.seqs, s.device)
    out = batch.kv_lens if lens_out is None else _vector(lens_out, "lens_out", batch.seqs, s.device)
    n = _bytes(B.effort_kv_accept_workspace_bytes, batch.seqs) if batch.parents is not None else 0
    # rows of the call: as many as a call may have, and no more than the parents, where there are any
    tokens = 1 << 24 if batch.parents is None else min(1 << 24, batch.parents.shape[0])

    def call(handle):
        ws = leaf.new_empty(n, dtype=torch.uint8) if n else None
        B.effort_kv_accept(s.descs, s.count, batch.desc(tokens), batch.parents, leaf, out, ws, n, handle)
        return out

    return _run(s.device, stream, call)


def beam_select(logits, scores, keep=None, ended=None, end_token: int = 0, out=None, stream=None):
    """Beam search's selection.  scores float32 [items][beams], logits
    [items * beams][vocab] or [items][beams][vocab]; of an item's beams b and
    tokens t the `keep` (default: beams) best by scores[b] + log_softmax(logits[b])[t],
    the best first; equal ones in the order of beams and tokens.  A beam with
    ended[b] (bool [items][beams]) continues with itself alone, its score
    unchanged and its token `end_token`.  Tokens with a logit of -inf, beams
    whose score is not finite and rows with a NaN or +inf are no candidates;
    where there are fewer than `keep`, the rest are -inf, -1, -1.  (Forbid tokens
    with -inf, not with the lowest number: a row of nothing else is no dead end,
    and beside it the logarithm of its length is lost.)  Returns
    (scores, parents, tokens), [items][keep]: parents are rows of the logits, as
    KVPages.fork takes them.  `out`: three tensors to write to; out[0] may be
    scores itself if keep == beams."""
    if scores.dim() != 2 or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be a contiguous float32 tensor [items][beams]")
    (items, beams), dev = scores.shape, scores.device
    dt = _dtype(logits, "logits")
    shape, strides = logits.shape, logits.stride()
    if len(shape) == 2 and shape[0] == items * beams:
        stride = strides[0]
    elif len(shape) == 3 and shape[:2] == (items, beams):
        if items > 1 and beams > 1 and strides[0] != beams * strides[1]:
            raise ValueError("logits: rows must be one distance apart (strides %s)" % (strides,))
        stride = strides[1] if beams > 1 else strides[0]
    else:
        raise ValueError("logits: shape %s, wanted [%d][vocab] or [%d][%d][vocab]" % (
            tuple(shape), items * beams, items, beams))
    vocab = shape[-1]
    if logits.device != dev or (vocab > 1 and strides[-1] != 1):
        raise ValueError("logits must be on %s, their rows contiguous" % dev)
    if items * beams <= 1:
        stride = max(vocab, 1)
    if ended is not None and (ended.dtype not in (torch.bool, torch.uint8) or ended.shape != scores.shape or
                              ended.device != dev or not ended.is_contiguous()):
        raise ValueError("ended must be a contiguous bool tensor [items][beams] on %s" % dev)
    keep = beams if keep is None else keep
    _i32(keep, "keep")
    _i32(end_token, "end_token")
    n = _bytes(B.effort_beam_workspace_bytes, items, beams, vocab)

    def call(handle):
        if out is None:
            o = (scores.new_empty((items, keep)), *scores.new_empty((2, items, keep), dtype=torch.int32).unbind())
        else:
            o = tuple(out)
            if [t.dtype for t in o] != [torch.float32, torch.int32, torch.int32] or \
                    any(t.shape != (items, keep) or t.device != dev or not t.is_contiguous() for t in o):
                raise ValueError("out must be contiguous float32, int32, int32 tensors [%d][%d] on %s" % (
                    items, keep, dev))
        ws = scores.new_empty(n, dtype=torch.uint8) if n else None
        B.effort_beam_select(dt, logits, stride, scores, ended, end_token, items, beams, vocab, keep, *o, ws, n, handle)
        return o

    return _run(dev, stream, call)
