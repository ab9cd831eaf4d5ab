"""Around the decode step: Python face of ``include/nmserve.h``.

Tensors, streams and results are handled as in ``attention.py``.
"""
import ctypes

import torch

from ._lib import NM_OK, KvPagesStruct, NmError, serve_lib
from .attention import _cache, _check, _dtype, _empty, _fit, _other, _refuse, _rows, _size, _stream

_lib = None


def _load():
    global _lib
    _lib = serve_lib()
    return _lib


class KVPages:
    """The book of a cache's pages for ``sequences`` sequences of up to ``width`` pages each, on the device:
    ``table`` int32 [sequences][width] and ``lens`` int32 [sequences] as attn_decode takes them (a negative length
    is a padding row), ``free`` int32 [n_pages], a stack of free pages, ``n_free`` int32 [1] of them, the top one
    last.  New: nobody has a token, all pages are free, page 0 on top.  The tensors may be written to, not
    replaced.  Calls on one book must follow each other."""

    __slots__ = ("_buffers", "_struct", "_ref", "_index", "device", "sequences", "width", "n_pages", "page_size")

    def __init__(self, sequences, width, n_pages, page_size, device="cuda"):
        lib = _lib or _load()
        sizes = (sequences, width, n_pages, page_size)
        scratch = lib.nm_kv_plan_scratch_bytes(sequences) if _fit(*sizes) else -1
        if scratch < 0 or not 1 <= width <= 2 ** 24 or sequences * width >= 2 ** 31 or n_pages < 1 or \
                page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"no book of {sequences} sequences of {width} pages, {n_pages} pages of {page_size} tokens")
        table = torch.zeros((sequences, width), dtype=torch.int32, device=device)
        lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
        n_free = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        room = torch.empty(scratch, dtype=torch.uint8, device=device)
        self._buffers = (table, lens, free, n_free, room)
        self.device, self._index = table.device, table.get_device()
        self.sequences, self.width, self.n_pages, self.page_size = sizes
        self._struct = KvPagesStruct(*(t.data_ptr() for t in self._buffers), sequences, width, n_pages, page_size)
        self._ref = ctypes.addressof(self._struct)

    # Fixed, since the handle holds their addresses.
    @property
    def table(self):
        return self._buffers[0]

    @property
    def lens(self):
        return self._buffers[1]

    @property
    def free(self):
        return self._buffers[2]

    @property
    def n_free(self):
        return self._buffers[3]


def kv_plan(pages, adds, rows, out=None, stream=None):
    """One step of a KVPages book: sequence b gets adds[b] more tokens (int32 [sequences]; negative: so many fewer,
    all it has at most), pages of dropped tokens going back onto the stack first and new ones coming off its top,
    in order, until pages or the ``rows`` rows run out (no sequence is overtaken; one whose row of the table is too
    short gets none).  Brings pages.table, .lens, .free and .n_free up to date and returns (starts, slots,
    positions, granted): rows starts[b] .. starts[b+1] - 1 (int32 [sequences + 1]) are b's new tokens, slots (int64
    [rows]) and positions (int32 [rows]) theirs in the cache and the sequence (-1 and 0 behind the last), granted
    (int32 [sequences]) what each got or lost.  ``out`` is such a tuple.  New rows are packed, without gaps for
    sequences that get nothing; attn_decode and attn_tree take sequence b's N rows at b N: see include/nmserve.h for
    the layout of a step in which some may get nothing."""
    if not isinstance(pages, KVPages):
        raise TypeError("pages must be a KVPages")
    p = pages
    dev, B = p._index, p.sequences
    ap = _check(adds, "adds", dev, torch.int32, (B,))
    if not 0 <= rows < 2 ** 31:
        raise ValueError(f"{rows} rows")
    other = _other(dev, stream)
    try:
        if out is None:
            out = (adds.new_empty(B + 1), adds.new_empty(rows, dtype=torch.int64), adds.new_empty(rows),
                   torch.empty_like(adds))
            at = [t.data_ptr() for t in out]
        else:
            at = [_check(t, f"out[{i}]", dev, dt, shape) for i, (t, dt, shape) in
                  enumerate(zip(out, (torch.int32, torch.int64, torch.int32, torch.int32),
                                ((B + 1,), (rows,), (rows,), (B,)), strict=True))]
        st = (_lib or _load()).nm_kv_plan(p._ref, ap, rows, *at, _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_kv_plan", st)
    return tuple(out)


def attn_prompt_workspace(T, Tk, B, heads_q, heads, D, device="cuda"):
    """A workspace for attn_prompt calls of T queries and Tk keys in B sequences, or of no larger
    T, Tk and B (any contents; calls that may run at the same time need one each)."""
    sizes = (T, Tk, B, heads_q, heads, D)
    nbytes = (_lib or _load()).nm_attn_prompt_workspace_bytes(*sizes) if _fit(*sizes) else -1
    if nbytes < 0:
        raise ValueError(f"no such attention: {T} queries, {Tk} keys, {B} sequences, {heads_q} query heads on {heads} "
                         f"of {D} columns")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def attn_prompt(q, k, v, starts, k_starts=None, scale=None, out=None, lse=None, ws=None, stream=None):
    """Causal attention over packed prompts: sequence b's queries are rows starts[b] .. starts[b+1] - 1
    of q [T][Hq][D], its keys and values rows k_starts[b] .. k_starts[b+1] - 1 of k and v [Tk][heads][D]
    (k_starts None: starts; int32 [B + 1], device).  Its last query stands at its last key: query i of nq
    sees keys j <= i + nk - nq, so that more keys than queries are a piece of a prompt behind earlier
    tokens.  scale defaults to 1/sqrt(D).  Returns out [T][Hq][D], zeros where a query sees no key; rows
    that no sequence has are left as they are.  ``lse`` (float32 [T][Hq]) receives the log of the
    softmax's sum.  ``ws``: an attn_prompt_workspace(), or None to allocate what this call needs (often nothing)."""
    shape = _size(q, "q", 3)
    T, hq, D = shape
    Tk, heads, _ = _size(k, "k", 3)
    dev, dt = q.get_device(), q.dtype
    code = _dtype(dt)
    qp, qs = _rows(q, "q", dev, dt, shape)
    kp, ks = _rows(k, "k", dev, dt, (Tk, heads, D))
    vp, vs = _rows(v, "v", dev, dt, (Tk, heads, D))
    n, = _size(starts, "starts", 1)
    if n < 1:
        raise ValueError("starts must have an entry more than there are sequences")
    sp = _check(starts, "starts", dev, torch.int32, (n,))
    ksp = None if k_starts is None else _check(k_starts, "k_starts", dev, torch.int32, (n,))
    if k_starts is None and Tk != T:
        raise ValueError(f"{T} queries and {Tk} keys need k_starts")
    lsep = None if lse is None else _check(lse, "lse", dev, torch.float32, (T, hq))
    wsp, nbytes = None, 0
    if ws is not None:
        nbytes, = _size(ws, "ws", 1)
        wsp = _check(ws, "ws", dev, torch.uint8, (nbytes,))
    lib = _lib or _load()
    other = _other(dev, stream)
    try:
        if out is None:
            out = _empty(q, qs)
            op = out.data_ptr()
        else:
            op = _check(out, "out", dev, dt, shape)
        if ws is None:
            nbytes = lib.nm_attn_prompt_call_bytes(T, Tk, n - 1, hq, heads, D)
            if nbytes > 0:
                ws = q.new_empty(nbytes, dtype=torch.uint8)
                wsp = ws.data_ptr()
        st = lib.nm_attn_prompt(qp, qs, T, kp, ks, vp, vs, Tk, sp, ksp, n - 1, hq, heads, D, code,
                                D ** -0.5 if scale is None else scale, op, lsep, wsp, max(nbytes, 0), _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_attn_prompt", st)
    return out


def attn_tree_workspace(B, drafts, heads_q, cache, max_len):
    """A workspace for attn_tree calls of this shape, or of no larger B and max_len, on the cache's device (any
    contents; calls that may run at the same time need one each)."""
    c = _cache(cache)
    sizes = (B, drafts, heads_q, max_len)
    nbytes = (_lib or _load()).nm_attn_tree_workspace_bytes(B, drafts, heads_q, c.heads, c.D, c._format, max_len) \
        if _fit(*sizes) else -1
    if nbytes < 0:
        raise ValueError(f"no such attention: {B} sequences of {drafts} drafts, {heads_q} query heads on {c.heads}, "
                         f"{max_len} tokens")
    return torch.empty(nbytes, dtype=torch.uint8, device=c.device)


def attn_tree(q, cache, page_table, lens, visible, max_len=None, scale=None, out=None, lse=None, ws=None, stream=None):
    """Attention of a tree of drafted tokens per sequence, q [B][N][Hq][D], over the cache.  Sequence b holds lens[b]
    (int32 [B], device; at most max_len) tokens on its pages page_table[b] (int32 [B][pages]), the last N of which are
    the drafts: draft i sees all tokens before the drafts, and draft j where bit j of visible[b][i] (int64 [B][N]) is
    set.  lens[b] < 0 marks a padding row, which is left as it was: sequences to which kv_plan granted nothing go in as
    such.  scale defaults to 1/sqrt(D); max_len to the
    table's width.  Returns out [B][N][Hq][D]; ``lse`` (float32 [B][N][Hq]) receives the log of the softmax's sum.
    ``ws``: an attn_tree_workspace(), or None to allocate what this call needs (often nothing).  The rows of q may be strided
    (draft after draft, sequence after sequence at one stride).  A batch of no sequences gives an empty result."""
    c = _cache(cache)
    dev, dt = c._index, c.dtype
    B, N, hq, _ = _size(q, "q", 4)
    shape = (B, N, hq, c.D)
    if q.shape != shape:
        _refuse(q, "q", dev, dt, shape)
    rows = q.reshape(B * N, hq, c.D) if q.is_contiguous() else _drafts(q)
    qp, qs = _rows(rows, "q", dev, dt, (B * N, hq, c.D))
    lp = _check(lens, "lens", dev, torch.int32, (B,))
    vp = _check(visible, "visible", dev, torch.int64, (B, N))
    width = _size(page_table, "page_table", 2)[1]
    if page_table.is_contiguous():
        table, stride = _check(page_table, "page_table", dev, torch.int32, (B, width)), width
    else:
        if (width > 1 and page_table.stride(1) != 1) or page_table.get_device() != dev or \
                page_table.dtype != torch.int32 or page_table.shape[0] != B:
            _refuse(page_table, "page_table (rows)", dev, torch.int32, (B, width))
        table, stride = page_table.data_ptr(), page_table.stride(0)
    width *= c.page_size
    max_len = width if max_len is None else max_len
    if not 0 <= max_len <= width:
        raise ValueError(f"max_len {max_len} is not within what page_table holds ({width} tokens)")
    lsep = None if lse is None else _check(lse, "lse", dev, torch.float32, (B, N, hq))
    wsp, nbytes = None, 0
    if ws is not None:
        nbytes, = _size(ws, "ws", 1)
        wsp = _check(ws, "ws", dev, torch.uint8, (nbytes,))
    lib = _lib or _load()
    if B == 0:                                        # no sequence: nothing to launch
        attn_tree_workspace(1, N, hq, c, max_len)     # what the arguments alone can refuse
        if out is not None:
            _check(out, "out", dev, dt, shape)
        return torch.empty_like(q) if out is None else out
    other = _other(dev, stream)
    try:
        if out is None:
            out = torch.empty_like(q) if qs == hq * c.D else q.new_empty(shape)
            op = out.data_ptr()
        else:
            op = _check(out, "out", dev, dt, shape)
        if ws is None:
            nbytes = lib.nm_attn_tree_call_bytes(B, N, hq, c.heads, c.D, c._format, max_len)
            if nbytes > 0:
                ws = q.new_empty(nbytes, dtype=torch.uint8)
                wsp = ws.data_ptr()
        st = lib.nm_attn_tree(qp, qs, B, N, hq, c._ref, vp, table, stride, lp, max_len,
                              c.D ** -0.5 if scale is None else scale, op, lsep, wsp, max(nbytes, 0), _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_attn_tree", st)
    return out


def _drafts(q):
    """[B * N][Hq][D] of strided q [B][N][Hq][D] whose rows lie one after the other."""
    B, N, hq, D = q.shape
    s = q.stride()
    row = s[1] if N > 1 else s[0]
    if B > 1 and N > 1 and s[0] != N * s[1]:
        raise ValueError("q: drafts and sequences must follow each other at one stride")
    return q.as_strided((B * N, hq, D), (row, s[2], s[3]))
