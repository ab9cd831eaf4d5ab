"""Between a decode layer's q+k+v and o projections: Python face of
``include/nmattn.h``.

q, k and v are [rows][heads][D] tensors whose heads and columns are contiguous;
rows may be strided (views of a fused q+k+v buffer).  Work runs on ``stream``
(default: the current stream of the tensors' device); results and workspaces
that a call allocates belong to that stream.
"""
import ctypes
import math

import torch

from ._lib import (NM_BF16, NM_FP16, NM_KV_16, NM_KV_MX4, NM_KV_MX8, NM_OK, KvCacheStruct, NmError, attn_lib)

_DT = {torch.float16: NM_FP16, torch.bfloat16: NM_BF16}
_FORMATS = {"16": NM_KV_16, "mx8": NM_KV_MX8, "mx4": NM_KV_MX4}


def _dtype(dtype):
    if dtype not in _DT:
        raise TypeError(f"libnmspmv supports float16 and bfloat16, not {dtype}")
    return _DT[dtype]


def _refuse(t, name, device, dtype, shape, contiguous):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(t, name, device, dtype, shape, contiguous=True):
    """t is a tensor on the GPU `device` with `dtype` and `shape`."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.dtype == dtype and t.shape == shape and
            (not contiguous or t.is_contiguous())):
        _refuse(t, name, device, dtype, shape, contiguous)


def _size(t, name, dims):
    """The shape of a tensor of `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    return t.shape


def _rows(t, name, device, dtype, shape):
    """Row stride of strided rows [rows][heads][D] of that shape."""
    _check(t, name, device, dtype, shape, contiguous=False)
    rows, heads, D = shape
    if t.is_contiguous():
        return heads * D
    s0, s1, s2 = t.stride()
    if (D > 1 and s2 != 1) or (heads > 1 and s1 != D) or (rows > 1 and s0 < heads * D):
        raise ValueError(f"{name}: heads and columns must be contiguous, rows must not overlap")
    return s0 if rows > 1 else heads * D


class _On:
    """Makes `device` and the stream to launch on current (torch's allocator
    then hands out memory of that stream); gives the stream's handle."""

    __slots__ = ("guards", "handle")

    def __init__(self, device, stream):
        self.guards = []
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, not on {device}")
            self.guards.append(torch.cuda.stream(stream))       # sets the device as well
        elif device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        for g in self.guards:
            g.__enter__()
        self.handle = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        for g in self.guards:
            g.__exit__(*exc)


def _call(name, *args):
    st = getattr(attn_lib(), name)(*args)
    if st != NM_OK:
        raise NmError(name, st)


def qk_norm_rope(q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6, interleaved=False, out=None, stream=None):
    """Per-head RMS norms of q [T][Hq][D] and k [T][Hk][D] (weights wq, wk [D];
    None: no norm), then the rotation by positions[t] * inv_freq[i] of column
    pairs (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``; rot = 2 *
    len(inv_freq), further columns are not turned.  positions int32 [T],
    inv_freq float32.  Returns (q, k), contiguous; ``out`` is such a pair, and
    may be (q, k) themselves."""
    T, hq, D = _size(q, "q", 3)
    hk = _size(k, "k", 3)[1]
    pairs, = _size(inv_freq, "inv_freq", 1)
    dev, dt = q.device, q.dtype
    code = _dtype(dt)
    qs = _rows(q, "q", dev, dt, (T, hq, D))
    ks = _rows(k, "k", dev, dt, (T, hk, D))
    _check(positions, "positions", dev, torch.int32, (T,))
    _check(inv_freq, "inv_freq", dev, torch.float32, (pairs,))
    for w, name in ((wq, "wq"), (wk, "wk")):
        if w is not None:
            _check(w, name, dev, dt, (D,))
    if out is not None:
        _check(out[0], "out[0]", dev, dt, (T, hq, D))
        _check(out[1], "out[1]", dev, dt, (T, hk, D))
    with _On(dev, stream) as handle:
        if out is None:
            out = (torch.empty((T, hq, D), dtype=dt, device=dev), torch.empty((T, hk, D), dtype=dt, device=dev))
        _call("nm_qk_norm_rope", q.data_ptr(), qs, k.data_ptr(), ks, T, hq, hk, D, code,
              None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(), eps, positions.data_ptr(),
              inv_freq.data_ptr(), 2 * pairs, int(bool(interleaved)), out[0].data_ptr(),
              out[1].data_ptr(), handle)
    return out[0], out[1]


class KVCache:
    """A paged cache of keys and values: n_pages pages of page_size tokens,
    ``heads`` key heads of D columns.  format "16" keeps the 16-bit values,
    "mx8" and "mx4" keep 8- and 4-bit floats (e4m3, e2m1) with one power-of-two
    scale per 32 columns.  A slot is page * page_size + place in the page."""

    __slots__ = ("_buffers", "_struct", "_ref", "device", "dtype", "format", "n_pages", "page_size", "heads", "D")

    def __init__(self, n_pages, page_size, heads, D, dtype, format="16", device="cuda"):
        if format not in _FORMATS:
            raise ValueError(f"format must be one of {', '.join(_FORMATS)}, not {format}")
        code, fmt = _dtype(dtype), _FORMATS[format]
        nbytes = attn_lib().nm_kv_bytes(n_pages, page_size, heads, D, fmt)
        if nbytes < 0:
            raise ValueError(f"no cache of {n_pages} pages of {page_size} tokens, {heads} heads, {D} columns")
        sbytes = attn_lib().nm_kv_scale_bytes(n_pages, page_size, heads, D, fmt)
        k, v = (torch.zeros(nbytes, dtype=torch.uint8, device=device) for _ in range(2))
        k_scale, v_scale = (torch.zeros(sbytes, dtype=torch.uint8, device=device) if sbytes else None
                            for _ in range(2))
        self._buffers = (k, v, k_scale, v_scale)
        self.device, self.dtype, self.format = k.device, dtype, format
        self.n_pages, self.page_size, self.heads, self.D = n_pages, page_size, heads, D
        self._struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if sbytes else None,
                                     v_scale.data_ptr() if sbytes else None, n_pages, page_size, heads, D, code, fmt)
        self._ref = ctypes.addressof(self._struct)

    # The buffers, in the library's byte order (include/nmattn.h); fixed, since the handle holds their addresses.
    @property
    def k(self):
        return self._buffers[0]

    @property
    def v(self):
        return self._buffers[1]

    @property
    def k_scale(self):
        return self._buffers[2]

    @property
    def v_scale(self):
        return self._buffers[3]

    @property
    def nbytes(self):
        return sum(b.numel() for b in self._buffers if b is not None)


def _cache(cache):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    return cache


def kv_write(cache, k, v, slots, stream=None):
    """Row t of k and v [T][heads][D] into slot slots[t] (int64 [T]), quantised
    to the cache's format.  A negative slot, or one behind the last, is
    skipped; no slot twice in one call."""
    c = _cache(cache)
    T, = _size(slots, "slots", 1)
    _check(slots, "slots", c.device, torch.int64, (T,))
    shape = (T, c.heads, c.D)
    ks, vs = _rows(k, "k", c.device, c.dtype, shape), _rows(v, "v", c.device, c.dtype, shape)
    with _On(c.device, stream) as handle:
        _call("nm_kv_write", c._ref, k.data_ptr(), ks, v.data_ptr(), vs, T, slots.data_ptr(), handle)


def kv_read(cache, slots, out=None, stream=None):
    """(k, v) [T][heads][D] in the cache's dtype from slots (int64 [T]); zeros
    for a slot outside the cache."""
    c = _cache(cache)
    T, = _size(slots, "slots", 1)
    _check(slots, "slots", c.device, torch.int64, (T,))
    shape = (T, c.heads, c.D)
    if out is not None:
        _check(out[0], "out[0]", c.device, c.dtype, shape)
        _check(out[1], "out[1]", c.device, c.dtype, shape)
    with _On(c.device, stream) as handle:
        if out is None:
            out = tuple(torch.empty(shape, dtype=c.dtype, device=c.device) for _ in range(2))
        _call("nm_kv_read", c._ref, slots.data_ptr(), T, out[0].data_ptr(), out[1].data_ptr(), handle)
    return out[0], out[1]


def attn_workspace(B, heads_q, cache, max_len, prefix_len=0):
    """A workspace for attn_decode calls of this shape on the cache's device
    (any contents; calls that may run at the same time need one each)."""
    c = _cache(cache)
    nbytes = attn_lib().nm_attn_workspace_bytes(B, heads_q, c.heads, c.D, prefix_len, max_len)
    if nbytes < 0:
        raise ValueError(f"no such attention: {B} sequences, {heads_q} query heads on {c.heads}, {prefix_len} + "
                         f"{max_len} tokens")
    return torch.empty(nbytes, dtype=torch.uint8, device=c.device)


def attn_decode(q, cache, page_table, lens, max_len=None, prefix_pages=None, prefix_len=0, scale=None, out=None,
                lse=None, ws=None, stream=None):
    """Attention of one query token per sequence, q [B][Hq][D], over the cache.
    Sequence b sees the prefix (the first prefix_len tokens of prefix_pages,
    int32, shared by the batch and read once) and then lens[b] (int32 [B],
    device; at most max_len) tokens of its own pages page_table[b] (int32
    [B][pages]); lens[b] < 0 marks a padding row, which is left as it was.
    scale defaults to 1/sqrt(D); max_len to the table's width.  Returns out
    [B][Hq][D]; ``lse`` (float32 [B][Hq]) receives the log of the softmax's
    sum.  ``ws``: an attn_workspace(), or None to allocate one."""
    c = _cache(cache)
    dev, dt = c.device, c.dtype
    B, hq, _ = _size(q, "q", 3)
    qs = _rows(q, "q", dev, dt, (B, hq, c.D))
    _check(lens, "lens", dev, torch.int32, (B,))
    table, stride, width = None, 0, 0
    if page_table is not None:
        width = _size(page_table, "page_table", 2)[1]
        _check(page_table, "page_table", dev, torch.int32, (B, width), contiguous=False)
        stride = width
        if not page_table.is_contiguous():
            if width > 1 and page_table.stride(1) != 1:
                raise ValueError("page_table rows must be contiguous")
            stride = page_table.stride(0)
        table, width = page_table.data_ptr(), width * c.page_size
    max_len = width if max_len is None else max_len
    if max_len > width:
        raise ValueError(f"max_len {max_len} is more than page_table holds ({width} tokens)")
    if prefix_len:
        n, = _size(prefix_pages, "prefix_pages", 1)
        _check(prefix_pages, "prefix_pages", dev, torch.int32, (n,))
        if prefix_len > n * c.page_size:
            raise ValueError(f"prefix_len {prefix_len} is more than prefix_pages holds ({n * c.page_size} tokens)")
    if out is not None:
        _check(out, "out", dev, dt, (B, hq, c.D))
    if lse is not None:
        _check(lse, "lse", dev, torch.float32, (B, hq))
    if ws is not None:
        _check(ws, "ws", dev, torch.uint8, _size(ws, "ws", 1))
    need = attn_lib().nm_attn_workspace_bytes(B, hq, c.heads, c.D, prefix_len, max_len)
    with _On(dev, stream) as handle:
        if out is None:
            out = torch.empty((B, hq, c.D), dtype=dt, device=dev)
        if ws is None and need > 0:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _call("nm_attn_decode", q.data_ptr(), qs, B, hq, c._ref, None if prefix_len == 0 else prefix_pages.data_ptr(),
              prefix_len, table, stride, lens.data_ptr(), max_len, 1.0 / math.sqrt(c.D) if scale is None else scale,
              out.data_ptr(), None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
              0 if ws is None else ws.numel(), handle)
    return out
