"""Between a decode layer's q+k+v and o projections: Python face of
``include/nmattn.h``.

q, k and v are [rows][heads][D] tensors whose heads and columns are contiguous;
rows may be strided (views of a fused q+k+v buffer).  Work runs on ``stream``
(default: the current stream of the tensors' device); results and workspaces
that a call allocates belong to that stream.
"""
import ctypes

import torch

from ._lib import (NM_BF16, NM_FP16, NM_KV_16, NM_KV_MX4, NM_KV_MX8, NM_OK, KvCacheStruct, NmError, attn_lib)

_DT = {torch.float16: NM_FP16, torch.bfloat16: NM_BF16}
_FORMATS = {"16": NM_KV_16, "mx8": NM_KV_MX8, "mx4": NM_KV_MX4}


def _dtype(dtype):
    if dtype not in _DT:
        raise TypeError(f"libnmspmv supports float16 and bfloat16, not {dtype}")
    return _DT[dtype]


# Devices are numbers here (of a GPU; -1: the host), since comparing device objects
# is what a check of a tensor would spend most of its time on.

def _refuse(t, name, device, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(t, name, device, dtype, shape):
    """Address of t, which is a contiguous tensor on the GPU `device` with
    `dtype` and `shape`."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.shape == shape and
            t.is_contiguous()):
        _refuse(t, name, device, dtype, shape)
    return t.data_ptr()


def _size(t, name, dims):
    """The shape of a tensor of `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {len(shape)}")
    return shape


def _rows(t, name, device, dtype, shape):
    """Address and row stride of strided rows [rows][heads][D] of that shape."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.shape == shape):
        _refuse(t, name, device, dtype, shape)
    rows, heads, D = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * D
    s0, s1, s2 = t.stride()
    if (D > 1 and s2 != 1) or (heads > 1 and s1 != D) or (rows > 1 and s0 < heads * D):
        raise ValueError(f"{name}: heads and columns must be contiguous, rows must not overlap")
    return t.data_ptr(), s0 if rows > 1 else heads * D


# A decode step's calls take Python longer than the GPU, so the common case, the
# current stream of the current device, goes through torch's own shortcuts where it
# has them (a stream object alone costs 2 us).
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Other:
    """Another stream or device than the current ones, made current until
    close() (torch's allocator then hands out memory of that stream)."""

    def __init__(self, device, stream):
        if stream is not None and stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, not on cuda:{device}")
        self.guard = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)
        self.guard.__enter__()

    def close(self):
        self.guard.__exit__(None, None, None)


def _other(device, stream):
    """None where work goes to the current stream of the current device."""
    if device < 0:
        raise TypeError("tensors must be CUDA (HIP) tensors")
    return None if stream is None and device == _device() else _Other(device, stream)


_lib = None


def _load():
    global _lib
    _lib = attn_lib()
    return _lib


def _fit(*sizes):
    """Whether sizes are those of a C call's arguments: ctypes would cut others to their low bits."""
    return all(0 <= n < 2 ** 31 for n in sizes)


def _rot(pairs):
    """Columns that so many frequencies turn, as a C int (more than any head has where they do not fit)."""
    return 2 * min(pairs, 2 ** 30 - 1)


def _empty(like, stride):
    """A new contiguous tensor of the shape, dtype and device of the rows `like`,
    whose row stride _rows() found to be `stride`."""
    rows, heads, D = like.shape
    return torch.empty_like(like) if stride == heads * D else like.new_empty((rows, heads, D))


def qk_norm_rope(q, k, positions, inv_freq, wq=None, wk=None, eps=1e-6, interleaved=False, out=None, stream=None):
    """Per-head RMS norms of q [T][Hq][D] and k [T][Hk][D] (weights wq, wk [D];
    None: no norm), then the rotation by positions[t] * inv_freq[i] of column
    pairs (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``; rot = 2 *
    len(inv_freq), further columns are not turned.  positions int32 [T],
    inv_freq float32.  Returns (q, k), contiguous; ``out`` is such a pair, and
    may be (q, k) themselves."""
    shape = _size(q, "q", 3)
    T, hq, D = shape
    hk = _size(k, "k", 3)[1]
    pairs, = _size(inv_freq, "inv_freq", 1)
    dev, dt = q.get_device(), q.dtype
    code = _dtype(dt)
    qp, qs = _rows(q, "q", dev, dt, shape)
    kp, ks = _rows(k, "k", dev, dt, (T, hk, D))
    pos = _check(positions, "positions", dev, torch.int32, (T,))
    freq = _check(inv_freq, "inv_freq", dev, torch.float32, (pairs,))
    wqp = None if wq is None else _check(wq, "wq", dev, dt, (D,))
    wkp = None if wk is None else _check(wk, "wk", dev, dt, (D,))
    other = _other(dev, stream)
    try:
        if out is None:
            out = oq, ok = _empty(q, qs), _empty(k, ks)
            oqp, okp = oq.data_ptr(), ok.data_ptr()
        else:
            oqp = _check(out[0], "out[0]", dev, dt, shape)
            okp = _check(out[1], "out[1]", dev, dt, (T, hk, D))
        st = (_lib or _load()).nm_qk_norm_rope(qp, qs, kp, ks, T, hq, hk, D, code, wqp, wkp, eps, pos, freq,
                                               _rot(pairs), 1 if interleaved else 0, oqp, okp, _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_qk_norm_rope", st)
    return out[0], out[1]


class KVCache:
    """A paged cache of keys and values: n_pages pages of page_size tokens,
    ``heads`` key heads of D columns.  format "16" keeps the 16-bit values,
    "mx8" and "mx4" keep 8- and 4-bit floats (e4m3, e2m1) with one power-of-two
    scale per 32 columns.  A slot is page * page_size + place in the page."""

    __slots__ = ("_buffers", "_struct", "_ref", "_format", "_index", "device", "dtype", "format", "n_pages", "page_size", "heads", "D")

    def __init__(self, n_pages, page_size, heads, D, dtype, format="16", device="cuda"):
        if format not in _FORMATS:
            raise ValueError(f"format must be one of {', '.join(_FORMATS)}, not {format}")
        code, fmt = _dtype(dtype), _FORMATS[format]
        sizes = (n_pages, page_size, heads, D)
        nbytes = attn_lib().nm_kv_bytes(*sizes, fmt) if _fit(*sizes) else -1
        if nbytes < 0:
            raise ValueError(f"no cache of {n_pages} pages of {page_size} tokens, {heads} heads, {D} columns")
        sbytes = attn_lib().nm_kv_scale_bytes(n_pages, page_size, heads, D, fmt)
        k, v = (torch.zeros(nbytes, dtype=torch.uint8, device=device) for _ in range(2))
        k_scale, v_scale = (torch.zeros(sbytes, dtype=torch.uint8, device=device) if sbytes else None
                            for _ in range(2))
        self._buffers = (k, v, k_scale, v_scale)
        self.device, self.dtype, self.format, self._format = k.device, dtype, format, fmt
        self._index = k.get_device()
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
    dev, dt = c._index, c.dtype
    T, = _size(slots, "slots", 1)
    sp = _check(slots, "slots", dev, torch.int64, (T,))
    shape = (T, c.heads, c.D)
    kp, ks = _rows(k, "k", dev, dt, shape)
    vp, vs = _rows(v, "v", dev, dt, shape)
    other = _other(dev, stream)
    try:
        st = (_lib or _load()).nm_kv_write(c._ref, kp, ks, vp, vs, T, sp, _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_kv_write", st)


def kv_read(cache, slots, out=None, stream=None):
    """(k, v) [T][heads][D] in the cache's dtype from slots (int64 [T]); zeros
    for a slot outside the cache."""
    c = _cache(cache)
    dev, dt = c._index, c.dtype
    T, = _size(slots, "slots", 1)
    sp = _check(slots, "slots", dev, torch.int64, (T,))
    shape = (T, c.heads, c.D)
    other = _other(dev, stream)
    try:
        if out is None:
            k = slots.new_empty(shape, dtype=dt)
            out = k, torch.empty_like(k)
            kp, vp = k.data_ptr(), out[1].data_ptr()
        else:
            kp = _check(out[0], "out[0]", dev, dt, shape)
            vp = _check(out[1], "out[1]", dev, dt, shape)
        st = (_lib or _load()).nm_kv_read(c._ref, sp, T, kp, vp, _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_kv_read", st)
    return out[0], out[1]


def attn_workspace(B, heads_q, cache, max_len, prefix_len=0):
    """A workspace for attn_decode calls of this shape, or of no larger B,
    max_len and prefix_len, on the cache's device (any contents; calls that may
    run at the same time need one each)."""
    c = _cache(cache)
    nbytes = 0
    if B != 0:
        nbytes = attn_lib().nm_attn_workspace_bytes(B, heads_q, c.heads, c.D, c._format, prefix_len, max_len) \
            if _fit(B, heads_q, max_len, prefix_len) else -1
    if nbytes < 0:
        raise ValueError(f"no such attention: {B} sequences, {heads_q} query heads on {c.heads}, {prefix_len} + "
                         f"{max_len} tokens")
    return torch.empty(nbytes, dtype=torch.uint8, device=c.device)


def _no_sequences(q, c, max_len, prefix_len, out):
    """attn_decode of an empty batch: what the arguments alone can refuse, and an empty result."""
    attn_workspace(1, q.shape[1], c, max_len, prefix_len)
    if out is None:
        return torch.empty_like(q)
    _check(out, "out", c._index, c.dtype, q.shape)
    return out


def attn_decode(q, cache, page_table, lens, max_len=None, prefix_pages=None, prefix_len=0, scale=None, out=None,
                lse=None, ws=None, stream=None):
    """Attention of one query token per sequence, q [B][Hq][D], over the cache.
    Sequence b sees the prefix (the first prefix_len tokens of prefix_pages,
    int32, shared by the batch and read once) and then lens[b] (int32 [B],
    device; at most max_len) tokens of its own pages page_table[b] (int32
    [B][pages]); lens[b] < 0 marks a padding row, which is left as it was.
    scale defaults to 1/sqrt(D); max_len to the table's width.  Returns out
    [B][Hq][D]; ``lse`` (float32 [B][Hq]) receives the log of the softmax's
    sum.  ``ws``: an attn_workspace(), or None to allocate one.  A batch of no
    sequences gives an empty result."""
    c = _cache(cache)
    dev, dt = c._index, c.dtype
    B, hq, _ = _size(q, "q", 3)
    shape = (B, hq, c.D)
    qp, qs = _rows(q, "q", dev, dt, shape)
    lp = _check(lens, "lens", dev, torch.int32, (B,))
    table, stride, width = None, 0, 0
    if page_table is not None:
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
    pp = None
    if prefix_len:
        n, = _size(prefix_pages, "prefix_pages", 1)
        pp = _check(prefix_pages, "prefix_pages", dev, torch.int32, (n,))
        if not 0 < prefix_len <= n * c.page_size:
            raise ValueError(f"prefix_len {prefix_len} is not within what prefix_pages holds ({n * c.page_size} tokens)")
    lsep = None if lse is None else _check(lse, "lse", dev, torch.float32, (B, hq))
    wsp, nbytes = None, 0
    if ws is not None:
        nbytes, = _size(ws, "ws", 1)
        wsp = _check(ws, "ws", dev, torch.uint8, (nbytes,))
    if B == 0:                                        # no sequence: nothing to launch
        return _no_sequences(q, c, max_len, prefix_len, out)
    other = _other(dev, stream)
    try:
        if out is None:
            out = _empty(q, qs)
            op = out.data_ptr()
        else:
            op = _check(out, "out", dev, dt, shape)
        if ws is None:
            nbytes = (_lib or _load()).nm_attn_workspace_bytes(B, hq, c.heads, c.D, c._format, prefix_len, max_len)
            if nbytes > 0:
                ws = q.new_empty(nbytes, dtype=torch.uint8)
                wsp = ws.data_ptr()
        st = (_lib or _load()).nm_attn_decode(qp, qs, B, hq, c._ref, pp, prefix_len, table, stride, lp, max_len,
                                              c.D ** -0.5 if scale is None else scale, op, lsep, wsp, max(nbytes, 0),
                                              _stream(dev))
    finally:
        if other is not None:
            other.close()
    if st != NM_OK:
        raise NmError("nm_attn_decode", st)
    return out
