"""A serving cache in fewer bits, and attention of drafted tokens over it.

Marshalling over the C ABI, as in api.py: tensors are checked, outputs allocated with
torch, and the library's kernels do every step of the computation.
"""
from __future__ import annotations

import math

import torch

from . import binding as _b
from .api import _DTYPES, _call_on, _like, _scratch, _share, _stream_on

_FORMATS = {"bf16": _b.CACHE_BF16, "mxfp8": _b.CACHE_MXFP8, "mxfp4": _b.CACHE_MXFP4}
_BLOCK = 32


def _code_width(D: int, format: str) -> int:
    return D // 2 if format == "mxfp4" else D


class KVCache:
    """Rows of K and V for B sequences in one format.

    format "bf16": k, v [B, Hkv, capacity, D] bfloat16. "mxfp8": uint8 e4m3 codes
    [B, Hkv, capacity, D]; "mxfp4": two e2m1 codes per byte [B, Hkv, capacity, D/2]; both
    with k_scale, v_scale uint8 [B, Hkv, capacity, D/32] (the byte is the scale's exponent
    + 127). capacity is a multiple of 16. The tensors are the caller's: nothing is copied.
    """

    def __init__(self, format: str, k, v, k_scale=None, v_scale=None):
        if format not in _FORMATS:
            raise ValueError(f"format must be one of {sorted(_FORMATS)}")
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [B, Hkv, capacity, width] tensors of one shape")
        want = torch.bfloat16 if format == "bf16" else torch.uint8
        tensors = [k, v] if format == "bf16" else [k, v, k_scale, v_scale]
        self.D = k.shape[3] * (2 if format == "mxfp4" else 1)
        if format != "bf16":
            shape = (*k.shape[:3], self.D // _BLOCK)
            for s in (k_scale, v_scale):
                if s is None or tuple(s.shape) != shape or s.dtype != torch.uint8:
                    raise ValueError("k_scale and v_scale must be uint8 [B, Hkv, capacity, D/32]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        if k.dtype != want or v.dtype != want:
            raise ValueError(f"a {format} cache keeps its rows as {want}")
        if any(t.device != k.device for t in tensors):
            raise ValueError("the cache's tensors must be on one device")
        if not all(t.is_contiguous() for t in tensors):
            raise ValueError("the cache's tensors must be contiguous")
        self.format, self.k, self.v, self.k_scale, self.v_scale = format, k, v, k_scale, v_scale
        self.B, self.Hkv, self.capacity = k.shape[:3]

    @classmethod
    def allocate(cls, B: int, Hkv: int, capacity: int, D: int, format: str = "mxfp8", device="cuda") -> "KVCache":
        """A cache of uninitialised rows (capacity is rounded up to a multiple of 16)."""
        if format not in _FORMATS:
            raise ValueError(f"format must be one of {sorted(_FORMATS)}")
        if D not in (64, 128):
            raise ValueError("D must be 64 or 128")
        cap = (capacity + 15) // 16 * 16
        if format == "bf16":
            return cls(format, *(torch.empty(B, Hkv, cap, D, dtype=torch.bfloat16, device=device) for _ in range(2)))
        rows = [torch.empty(B, Hkv, cap, _code_width(D, format), dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.empty(B, Hkv, cap, D // _BLOCK, dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(format, *rows, *scales)

    def bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._tensors() if t is not None)

    def _tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale

    def _pointers(self):
        if self.k_scale is None:
            return self.k.data_ptr(), self.v.data_ptr(), 0, 0
        return self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr()


def _int_rows(t, shape, name, device) -> int:
    """Address of an int32 tensor of this shape (0 for None)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on the cache's device")
    return t.data_ptr()


def _required(t, name):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _strides(t):
    """Element strides of the first three dimensions (those of size 1 do not matter)."""
    (n0, n1, n2, _), (s0, s1, s2, _) = t.shape, t.stride()
    return s0 if n0 > 1 else 0, s1 if n1 > 1 else 0, s2 if n2 > 1 else 0


def _int31(x) -> int:
    """x for a C int in which everything past the largest sequence, or below 0, means the same."""
    return max(-1, min(int(x), 2 ** 31 - 1))


def _on_device(cache: KVCache):
    dev = cache.k.device
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    return dev


def cache_write(cache: KVCache, k_new, v_new, start, count=None, index=None, workspace=None, stream=None) -> None:
    """Write new rows into the cache in its format.

    k_new, v_new [B, Hkv, T, D] bf16 or fp32 with any strides that keep rows 16-byte
    aligned and the head dimension contiguous (a slice of a fused projection is fine).
    Cache row start[b] + i becomes new row i for i < count[b] (default: all T). With
    index [B, n] int32 there are n rows to write and row i comes from new row index[b, i].
    No other row is touched; rows that would fall outside the cache are skipped, which
    `status` reports for a given `workspace` (uint8, >= 256 bytes). The new rows must not be
    rows of the cache itself. Asynchronous on `stream`.
    """
    dev = _on_device(cache)
    for t in (k_new, v_new):
        if t.dim() != 4 or t.shape[0] != cache.B or t.shape[1] != cache.Hkv or t.shape[3] != cache.D:
            raise ValueError("k_new and v_new must be [B, Hkv, T, D] like the cache")
        if t.dtype not in _DTYPES or t.dtype != k_new.dtype or t.device != dev:
            raise ValueError("k_new and v_new must share dtype float32 or bfloat16 and the cache's device")
        if t.stride(3) != 1:
            raise ValueError("the head dimension of k_new and v_new must be contiguous")
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must have one shape")
    T_src = k_new.shape[2]
    T = T_src if index is None else index.shape[-1]
    p_start = _int_rows(_required(start, "start"), (cache.B,), "start", dev)
    p_count = _int_rows(count, (cache.B,), "count", dev)
    p_index = _int_rows(index, (cache.B, T), "index", dev)
    ws, ws_bytes = (0, 0) if workspace is None else (_scratch(workspace, 0, dev).data_ptr(), workspace.nbytes)
    if T == 0:  # nothing to write, which the status word has to say
        if workspace is not None:
            if ws_bytes < 256:
                raise _b.RingAttnError(_b.EWORKSPACE, "ring_attn_cache_write")
            with torch.cuda.stream(stream):
                workspace.reshape(-1).view(torch.uint8)[:4].zero_()
        return
    if T_src == 0:
        raise ValueError("index picks rows of k_new and v_new, which have none")
    rc = _call_on(dev, _b.ring_attn_cache_write, k_new.data_ptr(), v_new.data_ptr(),
                  (*_strides(k_new), *_strides(v_new)), _DTYPES[k_new.dtype], *cache._pointers(),
                  _FORMATS[cache.format], cache.B, cache.Hkv, cache.capacity, cache.D, T, T_src, p_start, p_count,
                  p_index, ws, ws_bytes, _stream_on(stream, dev))
    _b.check(rc, "ring_attn_cache_write")
    _share(stream, dev, (*cache._tensors(), k_new, v_new, start, count, index, workspace))


def cache_read(cache: KVCache, start, T: int, count=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """Read rows [start[b], start[b] + T) back as the values they stand for.

    Returns (k, v) [B, Hkv, T, D] in dtype (bf16 or fp32); rows i >= count[b] and rows
    outside the cache are zeros. Asynchronous on `stream`.
    """
    dev = _on_device(cache)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    shape = (cache.B, cache.Hkv, T, cache.D)
    k_out = _like(k_out, cache.k, "k_out", shape, dtype, stream)
    v_out = _like(v_out, cache.k, "v_out", shape, dtype, stream)
    if T == 0:
        return k_out, v_out
    p_start = _int_rows(_required(start, "start"), (cache.B,), "start", dev)
    p_count = _int_rows(count, (cache.B,), "count", dev)
    rc = _call_on(dev, _b.ring_attn_cache_read, *cache._pointers(), _FORMATS[cache.format], cache.B, cache.Hkv,
                  cache.capacity, cache.D, T, p_start, p_count, k_out.data_ptr(), v_out.data_ptr(), _DTYPES[dtype],
                  _stream_on(stream, dev))
    _b.check(rc, "ring_attn_cache_read")
    _share(stream, dev, (*cache._tensors(), start, count), (k_out, v_out))
    return k_out, v_out


def _tree_bytes(q, cache: KVCache) -> int:
    B, Hq, T, D = q.shape
    n = _b.ring_attn_tree_workspace_bytes(_FORMATS[cache.format], B, Hq, cache.Hkv, cache.capacity, D, T)
    if n == 0:
        raise _b.RingAttnError(_b.EINVAL, "ring_attn_tree_workspace_bytes")
    return n


def tree_workspace(q, cache: KVCache) -> torch.Tensor:
    """Scratch for tree_attention calls of q's shape over this cache (one call at a time)."""
    return _scratch(None, _tree_bytes(q, cache), cache.k.device)


def tree_attention(q, cache: KVCache, lengths, parents=None, counts=None, window: int = 0, sinks: int = 0,
                   scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of T drafted tokens per sequence over its cache (T = 1: ordinary decoding).

    q [B, Hq, T, D] bf16 (rows 16-byte aligned, any other strides). Sequence b holds
    lengths[b] committed rows; its drafted node j has been written to cache row
    lengths[b] + j. parents [B, T] int32 gives the tree (parent in [-1, j), -1 the last
    committed token; None: a chain). Node t sees all committed tokens, its ancestors and
    itself, or, with window > 0, of these the last `window` positions up to its own
    (lengths[b] + its depth) and the first `sinks`. counts [B] gives the live nodes; rows of
    dead ones are 0 with lse = -inf. Returns (out [B, Hq, T, D] bf16, lse [B, Hq, T] fp32).
    Asynchronous on `stream`.
    """
    dev = _on_device(cache)
    if q.dim() != 4 or q.shape[0] != cache.B or q.shape[3] != cache.D:
        raise ValueError("q must be [B, Hq, T, D] like the cache")
    if q.dtype != torch.bfloat16 or q.device != dev or q.stride(3) != 1:
        raise ValueError("q must be a bf16 tensor on the cache's device with a contiguous head dimension")
    B, Hq, T, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    out = _like(out, q, "out", (B, Hq, T, D), torch.bfloat16, stream)
    lse = _like(lse, q, "lse", (B, Hq, T), torch.float32, stream)
    p_len = _int_rows(_required(lengths, "lengths"), (B,), "lengths", dev)
    p_par = _int_rows(parents, (B, T), "parents", dev)
    p_cnt = _int_rows(counts, (B,), "counts", dev)
    workspace = _scratch(workspace, _tree_bytes(q, cache) if workspace is None else 0, dev, stream)
    rc = _call_on(dev, _b.ring_attn_tree, q.data_ptr(), _strides(q), *cache._pointers(), _FORMATS[cache.format],
                  out.data_ptr(), lse.data_ptr(), B, Hq, cache.Hkv, cache.capacity, D, T, p_len, p_par, p_cnt,
                  _int31(window), _int31(sinks), scale, workspace.data_ptr(), workspace.nbytes, _stream_on(stream, dev))
    _b.check(rc, "ring_attn_tree")
    _share(stream, dev, (*cache._tensors(), q, lengths, parents, counts, workspace), (out, lse))
    return out, lse
