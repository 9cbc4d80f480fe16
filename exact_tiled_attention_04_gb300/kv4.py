"""PyTorch conveniences for the 4-bit key/value cache and for the attention
weight of a prompt: tensor checks, allocation of outputs, and one call of the
C entry point each (include/fa.h documents format, results and errors).

Every call is enqueued on `stream` (default: the device's current stream), and
what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import binding as _b


torch = None  # PyTorch, imported by the first call (importing the package does not need it)


def _need_torch():
    global torch
    if torch is None:
        import torch as module
        torch = module


@functools.lru_cache(maxsize=None)
def _default_scale(d: int) -> float:
    return float(torch.tensor(1.0, dtype=torch.float32) / torch.sqrt(torch.tensor(float(d), dtype=torch.float32)))


def _scale(scale, d: int) -> float:
    if scale is None:
        return _default_scale(d)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    return float(scale)


def _empty(shape, dtype, device, stream, returned: bool = True):
    """Memory for a call on `stream` (None: the current one)."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    return _b._empty_on(stream, shape, dtype, device, returned)


def _call(where: str, function, device, stream, *args):
    """One C call on `stream` (None: the device's current one) with the
    device made current where it is not."""
    current = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        status = function(*args, current or None)
    else:
        with torch.cuda.device(device):
            status = function(*args, current or None)
    if status != _b.FA_OK:
        raise _b.FAError(status, where)


def _check(t, what: str, dtype, shape, device):
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what} must be a contiguous CUDA tensor on {device}")


def _rows(t, what: str, device) -> int:
    """Check 16-bit rows [batch, heads, rows, d]; their dtype code."""
    if t.dim() != 4:
        raise ValueError(f"{what} must be [batch, heads, rows, d], got {tuple(t.shape)}")
    dtype = t.dtype
    code = _b.FA_DTYPE_BF16 if dtype is torch.bfloat16 else _b.FA_DTYPE_F16 if dtype is torch.float16 else None
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float16, got {dtype}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor on {device}")
    return code


class KV4Cache:
    """A 4-bit key/value cache: the caller's tensors and their addresses.

    k_codes, v_codes [B, H_kv, capacity, d // 2] and k_scales, v_scales
    [B, H_kv, capacity, d // 16] uint8; counts int32 [2, B] (length, tokens
    appended); pos int32 and weight fp32 [B, H_kv, capacity], each optional.
    capacity is a multiple of 128, d is 64 or 128.  The tensors are checked
    here once; replace none of them afterwards.

    Blocks of 16 channels below 0.006 in magnitude are stored as zeros, below
    0.094 with fewer bits, above 2688 saturated: multiply keys or values out of
    that range by a power of two before storing them, and `scale` or the output
    by its inverse.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, counts, pos=None, weight=None):
        _need_torch()
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes must be [B, H_kv, capacity, d // 2], got {tuple(k_codes.shape)}")
        B, H_kv, capacity, half = (int(x) for x in k_codes.shape)
        d, dev = 2 * half, k_codes.device
        if d not in (64, 128) or capacity < 1 or capacity % 128:
            raise ValueError(f"d must be 64 or 128 and capacity a multiple of 128, got {d} and {capacity}")
        for t, what, dtype, shape in ((k_codes, "k_codes", torch.uint8, (B, H_kv, capacity, half)),
                                      (v_codes, "v_codes", torch.uint8, (B, H_kv, capacity, half)),
                                      (k_scales, "k_scales", torch.uint8, (B, H_kv, capacity, d // 16)),
                                      (v_scales, "v_scales", torch.uint8, (B, H_kv, capacity, d // 16)),
                                      (counts, "counts", torch.int32, (2, B)),
                                      (pos, "pos", torch.int32, (B, H_kv, capacity)),
                                      (weight, "weight", torch.float32, (B, H_kv, capacity))):
            if t is not None:
                _check(t, what, dtype, shape, dev)
        if dev.type != "cuda":
            raise ValueError(f"k_codes must be a contiguous CUDA tensor, is on {dev}")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.counts, self.pos, self.weight = counts, pos, weight
        self.B, self.H_kv, self.capacity, self.d, self.device = B, H_kv, capacity, d, dev
        self._struct = _b.fa_kv4_cache_t(
            k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
            weight.data_ptr() if weight is not None else None, pos.data_ptr() if pos is not None else None,
            counts.data_ptr(), B, H_kv, capacity, d)
        self._ref = ctypes.pointer(self._struct)
        self._need = {}

    @classmethod
    def empty(cls, B: int, H_kv: int, capacity: int, d: int, device="cuda", pos: bool = True, weight: bool = True):
        """An empty cache of at least `capacity` slots (rounded up to a multiple of 128)."""
        _need_torch()
        cap = max(128, -(-capacity // 128) * 128)
        new = functools.partial(torch.zeros, device=device)
        return cls(new((B, H_kv, cap, d // 2), dtype=torch.uint8), new((B, H_kv, cap, d // 16), dtype=torch.uint8),
                   new((B, H_kv, cap, d // 2), dtype=torch.uint8), new((B, H_kv, cap, d // 16), dtype=torch.uint8),
                   new((2, B), dtype=torch.int32), pos=new((B, H_kv, cap), dtype=torch.int32) if pos else None,
                   weight=new((B, H_kv, cap), dtype=torch.float32) if weight else None)

    @property
    def lengths(self):
        """int32 [B]: slots in use (a view of counts)."""
        return self.counts[0]

    def workspace_size(self, H: int, N_q: int, with_weight: bool) -> int:
        """Bytes kv4_attention needs for these sizes on the cache's device."""
        key = (H, N_q, bool(with_weight))
        if key not in self._need:
            with torch.cuda.device(self.device):
                self._need[key] = _b.fa_kv4_fwd_workspace_size(self.B, H, self.H_kv, N_q, self.capacity, self.d,
                                                               int(with_weight))
        return self._need[key]


def kv4_append(cache: KV4Cache, k, v, counts_out=None, stream=None):
    """Store k, v [B, H_kv, n, d] (bf16 or fp16) behind the cache's last
    entries; the counts advance in place, or go to `counts_out` (int32
    [2, B]).  Rows past the capacity are dropped and reported by
    fa_device_status (FA_ERR_CAPACITY).  Returns the advanced counts."""
    code = _rows(k, "k", cache.device)
    if v.dtype != k.dtype:
        raise TypeError("k and v must share a dtype")
    _check(v, "v", k.dtype, k.shape, cache.device)
    B, H_kv, n, d = k.shape
    if B != cache.B or H_kv != cache.H_kv or d != cache.d:
        raise ValueError(f"k must be [{cache.B}, {cache.H_kv}, n, {cache.d}], got {tuple(k.shape)}")
    if counts_out is None:
        counts_out = cache.counts
    else:
        _check(counts_out, "counts_out", torch.int32, (2, B), cache.device)
    _call("fa_kv4_append", _b.load().fa_kv4_append, cache.device, stream,
          cache._ref, k.data_ptr(), v.data_ptr(), n, code, counts_out.data_ptr())
    return counts_out


def kv4_read(cache: KV4Cache, count: int, first=None, dtype=None, k=None, v=None, stream=None):
    """The values (k, v) [B, H_kv, count, d] of `count` slots from first[b] on
    (int32 [B]; default 0), exactly as attention sees them.  dtype: bfloat16
    (default) or float16."""
    if dtype is None or dtype == torch.bfloat16:
        dtype, code = torch.bfloat16, _b.FA_DTYPE_BF16
    elif dtype == torch.float16:
        code = _b.FA_DTYPE_F16
    else:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    shape = (cache.B, cache.H_kv, count, cache.d)
    if k is None:
        k = _empty(shape, dtype, cache.device, stream)
    else:
        _check(k, "k", dtype, shape, cache.device)
    if v is None:
        v = _empty(shape, dtype, cache.device, stream)
    else:
        _check(v, "v", dtype, shape, cache.device)
    if first is not None:
        _check(first, "first", torch.int32, (cache.B,), cache.device)
    _call("fa_kv4_read", _b.load().fa_kv4_read, cache.device, stream,
          cache._ref, first.data_ptr() if first is not None else None, count, k.data_ptr(), v.data_ptr(), code)
    return k, v


def kv4_attention(q, cache: KV4Cache, scale: float | None = None, causal: bool = False, out=None, lse=None,
                  with_lse: bool = True, weight_out=None, workspace=None, stream=None):
    """O = softmax(scale * Q K^T) V for q [B, H, N_q, d] (bf16 or fp16) over
    the cache's entries; H a multiple of H_kv, N_q * H / H_kv <= 128.

    Returns (out, lse) as `attention` does.  causal: query i sees slots
    j < length - (N_q - 1 - i).  weight_out: fp32 [B, H_kv, capacity], gets
    cache.weight (or 0) plus each entry's softmax weights (pass cache.weight
    to accumulate in place).  `workspace` (uint8, cache.workspace_size(...)
    bytes) is allocated when not given."""
    device = cache.device
    code = _rows(q, "q", device)
    B, H, N_q, d = q.shape
    if B != cache.B or d != cache.d or H % cache.H_kv:
        raise ValueError(f"q must be [{cache.B}, a multiple of {cache.H_kv}, N_q, {cache.d}], got {tuple(q.shape)}")
    if out is None:
        out = _empty((B, H, N_q, d), q.dtype, device, stream)
    else:
        _check(out, "out", q.dtype, q.shape, device)
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, H, N_q), device)
    elif with_lse:
        lse = _empty((B, H, N_q), torch.float32, device, stream)
    if weight_out is not None:
        _check(weight_out, "weight_out", torch.float32, (B, cache.H_kv, cache.capacity), device)
    if workspace is None:
        size = max(cache.workspace_size(H, N_q, weight_out is not None), 16)
        workspace = _empty(size, torch.uint8, device, stream, returned=False)
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
    _call("fa_kv4_fwd", _b.load().fa_kv4_fwd, device, stream,
          cache._ref, q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
          weight_out.data_ptr() if weight_out is not None else None, H, N_q, _scale(scale, d),
          code | _b.FA_FLAG_CAUSAL if causal else code, workspace.data_ptr(), size)
    return out, lse


def kv4_evict(cache: KV4Cache, keep: int, sinks: int = 0, recent: int = 0, weight=None, out: KV4Cache | None = None,
              counts_out=None, src=None, stream=None):
    """Keep each head's `keep` entries of largest weight (`weight` fp32
    [B, H_kv, capacity], default cache.weight), and first of all those with
    pos < sinks or among the `recent` newest.  In place, or into the cache
    `out`; the new counts go to the cache that holds the result, or to
    `counts_out`.  Returns src int32 [B, H_kv, keep]: the slot each slot's
    entry came from, -1 behind the last."""
    if keep < 1:
        raise ValueError(f"keep must be at least 1, got {keep}")
    if weight is not None:
        _check(weight, "weight", torch.float32, (cache.B, cache.H_kv, cache.capacity), cache.device)
    if src is None:
        src = _empty((cache.B, cache.H_kv, keep), torch.int32, cache.device, stream)
    else:
        _check(src, "src", torch.int32, (cache.B, cache.H_kv, keep), cache.device)
    if counts_out is None:
        counts_out = (cache if out is None else out).counts
    else:
        _check(counts_out, "counts_out", torch.int32, (2, cache.B), cache.device)
    if out is not None and out.device != cache.device:
        raise ValueError(f"out must be on {cache.device}")
    _call("fa_kv4_evict", _b.load().fa_kv4_evict, cache.device, stream,
          cache._ref, keep, sinks, recent, weight.data_ptr() if weight is not None else None,
          out._ref if out is not None else None, src.data_ptr(), counts_out.data_ptr())
    return src


def _weight_stride(t, what: str, shape, device) -> int:
    """Distance between the heads' rows of a [B, H_kv, N_kv] tensor whose
    rows are contiguous and equally far apart."""
    if t.dtype != torch.float32 or t.shape != shape or t.device != device:
        raise ValueError(f"{what} must be fp32 {shape} on {device}")
    B, H_kv, N_kv = shape
    s0, s1, s2 = t.stride()
    # a dimension of size 1 has no stride of its own
    row = s1 if H_kv > 1 else s0 if B > 1 else N_kv
    if (N_kv > 1 and s2 != 1) or (B > 1 and s0 != H_kv * row) or row < N_kv:
        raise ValueError(f"{what} must have contiguous rows, equally far apart")
    return row


def attention_weights(q, k, lse, scale: float | None = None, causal: bool = False, first_query: int = 0,
                      weight_in=None, out=None, stream=None):
    """The attention weight each key of a prompt receives: `weight_in` (or 0)
    plus the sum over a group's query heads and the queries from `first_query`
    on of exp(scale q.k - lse), fp32 [B, H_kv, N_kv].  q [B, H, N_q, d],
    k [B, H_kv, N_kv, d] (bf16 or fp16) and lse [B, H, N_q] as `attention`
    took and returned them.  `out` and `weight_in` may be the first N_kv
    columns of a cache's weight (same strides), and the same tensor."""
    _need_torch()
    device = q.device
    if device.type != "cuda":
        raise ValueError(f"q must be a contiguous CUDA tensor, is on {device}")
    code = _rows(q, "q", device)
    _rows(k, "k", device)
    if k.dtype != q.dtype:
        raise TypeError("q and k must share a dtype")
    B, H, N_q, d = q.shape
    _, H_kv, N_kv, _ = k.shape
    if k.shape[0] != B or k.shape[3] != d or H_kv < 1 or H % H_kv:
        raise ValueError(f"incompatible q and k shapes: {tuple(q.shape)} {tuple(k.shape)}")
    _check(lse, "lse", torch.float32, (B, H, N_q), device)
    shape = (B, H_kv, N_kv)
    if out is None:
        out = _empty(shape, torch.float32, device, stream)
    stride = _weight_stride(out, "out", shape, device)
    if weight_in is not None and _weight_stride(weight_in, "weight_in", shape, device) != stride:
        raise ValueError("weight_in and out must have the same strides")
    _call("fa_fwd_weights", _b.load().fa_fwd_weights, device, stream,
          q.data_ptr(), k.data_ptr(), lse.data_ptr(), weight_in.data_ptr() if weight_in is not None else None,
          out.data_ptr(), stride, B, H, H_kv, N_q, N_kv, d, first_query, _scale(scale, d),
          code | _b.FA_FLAG_CAUSAL if causal else code)
    return out
