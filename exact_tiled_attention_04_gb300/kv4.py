"""PyTorch conveniences for the 4-bit key/value cache and for the attention
weight of a prompt: tensor checks, allocation of outputs, and one call of the
C entry point each (include/fa.h documents format, results and errors).
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import binding as _b


@functools.lru_cache(maxsize=None)
def _default_scale(d: int) -> float:
    import torch
    return float(torch.tensor(1.0, dtype=torch.float32) / torch.sqrt(torch.tensor(float(d), dtype=torch.float32)))


def _scale(scale, d: int) -> float:
    if scale is None:
        return _default_scale(d)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    return float(scale)


class _On:
    """The tensors' device as the current one, switched only when it is not."""

    def __init__(self, device):
        import torch
        self.guard = torch.cuda.device(device) if torch.cuda.current_device() != device.index else None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _stream(stream, device, *made):
    """The stream to launch on.  `made`: tensors allocated for this call, whose
    memory the allocator must not hand out again before another stream is done."""
    import torch
    current = torch.cuda.current_stream(device)
    if stream is None or stream == current:
        return current.cuda_stream
    for t in made:
        t.record_stream(stream)
    return stream.cuda_stream


def _check(t, what: str, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor on {device}")


def _rows(t, what: str, device):
    import torch
    if t.dim() != 4:
        raise ValueError(f"{what} must be [batch, heads, rows, d], got {tuple(t.shape)}")
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{what} must be bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda or (device is not None and t.device != device) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor" + (f" on {device}" if device is not None else ""))


def _done(status: int, where: str):
    if status != _b.FA_OK:
        raise _b.FAError(status, where)


class KV4Cache:
    """A 4-bit key/value cache: the caller's tensors and their addresses.

    k_codes, v_codes [B, H_kv, capacity, d // 2] and k_scales, v_scales
    [B, H_kv, capacity, d // 16] uint8; counts int32 [2, B] (length, tokens
    appended); pos int32 and weight fp32 [B, H_kv, capacity], each optional.
    capacity is a multiple of 128, d is 64 or 128.  The tensors are checked
    here once; replace none of them afterwards.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, counts, pos=None, weight=None):
        import torch
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
        import torch
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
            with _On(self.device):
                self._need[key] = _b.fa_kv4_fwd_workspace_size(self.B, H, self.H_kv, N_q, self.capacity, self.d,
                                                               int(with_weight))
        return self._need[key]


def kv4_append(cache: KV4Cache, k, v, counts_out=None, stream=None):
    """Store k, v [B, H_kv, n, d] (bf16 or fp16) behind the cache's last
    entries; the counts advance in place, or go to `counts_out` (int32
    [2, B]).  Rows past the capacity are dropped and reported by
    fa_device_status (FA_ERR_CAPACITY).  Returns the advanced counts."""
    import torch
    _rows(k, "k", cache.device)
    if v.dtype != k.dtype:
        raise TypeError("k and v must share a dtype")
    _check(v, "v", k.dtype, k.shape, cache.device)
    if (k.shape[0], k.shape[1], k.shape[3]) != (cache.B, cache.H_kv, cache.d):
        raise ValueError(f"k must be [{cache.B}, {cache.H_kv}, n, {cache.d}], got {tuple(k.shape)}")
    counts = cache.counts
    if counts_out is not None:
        _check(counts_out, "counts_out", torch.int32, (2, cache.B), cache.device)
        counts = counts_out
    with _On(cache.device):
        _done(_b.fa_kv4_append(cache._ref, k.data_ptr(), v.data_ptr(), k.shape[2], _b._dtype_code(k),
                               counts.data_ptr(), _stream(stream, cache.device)), "fa_kv4_append")
    return counts


def kv4_read(cache: KV4Cache, count: int, first=None, dtype=None, k=None, v=None, stream=None):
    """The values (k, v) [B, H_kv, count, d] of `count` slots from first[b] on
    (int32 [B]; default 0), exactly as attention sees them.  dtype: bfloat16
    (default) or float16."""
    import torch
    dtype = dtype or torch.bfloat16
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    shape = (cache.B, cache.H_kv, int(count), cache.d)
    made = []
    if k is None:
        made.append(k := torch.empty(shape, dtype=dtype, device=cache.device))
    else:
        _check(k, "k", dtype, shape, cache.device)
    if v is None:
        made.append(v := torch.empty(shape, dtype=dtype, device=cache.device))
    else:
        _check(v, "v", dtype, shape, cache.device)
    if first is not None:
        _check(first, "first", torch.int32, (cache.B,), cache.device)
    with _On(cache.device):
        _done(_b.fa_kv4_read(cache._ref, first.data_ptr() if first is not None else None, int(count), k.data_ptr(),
                             v.data_ptr(), _b._dtype_code(k), _stream(stream, cache.device, *made)), "fa_kv4_read")
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
    import torch
    _rows(q, "q", cache.device)
    B, H, N_q, d = q.shape
    if B != cache.B or d != cache.d or H % cache.H_kv:
        raise ValueError(f"q must be [{cache.B}, a multiple of {cache.H_kv}, N_q, {cache.d}], got {tuple(q.shape)}")
    made = []
    if out is None:
        made.append(out := torch.empty_like(q))
    else:
        _check(out, "out", q.dtype, q.shape, cache.device)
    if lse is not None:
        _check(lse, "lse", torch.float32, q.shape[:3], cache.device)
    elif with_lse:
        made.append(lse := torch.empty((B, H, N_q), dtype=torch.float32, device=cache.device))
    if weight_out is not None:
        _check(weight_out, "weight_out", torch.float32, (B, cache.H_kv, cache.capacity), cache.device)
    if workspace is None:
        need = cache.workspace_size(H, N_q, weight_out is not None)
        made.append(workspace := torch.empty(max(need, 16), dtype=torch.uint8, device=cache.device))
    elif workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {cache.device}")
    with _On(cache.device):
        _done(_b.fa_kv4_fwd(cache._ref, q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
                            weight_out.data_ptr() if weight_out is not None else None, H, N_q, _scale(scale, d),
                            _b._dtype_code(q) | (_b.FA_FLAG_CAUSAL if causal else 0), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream(stream, cache.device, *made)),
              "fa_kv4_fwd")
    return out, lse


def kv4_evict(cache: KV4Cache, keep: int, sinks: int = 0, recent: int = 0, weight=None, out: KV4Cache | None = None,
              counts_out=None, src=None, stream=None):
    """Keep each head's `keep` entries of largest weight (`weight` fp32
    [B, H_kv, capacity], default cache.weight), and first of all those with
    pos < sinks or among the `recent` newest.  In place, or into the cache
    `out`; the new counts go to the cache that holds the result, or to
    `counts_out`.  Returns src int32 [B, H_kv, keep]: the slot each slot's
    entry came from, -1 behind the last."""
    import torch
    if keep < 1:
        raise ValueError(f"keep must be at least 1, got {keep}")
    if weight is not None:
        _check(weight, "weight", torch.float32, (cache.B, cache.H_kv, cache.capacity), cache.device)
    made = []
    if src is None:
        made.append(src := torch.empty((cache.B, cache.H_kv, keep), dtype=torch.int32, device=cache.device))
    else:
        _check(src, "src", torch.int32, (cache.B, cache.H_kv, keep), cache.device)
    if counts_out is None:
        counts_out = (cache if out is None else out).counts
    else:
        _check(counts_out, "counts_out", torch.int32, (2, cache.B), cache.device)
    if out is not None and out.device != cache.device:
        raise ValueError(f"out must be on {cache.device}")
    with _On(cache.device):
        _done(_b.fa_kv4_evict(cache._ref, keep, sinks, recent, weight.data_ptr() if weight is not None else None,
                              out._ref if out is not None else None, src.data_ptr(), counts_out.data_ptr(),
                              _stream(stream, cache.device, *made)), "fa_kv4_evict")
    return src


def _weight_stride(t, what: str, shape, device) -> int:
    """Distance between the heads' rows of a [B, H_kv, N_kv] tensor whose
    rows are contiguous and equally far apart."""
    import torch
    if t.dtype != torch.float32 or tuple(t.shape) != shape or t.device != device:
        raise ValueError(f"{what} must be fp32 {shape} on {device}")
    B, H_kv, N_kv = shape
    # a dimension of size 1 has no stride of its own
    row = t.stride(1) if H_kv > 1 else t.stride(0) if B > 1 else N_kv
    if (N_kv > 1 and t.stride(2) != 1) or (B > 1 and t.stride(0) != H_kv * row) or row < N_kv:
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
    import torch
    _rows(q, "q", None)
    _rows(k, "k", q.device)
    if k.dtype != q.dtype:
        raise TypeError("q and k must share a dtype")
    B, H, N_q, d = q.shape
    if k.shape[0] != B or k.shape[3] != d or H % k.shape[1]:
        raise ValueError(f"incompatible q and k shapes: {tuple(q.shape)} {tuple(k.shape)}")
    H_kv, N_kv = k.shape[1], k.shape[2]
    _check(lse, "lse", torch.float32, (B, H, N_q), q.device)
    made = []
    if out is None:
        made.append(out := torch.empty((B, H_kv, N_kv), dtype=torch.float32, device=q.device))
    stride = _weight_stride(out, "out", (B, H_kv, N_kv), q.device)
    if weight_in is not None and _weight_stride(weight_in, "weight_in", (B, H_kv, N_kv), q.device) != stride:
        raise ValueError("weight_in and out must have the same strides")
    with _On(q.device):
        _done(_b.fa_fwd_weights(q.data_ptr(), k.data_ptr(), lse.data_ptr(),
                                weight_in.data_ptr() if weight_in is not None else None, out.data_ptr(), stride, B, H,
                                H_kv, N_q, N_kv, d, first_query, _scale(scale, d),
                                _b._dtype_code(q) | (_b.FA_FLAG_CAUSAL if causal else 0),
                                _stream(stream, q.device, *made)), "fa_fwd_weights")
    return out
