"""PyTorch conveniences for attention over packed sequences: tensor checks,
allocation of outputs, and one call of the C entry point each (include/fa.h
documents layout, results and errors).

Every call is enqueued on `stream` (default: the device's current stream), and
what it allocates belongs to that stream.
"""
from __future__ import annotations

from . import binding as _b
from . import kv4 as _k

_rows_t = _b.fa_rows_t


def _call_with_workspace(where: str, function, device, stream, size: int, *args):
    """`kv4._call` with a workspace of `size` bytes that belongs to the call: from
    the stream's memory, and free for what is queued behind it (without a tensor
    around it, which takes longer to make than the kernels' launches)."""
    torch_c = _k.torch._C
    if torch_c._cuda_getDevice() != device.index:
        with _k.torch.cuda.device(device):
            return _call_with_workspace(where, function, device, stream, size, *args)
    current = torch_c._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    memory = torch_c._cuda_cudaCachingAllocator_raw_alloc(max(size, 16), current)
    try:
        status = function(*args, memory, size, current or None)
    finally:
        torch_c._cuda_cudaCachingAllocator_raw_delete(memory)
    if status != _b.FA_OK:
        raise _b.FAError(status, where)


def _new(rows: int, heads: int, d: int, dtype, device, stream):
    """An output [rows, heads, d] and its C view."""
    t = _k._empty((rows, heads, d), dtype, device, stream)
    return t, _rows_t(t.data_ptr() or None, heads * d, d)


def _view(t, what: str, shape, dtype, device):
    """The C view of a [rows, heads, d] tensor whose rows may lie apart."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, is on {t.device}")
    row, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{what} must have contiguous channels")
    return _rows_t(t.data_ptr() or None, row, head)


def _offsets(cu, what: str, device, B=None):
    torch = _k.torch
    if cu.dtype is not torch.int32:
        raise TypeError(f"{what} must be int32, got {cu.dtype}")
    if cu.dim() != 1 or cu.shape[0] < 2 or (B is not None and cu.shape[0] != B + 1):
        raise ValueError(f"{what} must be [sequences + 1], got {tuple(cu.shape)}")
    if cu.device != device or not cu.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor on {device}")
    return cu.shape[0] - 1


def _inputs(q, k, v, cu_q, cu_k):
    """Checked sizes (B, T_q, T_k, H, H_kv, d), dtype code and views of q, k, v."""
    _k._need_torch()
    torch = _k.torch
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q and k must be [rows, heads, d], got {tuple(q.shape)} and {tuple(k.shape)}")
    device, dtype = q.device, q.dtype
    if device.type != "cuda":
        raise ValueError(f"q must be a CUDA tensor, is on {device}")
    code = _b.FA_DTYPE_BF16 if dtype is torch.bfloat16 else _b.FA_DTYPE_F16 if dtype is torch.float16 else None
    if code is None:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    T_q, H, d = q.shape
    T_k, H_kv, _ = k.shape
    if H_kv < 1 or H % H_kv:
        raise ValueError(f"the heads of q must be a multiple of k's, got {H} and {H_kv}")
    kv = (T_k, H_kv, d)
    views = _view(q, "q", q.shape, dtype, device), _view(k, "k", kv, dtype, device), _view(v, "v", kv, dtype, device)
    B = _offsets(cu_q, "cu_q", device)
    if cu_k is not cu_q:
        _offsets(cu_k, "cu_k", device, B)
    return device, code, (B, T_q, T_k, H, H_kv, d), views


def packed_attention(q, k, v, cu_q, cu_k=None, scale: float | None = None, causal: bool = False, out=None, lse=None,
                     with_lse: bool = True, stream=None):
    """O = softmax(scale * Q K^T) V within each of a batch of packed sequences:
    q [T_q, H, d], k and v [T_k, H_kv, d] (bf16 or fp16, d = 64 or 128, H a
    multiple of H_kv), sequence s in rows cu_q[s] .. cu_q[s + 1] - 1 of q and
    cu_k[s] .. cu_k[s + 1] - 1 of k and v (int32 on the device; cu_k defaults to
    cu_q).  Rows and heads may lie apart (slices of one projection's output), at
    multiples of 8 elements.

    Returns (out, lse): out [T_q, H, d], lse fp32 [H, T_q] or None; rows of no
    sequence are not written.  causal: query i of a sequence sees keys
    j <= i + n_k - n_q."""
    if cu_k is None:
        cu_k = cu_q
    device, code, sizes, views = _inputs(q, k, v, cu_q, cu_k)
    _, T_q, _, H, _, d = sizes
    torch = _k.torch
    if out is None:
        out, view = _new(T_q, H, d, q.dtype, device, stream)
    else:
        view = _view(out, "out", q.shape, q.dtype, device)
    if lse is not None:
        _k._check(lse, "lse", torch.float32, (H, T_q), device)
    elif with_lse:
        lse = _k._empty((H, T_q), torch.float32, device, stream)
    _k._call("fa_packed_fwd", _b.load().fa_packed_fwd, device, stream, *views, view,
             lse.data_ptr() or None if lse is not None else None, cu_q.data_ptr(), cu_k.data_ptr(), *sizes,
             _k._scale(scale, d), code | _b.FA_FLAG_CAUSAL if causal else code)
    return out, lse


def packed_attention_backward(q, k, v, o, lse, dout, cu_q, cu_k=None, scale: float | None = None, causal: bool = False,
                              dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of `packed_attention` for its o and lse and the
    upstream gradient dout [T_q, H, d]; arguments as there.  dq, dk and dv may be
    slices of one tensor.  `workspace` (uint8, fa_packed_bwd_workspace_size
    bytes) is allocated when not given."""
    if cu_k is None:
        cu_k = cu_q
    device, code, sizes, (vq, vk, vv) = _inputs(q, k, v, cu_q, cu_k)
    B, T_q, T_k, H, H_kv, d = sizes
    dtype, torch = q.dtype, _k.torch
    _k._check(lse, "lse", torch.float32, (H, T_q), device)
    outputs = []
    for x, what, rows, heads in ((dq, "dq", T_q, H), (dk, "dk", T_k, H_kv), (dv, "dv", T_k, H_kv)):
        outputs.append(_new(rows, heads, d, dtype, device, stream) if x is None
                       else (x, _view(x, what, (rows, heads, d), dtype, device)))
    (dq, vdq), (dk, vdk), (dv, vdv) = outputs
    args = (vq, vk, vv, _view(o, "o", q.shape, dtype, device), _view(dout, "dout", q.shape, dtype, device),
            lse.data_ptr() or None, vdq, vdk, vdv, cu_q.data_ptr(), cu_k.data_ptr(), *sizes, _k._scale(scale, d),
            code | _b.FA_FLAG_CAUSAL if causal else code)
    function = _b.load().fa_packed_bwd
    if workspace is None:
        _call_with_workspace("fa_packed_bwd", function, device, stream, _b.fa_packed_bwd_workspace_size(B, T_q, H, d), *args)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        _k._call("fa_packed_bwd", function, device, stream, *args, workspace.data_ptr(),
                 workspace.numel() * workspace.element_size())
    return dq, dk, dv
