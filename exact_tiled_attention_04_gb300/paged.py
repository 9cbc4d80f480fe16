"""PyTorch conveniences for the paged key/value cache: tensor checks,
allocation of outputs, and one call of the C entry point each (include/fa.h
documents layout, results and errors).

Every call is enqueued on `stream` (default: the device's current stream), and
what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

from . import binding as _b
from . import kv4 as _k
from .packed import _call_with_workspace, _new, _offsets, _view


def rotary_table(rows: int, rot: int, base: float = 10000.0, device="cuda"):
    """fp32 [rows, rot]: for each position the cosines of its rot / 2 angles
    position * base ** (-2 j / rot), then their sines; the angles in 64 bits."""
    _k._need_torch()
    torch = _k.torch
    if rows < 1 or rot < 16 or rot % 16:
        raise ValueError(f"rows must be at least 1 and rot a multiple of 16, got {rows} and {rot}")
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


class PagedKVCache:
    """A paged key/value cache: the caller's tensors and their addresses.

    k_pages, v_pages [num_pages, H_kv, page_size, d] (bf16 or fp16, page_size 16,
    32, 64 or 128, d 64 or 128); block_table int32 [B, max_pages], the page of each
    sequence's slots s // page_size; lengths int32 [B], the slots in use.  The
    tensors are checked here once; replace none of them afterwards (their contents
    are read by every call)."""

    def __init__(self, k_pages, v_pages, block_table, lengths):
        _k._need_torch()
        torch = _k.torch
        if k_pages.dim() != 4 or block_table.dim() != 2:
            raise ValueError(f"k_pages must be [num_pages, H_kv, page_size, d] and block_table [B, max_pages], got "
                             f"{tuple(k_pages.shape)} and {tuple(block_table.shape)}")
        num_pages, H_kv, page, d = (int(x) for x in k_pages.shape)
        B, max_pages = (int(x) for x in block_table.shape)
        device, dtype = k_pages.device, k_pages.dtype
        if device.type != "cuda":
            raise ValueError(f"k_pages must be a contiguous CUDA tensor, is on {device}")
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"k_pages must be bfloat16 or float16, got {dtype}")
        if d not in (64, 128) or page not in (16, 32, 64, 128):
            raise ValueError(f"d must be 64 or 128 and page_size 16, 32, 64 or 128, got {d} and {page}")
        if min(num_pages, H_kv, B, max_pages) < 1:
            raise ValueError("a cache has at least one page, head and sequence")
        for t, what, kind, shape in ((k_pages, "k_pages", dtype, k_pages.shape), (v_pages, "v_pages", dtype, k_pages.shape),
                                     (block_table, "block_table", torch.int32, (B, max_pages)),
                                     (lengths, "lengths", torch.int32, (B,))):
            _k._check(t, what, kind, shape, device)
        self.k_pages, self.v_pages, self.block_table, self.lengths = k_pages, v_pages, block_table, lengths
        self.num_pages, self.page_size, self.B, self.max_pages, self.H_kv, self.d = num_pages, page, B, max_pages, H_kv, d
        self.device, self.dtype = device, dtype
        self._code = _b.FA_DTYPE_BF16 if dtype is torch.bfloat16 else _b.FA_DTYPE_F16
        self._struct = _b.fa_paged_cache_t(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                           lengths.data_ptr(), num_pages, page, B, max_pages, H_kv, d)
        self._ref = ctypes.pointer(self._struct)
        self._need = {}

    @property
    def capacity(self) -> int:
        """Slots a sequence can have."""
        return self.max_pages * self.page_size

    def workspace_size(self, H: int, N_q: int, prefix_length: int = 0) -> int:
        """Bytes paged_attention needs for these sizes on the cache's device."""
        key = (H, N_q, prefix_length)
        if key not in self._need:
            with _k.torch.cuda.device(self.device):
                self._need[key] = _b.fa_paged_fwd_workspace_size(self.B, H, self.H_kv, N_q, self.capacity, self.d,
                                                                 prefix_length)
        return self._need[key]


def paged_append(cache: PagedKVCache, k, v, cu=None, q=None, table=None, positions=None, first_position: int = 0,
                 interleaved: bool = False, q_out=None, k_out=None, lengths_out=None, stream=None):
    """Store k, v [T, H_kv, d] behind the sequences' last slots, keys rotated by
    their positions, and rotate q [T, H, d] beside them.  Rows cu[b] .. cu[b + 1] - 1
    are sequence b's (int32 on the device; None: T / B rows each).

    table: `rotary_table`, or None for no rotation; positions: int32 [T], or None:
    first_position (a shared prefix's length, say) + the slot.  interleaved: pairs of
    neighbouring channels.  k_out: [T, H_kv, d], gets the rotated keys too.  The
    lengths advance in place, or go to `lengths_out` (int32 [B]).  Rows past the
    capacity are dropped and reported by fa_device_status (FA_ERR_CAPACITY), as are
    page numbers and positions out of range (FA_ERR_RANGE).

    Returns the rotated q (`q_out`, allocated when not given; None without q); rows of
    no sequence are not written."""
    device, dtype, torch = cache.device, cache.dtype, _k.torch
    if k.dim() != 3:
        raise ValueError(f"k must be [rows, heads, d], got {tuple(k.shape)}")
    T = k.shape[0]
    kv = (T, cache.H_kv, cache.d)
    vk, vv = _view(k, "k", kv, dtype, device), _view(v, "v", kv, dtype, device)
    if cu is not None:
        _offsets(cu, "cu", device, cache.B)
    elif T % cache.B:
        raise ValueError(f"without cu every sequence gets as many rows, but {T} rows are for {cache.B} sequences")
    H, vq, vq_out = 0, None, None
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [rows, heads, d], got {tuple(q.shape)}")
        H = q.shape[1]
        shape = (T, H, cache.d)
        vq = _view(q, "q", shape, dtype, device)
        if q_out is None:
            q_out, vq_out = _new(T, H, cache.d, dtype, device, stream)
        else:
            vq_out = _view(q_out, "q_out", shape, dtype, device)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    vk_out = _view(k_out, "k_out", kv, dtype, device) if k_out is not None else None
    rows = rot = 0
    if table is not None:
        if table.dim() != 2:
            raise ValueError(f"table must be [positions, rot], got {tuple(table.shape)}")
        rows, rot = table.shape
        _k._check(table, "table", torch.float32, (rows, rot), device)
    if positions is not None:
        _k._check(positions, "positions", torch.int32, (T,), device)
    if lengths_out is None:
        lengths_out = cache.lengths
    else:
        _k._check(lengths_out, "lengths_out", torch.int32, (cache.B,), device)
    _k._call("fa_paged_append", _b.load().fa_paged_append, device, stream, cache._ref, vk, vv,
             cu.data_ptr() if cu is not None else None, T, vq, vq_out, H, vk_out,
             table.data_ptr() if table is not None else None, rows, rot,
             positions.data_ptr() or None if positions is not None else None, first_position, lengths_out.data_ptr(),
             cache._code | _b.FA_FLAG_INTERLEAVED if interleaved else cache._code)
    return q_out


def paged_attention(q, cache: PagedKVCache, scale: float | None = None, causal: bool = False, prefix_pages=None,
                    prefix_length: int = 0, out=None, lse=None, with_lse: bool = True, workspace=None, stream=None):
    """O = softmax(scale * Q K^T) V for q [B, H, N_q, d] over the sequences' slots;
    H a multiple of H_kv, N_q * H / H_kv <= 128.  (`paged_append` returns queries as
    [rows, heads, d]: with N_q above 1 they are transposed in between.)

    prefix_pages (int32, of the same pool) and prefix_length: slots that come
    before every sequence's own, read once for up to 256 rows a key/value head.  causal: query i
    sees the prefix and the own slots j < length - (N_q - 1 - i).  Returns
    (out, lse) as `attention` does.  `workspace` (uint8, cache.workspace_size(...)
    bytes) is allocated when not given."""
    device, torch = cache.device, _k.torch
    if q.dim() != 4:
        raise ValueError(f"q must be [batch, heads, rows, d], got {tuple(q.shape)}")
    B, H, N_q, d = q.shape
    if B != cache.B or d != cache.d or H < 1 or H % cache.H_kv:
        raise ValueError(f"q must be [{cache.B}, a multiple of {cache.H_kv}, N_q, {cache.d}], got {tuple(q.shape)}")
    _k._check(q, "q", cache.dtype, (B, H, N_q, d), device)
    if prefix_length < 0 or (prefix_length > 0) != (prefix_pages is not None):
        raise ValueError("prefix_pages and a positive prefix_length come together")
    if prefix_pages is not None:
        _k._check(prefix_pages, "prefix_pages", torch.int32, (-(-prefix_length // cache.page_size),), device)
    if out is None:
        out = _k._empty((B, H, N_q, d), q.dtype, device, stream)
    else:
        _k._check(out, "out", q.dtype, q.shape, device)
    if lse is not None:
        _k._check(lse, "lse", torch.float32, (B, H, N_q), device)
    elif with_lse:
        lse = _k._empty((B, H, N_q), torch.float32, device, stream)
    args = (cache._ref, q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None, H, N_q,
            prefix_pages.data_ptr() if prefix_pages is not None else None, prefix_length, _k._scale(scale, d),
            cache._code | _b.FA_FLAG_CAUSAL if causal else cache._code)
    function = _b.load().fa_paged_fwd
    if workspace is None:
        _call_with_workspace("fa_paged_fwd", function, device, stream, cache.workspace_size(H, N_q, prefix_length), *args)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        _k._call("fa_paged_fwd", function, device, stream, *args, workspace.data_ptr(),
                 workspace.numel() * workspace.element_size())
    return out, lse
