"""The paged key/value cache on the GPU against 64 bits: rows rotated and
stored, attention over pages (row counts, head layouts, page sizes, lengths from
none to many runs, masks, shared prefixes, what other slots hold), numbers out
of range, and the calls together as a serving loop makes them."""
import math

import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from . import packed_ref as R  # noqa: E402
from .test_packed_gpu import TORCH, int32, rng, rows, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert fa.fa_device_status(None) == fa.FA_OK


def cache_of(g, lengths, H_kv, d, page, dtype="bf16", room=0, prefix=0, poison=True):
    """A cache with its sequences' pages in shuffled order, `room` free slots behind each length; slots that nothing
    holds are NaN.  Also the prefix's page numbers."""
    need = [max(1, -(-(n + room) // page)) for n in lengths]
    shared = -(-prefix // page)
    pool = sum(need) + shared + 2
    order = torch.randperm(pool, generator=g, device="cuda").int()
    k, v = rows(g, pool, H_kv, page, d, dtype=dtype), rows(g, pool, H_kv, page, d, dtype=dtype)
    table = torch.full((len(lengths), max(need)), -7, dtype=torch.int32, device="cuda")  # numbers not looked at
    at = shared
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if poison:
        free = torch.ones(pool, page, dtype=torch.bool, device="cuda")
        for numbers, n in [(order[:shared], prefix)] + [(table[b], n) for b, n in enumerate(lengths)]:
            for s0 in range(0, n, page):
                free[int(numbers[s0 // page]), :n - s0] = False
        for x in (k, v):
            x.masked_fill_(free[:, None, :, None], math.nan)
    return fa.PagedKVCache(k, v, table, int32(lengths)), (order[:shared].contiguous() if prefix else None)


def gather(pages, numbers, n):
    """[n, H_kv, d] of the first n slots."""
    page = pages.shape[2]
    x = pages[numbers[:-(-n // page)].long()].transpose(1, 2).reshape(-1, pages.shape[1], pages.shape[3])
    return x[:n]


def reference(q, c, lengths, scale, causal, prefix_pages=None, prefix=0):
    half, tiny = R.HALF[q.dtype], R.TINY[q.dtype]
    B, H, N_q, d = q.shape
    group = H // c.H_kv
    f64 = dict(dtype=torch.float64, device="cuda")
    out, tol, lse, tol_l = (torch.zeros(s, **f64) for s in (q.shape, q.shape, q.shape[:3], q.shape[:3]))
    for b, n in enumerate(lengths):
        k, v = gather(c.k_pages, c.block_table[b], n), gather(c.v_pages, c.block_table[b], n)
        if prefix:
            k = torch.cat((gather(c.k_pages, prefix_pages, prefix), k))
            v = torch.cat((gather(c.v_pages, prefix_pages, prefix), v))
        see = torch.ones(N_q, prefix + n, dtype=torch.bool, device="cuda")
        if causal:
            for i in range(N_q):
                see[i, prefix + max(0, n - (N_q - 1 - i)):] = False
        for h in range(H):
            got = R.attend(q[b, h].double(), k[:, h // group].double(), v[:, h // group].double(), scale, see, half, tiny)
            out[b, h], lse[b, h], tol[b, h], tol_l[b, h] = got
    return out, lse, tol, tol_l


def check(g, c, lengths, H, N_q, causal=False, scale=None, prefix_pages=None, prefix=0, q=None, **kw):
    d = c.d
    q = (torch.randn(len(lengths), H, N_q, d, generator=g, device="cuda").to(c.dtype)) if q is None else q
    out, lse = fa.paged_attention(q, c, causal=causal, scale=scale, prefix_pages=prefix_pages, prefix_length=prefix, **kw)
    s = 1 / math.sqrt(d) if scale is None else scale
    want_o, want_l, tol_o, tol_l = reference(q, c, lengths, s, causal, prefix_pages, prefix)
    within(lse, want_l, tol_l, "lse")
    within(out, want_o, tol_o, "out")
    return out, lse


# ------------------------------------------------------------------ append
def rotated(x, table, positions, interleaved):
    """64-bit rotation of rows x [T, heads, d] and the tolerance of the kernel's: fp32 products and sums, one rounding."""
    half = R.HALF[x.dtype]
    x = x.double()
    if table is None:
        return x, torch.zeros_like(x)
    rot = table.shape[1]
    cos, sin = (t.double()[:, None] for t in table[positions].split(rot // 2, 1))
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out, tol = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, a * sin + b * cos
    size = a.abs() + b.abs()
    for j in (first, second):
        tol[..., j] = half * out[..., j].abs() + (1 + half) * 2.0 ** -22 * size + R.TINY[torch.float16]
    return out, tol


def check_append(g, c, lens, H, table=None, positions=None, interleaved=False, first=0, with_k=False, uniform=False,
                 in_place=True, views=None, q_out=None):
    held = c.lengths.tolist()
    T = sum(lens)
    dtype = "bf16" if c.dtype == torch.bfloat16 else "f16"
    if views is None:
        k, v = rows(g, T, c.H_kv, c.d, dtype=dtype), rows(g, T, c.H_kv, c.d, dtype=dtype)
        q = rows(g, T, H, c.d, dtype=dtype) if H else None
    else:
        q, k, v = views
    k0, v0 = k.clone(), v.clone()
    q0 = q.clone() if H else None
    cu = None if uniform else int32(R.offsets(lens))
    k_out = torch.full_like(k0, math.nan) if with_k else None
    before = [c.k_pages.clone(), c.v_pages.clone()]
    lengths_out = None if in_place else torch.full_like(c.lengths, -1)
    got = fa.paged_append(c, k, v, cu=cu, q=q, table=table, positions=positions, first_position=first,
                          interleaved=interleaved, k_out=k_out, lengths_out=lengths_out, q_out=q_out)
    new = [min(a + b, c.capacity) for a, b in zip(held, lens)]
    assert (c.lengths if in_place else lengths_out).tolist() == new
    if not in_place:
        assert c.lengths.tolist() == held
    slots = torch.cat([torch.arange(n, device="cuda") + a for a, n in zip(held, lens)])
    pos = positions.long() if positions is not None else slots + first
    want_k, tol_k = rotated(k0, table, pos, interleaved)
    if H:
        within(got, *rotated(q0, table, pos, interleaved), "q")
    if with_k:
        within(k_out, want_k, tol_k, "k_out")
    at = 0
    for b, n in enumerate(lens):
        keep = min(held[b] + n, c.capacity) - held[b]
        for name, want, tol in (("k", want_k, tol_k), ("v", v0.double(), torch.zeros_like(tol_k))):
            x = gather(c.k_pages if name == "k" else c.v_pages, c.block_table[b], held[b] + keep)[held[b]:]
            within(x, want[at:at + keep], tol[at:at + keep], name)
        for s in range(held[b], held[b] + keep):  # then put back what was there
            p, r = int(c.block_table[b, s // c.page_size]), s % c.page_size
            before[0][p, :, r], before[1][p, :, r] = c.k_pages[p, :, r], c.v_pages[p, :, r]
        at += n
    for x, y in zip((c.k_pages, c.v_pages), before):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))  # nothing else was written
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f16"), (128, "f16")])
def test_append_types_and_pages(page, d, dtype):
    g = rng(1)
    lens = [1, 0, 37, 130, 5]
    c, _ = cache_of(g, [15, 3, 0, 127, 700], 2, d, page, dtype, room=130, poison=False)
    check_append(g, c, lens, 6, fa.rotary_table(900, d), with_k=True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 112)])
def test_append_rotations(d, rot, interleaved):
    g = rng(2)
    c, _ = cache_of(g, [15, 300], 3, d, 16, room=40, poison=False)
    pos = torch.randint(0, 100000, (41,), generator=g, device="cuda", dtype=torch.int32)
    check_append(g, c, [40, 1], 3, fa.rotary_table(100000, rot), pos, interleaved, with_k=True)


@pytest.mark.parametrize("uniform", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,n,H,H_kv", [(1, 1, 1, 1), (3, 1, 32, 8), (40, 1, 8, 2), (70, 3, 4, 4), (2, 700, 5, 5), (5, 2, 64, 8)])
def test_append_grids(B, n, H, H_kv, uniform, in_place):
    g = rng(3)
    c, _ = cache_of(g, [(13 * b) % 50 for b in range(B)], H_kv, 128, 32, room=n, poison=False)
    check_append(g, c, [n] * B, H, fa.rotary_table(800, 128), first=7, uniform=uniform, in_place=in_place)


def test_append_without_queries_or_table():
    g = rng(4)
    c, _ = cache_of(g, [15, 300], 3, 64, 16, room=40, poison=False)
    check_append(g, c, [40, 1], 0)
    check_append(g, c, [0, 0], 2)


def test_append_views_of_one_projection_in_place():
    g = rng(5)
    c, _ = cache_of(g, [15, 300], 2, 128, 64, room=40, poison=False)
    qkv = rows(g, 41, 6 + 2 + 2, 128)
    q, k, v = qkv.split([6, 2, 2], 1)
    got = check_append(g, c, [40, 1], 6, fa.rotary_table(400, 128), views=(q, k, v), q_out=q)
    assert got is q


def test_append_past_the_capacity():
    g = rng(6)
    c, _ = cache_of(g, [30, 2], 2, 64, 16, poison=False)  # 32 slots each
    check_append(g, c, [10, 3], 2, fa.rotary_table(100, 64))
    assert fa.fa_device_status(None) == fa.FA_ERR_CAPACITY
    assert fa.fa_device_status(None) == fa.FA_OK


def test_append_numbers_out_of_range():
    """Rows whose page is outside the pool are dropped; positions outside the table are taken as its ends."""
    g = rng(7)
    c, _ = cache_of(g, [0, 0, 0], 1, 64, 16, room=20, poison=False)
    c.block_table[0, 1] = c.num_pages
    c.block_table[2, 0] = -1
    before = c.k_pages.clone()
    k, v, q = (rows(g, 60, 1, 64) for _ in range(3))
    table = fa.rotary_table(16, 64)
    got = fa.paged_append(c, k, v, q=q, table=table)
    assert fa.fa_device_status(None) == fa.FA_ERR_RANGE
    pos = torch.arange(20, device="cuda").clamp(max=15).repeat(3)
    within(got, *rotated(q, table, pos, False))
    want, tol = rotated(k, table, pos, False)
    for b, s, n in ((0, 0, 16), (1, 0, 16), (1, 16, 4), (2, 16, 4)):
        p = int(c.block_table[b, s // 16])
        within(c.k_pages[p, :, :n].transpose(0, 1), want[20 * b + s:20 * b + s + n], tol[20 * b + s:20 * b + s + n])
        before[p, :, :n] = c.k_pages[p, :, :n]
    assert torch.equal(c.k_pages, before)
    assert c.lengths.tolist() == [20, 20, 20]


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("N_q,G", [(1, 1), (1, 3), (2, 4), (1, 8), (4, 4), (17, 1), (3, 7), (5, 8), (16, 8)])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
def test_row_counts(N_q, G, d, dtype, causal):
    g = rng(10)
    lengths = [300, 1, 129]
    c, _ = cache_of(g, lengths, 2, d, 16, dtype)
    check(g, c, lengths, 2 * G, N_q, causal)


@pytest.mark.parametrize("lengths", [[1], [127, 128, 129], [0, 5, 0, 128], [15, 16, 17, 31, 33, 0, 1000], [2500], [0, 0], [40000]],
                         ids=str)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_and_pages(lengths, page, d):
    g = rng(11)
    c, _ = cache_of(g, lengths, 2, d, page)
    check(g, c, lengths, 4, 1)


@pytest.mark.parametrize("B", [33, 70, 300])
def test_many_sequences(B):
    g = rng(12)
    lengths = [(37 * b * b) % 260 for b in range(B)]
    c, _ = cache_of(g, lengths, 2, 64, 16)
    check(g, c, lengths, 8, 1)


@pytest.mark.parametrize("prefix", [1, 100, 128, 1000, 5000])
@pytest.mark.parametrize("B,H,H_kv,N_q", [(1, 1, 1, 1), (3, 8, 2, 1), (40, 8, 2, 1), (9, 16, 1, 1), (5, 8, 1, 16), (70, 4, 2, 2)])
@pytest.mark.parametrize("d,dtype,page", [(64, "f16", 16), (128, "bf16", 64)])
def test_shared_prefix(prefix, B, H, H_kv, N_q, d, dtype, page):
    g = rng(13)
    lengths = [(53 * b) % 300 for b in range(B)]
    c, pages = cache_of(g, lengths, H_kv, d, page, dtype, prefix=prefix)
    check(g, c, lengths, H, N_q, causal=N_q > 1, prefix_pages=pages, prefix=prefix)
