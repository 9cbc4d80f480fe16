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


@pytest.mark.parametrize("cu", [[-2 ** 31, 5, 20, 41], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 41], [30, 10, 50, 2 ** 31 - 1], [41, 0, 0, 0]])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_offsets_that_are_none(cu, in_place):
    """Offsets out of range or order: other pages and rows are not touched, lengths stay within the capacity, and the
    next call is as ever."""
    g = rng(22)
    c, _ = cache_of(g, [15, 3, 100], 2, 64, 16, room=60, poison=False)
    mine = [int(x) for x in c.block_table.flatten() if x >= 0]
    other = [i for i in range(c.num_pages) if i not in mine]
    was = [x[other].clone() for x in (c.k_pages, c.v_pages)]
    held = c.lengths.clone()
    table = fa.rotary_table(200, 64)
    guard = torch.full((2, 141, 2, 64), 5.0, device="cuda").bfloat16()
    x = rows(g, 41, 2, 64)
    out = torch.empty_like(c.lengths)
    fa.paged_append(c, x, x, cu=int32(cu), q=x, q_out=guard[0, 50:91], k_out=guard[1, 50:91], table=table,
                    lengths_out=None if in_place else out)
    got = c.lengths if in_place else out
    assert fa.fa_device_status(None) in (fa.FA_OK, fa.FA_ERR_CAPACITY, fa.FA_ERR_RANGE)
    assert (got >= held).all() and (got <= c.capacity).all()
    assert (guard[:, :50] == 5).all() and (guard[:, 91:] == 5).all()
    for a, b in zip(was, (c.k_pages, c.v_pages)):
        assert torch.equal(a, b[other])
    c.lengths.copy_(held)
    check_append(g, c, [3, 0, 38], 2, table)


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


@pytest.mark.parametrize("H,H_kv,N_q,prefix", [(1, 1, 1, 0), (8, 2, 1, 0), (6, 2, 3, 0), (2, 1, 1, 100)])
@pytest.mark.parametrize("B", [256, 257, 600])
def test_more_sequences_than_a_warp_reads_alone(B, H, H_kv, N_q, prefix):
    """Blocks of the second kernel whose rows are of one sequence, of several, of eight; long sequences among short and
    empty ones."""
    g = rng(23)
    lengths = [(37 * b * b) % 200 if b % 3 else 3000 * (b % 60 == 0) for b in range(B)]
    c, pages = cache_of(g, lengths, H_kv, 64, 64, prefix=prefix)
    check(g, c, lengths, H, N_q, causal=N_q > 1, prefix_pages=pages, prefix=prefix)


@pytest.mark.parametrize("prefix", [1, 100, 128, 1000, 5000])
@pytest.mark.parametrize("B,H,H_kv,N_q", [(1, 1, 1, 1), (3, 8, 2, 1), (40, 8, 2, 1), (9, 16, 1, 1), (5, 8, 1, 16), (70, 4, 2, 2)])
@pytest.mark.parametrize("d,dtype,page", [(64, "f16", 16), (128, "bf16", 64)])
def test_shared_prefix(prefix, B, H, H_kv, N_q, d, dtype, page):
    g = rng(13)
    lengths = [(53 * b) % 300 for b in range(B)]
    c, pages = cache_of(g, lengths, H_kv, d, page, dtype, prefix=prefix)
    check(g, c, lengths, H, N_q, causal=N_q > 1, prefix_pages=pages, prefix=prefix)


@pytest.mark.parametrize("N_q,length", [(4, 2), (4, 4), (4, 5), (8, 1), (3, 0), (4, 127), (4, 130), (2, 640)])
@pytest.mark.parametrize("prefix", [0, 33])
@pytest.mark.parametrize("d", [64, 128])
def test_causal_drafts(N_q, length, prefix, d):
    """Drafts longer than what they follow: rows that see nothing (or the prefix alone)."""
    g = rng(14)
    lengths = [length, 300]
    c, pages = cache_of(g, lengths, 2, d, 16, prefix=prefix)
    check(g, c, lengths, 4, N_q, causal=True, prefix_pages=pages, prefix=prefix)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("prefix", [0, 200])
def test_scales(scale, prefix):
    g = rng(15)
    lengths = [300, 17]
    c, pages = cache_of(g, lengths, 2, 64, 32, prefix=prefix)
    check(g, c, lengths, 6, 1, scale=scale, prefix_pages=pages, prefix=prefix)


@pytest.mark.parametrize("G", [4, 8, 16, 32])  # rows of a block
@pytest.mark.parametrize("prefix", [0, 1500])
def test_growing_scores(G, prefix):
    """Every tile's scores are far above the one's before it: the reference moves each time."""
    g = rng(16)
    lengths = [2000, 900]
    c, pages = cache_of(g, lengths, 1, 64, 64, prefix=prefix)
    q = torch.ones(2, G, 1, 64, device="cuda").bfloat16() * torch.linspace(0.2, 1, G, device="cuda").bfloat16()[None, :, None, None]
    for numbers, n, base in [(pages, prefix, 0)] * (prefix > 0) + [(c.block_table[b], n, prefix) for b, n in enumerate(lengths)]:
        for s in range(0, n, 64):
            c.k_pages[int(numbers[s // 64]), :, :n - s] = (base + s) / 512
    check(g, c, lengths, G, 1, prefix_pages=pages, prefix=prefix, q=q)


def test_lengths_outside_the_cache_are_clamped():
    g = rng(17)
    c, _ = cache_of(g, [64, 64, 64], 2, 64, 16, poison=False)
    q = torch.randn(3, 4, 1, 64, generator=g, device="cuda").bfloat16()
    want = fa.paged_attention(q, c)
    c.lengths.copy_(int32([64, 1 << 30, -5]))
    out, lse = fa.paged_attention(q, c)
    assert torch.equal(out[:2], want[0][:2]) and torch.equal(lse[:2], want[1][:2])
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("prefix", [0, 64])
def test_pages_outside_the_pool_read_as_zeros(prefix):
    g = rng(18)
    c, pages = cache_of(g, [100, 40], 2, 128, 16, poison=False, prefix=prefix)
    c.block_table[0, 2], c.block_table[1, 0] = c.num_pages + 5, -3
    if prefix:
        pages[1] = 1 << 30
    q = torch.randn(2, 4, 1, 128, generator=g, device="cuda").bfloat16()
    got = fa.paged_attention(q, c, prefix_pages=pages, prefix_length=prefix)
    # the same with a page of zeros
    zero = torch.zeros(1, *c.k_pages.shape[1:], device="cuda").bfloat16()
    k, v = torch.cat((c.k_pages, zero)), torch.cat((c.v_pages, zero))
    bad = (c.block_table < 0) | (c.block_table >= c.num_pages)
    c2 = fa.PagedKVCache(k, v, torch.where(bad, c.num_pages, c.block_table).int(), c.lengths)
    if prefix:
        pages = torch.where(pages >= c.num_pages, c.num_pages, pages).int()
    want = fa.paged_attention(q, c2, prefix_pages=pages, prefix_length=prefix)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_page_in_many_sequences():
    """A prompt's pages in several block tables, and the same page twice in one."""
    g = rng(19)
    c, _ = cache_of(g, [160, 96], 2, 64, 32)
    c.block_table[1, :2] = c.block_table[0, 3]
    check(g, c, [160, 96], 4, 1)


def test_pools_pass_32_bits():
    """Pages behind 2^32 elements of the pool, written and attended to."""
    g = rng(20)
    H_kv, page, d = 8, 128, 128
    num = 2 ** 32 // (H_kv * page * d) + 40
    k = torch.zeros(num, H_kv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.arange(num - 8, num, device="cuda").int().flip(0).reshape(2, 4).contiguous()
    c = fa.PagedKVCache(k, v, table, int32([0, 0]))
    lens = [500, 130]
    check_append(g, c, lens, 16, fa.rotary_table(512, d))
    check(g, c, lens, 16, 1)
    check(g, c, lens, 16, 1, prefix_pages=table[0, :2].contiguous(), prefix=200)
    assert not k[:num - 8].any()


def test_long_cache():
    """One sequence over many CTAs, every SM's run a part of it."""
    g = rng(21)
    lengths = [150000]
    c, _ = cache_of(g, lengths, 1, 64, 128)
    check(g, c, lengths, 4, 1)


# ------------------------------------------------- streams, captured calls, calls at once
@pytest.mark.parametrize("prefix", [0, 700])
def test_repeats_and_another_stream(prefix):
    g = rng(22)
    c, pages = cache_of(g, [300, 5, 7000, 0], 2, 128, 64, prefix=prefix)
    q = torch.randn(4, 8, 2, 128, generator=g, device="cuda").bfloat16()
    want = fa.paged_attention(q, c, causal=True, prefix_pages=pages, prefix_length=prefix)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        got = fa.paged_attention(q, c, causal=True, prefix_pages=pages, prefix_length=prefix, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_do_not_depend_on_the_workspace():
    g = rng(23)
    c, pages = cache_of(g, [300, 5, 7000, 0], 2, 128, 64, prefix=300)
    q = torch.randn(4, 8, 1, 128, generator=g, device="cuda").bfloat16()
    want = None
    for fill in (0, 255):
        ws = torch.full((c.workspace_size(8, 1, 300),), fill, dtype=torch.uint8, device="cuda")
        got = fa.paged_attention(q, c, prefix_pages=pages, prefix_length=300, workspace=ws)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_at_once():
    jobs = []
    for i, (lengths, prefix) in enumerate((([5000, 1, 400], 0), ([100] * 30, 1000), ([20000], 0), ([64, 3000], 77))):
        g = rng(30 + i)
        c, pages = cache_of(g, lengths, 2, 128, 16, prefix=prefix)
        q = torch.randn(len(lengths), 8, 1, 128, generator=g, device="cuda").bfloat16()
        jobs.append((q, c, pages, prefix, fa.paged_attention(q, c, prefix_pages=pages, prefix_length=prefix)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = []
        for s, (q, c, pages, prefix, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(fa.paged_attention(q, c, prefix_pages=pages, prefix_length=prefix))
        torch.cuda.synchronize()
        for a, (_, _, _, _, want) in zip(got, jobs):
            assert all(torch.equal(x, y) for x, y in zip(a, want))


# ---------------------------------------------------------- a serving loop
@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("d,dtype,page", [(64, "f16", 16), (128, "bf16", 64)])
def test_prompts_then_captured_steps(prefix, d, dtype, page):
    """Prompts of different lengths rotated, stored and attended to, then decode steps in a captured graph that advances
    the lengths, against 64-bit attention over the rotated rows that the cache holds."""
    g = rng(40)
    H, H_kv, steps = 8, 2, 5
    lens = [130, 1, 77]
    c, pages = cache_of(g, [0, 0, 0], H_kv, d, page, dtype, room=max(lens) + steps, prefix=prefix)
    table = fa.rotary_table(prefix + max(lens) + steps, d)
    T, cu = sum(lens), int32(R.offsets(lens))
    q, k, v = (rows(g, T, h, d, dtype=dtype) for h in (H, H_kv, H_kv))
    k_rot = torch.empty_like(k)
    q_rot = fa.paged_append(c, k, v, cu=cu, q=q, table=table, first_position=prefix, k_out=k_rot)
    assert c.lengths.tolist() == lens
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens]) + prefix
    within(q_rot, *rotated(q, table, pos, False))
    within(k_rot, *rotated(k, table, pos, False))
    for b, n in enumerate(lens):  # the cache holds the rows that the prompt attends over
        at = R.offsets(lens)[b]
        assert torch.equal(gather(c.k_pages, c.block_table[b], n), k_rot[at:at + n])
        assert torch.equal(gather(c.v_pages, c.block_table[b], n), v[at:at + n])
    out, lse = fa.packed_attention(q_rot, k_rot, v, cu, causal=True)
    want_o, want_l, tol_o, tol_l = R.forward(q_rot, k_rot, v, R.offsets(lens), R.offsets(lens), 1 / math.sqrt(d), True)
    within(out, want_o, tol_o)
    within(lse, want_l, tol_l)

    new = [[rows(g, 3, h, d, dtype=dtype) for h in (H, H_kv, H_kv)] for _ in range(steps)]
    q1, k1, v1 = (torch.zeros_like(x) for x in new[0])
    ws = torch.empty(c.workspace_size(H, 1, prefix), dtype=torch.uint8, device="cuda")

    def step():
        q1_rot = fa.paged_append(c, k1, v1, q=q1, table=table, first_position=prefix)
        return q1_rot, *fa.paged_attention(q1_rot.view(3, H, 1, d), c, prefix_pages=pages, prefix_length=prefix, workspace=ws)

    held = c.lengths.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q1_rot, out, lse = step()
    c.lengths.copy_(held)
    for i in range(steps):
        for x, y in zip((q1, k1, v1), new[i]):
            x.copy_(y)
        graph.replay()
        lengths = [n + i + 1 for n in lens]
        assert c.lengths.tolist() == lengths
        within(q1_rot, *rotated(q1, table, torch.tensor(lengths, device="cuda") - 1 + prefix, False))
        want_o, want_l, tol_o, tol_l = reference(q1_rot.view(3, H, 1, d), c, lengths, 1 / math.sqrt(d), False, pages, prefix)
        within(out, want_o, tol_o)
        within(lse, want_l, tol_l)


def test_a_prefix_is_as_if_each_sequence_held_it():
    g = rng(41)
    prefix, lengths, page = 200, [50, 130, 1], 32
    c, pages = cache_of(g, lengths, 2, 64, page, prefix=prefix)
    q = torch.randn(3, 8, 1, 64, generator=g, device="cuda").bfloat16()
    out, lse = fa.paged_attention(q, c, prefix_pages=pages, prefix_length=prefix)
    # copies of prefix and own slots, page after page
    k, v = [], []
    for b, n in enumerate(lengths):
        for to, x in ((k, c.k_pages), (v, c.v_pages)):
            to.append(torch.cat((gather(x, pages, prefix), gather(x, c.block_table[b], n))).float())
    most = max(len(x) for x in k)
    cap = -(-most // page)
    kp, vp = (torch.zeros(3 * cap, 2, page, 64, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(3 * cap, device="cuda").int().view(3, cap)
    for b in range(3):
        for pool, x in ((kp, k[b]), (vp, v[b])):
            full = torch.zeros(cap * page, 2, 64, device="cuda")
            full[:len(x)] = x
            pool[b * cap:(b + 1) * cap] = full.view(cap, page, 2, 64).transpose(1, 2).bfloat16()
    one = fa.PagedKVCache(kp, vp, table, int32([len(x) for x in k]))
    o2, l2 = fa.paged_attention(q, one)
    _, _, tol, tol_l = reference(q, c, lengths, 1 / 8, False, pages, prefix)
    within(o2, out.double(), 2 * tol)
    within(l2, lse.double(), 2 * tol_l)
