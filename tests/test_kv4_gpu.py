"""The 4-bit key/value cache on the GPU against its 64-bit restatement:
storing and reading back, attention (row counts, head layouts, lengths from
none to many, masks, NaN behind the mask), accumulated weights of decode steps
and of prompts, eviction in place and into another cache, and the calls
together as a serving loop makes them, eager and captured."""
import threading

import numpy as np
import pytest

import exact_tiled_attention_04_gb300 as fa

from . import kv4_ref as R
from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
ARRAYS = ("k_codes", "k_scales", "v_codes", "v_scales", "pos", "weight")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert fa.fa_device_status(None) == fa.FA_OK


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, *shape, dtype="bf16", gain=1.0):
    return (gain * torch.randn(shape, generator=g, device="cuda")).to(TORCH[dtype])


def np64(t):
    return t.double().cpu().numpy()


def int32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(g, B, H_kv, lengths, d, capacity=None):
    """A cache whose every slot holds something; the scales behind a length are NaN."""
    c = fa.KV4Cache.empty(B, H_kv, capacity or max(lengths), d)
    fa.kv4_append(c, rows(g, B, H_kv, c.capacity, d), rows(g, B, H_kv, c.capacity, d),
                  counts_out=torch.empty_like(c.counts))
    c.counts.copy_(int32(lengths, lengths))
    c.weight.copy_(torch.rand(c.weight.shape, generator=g, device="cuda"))
    for b, n in enumerate(lengths):
        c.k_scales[b, :, n:] = 0x7F
        c.v_scales[b, :, n:] = 0xFF
    return c


def held(c):
    return (R.unpack(c.k_codes.cpu().numpy(), c.k_scales.cpu().numpy()),
            R.unpack(c.v_codes.cpu().numpy(), c.v_scales.cpu().numpy()))


# ------------------------------------------------------------ store and read
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H_kv,n,start", [(1, 1, 1, 0), (3, 2, 1, 77), (2, 5, 67, 61), (1, 8, 300, 84)])
def test_append_and_read(dtype, d, B, H_kv, n, start):
    g = rng(100 + n + d)
    c = fa.KV4Cache.empty(B, H_kv, start + n + 1, d)
    c.counts.copy_(int32([start] * B, [start + 9] * B))
    c.pos.fill_(-7)
    c.weight.fill_(3.0)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    # magnitudes from far below the smallest scale to past the largest
    gain = torch.exp2(torch.randint(-16, 12, (B, H_kv, n, d // 16, 1), generator=g, device="cuda").float())
    k = (rows(g, B, H_kv, n, d).float().reshape(B, H_kv, n, -1, 16) * gain).reshape(B, H_kv, n, d).to(TORCH[dtype])
    v = rows(g, B, H_kv, n, d, dtype=dtype)
    got = fa.kv4_append(c, k, v)
    assert got is c.counts and c.counts.tolist() == [[start + n] * B, [start + 9 + n] * B]
    for read in ("bf16", "f16"):
        rk, rv = fa.kv4_read(c, n, first=int32(*[start] * B), dtype=TORCH[read])
        assert np.array_equal(np64(rk), R.stored(np64(k)))
        assert np.array_equal(np64(rv), R.stored(np64(v)))
    assert c.pos[:, :, start:start + n].eq(torch.arange(start + 9, start + 9 + n, device="cuda")).all()
    assert c.weight[:, :, start:start + n].eq(0).all()
    for t, old in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
        assert torch.equal(t[:, :, :start], old[:, :, :start]) and torch.equal(t[:, :, start + n:], old[:, :, start + n:])
    assert c.pos[:, :, start + n:].eq(-7).all() and c.pos[:, :, :start].eq(-7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_rows_on_16_byte_boundaries(d):
    g = rng(105)

    def shifted(dtype="bf16"):  # 16 bytes behind a 32-byte boundary
        t = rows(g, 2 * 3 * 70 * d + 8, dtype=dtype)[8:].view(2, 3, 70, d)
        assert t.data_ptr() % 32 == 16
        return t

    c = fa.KV4Cache.empty(2, 3, 70, d)
    k, v = shifted(), shifted()
    fa.kv4_append(c, k, v)
    for rk, rv in (fa.kv4_read(c, 70), fa.kv4_read(c, 70, k=shifted(), v=shifted()),
                   fa.kv4_read(c, 70, dtype=torch.float16, k=shifted("f16"), v=shifted("f16"))):
        assert np.array_equal(np64(rk), R.stored(np64(k))) and np.array_equal(np64(rv), R.stored(np64(v)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_value_of_the_type(dtype):
    """Blocks whose largest is any finite value of the type and whose others sit at the codes'
    midpoints and points: scales and codes round as defined."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(TORCH[dtype])
    x = x[torch.isfinite(x)].float()
    frac = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, .5, 1, 2, 3, -6, -5, 0, -.25]) / 6
    blocks = (x[:, None] * frac).to(TORCH[dtype])
    n = blocks.shape[0] // 4
    k = blocks[:4 * n].reshape(1, 1, n, 64).cuda().contiguous()
    c = fa.KV4Cache.empty(1, 1, n, 64, pos=False, weight=False)
    fa.kv4_append(c, k, k)
    rk, rv = fa.kv4_read(c, n, dtype=torch.bfloat16)
    assert np.array_equal(np64(rk), R.stored(np64(k))) and torch.equal(rk, rv)


def test_non_finite_blocks_read_as_nan():
    k = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0, 3], k[0, 0, 0, 20], k[0, 0, 1, 63] = float("inf"), float("nan"), float("-inf")
    c = fa.KV4Cache.empty(1, 1, 128, 64)
    fa.kv4_append(c, k, k)
    rk, _ = fa.kv4_read(c, 2)
    assert np.array_equal(np64(rk), R.stored(np64(k)), equal_nan=True)
    assert torch.isnan(rk[0, 0, 0, :32]).all() and torch.isfinite(rk[0, 0, 0, 32:]).all()


def test_read_outside_the_capacity_is_zero():
    c = filled(rng(3), 2, 1, [128, 128], 64)
    k, v = fa.kv4_read(c, 6, first=int32(-3, 126))
    hk, _ = held(c)
    assert (k[0, :, :3] == 0).all() and (v[0, :, :3] == 0).all() and (k[1, :, 2:] == 0).all()
    assert np.array_equal(np64(k[0, :, 3:]), hk[0, :, :3]) and np.array_equal(np64(k[1, :, :2]), hk[1, :, 126:])


@pytest.mark.parametrize("n", [1, 5, 700])
def test_append_past_the_capacity(n):
    g = rng(4)
    c = fa.KV4Cache.empty(2, 2, 128, 64)
    c.counts.copy_(int32([126, 128], [126, 128]))
    old = c.k_codes.clone()
    k = rows(g, 2, 2, n, 64)
    fa.kv4_append(c, k, k)
    assert fa.fa_device_status(None) == fa.FA_ERR_CAPACITY  # the second sequence is full
    assert fa.fa_device_status(None) == fa.FA_OK
    assert c.counts.tolist() == [[min(126 + n, 128), 128], [126 + n, 128 + n]]
    got, _ = fa.kv4_read(c, 2, first=int32(126, 126))
    m = min(n, 2)
    assert np.array_equal(np64(got[0, :, :m]), R.stored(np64(k[0, :, :m])))
    assert torch.equal(c.k_codes[1], old[1]) and torch.equal(c.k_codes[0, :, :126], old[0, :, :126])


# ----------------------------------------------------------------- attention
def check_attention(c, q, dtype, causal=False, scale=None, weight=True):
    """fa.kv4_attention on poisoned outputs against 64 bits; returns (out, lse, weight_out)."""
    d = q.shape[3]
    lengths = [min(max(n, 0), c.capacity) for n in c.lengths.tolist()]
    hk, hv = held(c)
    sc = float(np.float32(1 / np.sqrt(d))) if scale is None else scale
    o_ref, l_ref, w_ref, av, big = R.attend(np64(q), hk, hv, lengths, sc, causal)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    w_out = torch.full_like(c.weight, -5.0) if weight else None
    ws = torch.full((c.workspace_size(q.shape[1], q.shape[2], weight) // 4 + 4,), float("nan"), device="cuda")
    w_in = np64(c.weight)
    fa.kv4_attention(q, c, scale=scale, causal=causal, out=out, lse=lse, weight_out=w_out, workspace=ws)
    assert fa.fa_device_status(None) == fa.FA_OK
    o, l = np64(out), np64(lse)
    vmax = max(np.abs(hv[b, :, :n]).max() if n else 0.0 for b, n in enumerate(lengths))
    tol = R.tol_out(o_ref, av, big, max(lengths), vmax, d, dtype)
    assert np.isfinite(o).all() and (np.abs(o - o_ref) <= tol).all(), np.max(np.abs(o - o_ref) / tol)
    empty = np.isneginf(l_ref)
    assert np.array_equal(empty, np.isneginf(l)) and (o[empty] == 0).all()
    tl = R.tol_lse(l_ref, big, d)
    assert (np.abs(l[~empty] - l_ref[~empty]) <= tl[~empty]).all(), np.max(np.abs(l[~empty] - l_ref[~empty]) / tl[~empty])
    if weight:
        w = np64(w_out)
        for b, n in enumerate(lengths):
            assert (w[b, :, n:] == -5.0).all()
            tw = R.tol_weight(w_ref[b, :, :n], big, l_ref, d, w_in[b, :, :n])
            err = np.abs(w[b, :, :n] - w_in[b, :, :n] - w_ref[b, :, :n])
            assert (err <= tw).all(), np.max(err / tw)
    return out, lse, w_out


# Caches of up to 512 slots get a block per head, longer ones are cut into runs that blocks share:
# both, whatever the lengths in them.
CAPACITY = pytest.mark.parametrize("capacity", [None, 2048], ids=["short", "cut"])


# (N_q, group): rows 1, 3, 8 (one tile of 8), 9, 16 (two), 17, 40, 128 (blocks of 16)
@pytest.mark.parametrize("N_q,G", [(1, 1), (1, 3), (2, 4), (1, 8), (3, 3), (4, 4), (17, 1), (5, 8), (16, 8)])
@pytest.mark.parametrize("d", [64, 128])
@CAPACITY
def test_row_counts(N_q, G, d, capacity):
    g = rng(200 + N_q * 10 + G)
    c = filled(g, 2, 2, [333, 70], d, capacity)
    check_attention(c, rows(g, 2, 2 * G, N_q, d), "bf16")
    check_attention(c, rows(g, 2, 2 * G, N_q, d, dtype="f16"), "f16", causal=True)


@pytest.mark.parametrize("lengths", [[1], [31, 32, 33], [0, 5, 0, 128], [127, 1, 129, 256, 0, 64, 1000], [2500], [0, 0]])
@pytest.mark.parametrize("d", [64, 128])
@CAPACITY
def test_lengths(lengths, d, capacity):
    g = rng(300 + sum(lengths))
    c = filled(g, len(lengths), 3, lengths, d, max(capacity or 0, max(lengths)))
    check_attention(c, rows(g, len(lengths), 6, 1, d), "bf16")


@pytest.mark.parametrize("B", [33, 70])
@CAPACITY
def test_many_sequences(B, capacity):
    """More sequences than the warp that looks for its first one holds."""
    g = rng(310 + B)
    lengths = [(37 * b) % 151 if b % 5 else 0 for b in range(B)]
    c = filled(g, B, 1, lengths, 64, capacity)
    check_attention(c, rows(g, B, 2, 1, 64, dtype="f16"), "f16")


@pytest.mark.parametrize("d,G", [(64, 4), (128, 8)])
def test_as_many_heads_as_blocks(d, G):
    """Caches of 513 to 1024 slots that one block reads whole."""
    g = rng(315 + d)
    lengths = [(331 * b) % 1025 for b in range(39)] + [1024]
    c = filled(g, 40, 8, lengths, d, 1024)
    check_attention(c, rows(g, 40, 8 * G, 1, d), "bf16")


@pytest.mark.parametrize("d,G", [(64, 4), (128, 4), (128, 8), (128, 16)])
def test_runs_that_count_the_ends_of_heads(d, G):
    """More than two groups of slots per block: runs begin and end anywhere, behind a head's last slot, too."""
    g = rng(317 + d + G)
    c = filled(g, 6, 8, [6000, 1, 0, 4097, 33, 5999], d)
    check_attention(c, rows(g, 6, 8 * G, 1, d), "bf16")
    c = filled(g, 1, 1, [300], d, 200000)  # short, in a long cache
    check_attention(c, rows(g, 1, G, 1, d), "bf16")


@pytest.mark.parametrize("d,G", [(64, 4), (128, 3), (128, 16)])
@pytest.mark.parametrize("n", [5000, 20000, 77000])  # 20, 79 and 301 parts of each row at four rows a head
def test_rows_of_many_parts(d, G, n):
    g = rng(319 + d + G)
    c = filled(g, 1, 1, [n], d)
    check_attention(c, rows(g, 1, G, 1, d), "bf16")


@pytest.mark.parametrize("N_q,length", [(4, 2), (4, 4), (4, 5), (8, 1), (3, 0), (4, 100), (2, 33), (4, 640)])
@pytest.mark.parametrize("d", [64, 128])
@CAPACITY
def test_causal_drafts(N_q, length, d, capacity):
    """Rows that see fewer slots, or none (the draft is longer than the cache)."""
    g = rng(320 + N_q + length)
    c = filled(g, 2, 2, [length, 200], d, capacity)
    check_attention(c, rows(g, 2, 4, N_q, d), "bf16", causal=True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_scales(scale):
    g = rng(330)
    c = filled(g, 1, 2, [777], 64)
    check_attention(c, rows(g, 1, 8, 1, 64), "bf16", scale=scale)


@pytest.mark.parametrize("dtype,gain", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 3e4), ("f16", 1e-6)])
def test_query_magnitudes(dtype, gain):
    """Queries at the ends of their type's range, with a scale that undoes the gain."""
    g = rng(340)
    c = filled(g, 1, 1, [500], 128)
    q = ((torch.rand(1, 4, 1, 128, generator=g, device="cuda") * 2 - 1) * gain).to(TORCH[dtype])
    check_attention(c, q, dtype, scale=float(0.2 / gain), weight=False)


@pytest.mark.parametrize("G", [4, 8, 12])  # the three layouts
@pytest.mark.parametrize("n", [900, 3000])
def test_growing_scores(G, n):
    """Scores that keep rising along the cache: every warp moves its reference many times."""
    g = rng(350)
    c = fa.KV4Cache.empty(1, 2, n, 128)
    ramp = torch.linspace(0.1, 8.0, n, device="cuda")[None, None, :, None]
    u = torch.randn(1, 2, 1, 128, generator=g, device="cuda")
    fa.kv4_append(c, (u * ramp).bfloat16(), rows(g, 1, 2, n, 128))
    q = (u.repeat_interleave(G, 1) + 0.1 * torch.randn(1, 2 * G, 1, 128, generator=g, device="cuda")).bfloat16()
    check_attention(c, q, "bf16")


def test_dominant_and_tiny_weights():
    """One key above 20000 others by 2^24 each: what they add up to is 2^-10 of the output and is kept."""
    n, d = 20000, 64
    c = fa.KV4Cache.empty(1, 1, n, d)
    k = torch.zeros(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 7, :16] = 6.0
    v[0, 0, 7] = -1.0
    fa.kv4_append(c, k, v)
    q = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., :16] = 1.0
    check_attention(c, q, "bf16", scale=float(24 * np.log(2) / 96))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("at", [7, 263])  # its warp's first slab, where the reference begins, and the second, which moves it
@pytest.mark.parametrize("G", [4, 8, 12])  # the three layouts
@pytest.mark.parametrize("d", [64, 128])
def test_tiny_weights_beside_a_dominant_one(d, G, at, dtype):
    """One key whose weight is 2^24 times the others' and whose value is 0: the output is the tiny
    weights of the keys that its warp holds (slots 0 to 31 and 256 to 287 of a cache that one block
    reads), and they are kept to fp16's 2^-25 below a weight of 2^7."""
    n = 512
    c = fa.KV4Cache.empty(1, 1, n, d)
    k, v = (torch.zeros(1, 1, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[0, 0, at, :16] = 6.0
    v[0, 0, :32] = v[0, 0, 256:288] = 1.0
    v[0, 0, at] = 0.0
    fa.kv4_append(c, k, v)
    q = torch.zeros(1, G, 1, d, dtype=TORCH[dtype], device="cuda")
    q[..., :16] = 1.0
    out, _, _ = check_attention(c, q, dtype, scale=float(24 * np.log(2) / 96))
    # 63 * 2^-24 / (1 + 511 * 2^-24); without the tiny weights it is 0, ten times what the check lets pass
    assert (out.float() > 0.8 * 63 * 2.0 ** -24).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4])  # 3, 6 and 12 rows: the three layouts
@CAPACITY
def test_nan_behind_the_mask(d, G, capacity):
    """A NaN entry that only the last row of a draft sees leaves the other rows as they were."""
    g = rng(360)
    c = filled(g, 1, 1, [100], d, capacity)
    q = rows(g, 1, G, 3, d)
    good, _ = fa.kv4_attention(q, c, causal=True)
    old = c.v_scales[0, 0, 99, 1].clone()
    c.v_scales[0, 0, 99, 1] = 0x7F
    out, lse = fa.kv4_attention(q, c, causal=True)
    assert torch.equal(out[:, :, :2], good[:, :, :2])
    assert torch.isnan(out[:, :, 2, 16:32]).all() and torch.equal(out[:, :, 2, :16], good[:, :, 2, :16])
    assert torch.equal(out[:, :, 2, 32:], good[:, :, 2, 32:]) and torch.isfinite(lse).all()
    c.v_scales[0, 0, 99, 1] = old
    c.k_scales[0, 0, 99, 0] = 0x7F
    w = torch.zeros_like(c.weight)
    out, lse = fa.kv4_attention(q, c, causal=True, weight_out=w)
    assert torch.equal(out[:, :, :2], good[:, :, :2]) and torch.isnan(out[:, :, 2]).all()
    assert torch.isfinite(lse[:, :, :2]).all() and torch.isnan(lse[:, :, 2]).all()
    # every row sees slot 0
    c.k_scales[0, 0, 0, 0] = 0xFF
    out, _ = fa.kv4_attention(q, c, causal=True)
    assert torch.isnan(out).all()


def test_lengths_outside_the_cache_are_clamped():
    g = rng(370)
    c = filled(g, 2, 1, [256, 0], 64, capacity=256)
    q = rows(g, 2, 2, 1, 64)
    want, _ = fa.kv4_attention(q, c)
    c.counts[0] = int32(9999, -4)
    got, lse = fa.kv4_attention(q, c)
    assert torch.equal(got, want) and torch.isneginf(lse[1]).all()


def test_matches_the_16_bit_attention_on_the_stored_values():
    g = rng(380)
    c = filled(g, 2, 2, [512, 512], 128)
    q = rows(g, 2, 8, 1, 128)
    k, v = fa.kv4_read(c, 512)
    want, wl = fa.attention(q, k, v)
    got, gl = fa.kv4_attention(q, c)
    assert (got.float() - want.float()).abs().max() <= 2 * 1.5e-2 and (gl - wl).abs().max() <= 1e-3


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_is_as_near_the_16_bit_attention_as_roundings_allow(dtype):
    """The two attentions on the same stored values differ by their own roundings only: this one's
    (R.tol_out), and the other's weights (half a step of their type, in numerator and denominator),
    scores and output."""
    g = rng(381)
    c = filled(g, 2, 2, [512, 512], 128)
    q = rows(g, 2, 8, 1, 128, dtype=dtype)
    k, v = fa.kv4_read(c, 512, dtype=TORCH[dtype])
    want, wl = fa.attention(q, k, v)
    got, gl = fa.kv4_attention(q, c)
    hk, hv = held(c)
    o, lse, _, av, big = R.attend(np64(q), hk, hv, [512, 512], float(np.float32(1 / np.sqrt(128))), False)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    mine = R.tol_out(o, av, big, 512, np.abs(hv).max(), 128, dtype)
    rel = 2 * half + 2 * R.score_error(big, 128)[..., None] + 2.0 ** -20
    other = half * np.abs(o) + (1 + half) * rel * (av + np.abs(o)) + 2.0 ** -24
    err = np.abs(np64(got) - np64(want))
    assert (err <= mine + other).all(), np.max(err / (mine + other))
    assert (np.abs(np64(gl) - np64(wl)) <= 2 * R.tol_lse(lse, big, 128)).all()


def test_long_cache_offsets_pass_32_bits():
    """Slots whose byte offsets pass 2^32: 2 x 4 heads of 17.3 million slots."""
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 25 GB")
    B, H_kv, d, cap = 2, 4, 64, 17_301_504
    assert B * H_kv * cap * (d // 2) > 2 ** 32
    c = fa.KV4Cache.empty(B, H_kv, cap, d, pos=False, weight=False)
    g = rng(390)
    n = 300
    base = int32(5, cap - n)
    c.counts[0] = base
    c.counts[1] = base
    kk, vv = rows(g, B, H_kv, n, d), rows(g, B, H_kv, n, d)
    fa.kv4_append(c, kk, vv)
    k, v = fa.kv4_read(c, n, first=base)
    assert np.array_equal(np64(k), R.stored(np64(kk))) and np.array_equal(np64(v), R.stored(np64(vv)))
    # a length of cap: all but the last n keys and values are zero (their scales are)
    q = rows(g, B, H_kv, 1, d)
    out, lse = fa.kv4_attention(q, c)
    p = torch.exp(torch.einsum("hd,hnd->hn", q[1, :, 0].double(), k[1].double()) / 8)
    z = p.sum(-1) + (cap - n)
    want = torch.einsum("hn,hnd->hd", p, v[1].double()) / z[:, None]
    # weights near 1 / cap: a bf16 rounding, and the fp16 weights' 2^-11 of sum p |v|, twice
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -9 * torch.einsum("hn,hnd->hd", p, v[1].double().abs()) / z[:, None] + 1e-9
    # fp32 sums: 17 million terms, a lane's share of them (under 2^13) added one by one: 2^-11
    assert ((out[1, :, 0].double() - want).abs() <= tol + 2.0 ** -11 * want.abs()).all()
    assert ((lse[1, :, 0].double() - torch.log(z)).abs() <= 2.0 ** -11).all()


def test_repeats_bit_for_bit_and_on_another_stream():
    g = rng(400)
    c = filled(g, 5, 4, [3000, 17, 900, 2048, 64], 128)
    q = rows(g, 5, 16, 1, 128)
    w = torch.zeros_like(c.weight)
    first = [t.clone() for t in (*fa.kv4_attention(q, c, weight_out=w), w)]
    for _ in range(3):
        w2 = torch.zeros_like(w)
        for a, b in zip(first, (*fa.kv4_attention(q, c, weight_out=w2), w2)):
            assert torch.equal(a, b)
    w3 = torch.zeros_like(w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = fa.kv4_attention(q, c, weight_out=w3, stream=s)
    s.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and torch.equal(w3, first[2])


def test_two_calls_at_once():
    g = rng(410)
    cs = [filled(g, 2, 2, [2000 + i, 31], 64) for i in range(2)]
    qs = [rows(g, 2, 8, 1, 64) for _ in range(2)]
    want = [fa.kv4_attention(q, c)[0].clone() for q, c in zip(qs, cs)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [fa.kv4_attention(q, c, stream=s)[0] for q, c, s in zip(qs, cs, ss)]
        for s in ss:
            s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def calls_on_a_stream():
    """Each call that allocates, with `stream` as its argument; and the bytes of its workspace."""
    g = rng(420)
    c = filled(g, 2, 2, [2000, 300], 64)
    to = fa.KV4Cache.empty(2, 2, 256, 64)
    q, pq, pk, pv = (rows(g, 2, h, n, 64) for h, n in ((8, 1), (4, 300), (2, 300), (2, 300)))
    _, lse = fa.attention(pq, pk, pv, causal=True)
    return {"attention": (lambda s: fa.kv4_attention(q, c, stream=s), c.workspace_size(8, 1, False)),
            "read": (lambda s: fa.kv4_read(c, 300, stream=s), 0),
            "evict": (lambda s: (fa.kv4_evict(c, 200, out=to, stream=s),), 0),
            "weights": (lambda s: (fa.attention_weights(pq, pk, lse, causal=True, stream=s),), 0)}


CALLS = pytest.mark.parametrize("name", ["attention", "read", "evict", "weights"])


@CALLS
def test_memory_of_a_call_on_another_stream(name):
    """Nothing the call allocates was freed on the current stream, whose queued kernels still write it."""
    call, bytes_ = calls_on_a_stream()[name]
    want = [t.clone() for t in call(None)]
    for t in (*want, torch.empty(16, dtype=torch.uint8, device="cuda")):
        torch.empty_like(t).fill_(77)  # loads the fills' kernels ahead of the pause
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)  # 0.2 s
    freed = [torch.empty_like(t) for t in want] + [torch.empty(max(bytes_, 16), dtype=torch.uint8, device="cuda")]
    for t in freed:
        t.fill_(77)
    at = {t.data_ptr() for t in freed}
    del freed, t
    got = call(s)
    assert not at & {t.data_ptr() for t in got}
    s.synchronize()
    assert not torch.cuda.current_stream().query()  # the fills are still to come
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@CALLS
def test_freed_results_of_a_call_on_another_stream(name):
    """A result that the caller frees while the current stream has its copy queued is not written again before that."""
    call, _ = calls_on_a_stream()[name]
    want = [t.clone() for t in call(None)]
    copies = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(400_000_000)
    for a, b in zip(copies, got):
        a.copy_(b)
    at = {t.data_ptr() for t in got}
    del got, b
    with torch.cuda.stream(s):
        again = [torch.full_like(t, 77) for t in want]
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


# ------------------------------------------------------------ prompt weights
def check_weights(B, H, H_kv, N_q, N_kv, d, dtype, causal, first, seed, w_in=True):
    g = rng(seed)
    q, k = rows(g, B, H, N_q, d, dtype=dtype), rows(g, B, H_kv, N_kv, d, dtype=dtype)
    v = rows(g, B, H_kv, N_kv, d, dtype=dtype)
    _, lse = fa.attention(q, k, v, causal=causal, num_splits=1)
    base = torch.rand(B, H_kv, N_kv, generator=g, device="cuda") if w_in else None
    out = fa.attention_weights(q, k, lse, causal=causal, first_query=first, weight_in=base)
    assert fa.fa_device_status(None) == fa.FA_OK
    scale = float(np.float32(1 / np.sqrt(d)))
    qn, kn, ln = np64(q), np64(k), np64(lse)
    ref, big = np.zeros((B, H_kv, N_kv)), 0.0
    seen = np.arange(N_kv)[None] <= np.arange(N_q)[:, None] + (N_kv - N_q)
    for b in range(B):
        for h in range(H):
            s = qn[b, h] @ kn[b, h // (H // H_kv)].T * scale
            big = max(big, float((np.abs(qn[b, h]) @ np.abs(kn[b, h // (H // H_kv)]).T).max()) * scale)
            with np.errstate(over="ignore", invalid="ignore"):
                p = np.where(np.isneginf(ln[b, h])[:, None], 0.0, np.exp(s - ln[b, h][:, None]))
            if causal:
                p = np.where(seen, p, 0.0)
            ref[b, h // (H // H_kv)] += p[first:].sum(0)
    wi = np64(base) if w_in else 0.0
    tol = R.tol_weight(ref, np.array([big]), ln, d, wi)
    err = np.abs(np64(out) - wi - ref)
    assert (err <= tol).all(), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
    return q, k, lse, out


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N_q,N_kv,first", [(1, 1, 0), (5, 129, 0), (128, 128, 100), (300, 300, 0), (257, 700, 256),
                                            (700, 257, 0), (640, 640, 200)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f16"), (128, "f16")])
def test_prompt_weights(causal, N_q, N_kv, first, d, dtype):
    check_weights(2, 4, 2, N_q, N_kv, d, dtype, causal, first, 500 + N_q + N_kv, w_in=first > 0)


def test_prompt_weights_head_layouts():
    check_weights(1, 6, 1, 200, 333, 64, "bf16", True, 0, 510)
    check_weights(3, 5, 5, 150, 150, 128, "f16", False, 10, 511)
    check_weights(1, 1, 1, 3000, 3000, 64, "bf16", True, 0, 512)   # key blocks shared by a cluster
    check_weights(2, 40, 20, 260, 1025, 64, "bf16", True, 0, 513)  # more blocks than SMs


def test_prompt_weights_into_a_cache():
    """weight_out as the first columns of a cache's weight, in place; the other columns stay."""
    q, k, lse, out = check_weights(2, 4, 2, 200, 200, 64, "bf16", True, 0, 520, w_in=False)
    w = torch.full((2, 2, 384), 2.0, device="cuda")
    got = fa.attention_weights(q, k, lse, causal=True, weight_in=w[:, :, :200], out=w[:, :, :200])
    assert got.data_ptr() == w.data_ptr() and w[:, :, 200:].eq(2.0).all()
    assert torch.equal(w[:, :, :200], 2.0 + out)
    assert torch.equal(fa.attention_weights(q, k, lse, causal=True), out)


def test_prompt_weights_masked_nan():
    """A NaN query row or key reaches only the weights it takes part in."""
    g = rng(530)
    q, k, v = (rows(g, 1, 1, 300, 64) for _ in range(3))
    _, lse = fa.attention(q, k, v, causal=True)
    good = fa.attention_weights(q, k, lse, causal=True)
    k2 = k.clone()
    k2[0, 0, 299] = float("nan")
    got = fa.attention_weights(q, k2, lse, causal=True)
    assert torch.equal(got[..., :299], good[..., :299]) and torch.isnan(got[..., 299]).all()
    q2 = q.clone()
    q2[0, 0, 50] = float("nan")
    got = fa.attention_weights(q2, k, lse, causal=True)
    assert torch.isnan(got[..., :51]).all() and torch.equal(got[..., 51:], good[..., 51:])


# ------------------------------------------------------------------ eviction
def bits(c, name):
    """An array of the cache as whole numbers (a NaN equals itself)."""
    t = getattr(c, name)
    return t.view(torch.int32) if name == "weight" else t


def check_evict(c, keep, sinks=0, recent=0, weight=None, out=None):
    n = [min(max(x, 0), c.capacity) for x in c.lengths.tolist()]
    seen = c.counts[1].tolist()
    old = {a: bits(c, a).clone() for a in ARRAYS if getattr(c, a) is not None}
    to = out if out is not None else c
    to_old = {a: bits(to, a).clone() for a in ARRAYS if getattr(to, a) is not None}
    w = (weight if weight is not None else c.weight).cpu().numpy()
    pos = c.pos.cpu().numpy() if c.pos is not None else None
    src = fa.kv4_evict(c, keep, sinks=sinks, recent=recent, weight=weight, out=out)
    for b in range(c.B):
        new = min(n[b], keep)
        for h in range(c.H_kv):
            want = R.select(w[b, h], pos[b, h] if pos is not None else None, n[b], seen[b], keep, sinks, recent)
            assert src[b, h, :new].tolist() == want and src[b, h, new:].eq(-1).all()
            at = torch.tensor(want, dtype=torch.long, device="cuda")
            for a in to_old:
                if a in old:
                    assert torch.equal(bits(to, a)[b, h, :new], old[a][b, h][at]), a
                assert torch.equal(bits(to, a)[b, h, new:], to_old[a][b, h, new:]), a
    assert to.counts.tolist() == [[min(x, keep) for x in n], seen]
    if out is not None:
        for a in old:
            assert torch.equal(bits(c, a), old[a])
    return src


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,keep,sinks,recent", [
    ([1], 1, 0, 0), ([2, 1, 0], 1, 0, 0), ([130, 128, 129], 128, 4, 16), ([300, 77, 0, 512], 100, 0, 0),
    ([1000, 999], 999, 4, 0), ([700], 20, 30, 40), ([513, 31], 512, 0, 100), ([64], 128, 4, 4)])
def test_evict_in_place(d, lengths, keep, sinks, recent):
    g = rng(600 + sum(lengths) + keep)
    check_evict(filled(g, len(lengths), 2, lengths, d), keep, sinks, recent)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length,keep", [(500, 100), (2500, 2000), (90, 128), (5000, 1)])
def test_evict_into_another_cache(d, length, keep):
    g = rng(620 + length)
    c = filled(g, 2, 3, [length, length // 2], d)
    to = filled(g, 2, 3, [3, 4], d, capacity=keep + 128)
    check_evict(c, keep, 4, min(16, keep), out=to)


@pytest.mark.parametrize("length,keep", [(300, 5000), (1, 129), (128, 100000)])
def test_evict_into_a_larger_cache(length, keep):
    """More than the first cache has slots may be asked for: all its entries are taken over."""
    g = rng(622 + length)
    c = filled(g, 2, 2, [length, 0], 64)
    check_evict(c, keep, 4, 16, out=filled(g, 2, 2, [7, 8], 64, capacity=keep + 100))


@pytest.mark.parametrize("length", [17, 300, 4100, 40010])
@pytest.mark.parametrize("e", [1, 2, 5, 15, 16, 17])
def test_evict_a_few(length, e):
    """As many as are found one by one, and one more; mostly ties; with protected ones among the last."""
    if e >= length:
        return
    g = rng(625 + length + e)
    c = filled(g, 1, 3, [length], 64)
    c.weight[0, 1].copy_(torch.randint(0, 2, c.weight[0, 1].shape, generator=g, device="cuda").float())
    c.weight[0, 2].zero_()
    check_evict(c, length - e, 3, min(4, length - e))


def test_evict_ties_and_odd_weights():
    """Ties by slot, signed zeros equal, infinities and NaN in order, over several warps' shares."""
    g = rng(630)
    c = filled(g, 1, 2, [3000], 64)
    c.weight.copy_(torch.randint(0, 3, c.weight.shape, generator=g, device="cuda").float())
    check_evict(c, 1500)
    c = filled(g, 1, 2, [3000], 64)
    c.weight.zero_()
    c.weight[:, :, ::2] = -0.0
    check_evict(c, 700, sinks=3, recent=5)
    c = filled(g, 1, 2, [2000], 64)
    c.weight[0, 0, 5], c.weight[0, 0, 1999], c.weight[0, 1, 1500] = float("nan"), float("inf"), -float("nan")
    c.weight[0, 1, 3] = -float("inf")
    check_evict(c, 2, sinks=1)
    c = filled(g, 1, 1, [2000], 64)
    c.weight.neg_()
    check_evict(c, 1999)


def test_evict_by_other_weights_and_without_pos():
    g = rng(640)
    c = filled(g, 2, 2, [400, 300], 128)
    w = torch.rand(c.weight.shape, generator=g, device="cuda")
    check_evict(c, 250, weight=w)
    bare = fa.KV4Cache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.counts)
    check_evict(bare, 100, weight=w)


def test_evict_long_rows_on_one_and_many_clusters():
    g = rng(650)
    c = filled(g, 1, 1, [60000], 64)
    check_evict(c, 30000, 4, 100)
    c = filled(g, 40, 8, [900] * 40, 64)  # more heads than SMs
    check_evict(c, 899)


@pytest.mark.parametrize("length,keep,levels", [(33000, 32990, 0), (45001, 20000, 0), (49152, 6000, 5),
                                                (300001, 250000, 0), (393216, 1000, 3)])
def test_evict_slices_of_more_words_than_threads(length, keep, levels):
    g = rng(655)
    c = filled(g, 1, 1, [length], 64)
    if levels:  # mostly ties
        c.weight.copy_(torch.randint(0, levels, c.weight.shape, generator=g, device="cuda").float())
    check_evict(c, keep, 4, 100)


@pytest.mark.parametrize("keep", [395, 250])  # few leaving entries, and many
def test_evict_by_weights_on_4_byte_boundaries(keep):
    g = rng(657)
    c = filled(g, 2, 2, [400, 300], 64)
    w = torch.rand(c.weight.numel() + 1, generator=g, device="cuda")[1:].view(c.weight.shape)
    assert w.data_ptr() % 16 == 4
    check_evict(c, keep, weight=w)


def test_evict_ranks_by_protected_positions_after_moves():
    """Positions move with their entries: the newest stay protected wherever they are."""
    g = rng(660)
    c = filled(g, 1, 2, [200], 64)
    c.pos.copy_(torch.arange(c.capacity, dtype=torch.int32, device="cuda").expand_as(c.pos))
    for keep in (150, 60):
        check_evict(c, keep, sinks=4, recent=20)
        for p in (0, 1, 2, 3, *range(180, 200)):
            assert (c.pos[:, :, :keep] == p).any(-1).all()


# ------------------------------------------------------------ as a user runs it
def serve(c, steps, keep, q, k, v):
    """`steps` decode steps: store the new token, attend and add weights, evict to `keep`."""
    outs = []
    for i in range(steps):
        fa.kv4_append(c, k[i], v[i])
        outs.append(fa.kv4_attention(q[i], c, weight_out=c.weight)[0])
        fa.kv4_evict(c, keep, sinks=2, recent=8)
    return outs


@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
def test_serving_loop(d, dtype):
    """A prompt read and stored, its weights counted, the cache compressed into a smaller one, then
    decode steps that store, attend, count and evict: each step against 64 bits on the cache's state."""
    g = rng(700 + d)
    B, H, H_kv, N, keep = 2, 8, 2, 300, 128
    q, k, v = rows(g, B, H, N, d, dtype=dtype), rows(g, B, H_kv, N, d, dtype=dtype), rows(g, B, H_kv, N, d, dtype=dtype)
    long = fa.KV4Cache.empty(B, H_kv, N, d)
    fa.kv4_append(long, k, v)
    ks, vs = fa.kv4_read(long, N, dtype=TORCH[dtype])
    _, lse = fa.attention(q, ks, vs, causal=True)
    fa.attention_weights(q, ks, lse, causal=True, out=long.weight[:, :, :N], weight_in=long.weight[:, :, :N])
    c = fa.KV4Cache.empty(B, H_kv, keep + 4, d)
    check_evict(long, keep, sinks=2, recent=8, out=c)
    # every query of every head of a group added 1 in all
    assert abs(float(long.weight.double().sum()) - B * H * N) <= 1e-3 * B * H * N
    for i in range(5):
        k1, v1, q1 = (rows(g, B, h, 1, d, dtype=dtype) for h in (H_kv, H_kv, H))
        fa.kv4_append(c, k1, v1)
        assert c.counts.tolist() == [[keep + 1] * B, [N + i + 1] * B]
        _, _, w = check_attention(c, q1, dtype)
        before = c.weight.clone()
        fa.kv4_attention(q1, c, weight_out=c.weight)
        assert torch.equal(c.weight[:, :, :keep + 1], w[:, :, :keep + 1])
        assert torch.equal(c.weight[:, :, keep + 1:], before[:, :, keep + 1:])
        check_evict(c, keep, sinks=2, recent=8)
        assert c.pos[:, :, :keep].max(-1).values.eq(N + i).all()


def test_captured_steps_follow_the_counts():
    """One decode step captured in a graph and replayed: counts advance on the device; results equal
    the same steps run eagerly, bit for bit."""
    g = rng(710)
    B, H, H_kv, d, keep, steps = 3, 8, 2, 64, 140, 6
    qs, ks, vs = (torch.stack([rows(g, B, h, 1, d) for _ in range(steps)]) for h in (H, H_kv, H_kv))
    eager, graph = (filled(rng(711), B, H_kv, [137, 20, 139], d, capacity=256) for _ in range(2))
    outs = [o.clone() for o in serve(eager, steps, keep, qs, ks, vs)]
    q, k, v, out = qs[0].clone(), ks[0].clone(), vs[0].clone(), torch.empty_like(qs[0])
    ws = torch.empty(graph.workspace_size(H, 1, True), dtype=torch.uint8, device="cuda")
    src = torch.empty(B, H_kv, keep, dtype=torch.int32, device="cuda")

    def step():
        fa.kv4_append(graph, k, v)
        fa.kv4_attention(q, graph, out=out, weight_out=graph.weight, workspace=ws)
        fa.kv4_evict(graph, keep, sinks=2, recent=8, src=src)

    state = [getattr(graph, a) for a in (*ARRAYS, "counts")]
    saved = [t.clone() for t in state]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # warm-up, undone below
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for t, old in zip(state, saved):
        t.copy_(old)
    for i in range(steps):
        q.copy_(qs[i]), k.copy_(ks[i]), v.copy_(vs[i])
        gr.replay()
        assert torch.equal(out, outs[i]), i
    assert torch.equal(eager.counts, graph.counts)
    for a in ARRAYS:
        x, y = getattr(eager, a), getattr(graph, a)
        for b, n in enumerate(eager.lengths.tolist()):
            assert torch.equal(x[b, :, :n], y[b, :, :n]), a


def test_captured_across_streams():
    """A captured step whose row and query come from another captured stream, beside which the
    append runs, and whose output a third kernel reads."""
    g = rng(720)
    B, H, H_kv, d = 2, 8, 2, 128
    c = filled(g, B, H_kv, [1500, 1100], d, capacity=2048)
    k, v, q = (rows(g, B, h, 1, d) for h in (H_kv, H_kv, H))
    q2, out, twice = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(c.workspace_size(H, 1, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.mul(q, 2, out=q2)
        fa.kv4_append(c, k, v)
        here.wait_stream(side)
        fa.kv4_attention(q2, c, out=out, weight_out=c.weight, workspace=ws)
        torch.mul(out, 2, out=twice)

    state = [t.clone() for t in (c.counts, c.weight)]
    step()
    torch.cuda.synchronize()
    want, weight = twice.clone(), c.weight.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for _ in range(3):
        c.counts.copy_(state[0]), c.weight.copy_(state[1])
        for t in (q2, out, twice):
            t.zero_()
        gr.replay()
        assert torch.equal(twice, want) and torch.equal(c.weight, weight)


def test_prompt_into_cache_behind_the_forward_pass():
    """The forward pass, the keys' weights from its lse, storing and attending follow one another
    without a wait in between, and match the same calls made one at a time."""
    g = rng(730)
    B, H, H_kv, N, d = 1, 8, 2, 2500, 128  # a last wave that the forward pass splits
    q, k, v = (rows(g, B, h, N, d) for h in (H, H_kv, H_kv))
    want = None
    for apart in (True, False, False):
        def step():
            if apart:
                torch.cuda.synchronize()
        c = fa.KV4Cache.empty(B, H_kv, N + 1, d)
        c.weight.zero_()
        x = (k * 1).contiguous()
        step()
        o, lse = fa.attention(q, x, v, causal=True)
        step()
        fa.kv4_append(c, x, v)
        step()
        fa.attention_weights(q, x, lse, causal=True, weight_in=c.weight[:, :, :N], out=c.weight[:, :, :N])
        step()
        w = c.weight[:, :, :N].clone()
        step()
        out, _ = fa.kv4_attention(q[:, :, -1:].contiguous(), c, weight_out=c.weight)
        torch.cuda.synchronize()
        got = [o, lse, w, out, c.weight[:, :, :N].clone()]
        want = want or got
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_serving_loops_at_once():
    """Loops on three streams, with the prompt's kernels between them, equal the same loops one after another."""
    g = rng(740)
    H, H_kv, d, steps, N = 8, 2, 64, 12, 1300
    sizes = [(3, [1500, 20, 700], 1499), (1, [9000], 8900), (8, [600, 0, 31, 512, 511, 64, 1, 600], 600)]
    token = [tuple(torch.stack([rows(g, B, h, 1, d) for _ in range(steps)]) for h in (H, H_kv, H_kv)) for B, _, _ in sizes]
    pq, pk, pv = (rows(g, 1, h, N, d) for h in (H, H_kv, H_kv))

    def caches():
        return [filled(rng(741 + i), B, H_kv, lengths, d, max(lengths) + steps) for i, (B, lengths, _) in enumerate(sizes)]

    def loop(c, size, t):
        _, lse = fa.attention(pq, pk, pv, causal=True)
        w = fa.attention_weights(pq, pk, lse, causal=True)
        return [*serve(c, steps, size[2], *t), w, lse]

    want = caches()
    outs = [[x.clone() for x in loop(c, s, t)] for c, s, t in zip(want, sizes, token)]
    for _ in range(3):
        got = caches()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in sizes]
        res = []
        for c, s, t, stream in zip(got, sizes, token, streams):
            with torch.cuda.stream(stream):
                res.append(loop(c, s, t))
        torch.cuda.synchronize()
        for a, b in zip(outs, res):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        for x, y in zip(want, got):
            assert torch.equal(x.counts, y.counts)
            for name in ARRAYS:
                for b, n in enumerate(x.lengths.tolist()):
                    assert torch.equal(bits(x, name)[b, :, :n], bits(y, name)[b, :, :n]), name


def test_lengths_advanced_just_before_the_call():
    """Appends whose blocks read the lengths on every SM and whose second kernel advances them, each
    followed at once by attention with weights: the same as with a wait after every call."""
    g = rng(750)
    H, H_kv, d, n, steps = 32, 8, 128, 600, 3
    k, v, q = (rows(g, 1, h, x, d) for h, x in ((H_kv, n), (H_kv, n), (H, 1)))
    c = fa.KV4Cache.empty(1, H_kv, steps * n + 100, d)

    def run(wait):
        c.counts.zero_()
        got = []
        for i in range(1, steps + 1):
            fa.kv4_append(c, k, v)
            wait()
            got += fa.kv4_attention(q, c, weight_out=c.weight)
            wait()
            got.append(c.weight[:, :, :i * n].clone())  # behind the length: what earlier rounds left
        return got

    want = run(torch.cuda.synchronize)
    for _ in range(20):
        for a, b in zip(want, run(lambda: None)):
            assert torch.equal(a, b)


def test_evictions_of_several_host_threads():
    """Threads that evict from caches of different sizes: none changes what the others may launch."""
    sizes = (128, 40960) * 4
    barrier = threading.Barrier(len(sizes))
    status = []

    def loop(capacity):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            c = filled(rng(760), 1, 2, [capacity], 64)
            src = torch.empty(1, 2, capacity - 1, dtype=torch.int32, device="cuda")
            counts = torch.empty_like(c.counts)
        stream.synchronize()
        call = (c._struct, capacity - 1, 0, 0, None, None, src.data_ptr(), counts.data_ptr(), stream.cuda_stream)
        barrier.wait()
        status.extend(fa.fa_kv4_evict(*call) for _ in range(2000))
        stream.synchronize()

    threads = [threading.Thread(target=loop, args=(n,)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert status == [fa.FA_OK] * (2000 * len(sizes))
