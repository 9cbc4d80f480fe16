"""Attention over packed sequences on the GPU against its 64-bit restatement:
lengths from none to many tiles, head layouts, keys of other lengths, strided
views, what other rows hold, gradients, captured calls, calls at once."""
import math

import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from . import packed_ref as R  # noqa: E402

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


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


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def batch(seed, lens, H, H_kv, d, dtype, lens_k=None, gain=1.0):
    """q, k, v and the offsets as lists."""
    g, lens_k = rng(seed), lens if lens_k is None else lens_k
    return (rows(g, sum(lens), H, d, dtype=dtype, gain=gain), rows(g, sum(lens_k), H_kv, d, dtype=dtype),
            rows(g, sum(lens_k), H_kv, d, dtype=dtype), R.offsets(lens), R.offsets(lens_k))


def within(got, want, tol, what=""):
    """Where `want` is finite `got` is within `tol`, and -inf where it is that; NaN wants are not looked at."""
    got = got.double()
    assert torch.equal(got[want == -math.inf], want[want == -math.inf])
    at = torch.isfinite(want)
    bad = ~((got - want).abs() <= tol) & at
    worst = ((got - want).abs() / tol)[at].max() if at.any() else 0.0
    assert not bad.any(), (what, int(bad.sum()), float(worst), bad.nonzero()[:4].tolist())


def check_forward(q, k, v, cu_q, cu_k, causal, scale=None, **kw):
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse = fa.packed_attention(q, k, v, int32(cu_q), int32(cu_k), scale=scale, causal=causal, **kw)
    want_o, want_l, tol_o, tol_l = R.forward(q, k, v, cu_q, cu_k, s, causal)
    within(lse, want_l, tol_l, "lse")
    within(out, want_o, tol_o, "out")
    return out, lse


def check_backward(q, k, v, cu_q, cu_k, causal, scale=None, seed=99, **kw):
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse = check_forward(q, k, v, cu_q, cu_k, causal, scale)
    dout = torch.randn(q.shape, generator=rng(seed), device="cuda").to(q.dtype)
    got = fa.packed_attention_backward(q, k, v, out, lse, dout, int32(cu_q), int32(cu_k), scale=scale, causal=causal, **kw)
    want = R.backward(q, k, v, out, lse, dout, cu_q, cu_k, s, causal)
    for name, x in zip(("dq", "dk", "dv"), got):
        within(x, *want[name], name)
    return got


LENS = [[1], [64], [127, 128, 129], [256, 1, 0, 300], [0, 0], [700, 3, 513]]
TYPES = [(64, "bf16"), (128, "bf16"), (64, "f16"), (128, "f16")]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_forward_lengths(lens, causal, d, dtype):
    check_forward(*batch(1, lens, 4, 2, d, dtype), causal)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 3), (3, 1), (4, 1), (6, 2), (16, 2), (5, 5)])
@pytest.mark.parametrize("causal", [False, True])
def test_forward_heads(H, H_kv, causal):
    check_forward(*batch(2, [130, 40, 385], H, H_kv, 64, "bf16"), causal)


KEYS = [([100, 33, 257, 1], [300, 0, 128, 77]), ([300, 129, 5], [200, 1, 4]), ([1, 1, 1], [640, 0, 129]), ([0, 50], [70, 0]),
        ([400], [100])]


@pytest.mark.parametrize("lens,lens_k", KEYS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("H", [2, 4])  # groups of one head (blocks of 256 rows) and of two
def test_forward_keys_of_other_lengths(lens, lens_k, causal, d, dtype, H):
    check_forward(*batch(3, lens, H, 2, d, dtype, lens_k), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B", [31, 32, 33, 150])
def test_forward_many_sequences(B, causal):
    lens = [(7 * i * i + 3 * i) % 200 for i in range(B)]
    check_forward(*batch(4, lens, 2, 1, 64, "bf16"), causal)


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", TYPES)
def test_backward_lengths(lens, causal, d, dtype):
    check_backward(*batch(5, lens, 4, 2, d, dtype), causal)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 1), (6, 2), (8, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_backward_heads(H, H_kv, causal):
    check_backward(*batch(6, [130, 40, 385], H, H_kv, 128, "bf16"), causal)


@pytest.mark.parametrize("lens,lens_k", KEYS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_backward_keys_of_other_lengths(lens, lens_k, causal, d, dtype):
    check_backward(*batch(7, lens, 4, 2, d, dtype, lens_k), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B", [32, 33, 150])
def test_backward_many_sequences(B, causal):
    lens = [(7 * i * i + 3 * i) % 200 for i in range(B)]
    check_backward(*batch(8, lens, 2, 1, 64, "bf16"), causal)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (4, 2)])  # blocks of 256 rows of a head, of 128 of two
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,first", [(64, 0), (65, 0), (65, 300), (700, 0)])
def test_sequences_in_order(B, first, causal, H, H_kv):
    """Batches of more sequences than are ordered by their work: empty ones, long ones among short ones, rows of no
    sequence before and behind them, keys of other lengths."""
    lens = [(0, 1, 700, 7, 128, 3, 129, 0, 31, 257)[(i * i + i // 7) % 10 if i % 13 == 0 else i % 2 + 3 * (i % 3 == 0)]
            for i in range(B)]
    lens_k = [n + (0, 5, 130)[i % 3] if i % 11 else 0 for i, n in enumerate(lens)]
    g = rng(30)
    Tq, Tk = sum(lens) + first + 40, sum(lens_k) + first + 40
    q, k, v = rows(g, Tq, H, 64), rows(g, Tk, H_kv, 64), rows(g, Tk, H_kv, 64)
    cu_q, cu_k = R.offsets(lens, first), R.offsets(lens_k, first)
    dx = [torch.full(x.shape, 5.0, device="cuda").bfloat16() for x in (q, k, v)]
    check_backward(q, k, v, cu_q, cu_k, causal, dq=dx[0], dk=dx[1], dv=dx[2])
    for x, cu in zip(dx, (cu_q, cu_k, cu_k)):
        assert (x[:first] == 5).all() and (x[cu[-1]:] == 5).all()


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_many_offsets_that_are_none(seed):
    g = rng(31 + seed)
    q, k, v, good, _ = batch(32, [100, 100, 200], 2, 2, 64, "bf16")
    cu = torch.randint(-500, 1000, (100,), generator=g, device="cuda").int()
    if seed == 1:
        cu = torch.randint(-2 ** 31, 2 ** 31 - 1, (100,), generator=g, device="cuda").int()
    if seed == 2:
        cu = cu.sort(descending=True)[0]
    guard = torch.full((3, 500, 2, 64), 5.0, device="cuda").bfloat16()
    out, lse = fa.packed_attention(q, k, v, cu, causal=True, out=guard[0, 50:450])
    fa.packed_attention_backward(q, k, v, out, lse, q, cu, causal=True, dq=guard[1, 50:450], dk=guard[2, 50:450])
    assert (guard[:, :50] == 5).all() and (guard[:, 450:] == 5).all()
    check_backward(q, k, v, good, good, True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_scales(scale, d, causal):
    check_backward(*batch(9, [200, 1, 130], 4, 2, d, "bf16"), causal, scale)


# ------------------------------------------------- layouts, and what other rows hold
def test_slices_of_one_projection():
    """q, k and v as slices of one tensor, the gradients into slices of another."""
    g = rng(10)
    lens = [200, 1, 0, 333]
    T, cu = sum(lens), R.offsets(lens)
    qkv, grad = rows(g, T, 6 + 2 + 2, 128), torch.full((T, 10, 128), math.nan, device="cuda").bfloat16()
    dq, dk, dv = grad.split([6, 2, 2], 1)
    got = check_backward(*qkv.split([6, 2, 2], 1), cu, cu, True, dq=dq, dk=dk, dv=dv)
    assert all(a is b for a, b in zip(got, (dq, dk, dv))) and torch.isfinite(grad).all()


def test_heads_before_rows():
    """[heads, rows, d] memory, and rows further apart than they are long."""
    g = rng(11)
    lens = [200, 1, 131]
    T, cu = sum(lens), R.offsets(lens)
    q = rows(g, 4, T, 64, dtype="f16").transpose(0, 1)
    k, v = (rows(g, T, 2, 96, dtype="f16")[..., 16:80] for _ in range(2))
    out = torch.full((T, 4, 128), math.nan, device="cuda").half()[..., 64:]
    check_forward(q, k, v, cu, cu, False, out=out)
    check_backward(q, k, v, cu, cu, True, dq=torch.empty(4, T, 64, device="cuda").half().transpose(0, 1))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 4])
def test_rows_of_no_sequence(causal, d, H):
    """Rows ahead of the first sequence and behind the last are neither read nor written."""
    lens, lens_k = [70, 0, 129, 300], [128, 31, 0, 260]
    q, k, v, _, _ = batch(12, [37] + lens + [91], H, 2, d, "bf16", [5] + lens_k + [200])
    cu_q, cu_k = R.offsets(lens, 37), R.offsets(lens_k, 5)
    dout = rows(rng(13), *q.shape)
    for x, cu in ((q, cu_q), (k, cu_k), (v, cu_k), (dout, cu_q)):
        x[:cu[0]], x[cu[-1]:] = math.nan, math.inf
    out, lse = torch.full_like(q, 7), torch.full((H, len(q)), 7.0, device="cuda")
    check_forward(q, k, v, cu_q, cu_k, causal, out=out, lse=lse)
    s = 1 / math.sqrt(d)
    want = R.backward(q, k, v, out, lse, dout, cu_q, cu_k, s, causal)
    got = fa.packed_attention_backward(q, k, v, out, lse, dout, int32(cu_q), int32(cu_k), causal=causal,
                                       dq=torch.full_like(q, 7), dk=torch.full_like(k, 7), dv=torch.full_like(v, 7))
    for name, x in zip(("dq", "dk", "dv"), got):
        within(x, *want[name], name)
    for x, cu in ((out, cu_q), (lse.T, cu_q), (got[0], cu_q), (got[1], cu_k), (got[2], cu_k)):
        assert (x[:cu[0]] == 7).all() and (x[cu[-1]:] == 7).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_another_sequences_infinities(causal, d):
    """What is not finite stays in its sequence, forward and backward."""
    lens = [150, 90, 40, 333]
    q, k, v, cu, _ = batch(14, lens, 4, 2, d, "bf16")
    dout = rows(rng(15), *q.shape)
    bad = slice(cu[1], cu[2])
    for x, value in ((q, math.nan), (k, math.inf), (v, -math.inf), (dout, math.nan)):
        x[bad] = value
    out, lse = fa.packed_attention(q, k, v, int32(cu), causal=causal)
    got = (out, lse.T) + tuple(fa.packed_attention_backward(q, k, v, out, lse, dout, int32(cu), causal=causal))
    for x in (q, k, v, dout):
        x[bad] = 1.0
    out2, lse2 = fa.packed_attention(q, k, v, int32(cu), causal=causal)
    want = (out2, lse2.T) + tuple(fa.packed_attention_backward(q, k, v, out2, lse2, dout, int32(cu), causal=causal))
    good = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    good[bad] = False
    for i, (a, b) in enumerate(zip(got, want)):
        if i == 2:  # dq's parts are added in any order
            assert torch.allclose(a[good].float(), b[good].float(), rtol=2.0 ** -7, atol=1e-5)
        else:
            assert torch.equal(a[good], b[good])


@pytest.mark.parametrize("gain", [20.0, 1e4])
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores(gain, d):
    """Scores that move the reference from tile to tile, and weights that are 0 or 1."""
    check_forward(*batch(16, [700, 130], 2, 1, d, "bf16", gain=gain), True)


def test_masked_keys_above_the_visible_ones():
    """A hidden key's score is far above every visible one."""
    q, k, v, cu, _ = batch(17, [256], 2, 1, 64, "bf16")
    k[200:] *= 100
    check_forward(q, k, v, cu, cu, True)


def test_no_rows():
    q, k = torch.empty(0, 4, 64, device="cuda").half(), torch.empty(0, 2, 64, device="cuda").half()
    cu = int32([0, 0, 0])
    out, lse = fa.packed_attention(q, k, k, cu)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    got = fa.packed_attention_backward(q, k, k, out, lse, q, cu)
    assert [x.shape for x in got] == [q.shape, k.shape, k.shape]
    # queries without keys, keys without queries
    g = rng(18)
    q1 = rows(g, 100, 4, 64, dtype="f16")
    out, lse = fa.packed_attention(q1, k, k, int32([0, 30, 100]), cu)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, _, _ = fa.packed_attention_backward(q1, k, k, out, lse, q1, int32([0, 30, 100]), cu)
    assert (dq == 0).all()
    k1 = rows(g, 100, 2, 64, dtype="f16")
    out, lse = fa.packed_attention(q, k1, k1, cu, int32([0, 30, 100]))
    _, dk, dv = fa.packed_attention_backward(q, k1, k1, out, lse, q, cu, int32([0, 30, 100]))
    assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("cu", [[0, 300, 100, 400], [-50, 100, 900, 300], [400, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 5, 7]])
def test_offsets_that_are_none(cu):
    """Offsets out of range or order: nothing outside the tensors is touched, and the next call is as ever."""
    q, k, v, good, _ = batch(19, [100, 100, 200], 2, 2, 64, "bf16")
    guard = torch.full((3, 500, 2, 64), 5.0, device="cuda").bfloat16()
    out, lse = fa.packed_attention(q, k, v, int32(cu), causal=True, out=guard[0, 50:450])
    fa.packed_attention_backward(q, k, v, out, lse, q, int32(cu), causal=True, dq=guard[1, 50:450], dk=guard[2, 50:450])
    assert (guard[:, :50] == 5).all() and (guard[:, 450:] == 5).all()
    check_backward(q, k, v, good, good, True)


def test_offsets_pass_32_bits():
    """Sequences behind 2^31 elements of every tensor."""
    T, H, d = 530000, 32, 128
    assert T * H * d > 2 ** 31 + 2 ** 24
    g = rng(20)
    q = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    k, v, out, dq, dk, dv, dout = (torch.zeros_like(q) for _ in range(7))
    first, lens = T - 400, [130, 1, 269]
    cu = R.offsets(lens, first)
    for x in (q, k, v, dout):
        x[first:] = rows(g, 400, H, d)
    lse = torch.zeros(H, T, device="cuda")
    fa.packed_attention(q, k, v, int32(cu), causal=True, out=out, lse=lse)
    fa.packed_attention_backward(q, k, v, out, lse, dout, int32(cu), causal=True, dq=dq, dk=dk, dv=dv)
    near = [x[first:] for x in (q, k, v, out, dout)]
    at, s = R.offsets(lens), 1 / math.sqrt(d)
    want_o, want_l, tol_o, tol_l = R.forward(*near[:3], at, at, s, True)
    within(out[first:], want_o, tol_o)
    within(lse[:, first:], want_l, tol_l)
    want = R.backward(*near[:4], lse[:, first:], near[4], at, at, s, True)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        within(x[first:], *want[name], name)
        assert not x[:first].any()


# ------------------------------------------------- streams, captured calls, calls at once
def test_repeats_and_another_stream():
    q, k, v, cu, _ = batch(21, [300, 5, 700], 4, 2, 128, "bf16")
    c = int32(cu)
    out, lse = fa.packed_attention(q, k, v, c, causal=True)
    grads = fa.packed_attention_backward(q, k, v, out, lse, q, c, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        o2, l2 = fa.packed_attention(q, k, v, c, causal=True, stream=stream)
        g2 = fa.packed_attention_backward(q, k, v, out, lse, q, c, causal=True, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert torch.equal(grads[1], g2[1]) and torch.equal(grads[2], g2[2])
        assert torch.allclose(grads[0].float(), g2[0].float(), rtol=2.0 ** -7, atol=1e-5)


def test_captured_calls_follow_the_offsets():
    """A captured forward and backward pass over other lengths, each time against a fresh call."""
    g = rng(22)
    q, k, v, dout = (rows(g, 600, h, 64, dtype="f16") for h in (4, 2, 2, 4))
    cu = int32([0, 200, 400, 600])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = fa.packed_attention(q, k, v, cu, causal=True)
        fa.packed_attention_backward(q, k, v, out, lse, dout, cu, causal=True)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fa.packed_attention(q, k, v, cu, causal=True)
        grads = fa.packed_attention_backward(q, k, v, out, lse, dout, cu, causal=True)
    for at in ([0, 200, 400, 600], [0, 1, 599, 600], [0, 0, 0, 600], [0, 128, 384, 600]):
        cu.copy_(int32(at))
        graph.replay()
        o2, l2 = fa.packed_attention(q, k, v, int32(at), causal=True)
        g2 = fa.packed_attention_backward(q, k, v, o2, l2, dout, int32(at), causal=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(a, b) for a, b in zip(grads[1:], g2[1:]))
        assert torch.allclose(grads[0].float(), g2[0].float(), rtol=2.0 ** -10, atol=1e-5)


def test_calls_at_once():
    """Forward and backward passes on four streams at once, each in its own memory."""
    jobs = []
    for i, (lens, d, causal) in enumerate((([900, 3, 300], 128, True), ([64] * 20, 64, False), ([2000], 128, False),
                                           ([1, 500, 0, 77], 64, True))):
        q, k, v, cu, _ = batch(30 + i, lens, 4, 2, d, "bf16")
        out, lse = fa.packed_attention(q, k, v, int32(cu), causal=causal)
        jobs.append((q, k, v, int32(cu), causal, out, lse, fa.packed_attention_backward(q, k, v, out, lse, q, int32(cu),
                                                                                         causal=causal)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for s, (q, k, v, cu, causal, out, lse, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                o2, l2 = fa.packed_attention(q, k, v, cu, causal=causal)
                got.append((o2, l2, fa.packed_attention_backward(q, k, v, out, lse, q, cu, causal=causal)))
        torch.cuda.synchronize()
        for (o2, l2, g2), (_, _, _, _, _, out, lse, grads) in zip(got, jobs):
            assert torch.equal(out, o2) and torch.equal(lse, l2)
            assert torch.equal(grads[1], g2[1]) and torch.equal(grads[2], g2[2])
            assert torch.allclose(grads[0].float(), g2[0].float(), rtol=2.0 ** -7, atol=1e-5)


def test_as_the_batched_attention():
    """Sequences of equal length are a batch: both calls' results, within the roundings of each."""
    B, H, H_kv, N, d = 3, 4, 2, 333, 128
    q, k, v, cu, _ = batch(40, [N] * B, H, H_kv, d, "bf16")
    out, lse, = check_forward(q, k, v, cu, cu, True)
    q4, k4, v4 = (x.view(B, N, -1, d).transpose(1, 2).contiguous() for x in (q, k, v))
    o4, l4 = fa.attention(q4, k4, v4, causal=True)
    _, _, tol, tol_l = R.forward(q, k, v, cu, cu, 1 / math.sqrt(d), True)
    within(o4.transpose(1, 2).reshape(q.shape), out.double(), 2 * tol)
    within(l4.transpose(0, 1).reshape(lse.shape), lse.double(), 2 * tol_l)
