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


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_scales(scale, d, causal):
    check_backward(*batch(9, [200, 1, 130], 4, 2, d, "bf16"), causal, scale)
