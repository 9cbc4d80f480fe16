"""Attention over packed sequences on the GPU: slices of one tensor in every
order of rows, heads and parts; how far a value row that is not finite reaches;
tensors with room for more rows than are in use; the longest sequences."""
import math

import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from . import packed_ref as R  # noqa: E402
from .test_packed_gpu import batch, check_backward, int32, rng, rows, within  # noqa: E402,F401
from .test_paged_gpu import cache_of, check_append  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert fa.fa_device_status(None) == fa.FA_OK


ORDERS = {"T H 3 d": lambda x: x.unbind(2), "H T 3 d": lambda x: [y.transpose(0, 1) for y in x.unbind(2)]}


@pytest.mark.parametrize("order", ORDERS)
def test_slices_with_the_parts_beside_each_head(order):
    """q, k and v, and the gradients, as parts of tensors that keep each head's three together."""
    g = rng(63)
    lens, H = [200, 1, 0, 131], 3
    T, cu = sum(lens), R.offsets(lens)
    shape = {"T H 3 d": (T, H, 3, 64), "H T 3 d": (H, T, 3, 64)}[order]
    q, k, v = ORDERS[order](rows(g, *shape))
    grads = torch.full(shape, math.nan, device="cuda").bfloat16()
    dq, dk, dv = ORDERS[order](grads)
    check_backward(q, k, v, cu, cu, True, dq=dq, dk=dk, dv=dv)
    assert torch.isfinite(grads).all()


@pytest.mark.parametrize("order", ORDERS)
def test_rows_rotated_in_place_beside_each_other(order):
    """q and k rotated where they lie, the parts of a head side by side; v stays as it was."""
    g = rng(64)
    c, _ = cache_of(g, [15, 300], 2, 64, 16, room=40, poison=False)
    shape = {"T H 3 d": (41, 2, 3, 64), "H T 3 d": (2, 41, 3, 64)}[order]
    q, k, v = ORDERS[order](rows(g, *shape))
    v0, table = v.clone(), fa.rotary_table(400, 64)
    k_rot = torch.empty_like(k)
    held = c.lengths.clone()
    fa.paged_append(c, k, v, cu=int32([0, 40, 41]), table=table, k_out=k_rot)
    c.lengths.copy_(held)
    k1 = k.clone()
    got = check_append(g, c, [40, 1], 2, table, views=(q, k, v), q_out=q)
    assert got is q and torch.equal(k, k1)
    c.lengths.copy_(held)
    fa.paged_append(c, k, v, cu=int32([0, 40, 41]), table=table, k_out=k)
    assert torch.equal(k, k_rot) and torch.equal(v, v0)


@pytest.mark.parametrize("H,H_kv", [(4, 2), (3, 3), (3, 1)])  # blocks of 128 rows of two heads, of 256 of one
@pytest.mark.parametrize("n_q,n_k", [(700, 700), (700, 701), (600, 728), (700, 760), (256, 257)])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_how_far_a_value_row_reaches(H, H_kv, n_q, n_k, d, dtype, value):
    """Queries that see the row are not finite; those that do not, from the distance on that the header gives, and the
    other sequence's are as without it, bit for bit."""
    q, k, v, cu_q, cu_k = batch(60, [40, n_q], H, H_kv, d, dtype, [40, n_k])
    want, want_l = fa.packed_attention(q, k, v, int32(cu_q), int32(cu_k), causal=True)
    last = torch.arange(n_q, device="cuda") + n_k - n_q  # the last key that each query sees
    reach = 128 + 128 * (H // H_kv % 2) + 127 * ((n_k - n_q) % 128 != 0)
    for key in [*range(0, n_k, 37), 255, n_k - 1] + [383] * (n_k > 383):
        w = v.clone()
        w[cu_k[1] + key] = value
        out, lse = fa.packed_attention(q, k, w, int32(cu_q), int32(cu_k), causal=True)
        assert torch.equal(lse, want_l) and torch.equal(out[:40], want[:40])
        out = out[40:]
        assert not torch.isfinite(out[last >= key]).any()
        far = last <= key - reach
        assert torch.equal(out[far], want[40:][far])


@pytest.mark.parametrize("H,H_kv,d", [(4, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("lens", [[130, 0, 300, 1], [14] * 70, [0, 0], [0] * 80], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_few_rows_in_use(lens, causal, H, H_kv, d):
    """Tensors with room for far more rows than the sequences have: results bit for bit those of tensors without it, and
    the other rows untouched; forward and backward, as a captured call whose offsets shrink has them."""
    g = rng(65)
    room, n = 20000, sum(lens)
    q, k, v, dout = (rows(g, room, h, d) for h in (H, H_kv, H_kv, H))
    cu = int32([0] + [room * (i + 1) // len(lens) for i in range(len(lens))])
    out, grads = torch.zeros_like(q), [torch.zeros_like(x) for x in (q, k, v)]
    lse = torch.zeros(H, room, device="cuda")

    def call():
        fa.packed_attention(q, k, v, cu, causal=causal, out=out, lse=lse)
        fa.packed_attention_backward(q, k, v, out, lse, dout, cu, causal=causal, dq=grads[0], dk=grads[1], dv=grads[2])

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    cu.copy_(int32(R.offsets(lens)))
    for x in (out, lse, *grads):
        x.fill_(7.0)
    graph.replay()
    for x in (out, lse.T, *grads):
        assert (x[n:] == 7).all()
    small = [x[:n].contiguous() for x in (q, k, v, dout)]
    want, want_l = fa.packed_attention(*small[:3], int32(R.offsets(lens)), causal=causal)
    assert torch.equal(out[:n], want) and torch.equal(lse[:, :n], want_l)
    dq, dk, dv = fa.packed_attention_backward(*small[:3], want, want_l, small[3], int32(R.offsets(lens)), causal=causal)
    assert torch.equal(grads[1][:n], dk) and torch.equal(grads[2][:n], dv)
    assert torch.allclose(grads[0][:n].float(), dq.float(), rtol=2.0 ** -7, atol=1e-5)


def test_forward_sweep_of_more_than_a_second():
    """One query over 2^27 + 1 keys of score 0, whose values take turns in sign: the last one over their number, exactly
    (powers of two; of values of one sign the sum would stop at 2^26 of them, below its last bits)."""
    n = 2 ** 27 + 1
    k = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    row = (2.0 ** (torch.arange(64, device="cuda") % 3) * (1 - 2 * (torch.arange(64, device="cuda") % 2))).bfloat16()
    v = row.repeat(n, 1)[:, None]
    v[1::2] *= -1
    q = rows(rng(66), 3, 1, 64)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, lse = fa.packed_attention(q, k, v, int32([0, 1, 3]), int32([0, n, n]))
    end.record()
    assert fa.fa_device_status(None) == fa.FA_OK
    assert torch.equal(out[0, 0], row * 2.0 ** -27) and abs(lse[0, 0].item() - math.log(n)) <= 2.0 ** -21 * math.log(n)
    assert not out[1:].any() and (lse[0, 1:] == -math.inf).all()
    assert start.elapsed_time(end) > 1000  # a wait for the block lasted longer than the limit of the others


def test_backward_sweep_of_more_than_a_second():
    """Gradients of 80 million queries, all of them zeros with zero gradients but the last, over 100 keys."""
    n, keys = 80_000_001, 100
    x = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[-1] = rows(rng(67), 1, 64)
    k, v = rows(rng(68), keys, 1, 64), rows(rng(69), keys, 1, 64)
    lse = torch.full((1, n), math.log(keys), device="cuda")
    cu_q, cu_k = int32([0, n]), int32([0, keys])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    dq, dk, dv = fa.packed_attention_backward(x, k, v, x, lse, x, cu_q, cu_k)
    end.record()
    assert fa.fa_device_status(None) == fa.FA_OK
    last = x[-1:].clone()
    want = R.backward(last, k, v, last, lse[:, -1:], last, [0, 1], [0, keys], 1 / 8, False)
    for name, got in (("dq", dq[-1:]), ("dk", dk), ("dv", dv)):
        within(got, *want[name], name)
    assert not dq[:-1].any()
    assert start.elapsed_time(end) > 1000


@pytest.mark.parametrize("n", [2 ** 18, 2 ** 20, 2 ** 22])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_long_sums(n, dtype):
    """Sums of n terms of one sign: forward over n keys of like weight, dV of n queries of like weight.  One accumulation in
    fp32 that loses up to a step for every 16 terms (n 2^-27), beside the roundings of the weights and of the result."""
    g = rng(70)
    x = (torch.rand(n, 1, 64, generator=g, device="cuda") + 0.5).to(dtype)
    zero, q = torch.zeros_like(x), rows(g, 2, 1, 64).to(dtype)
    out, lse = fa.packed_attention(q, zero, x, int32([0, 2]), int32([0, n]))
    half = R.HALF[dtype]
    mean = x.double().mean(0)
    assert ((out.double() - mean).abs() <= (2 * half + R.sums(n)) * mean).all()
    assert ((lse.double() - math.log(n)).abs() <= R.sums(n) + 2.0 ** -22 * math.log(n)).all()
    # every query has the weight 1/4 for each of four keys
    k = torch.zeros(4, 1, 64, dtype=dtype, device="cuda")
    lse = torch.full((1, n), math.log(4.0), device="cuda")
    _, dk, dv = fa.packed_attention_backward(zero, k, k, zero, lse, x, int32([0, n]), int32([0, 4]))
    want = x.double().sum(0) / 4
    if dtype == torch.bfloat16:  # (fp16 ends at 65504)
        assert ((dv.double() - want).abs() <= (2 * half + 2.0 ** -20 + R.sums(n)) * want).all()
    assert not dk.any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [5, 70])
@pytest.mark.parametrize("causal", [False, True])
def test_gradients_do_not_depend_on_the_workspace(causal, B, d):
    """Whatever the workspace held, with empty sequences and rows of none; nothing behind it is written."""
    g = rng(62)
    lens = [(0, 130, 1, 257, 40)[i % 5] if B == 5 else i * i % 60 for i in range(B)]
    T = 19 + sum(lens) + 300
    q, k, v, dout = (rows(g, T, h, d) for h in (4, 2, 2, 4))
    cu = R.offsets(lens, 19)
    out, lse = torch.zeros_like(q), torch.zeros(4, T, device="cuda")
    fa.packed_attention(q, k, v, int32(cu), causal=causal, out=out, lse=lse)
    want = R.backward(q, k, v, out, lse, dout, cu, cu, 1 / math.sqrt(d), causal)
    need = fa.fa_packed_bwd_workspace_size(B, T, 4, d)
    first = None
    for fill in (0, 255):  # zeros, NaN
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        ws[need:] = 77
        grads = [torch.full_like(x, 7) for x in (q, k, v)]
        got = fa.packed_attention_backward(q, k, v, out, lse, dout, int32(cu), causal=causal, workspace=ws[:need],
                                           dq=grads[0], dk=grads[1], dv=grads[2])
        for name, x in zip(("dq", "dk", "dv"), got):
            within(x[19:cu[-1]], *(t[19:cu[-1]] for t in want[name]), name)
            assert (x[:19] == 7).all() and (x[cu[-1]:] == 7).all()
        assert (ws[need:] == 77).all()
        first = first or got
        assert torch.equal(got[1], first[1]) and torch.equal(got[2], first[2])
