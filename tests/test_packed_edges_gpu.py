"""Attention over packed sequences on the GPU: slices of one tensor in every
order of rows, heads and parts."""
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
