"""Calls of the packed and the paged attention on a stream that is not the
current one: what they allocate belongs to that stream, and results may be freed
behind work queued on the current one."""
import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_packed_gpu import batch, int32, rng, rows  # noqa: E402
from .test_paged_gpu import cache_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


def calls_on_a_stream():
    """Each call that allocates, with `stream` as its argument; and the bytes of its workspace."""
    q, k, v, cu, _ = batch(50, [300, 41, 512], 4, 2, 64, "bf16")
    cu = int32(cu)
    o, lse = fa.packed_attention(q, k, v, cu, causal=True)
    g = rng(51)
    c, pages = cache_of(g, [5000, 300], 2, 128, 64, prefix=900, room=4, poison=False)
    q1 = torch.randn(2, 8, 1, 128, generator=g, device="cuda").bfloat16()
    k1, v1, lengths = rows(g, 2, 2, 128), rows(g, 2, 2, 128), torch.empty_like(c.lengths)
    table = fa.rotary_table(6000, 128)
    return {"packed": (lambda s: fa.packed_attention(q, k, v, cu, causal=True, stream=s), 16),
            "gradients": (lambda s: fa.packed_attention_backward(q, k, v, o, lse, o, cu, causal=True, stream=s),
                          fa.fa_packed_bwd_workspace_size(3, 853, 4, 64)),
            "paged": (lambda s: fa.paged_attention(q1, c, prefix_pages=pages, prefix_length=900, stream=s),
                      c.workspace_size(8, 1, 900)),
            "append": (lambda s: (fa.paged_append(c, k1, v1, q=q1.view(2, 8, 128), table=table, lengths_out=lengths, stream=s),), 16)}


CALLS = pytest.mark.parametrize("name", ["packed", "gradients", "paged", "append"])


def close(got, want, name):
    """Bit for bit; dQ's parts are added in any order."""
    if name != "gradients":
        return all(torch.equal(a, b) for a, b in zip(got, want))
    # fp32 sums in another order, rounded to bf16: an ulp (2^-7 relatively) of a value, and 2^-20 of the largest
    return all(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -20 * b.float().abs().max()).all()
               for a, b in zip(got, want))


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
    assert close(got, want, name)
    torch.cuda.synchronize()
    assert close(got, want, name)


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
    assert close(copies, want, name)
