"""Calls on a stream that is not the current one: what they allocate belongs to
that stream, and results may be freed behind work queued on the current one."""
import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


def calls_on_a_stream():
    """Each call that allocates, with `stream` as its argument; and the bytes of its workspace."""
    g = torch.Generator(device="cuda").manual_seed(40)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, k, v, dout = rows(1, 4, 700, 64), rows(1, 2, 700, 64), rows(1, 2, 700, 64), rows(1, 4, 700, 64)
    q1, kc, vc = rows(2, 8, 1, 128), rows(2, 2, 5000, 128), rows(2, 2, 5000, 128)
    o, lse = fa.attention(q, k, v, causal=True)
    return {"forward": (lambda s: fa.attention(q, k, v, causal=True, stream=s),
                        fa.fa_fwd_ex_workspace_size(1, 4, 700, 700, 64, 0)),
            "splits": (lambda s: fa.attention(q1, kc, vc, num_splits=20, stream=s),
                       fa.fa_fwd_ex_workspace_size(2, 8, 1, 5000, 128, 20)),
            "backward": (lambda s: fa.attention_backward(q, k, v, o, lse, dout, causal=True, stream=s),
                         fa.fa_bwd_workspace_size(1, 4, 700, 64))}


CALLS = pytest.mark.parametrize("name", ["forward", "splits", "backward"])


def close(got, want, name):
    """Bit for bit; the backward pass adds dQ's parts by atomics, in any order."""
    if name != "backward":
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
