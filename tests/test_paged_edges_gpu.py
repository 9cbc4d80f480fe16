"""The paged cache on the GPU: scores of -inf, and how many kernels each call launches."""
import math

import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from .test_packed_gpu import int32, rng, rows, within  # noqa: E402
from .test_paged_gpu import cache_of, reference  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert fa.fa_device_status(None) == fa.FA_OK


@pytest.mark.parametrize("G,N_q", [(1, 1), (8, 1), (4, 4), (32, 1)])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
def test_first_keys_without_weight(G, N_q, d, dtype):
    """The first 128 keys' scores are -inf and the others' about -100: the result is attention over the others."""
    g = rng(61)
    lengths = [300, 1000, 30000]
    c, _ = cache_of(g, lengths, 2, d, 64, dtype, poison=False)
    q = torch.randn(3, 2 * G, N_q, d, generator=g, device="cuda").to(c.dtype)
    q[..., 0] = 8.0
    c.k_pages[..., 0] = -12.5 * math.sqrt(d)
    for b in range(3):
        c.k_pages[c.block_table[b, :2].long(), ..., 0] = -math.inf
    out, lse = fa.paged_attention(q, c)
    rest = fa.PagedKVCache(c.k_pages, c.v_pages, c.block_table[:, 2:].contiguous(), c.lengths - 128)
    want_o, want_l, tol_o, tol_l = reference(q, rest, [n - 128 for n in lengths], 1 / math.sqrt(d), False)
    within(lse, want_l, tol_l, "lse")
    within(out, want_o, tol_o, "out")


def test_runs_without_weight():
    """One long sequence whose keys' scores are -inf but for the last ten's: most of its runs leave nothing."""
    g = rng(62)
    c, _ = cache_of(g, [40000], 1, 64, 64, "f16", poison=False)
    q = torch.randn(1, 4, 1, 64, generator=g, device="cuda").half()
    q[..., 0] = 8.0
    page = int(c.block_table[0, 39999 // 64])  # slots 39936 .. 39999
    c.k_pages[..., 0] = -math.inf
    c.k_pages[page, 0, 54:, 0] = -100.0
    out, lse = fa.paged_attention(q, c)
    k, v = (torch.zeros(1, 1, 16, 64, device="cuda").half() for _ in range(2))
    k[0, 0, :10], v[0, 0, :10] = c.k_pages[page, 0, 54:], c.v_pages[page, 0, 54:]
    rest = fa.PagedKVCache(k, v, int32([[0]]), int32([10]))
    want_o, want_l, tol_o, tol_l = reference(q, rest, [10], 1 / 8, False)
    within(lse, want_l, tol_l, "lse")
    within(out, want_o, tol_o, "out")


def kernels(call):
    """Kernels that a call launches: nodes of the graph it is captured into."""
    import ctypes
    call()  # (what is set up once)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t()
    cuda = ctypes.CDLL("libcuda.so.1")
    assert cuda.cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


def test_kernels_of_each_call():
    g = rng(71)
    c, pages = cache_of(g, [15, 300, 7], 2, 64, 16, room=100, prefix=40, poison=False)
    table, apart = fa.rotary_table(1000, 64), torch.empty_like(c.lengths)

    def append(T, **kw):
        x = rows(g, T, 2, 64)
        q = rows(g, T, 8, 64)
        return kernels(lambda: fa.paged_append(c, x, x, q=q, table=table, **kw))

    assert append(3) == 1 and append(3, lengths_out=apart) == 1  # a row each
    assert append(3, cu=int32([0, 1, 2, 3])) == 2 and append(3, cu=int32([0, 1, 2, 3]), lengths_out=apart) == 1
    assert append(60) == 2 and append(60, lengths_out=apart) == 1
    assert append(0) == 2 and append(0, lengths_out=apart) == 1
    q = rows(g, 3, 4, 64).view(3, 4, 1, 64)
    assert kernels(lambda: fa.paged_attention(q, c)) == 2
    assert kernels(lambda: fa.paged_attention(q, c, prefix_pages=pages, prefix_length=40)) == 3
    x, cu = rows(g, 50, 2, 64), int32([0, 20, 50])
    out, lse = fa.packed_attention(x, x, x, cu)
    assert kernels(lambda: fa.packed_attention(x, x, x, cu)) == 1
    assert kernels(lambda: fa.packed_attention_backward(x, x, x, out, lse, x, cu)) == 3


def test_drafts_stored_then_attended():
    """Three drafted tokens of each sequence rotated and stored, the queries transposed, causal attention behind a prefix."""
    g = rng(72)
    B, N, H, H_kv, d, prefix = 3, 3, 8, 2, 64, 40
    held = [15, 300, 0]
    c, pages = cache_of(g, held, H_kv, d, 16, room=N, prefix=prefix, poison=False)
    q, k, v = (rows(g, B * N, h, d) for h in (H, H_kv, H_kv))
    got = fa.paged_append(c, k, v, q=q, table=fa.rotary_table(400, d), first_position=prefix)
    q4 = got.view(B, N, H, d).transpose(1, 2).contiguous()
    out, lse = fa.paged_attention(q4, c, causal=True, prefix_pages=pages, prefix_length=prefix)
    want_o, want_l, tol_o, tol_l = reference(q4, c, [n + N for n in held], 1 / 8, True, pages, prefix)
    within(lse, want_l, tol_l, "lse")
    within(out, want_o, tol_o, "out")
