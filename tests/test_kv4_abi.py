"""Host-side checks of the 4-bit cache's entry points (no GPU needed): what
each call refuses, with which status, before any CUDA call; and of the Python
handle."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import exact_tiled_attention_04_gb300 as fa
from exact_tiled_attention_04_gb300 import binding as fab

from . import kv4_ref as R

# fake, aligned, far apart device addresses: validation never dereferences
A = [i << 36 for i in range(1, 24)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from exact_tiled_attention_04_gb300 import build
    build.build()
    return fab.load()


def cache(base=0, **kw):
    f = dict(k_codes=A[base], k_scales=A[base + 1], v_codes=A[base + 2], v_scales=A[base + 3], weight=A[base + 4],
             pos=A[base + 5], counts=A[base + 6], B=2, H_kv=2, capacity=256, d=128)
    f.update(kw)
    return ctypes.pointer(fab.fa_kv4_cache_t(**f))


CACHE_FAULTS = [
    (dict(k_codes=None), fab.FA_ERR_INVALID_ARG), (dict(k_scales=None), fab.FA_ERR_INVALID_ARG),
    (dict(v_codes=None), fab.FA_ERR_INVALID_ARG), (dict(v_scales=None), fab.FA_ERR_INVALID_ARG),
    (dict(counts=None), fab.FA_ERR_INVALID_ARG), (dict(B=0), fab.FA_ERR_INVALID_ARG),
    (dict(H_kv=-1), fab.FA_ERR_INVALID_ARG), (dict(capacity=0), fab.FA_ERR_INVALID_ARG),
    (dict(capacity=200), fab.FA_ERR_INVALID_ARG), (dict(d=0), fab.FA_ERR_INVALID_ARG),
    (dict(d=96), fab.FA_ERR_UNSUPPORTED), (dict(capacity=1 << 31), fab.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 40, H_kv=1 << 40), fab.FA_ERR_INVALID_ARG), (dict(k_codes=A[0] + 8), fab.FA_ERR_ALIGNMENT),
    (dict(v_scales=A[3] + 4), fab.FA_ERR_ALIGNMENT), (dict(pos=A[5] + 2), fab.FA_ERR_ALIGNMENT),
    (dict(v_codes=A[0] + 64), fab.FA_ERR_INVALID_ARG), (dict(weight=A[5]), fab.FA_ERR_INVALID_ARG),
]


def append(c, k=A[10], v=A[11], n=3, dtype=fab.FA_DTYPE_BF16, out=A[6]):
    return fab.fa_kv4_append_validate(c, k, v, n, dtype, out)


def read(c, first=A[12], count=3, k=A[10], v=A[11], dtype=fab.FA_DTYPE_F16):
    return fab.fa_kv4_read_validate(c, first, count, k, v, dtype)


def fwd(c, q=A[10], o=A[11], lse=A[12], w=A[13], H=8, Nq=2, scale=0.1, dtype=fab.FA_DTYPE_BF16, ws=A[14], size=1 << 34):
    return fab.fa_kv4_fwd_validate(c, q, o, lse, w, H, Nq, scale, dtype, ws, size)


def evict(c, keep=100, sinks=0, recent=0, rank=None, to=None, src=A[20], out=A[6]):
    return fab.fa_kv4_evict_validate(c, keep, sinks, recent, rank, to, src, out)


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_every_call_checks_the_cache(kw, status):
    c = cache(**kw)
    for call in (append, read, fwd, evict):
        assert call(c) == status
    assert append(None) == fab.FA_ERR_INVALID_ARG and fwd(None) == fab.FA_ERR_INVALID_ARG
    # the same before any CUDA call from the launching entry point
    assert fab.fa_kv4_append(c, A[10], A[11], 3, fab.FA_DTYPE_BF16, A[6], None) == status
    assert fab.fa_kv4_evict(cache(7), 100, 0, 0, None, c, A[20], A[21], None) == status


def test_append_arguments():
    c = cache()
    assert append(c) == fab.FA_OK and append(c, out=A[12]) == fab.FA_OK
    assert append(cache(weight=None, pos=None)) == fab.FA_OK
    for kw, st in ((dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(n=0), 1), (dict(n=-5), 1),
                   (dict(dtype=fab.FA_DTYPE_F32), 2), (dict(dtype=fab.FA_DTYPE_BF16 | fab.FA_FLAG_CAUSAL), 1),
                   (dict(dtype=9), 2), (dict(dtype=-1), 1), (dict(k=A[10] + 2), 3), (dict(out=A[12] + 1), 3),
                   (dict(k=A[0]), 1), (dict(v=A[6]), 1), (dict(out=A[6] + 4), 1), (dict(out=A[10] + 16), 1),
                   (dict(n=1 << 31), 2), (dict(n=1 << 60), 1)):
        assert append(c, **kw) == st, kw
    assert append(c, k=A[10], v=A[10]) == fab.FA_OK  # inputs may alias


def test_read_arguments():
    c = cache()
    assert read(c) == fab.FA_OK and read(c, first=None) == fab.FA_OK
    assert read(c, k=None) == fab.FA_OK and read(c, v=None) == fab.FA_OK
    for kw, st in ((dict(k=None, v=None), 1), (dict(count=0), 1), (dict(dtype=fab.FA_DTYPE_F32), 2),
                   (dict(k=A[10] + 8), 3), (dict(first=A[12] + 2), 3), (dict(v=A[10]), 1), (dict(v=A[2] + 32), 1),
                   (dict(first=A[10] + 16), 1), (dict(count=1 << 31), 2)):
        assert read(c, **kw) == st, kw


def test_attention_arguments():
    c = cache()
    assert fwd(c) == fab.FA_OK and fwd(c, lse=None, w=None) == fab.FA_OK
    assert fwd(c, w=A[4]) == fab.FA_OK  # adds in place
    assert fwd(c, H=2, Nq=128) == fab.FA_OK and fwd(c, dtype=fab.FA_DTYPE_F16 | fab.FA_FLAG_CAUSAL) == fab.FA_OK
    for kw, st in ((dict(q=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(H=0), 1), (dict(H=3), 1),
                   (dict(Nq=0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
                   (dict(dtype=fab.FA_DTYPE_F32), 2), (dict(dtype=0x201), 1), (dict(H=2, Nq=129), 2),
                   (dict(H=260, Nq=1), 2), (dict(H=64, Nq=5), 2), (dict(q=A[10] + 8), 3), (dict(o=A[11] + 4), 3),
                   (dict(ws=A[14] + 8), 3), (dict(lse=A[12] + 1), 3), (dict(size=100), 1), (dict(o=A[10]), 1),
                   (dict(o=A[0]), 1), (dict(lse=A[11] + 64), 1), (dict(w=A[5]), 1), (dict(w=A[4] + 4), 1),
                   (dict(ws=A[10]), 1), (dict(ws=A[2]), 1), (dict(ws=A[13]), 1)):
        assert fwd(c, **kw) == st, kw
    need = fab.fa_kv4_fwd_workspace_size(2, 8, 2, 2, 256, 128, 1)
    assert need > 0 and fwd(c, size=need) == fab.FA_OK and fwd(c, size=need - 1) == fab.FA_ERR_INVALID_ARG
    bare = fab.fa_kv4_fwd_workspace_size(2, 8, 2, 2, 256, 128, 0)
    assert need == bare + 2 * 2 * 256 * 8 * 4  # the scores
    for bad in ((0, 8, 2, 2, 256, 128), (2, 7, 2, 2, 256, 128), (2, 8, 2, 40, 256, 128), (2, 8, 2, 2, 250, 128),
                (2, 8, 2, 2, 256, 80), (1 << 40, 8, 2, 2, 1 << 30, 128)):
        assert fab.fa_kv4_fwd_workspace_size(*bad, 1) == 0


def test_evict_arguments():
    c, to = cache(), cache(7, capacity=128)
    assert evict(c) == fab.FA_OK and evict(c, sinks=4, recent=9) == fab.FA_OK and evict(c, keep=1000) == fab.FA_OK
    assert evict(c, rank=A[4]) == fab.FA_OK and evict(c, rank=A[18]) == fab.FA_OK
    assert evict(c, to=to) == fab.FA_OK and evict(c, to=to, out=A[13]) == fab.FA_OK
    bare = cache(weight=None, pos=None)
    assert evict(bare, rank=A[18]) == fab.FA_OK
    assert evict(bare) == fab.FA_ERR_INVALID_ARG                        # nothing to rank by
    assert evict(bare, rank=A[18], sinks=1) == fab.FA_ERR_INVALID_ARG   # no positions
    assert evict(bare, rank=A[18], recent=1) == fab.FA_ERR_INVALID_ARG
    for kw, st in ((dict(keep=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1), (dict(src=None), 1),
                   (dict(out=None), 1), (dict(src=A[20] + 2), 3), (dict(rank=A[18] + 1), 3), (dict(src=A[0]), 1),
                   (dict(src=A[4]), 1), (dict(rank=A[5]), 1), (dict(rank=A[4] + 4), 1), (dict(out=A[6] + 4), 1),
                   (dict(rank=A[18], src=A[18] + 16), 1), (dict(keep=200, to=to), 1), (dict(to=c), 1),
                   (dict(to=cache(7, d=64)), 1), (dict(to=cache(7, B=1)), 1), (dict(to=cache(7, pos=A[5])), 1),
                   (dict(to=cache(7, weight=A[18]), rank=A[18]), 1), (dict(to=cache(7, pos=A[20])), 1),
                   (dict(to=to, out=A[8]), 1), (dict(keep=1 << 31), 2)):
        assert evict(c, **kw) == st, kw
    assert evict(cache(capacity=393216)) == fab.FA_OK
    assert evict(cache(capacity=393216 + 128)) == fab.FA_ERR_UNSUPPORTED


def weights(q=A[0], k=A[1], lse=A[2], w_in=A[3], w=A[4], stride=400, B=2, H=4, H_kv=2, Nq=300, Nkv=400, d=64, first=0,
            scale=0.1, dtype=fab.FA_DTYPE_BF16):
    return fab.fa_fwd_weights_validate(q, k, lse, w_in, w, stride, B, H, H_kv, Nq, Nkv, d, first, scale, dtype)


def test_prompt_weights_arguments():
    assert weights() == fab.FA_OK and weights(w_in=None) == fab.FA_OK and weights(w_in=A[4]) == fab.FA_OK
    assert weights(stride=1000, dtype=fab.FA_DTYPE_F16 | fab.FA_FLAG_CAUSAL, d=128, first=299) == fab.FA_OK
    for kw, st in ((dict(q=None), 1), (dict(k=None), 1), (dict(lse=None), 1), (dict(w=None), 1), (dict(B=0), 1),
                   (dict(H=3), 1), (dict(Nq=0), 1), (dict(Nkv=0), 1), (dict(first=-1), 1), (dict(first=300), 1),
                   (dict(stride=399), 1), (dict(scale=math.nan), 1), (dict(dtype=fab.FA_DTYPE_F32), 2),
                   (dict(d=96), 2), (dict(dtype=0x801), 1), (dict(q=A[0] + 4), 3), (dict(w=A[4] + 2), 3),
                   (dict(w=A[0] + 64), 1), (dict(w=A[2]), 1), (dict(w_in=A[4] + 4), 1),
                   (dict(Nq=(1 << 31) - 1), 2), (dict(B=1 << 40, H=1 << 30), 1)):
        assert weights(**kw) == st, kw


def run_host(tmp_path, source):
    """Compile a C++ program against the library's internal headers, its CUDA calls the program's own; run it."""
    from exact_tiled_attention_04_gb300 import build
    (tmp_path / "t.cpp").write_text(source)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, "-I", build.INCLUDE, "-isystem", cuda,
                    "-o", str(tmp_path / "t"), str(tmp_path / "t.cpp")], check=True)
    subprocess.run([str(tmp_path / "t")], check=True)


def test_shared_memory_limit_is_set_once_per_context(tmp_path):
    """A device reset loses a kernel's limit: the next context gets it again, a failed call is not remembered."""
    run_host(tmp_path, r"""
#include "fa_kv4.h"
static int device = 0, calls = 0, limit = 0;
static unsigned long long context = 7;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) { ++calls; limit = v; return answer; }
unsigned long long fa::host::current_context_id() { return context; }
int main() {
    static fa::SmemAllowed done;
    int kernel = 0;
    auto allow = [&] { return fa::allow_smem(&kernel, 100000, done); };
    answer = cudaErrorInvalidValue;
    if (allow() != cudaErrorInvalidValue || calls != 1) return 1;
    answer = cudaSuccess;
    if (allow() != cudaSuccess || calls != 2 || limit != 100000) return 2;
    if (allow() != cudaSuccess || calls != 2) return 3;
    device = 1, context = 8;  // another device has a context of its own
    if (allow() != cudaSuccess || calls != 3) return 4;
    device = 0, context = 9;  // the first device was reset
    if (allow() != cudaSuccess || calls != 4 || allow() != cudaSuccess || calls != 4) return 5;
    context = 0;  // none current
    if (allow() != cudaSuccess || calls != 5) return 6;
    device = 1000, context = 10;  // past the remembered devices
    if (allow() != cudaSuccess || allow() != cudaSuccess || calls != 7) return 7;
    return 0;
}
""")


def test_blocks_of_the_copy_into_another_cache(tmp_path):
    """As many as hold the entries that can be kept, up to the largest `keep`."""
    run_host(tmp_path, r"""
#include "fa_kv4.h"
int main() {
    const int64_t capacities[] = {128, 256, 384, 40960, 393216}, keeps[] = {1, 255, 256, 257, 100000, 393216,
        (int64_t{1} << 31) - 300, (int64_t{1} << 31) - 256, (int64_t{1} << 31) - 255, (int64_t{1} << 31) - 1};
    for (int64_t c : capacities)
        for (int64_t k : keeps) {
            const int64_t n = k < c ? k : c, blocks = fa::kv4_copy_blocks(k, c);
            if (fa::kv4_kept_at_most(k, c) != n || blocks * 256 < n || (blocks - 1) * 256 >= n) return 1;
        }
    return 0;
}
""")


def test_handle_checks_its_tensors():
    torch = pytest.importorskip("torch")
    u8 = dict(dtype=torch.uint8)
    good = dict(k_codes=torch.zeros(1, 2, 128, 64, **u8), k_scales=torch.zeros(1, 2, 128, 8, **u8),
                v_codes=torch.zeros(1, 2, 128, 64, **u8), v_scales=torch.zeros(1, 2, 128, 8, **u8),
                counts=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.KV4Cache(**good)
    with pytest.raises(ValueError, match="multiple of 128"):
        fa.KV4Cache(**{**good, "k_codes": torch.zeros(1, 2, 100, 64, **u8)})
    with pytest.raises(ValueError, match="64 or 128"):
        fa.KV4Cache(**{**good, "k_codes": torch.zeros(1, 2, 128, 48, **u8)})
    with pytest.raises(ValueError, match="k_codes"):
        fa.KV4Cache(**{**good, "k_codes": torch.zeros(2, 128, 64, **u8)})
    with pytest.raises(TypeError, match="k_codes"):
        fa.KV4Cache(**{**good, "k_codes": torch.zeros(1, 2, 128, 64)})
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.attention_weights(torch.zeros(1, 1, 1, 64).half(), torch.zeros(1, 1, 1, 64).half(), torch.zeros(1, 1, 1))


def test_the_restatement_itself():
    """The reference's grids are the formats', its selection the documented order."""
    assert len(R.E4M3) == 127 and R.E4M3[-1] == 448 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[8] == 2.0 ** -6
    x = np.zeros((1, 16))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    assert R.stored(x)[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4]
    assert np.isnan(R.stored(np.full((1, 16), np.inf))).all() and (R.stored(np.full((1, 16), 1e-9)) == 0).all()
    w = np.array([1.0, np.nan, np.inf, 0.0, 5.0])
    assert R.select(w, None, 5, 5, 2, 0, 0) == [2, 1]
    assert R.select(w, np.arange(5), 5, 5, 2, 2, 1) == [0, 1]
    assert R.select(w, np.arange(5), 5, 5, 9, 0, 0) == [0, 1, 2, 3, 4]
    assert R.select(np.zeros(4), None, 4, 4, 2, 0, 0) == [0, 1]
    assert R.select(np.array([0.0, 1, 0, 2]), None, 4, 4, 2, 0, 0) == [3, 1]
