"""Host-side checks of attention over packed sequences and of the paged cache (no
GPU needed): what each call refuses, with which status, before any CUDA call;
what the Python layer refuses; and the gradients of the tests' restatement
against differences."""
import ctypes
import math

import pytest

import exact_tiled_attention_04_gb300 as fa
from exact_tiled_attention_04_gb300 import binding as fab

torch = pytest.importorskip("torch")

from . import packed_ref as R  # noqa: E402

OK, ARG, UNS, ALI = fab.FA_OK, fab.FA_ERR_INVALID_ARG, fab.FA_ERR_UNSUPPORTED, fab.FA_ERR_ALIGNMENT
# fake, aligned, far apart device addresses: validation never dereferences
A = [i << 36 for i in range(1, 30)]
BF16, F16, F32 = fab.FA_DTYPE_BF16, fab.FA_DTYPE_F16, fab.FA_DTYPE_F32


@pytest.fixture(scope="module", autouse=True)
def lib():
    from exact_tiled_attention_04_gb300 import build
    build.build()
    return fab.load()


def view(at, heads, d=64, row=None, head=None):
    return fab.fa_rows_t(at, heads * d if row is None else row, d if head is None else head)


def fwd(q=None, k=None, v=None, o=None, lse=A[5], cu_q=A[6], cu_k=A[7], B=3, T_q=100, T_k=90, H=4, H_kv=2, d=64,
        scale=0.1, dtype=BF16, call=fab.fa_packed_fwd_validate, **extra):
    views = [w if w is not None else view(at, h, d) for w, at, h in ((q, A[1], H), (k, A[2], H_kv), (v, A[3], H_kv), (o, A[4], H))]
    return call(*(None if w == "NULL" else w for w in views), lse, cu_q, cu_k, B, T_q, T_k, H, H_kv, d, scale, dtype, **extra)


FORWARD = [
    ({}, OK), (dict(dtype=F16 | fab.FA_FLAG_CAUSAL, d=128), OK), (dict(lse=None), OK), (dict(cu_k=A[6]), OK),
    (dict(T_q=0, T_k=0), OK), (dict(T_q=0, q=view(None, 4), o=view(None, 4), lse=None), OK), (dict(H=1, H_kv=1, T_q=1, T_k=1), OK),
    (dict(q="NULL"), ARG), (dict(o="NULL"), ARG), (dict(q=view(None, 4)), ARG), (dict(v=view(None, 2)), ARG), (dict(cu_q=None), ARG),
    (dict(cu_k=None), ARG), (dict(B=0), ARG), (dict(T_q=-1), ARG), (dict(T_k=-1), ARG), (dict(H=0), ARG), (dict(H_kv=0), ARG),
    (dict(H=3), ARG), (dict(d=0), ARG), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG),
    (dict(dtype=BF16 | 0x200), ARG), (dict(dtype=F32), UNS), (dict(dtype=7), UNS), (dict(d=96), UNS), (dict(d=256), UNS),
    (dict(T_q=1 << 31), UNS), (dict(T_k=1 << 62), UNS), (dict(B=1 << 40), UNS), (dict(B=1 << 23), UNS), (dict(H=65536, H_kv=65536), UNS),
    (dict(H=60000, H_kv=1, T_q=1 << 29), UNS), (dict(q=view(A[1], 4, row=1 << 39)), UNS),
    (dict(q=view(A[1] + 8, 4)), ALI), (dict(o=view(A[4] + 2, 4)), ALI), (dict(k=view(A[2], 2, row=132)), ALI),
    (dict(v=view(A[3], 2, head=68)), ALI), (dict(cu_q=A[6] + 2), ALI), (dict(lse=A[5] + 1), ALI),
    # rows that overlap within a view, and strides that are not positive
    (dict(q=view(A[1], 4, row=128)), ARG), (dict(q=view(A[1], 4, head=32)), ARG), (dict(k=view(A[2], 2, row=0)), ARG),
    (dict(k=view(A[2], 2, head=0)), ARG), (dict(q=view(A[1], 4, row=-256)), ARG),
    # heads before rows, and slices of one tensor
    (dict(q=view(A[1], 4, row=64, head=6400)), OK), (dict(q=view(A[1], 4, row=64, head=6000)), ARG),
    (dict(q=view(A[1], 4, row=512), k=view(A[1] + 512, 2, row=512), v=view(A[1] + 768, 2, row=512)), OK),
    (dict(q=view(A[1], 4, row=512), o=view(A[1] + 512, 4, row=512)), OK),
    (dict(q=view(A[1], 4, row=512), o=view(A[1] + 496, 4, row=512)), ARG),
    (dict(q=view(A[1], 4, row=512), o=view(A[1] + 512, 4, row=520)), ARG),
    (dict(o=view(A[1], 4)), ARG), (dict(o=view(A[2], 4)), ARG), (dict(o=view(A[3] + 64, 4)), ARG),
    (dict(lse=A[4]), ARG), (dict(lse=A[1]), ARG), (dict(cu_q=A[4] + 512), ARG), (dict(cu_k=A[5]), ARG),
]


@pytest.mark.parametrize("kw,status", FORWARD)
def test_packed_forward_arguments(kw, status):
    assert fwd(**kw) == status
    if status != OK:  # the same from the launching entry point, before any CUDA call
        assert fwd(call=fab.fa_packed_fwd, stream=None, **kw) == status


def bwd(dout=None, dq=None, dk=None, dv=None, lse=A[5], ws=A[15], size=1 << 32, call=fab.fa_packed_bwd_validate, tail=(), **kw):
    def go(q, k, v, o, lse_, cu_q, cu_k, B, T_q, T_k, H, H_kv, d, scale, dtype):
        more = [w if w is not None else view(at, h, d) for w, at, h in ((dout, A[10], H), (dq, A[11], H), (dk, A[12], H_kv), (dv, A[13], H_kv))]
        more = [None if w == "NULL" else w for w in more]
        return call(q, k, v, o, more[0], lse_, *more[1:], cu_q, cu_k, B, T_q, T_k, H, H_kv, d, scale, dtype, ws, size, *tail)
    return fwd(call=go, lse=lse, **kw)


BACKWARD = [
    ({}, OK), (dict(dtype=F16 | fab.FA_FLAG_CAUSAL, d=128), OK), (dict(T_q=0, lse=None), OK),
    (dict(lse=None), ARG), (dict(dout="NULL"), ARG), (dict(dq="NULL"), ARG), (dict(dv=view(None, 2)), ARG), (dict(ws=None), ARG),
    (dict(ws=A[15] + 8), ALI), (dict(dq=view(A[11] + 8, 4)), ALI), (dict(size=1000), ARG), (dict(dtype=F32), UNS), (dict(d=96), UNS),
    (dict(dq=view(A[1], 4)), ARG), (dict(dk=view(A[10], 2)), ARG), (dict(dv=view(A[12], 2)), ARG), (dict(dq=view(A[5], 4)), ARG),
    (dict(dq=view(A[11], 4, row=512), dk=view(A[11] + 512, 2, row=512), dv=view(A[11] + 768, 2, row=512)), OK),
    (dict(dq=view(A[11], 4, row=512), dk=view(A[11] + 384, 2, row=512)), ARG),
    (dict(ws=A[1]), ARG), (dict(ws=A[13]), ARG), (dict(ws=A[6]), ARG), (dict(lse=A[15] + 4096), ARG),
]


@pytest.mark.parametrize("kw,status", BACKWARD)
def test_packed_backward_arguments(kw, status):
    assert bwd(**kw) == status
    if status != OK:
        assert bwd(call=fab.fa_packed_bwd, tail=(None,), **kw) == status


def test_packed_backward_workspace():
    need = fab.fa_packed_bwd_workspace_size(3, 100, 4, 64)
    assert bwd(size=need) == OK and bwd(size=need - 1) == ARG
    # rows in whole blocks of 128 a sequence: an fp32 row of dQ and two statistics each
    assert need >= 4 * (100 // 128 + 3) * 128 * (64 * 4 + 8)
    for bad in ((0, 100, 4, 64), (3, -1, 4, 64), (3, 100, 0, 64), (3, 100, 4, 96), (3, 1 << 40, 4, 64)):
        assert fab.fa_packed_bwd_workspace_size(*bad) == 0


def cache(**kw):
    f = dict(k_pages=A[1], v_pages=A[2], block_table=A[3], lengths=A[4], num_pages=50, page_size=16, B=3, max_pages=7, H_kv=2, d=64)
    f.update(kw)
    return ctypes.pointer(fab.fa_paged_cache_t(**f))


def append(c=None, k=None, v=None, cu=A[9], T=30, q=None, q_out=None, H=4, k_out=None, table=A[14], rows=100, rot=64,
           positions=A[15], first=0, out=A[4], dtype=BF16, d=64, call=fab.fa_paged_append_validate, tail=()):
    views = [w if w is not None else view(at, h, d) for w, at, h in ((k, A[10], 2), (v, A[11], 2), (q, A[12], H), (q_out, A[13], H))]
    k, v, q, q_out = (None if w == "NULL" else w for w in views)
    return call(c or cache(d=d), k, v, cu, T, q, q_out, H, k_out, table, rows, rot, positions, first, out, dtype, *tail)


def attend(c=None, q=A[10], o=A[11], lse=A[12], H=8, N_q=2, pages=A[13], prefix=100, scale=0.1, dtype=BF16, ws=A[14], size=1 << 34):
    return fab.fa_paged_fwd_validate(c or cache(), q, o, lse, H, N_q, pages, prefix, scale, dtype, ws, size)


CACHE = [
    (dict(k_pages=None), ARG), (dict(v_pages=None), ARG), (dict(block_table=None), ARG), (dict(lengths=None), ARG), (dict(num_pages=0), ARG),
    (dict(page_size=0), ARG), (dict(B=0), ARG), (dict(max_pages=0), ARG), (dict(H_kv=-1), ARG), (dict(d=0), ARG), (dict(d=96), UNS),
    (dict(page_size=24), UNS), (dict(page_size=256), UNS), (dict(num_pages=1 << 31), UNS), (dict(max_pages=1 << 28), UNS),
    (dict(num_pages=1 << 60), ARG), (dict(B=1 << 30), UNS), (dict(k_pages=A[1] + 8), ALI), (dict(lengths=A[4] + 2), ALI),
    (dict(v_pages=A[1] + 64), ARG), (dict(lengths=A[3] + 4), ARG), (dict(block_table=A[2]), ARG),
]


@pytest.mark.parametrize("kw,status", CACHE)
def test_every_call_checks_the_cache(kw, status):
    c = cache(**kw)
    assert append(c) == status and attend(c) == status
    assert append(c, call=fab.fa_paged_append, tail=(None,)) == status
    assert fab.fa_paged_fwd(c, A[10], A[11], A[12], 8, 2, None, 0, 0.1, BF16, A[14], 1 << 34, None) == status


def test_null_cache():
    assert fab.fa_paged_append_validate(None, view(A[10], 2), view(A[11], 2), None, 3, None, None, 0, None, None, 0, 0, None, 0,
                                        A[4], BF16) == ARG
    assert fab.fa_paged_fwd_validate(None, A[10], A[11], None, 8, 1, None, 0, 0.1, BF16, A[14], 1 << 34) == ARG


APPEND = [
    ({}, OK), (dict(cu=None), OK), (dict(q="NULL", q_out="NULL"), OK), (dict(table=None, positions=None), OK), (dict(positions=None), OK),
    (dict(T=0), OK), (dict(out=A[16]), OK), (dict(k_out=view(A[16], 2)), OK), (dict(dtype=F16 | fab.FA_FLAG_INTERLEAVED), OK),
    (dict(rot=16), OK), (dict(q_out=view(A[12], 4)), OK), (dict(k_out=view(A[10], 2)), OK), (dict(first=-5), OK),
    (dict(k="NULL"), ARG), (dict(v="NULL"), ARG), (dict(q="NULL"), ARG), (dict(q_out="NULL"), ARG), (dict(out=None), ARG), (dict(T=-1), ARG),
    (dict(cu=None, T=31), ARG), (dict(H=0), ARG), (dict(rows=0), ARG), (dict(rot=8), ARG), (dict(rot=72), ARG), (dict(rot=80), ARG),
    (dict(table=None), ARG), (dict(first=1 << 41), ARG), (dict(dtype=BF16 | fab.FA_FLAG_CAUSAL), ARG), (dict(dtype=F32), UNS),
    (dict(T=1 << 31), UNS), (dict(table=A[14] + 4), ALI), (dict(cu=A[9] + 1), ALI), (dict(out=A[16] + 2), ALI), (dict(k=view(A[10] + 8, 2)), ALI),
    (dict(q=view(A[12], 4, row=260)), ALI),
    # what is written meets nothing else
    (dict(k=view(A[1] + 1024, 2)), ARG), (dict(q_out=view(A[2], 4)), ARG), (dict(q_out=view(A[10], 4)), ARG),
    (dict(q_out=view(A[12] + 128, 4)), ARG), (dict(k_out=view(A[11], 2)), ARG), (dict(k_out=view(A[13], 2)), ARG), (dict(out=A[3]), ARG),
    (dict(out=A[4] + 4), ARG), (dict(out=A[10]), ARG), (dict(out=A[15]), ARG), (dict(table=A[1]), ARG), (dict(q_out=view(A[14], 4)), ARG),
    (dict(positions=A[2]), ARG),
]


@pytest.mark.parametrize("kw,status", APPEND)
def test_append_arguments(kw, status):
    assert append(**kw) == status
    if status != OK:
        assert append(call=fab.fa_paged_append, tail=(None,), **kw) == status


ATTEND = [
    ({}, OK), (dict(prefix=0, pages=None), OK), (dict(lse=None), OK), (dict(dtype=F16 | fab.FA_FLAG_CAUSAL), OK), (dict(H=2, N_q=128), OK),
    (dict(q=None), ARG), (dict(o=None), ARG), (dict(ws=None), ARG), (dict(H=0), ARG), (dict(H=7), ARG), (dict(N_q=0), ARG), (dict(prefix=-1), ARG),
    (dict(prefix=0), ARG), (dict(pages=None), ARG), (dict(scale=math.nan), ARG), (dict(dtype=BF16 | 0x200), ARG), (dict(dtype=F32), UNS),
    (dict(N_q=33), UNS), (dict(H=258), UNS), (dict(prefix=1 << 31), UNS), (dict(q=A[10] + 8), ALI), (dict(ws=A[14] + 8), ALI),
    (dict(lse=A[12] + 2), ALI), (dict(pages=A[13] + 1), ALI), (dict(size=100), ARG), (dict(o=A[10]), ARG), (dict(lse=A[11]), ARG),
    (dict(ws=A[10]), ARG), (dict(o=A[1]), ARG), (dict(ws=A[3]), ARG), (dict(o=A[13]), ARG), (dict(lse=A[4]), ARG),
]


@pytest.mark.parametrize("kw,status", ATTEND)
def test_attention_arguments(kw, status):
    assert attend(**kw) == status


def test_attention_workspace():
    need = fab.fa_paged_fwd_workspace_size(3, 8, 2, 2, 112, 64, 100)
    assert need > fab.fa_paged_fwd_workspace_size(3, 8, 2, 2, 112, 64, 0) > 0
    assert attend(size=need) == OK and attend(size=need - 1) == ARG
    for bad in ((0, 8, 2, 2, 112, 64, 0), (3, 7, 2, 2, 112, 64, 0), (3, 8, 2, 33, 112, 64, 0), (3, 8, 2, 2, 112, 96, 0),
                (3, 8, 2, 2, 112, 64, -1), (1 << 22, 4096, 4096, 1, 1 << 20, 64, 0)):
        assert fab.fa_paged_fwd_workspace_size(*bad) == 0


def test_new_status_has_a_name():
    assert "range" in fab.fa_status_string(fab.FA_ERR_RANGE)


def test_python_refusals():
    """What the Python layer refuses ahead of the C call, on the CPU."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for bad in (lambda: fa.packed_attention(q, q, q, cu), lambda: fa.packed_attention(q[0], q, q, cu),
                lambda: fa.packed_attention_backward(q, q, q, q, q, q, cu),
                lambda: fa.PagedKVCache(torch.zeros(2, 1, 16, 64).bfloat16(), torch.zeros(2, 1, 16, 64).bfloat16(),
                                        torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)),
                lambda: fa.PagedKVCache(q, q, cu, cu), lambda: fa.rotary_table(0, 64, device="cpu"),
                lambda: fa.rotary_table(4, 24, device="cpu")):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_rotary_table():
    """Angles of far positions are formed in 64 bits."""
    t = fa.rotary_table(100001, 32, base=10000.0, device="cpu")
    assert t.shape == (100001, 32) and t.dtype == torch.float32
    for p, j in ((0, 3), (1, 0), (99999, 1), (100000, 15)):
        angle = p * 10000.0 ** (-2 * j / 32)
        assert abs(t[p, j].item() - math.cos(angle)) <= 2.0 ** -24 and abs(t[p, 16 + j].item() - math.sin(angle)) <= 2.0 ** -24


@pytest.mark.parametrize("causal", [False, True])
def test_restatements_gradients_against_differences(causal):
    """Central differences of sum(out * dout) in every coordinate (64 bits)."""
    g = torch.Generator().manual_seed(1)
    lens, lens_k, H, H_kv, d, scale = [3, 0, 4], [5, 2, 3], 4, 2, 8, 0.4
    cu_q, cu_k = R.offsets(lens), R.offsets(lens_k)
    q, k, v = (torch.randn(sum(n), h, d, generator=g, dtype=torch.float64) for n, h in ((lens, H), (lens_k, H_kv), (lens_k, H_kv)))
    dout = torch.randn(q.shape, generator=g, dtype=torch.float64)
    R.HALF[torch.float64], R.TINY[torch.float64] = 0.0, 0.0
    try:
        def loss(q, k, v):
            return (R.forward(q, k, v, cu_q, cu_k, scale, causal)[0] * dout).sum()

        out, lse, _, _ = R.forward(q, k, v, cu_q, cu_k, scale, causal)
        got = R.backward(q, k, v, out, lse, dout, cu_q, cu_k, scale, causal)
        for name, x in (("dq", q), ("dk", k), ("dv", v)):
            grad = torch.zeros_like(x)
            for i in range(x.numel()):
                at = x.view(-1)[i].item()
                x.view(-1)[i] = at + 1e-6
                up = loss(q, k, v)
                x.view(-1)[i] = at - 1e-6
                grad.view(-1)[i] = (up - loss(q, k, v)) / 2e-6
                x.view(-1)[i] = at
            assert (grad - got[name][0]).abs().max() <= 1e-8 * max(1.0, grad.abs().max()), name
    finally:
        del R.HALF[torch.float64], R.TINY[torch.float64]
