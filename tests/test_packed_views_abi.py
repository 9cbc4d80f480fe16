"""Host-side checks (no GPU needed) of views that are slices of one tensor: which
layouts share no element and are taken, which do and are refused."""
import itertools

import pytest

from exact_tiled_attention_04_gb300 import binding as fab

pytest.importorskip("torch")

from .test_packed_paged_abi import A, ARG, OK, append, bwd, cache, fwd, lib, view  # noqa: E402,F401


def slices(layout, T, H, d=64, parts=3):
    """(row, head, part) strides in elements of parts of one tensor."""
    return {"T H parts d": (H * parts * d, parts * d, d), "H T parts d": (parts * d, T * parts * d, d),
            "T parts H d": (parts * H * d, d, H * d), "parts T H d": (H * d, d, T * H * d),
            "parts H T d": (d, T * d, H * T * d)}[layout]


LAYOUTS = ["T H parts d", "H T parts d", "T parts H d", "parts T H d", "parts H T d"]


@pytest.mark.parametrize("T,H", [(100, 4), (1, 4), (100, 1), (1, 1)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradients_into_slices(layout, T, H):
    row, head, part = slices(layout, T, H)
    views = [view(A[11] + 2 * i * part, H, row=row, head=head) for i in range(3)]
    kw = dict(T_q=T, T_k=T, H=H, H_kv=H)
    for dq, dk, dv in itertools.permutations(views):
        assert bwd(dq=dq, dk=dk, dv=dv, **kw) == OK
    assert bwd(dq=views[0], dk=views[1], dv=views[1], **kw) == ARG
    near = view(A[11] + 2 * (part - 8), H, row=row, head=head)  # eight elements of the part before
    assert bwd(dq=views[0], dk=near, dv=views[2], **kw) == ARG


def test_strides_that_do_not_agree():
    q = view(A[11], 4, row=768, head=192)
    kw = dict(T_q=100, T_k=100, H=4, H_kv=4)
    for row, head, status in ((768, 192, OK), (776, 192, ARG), (768, 184, ARG), (1536, 192, OK), (192, 192 * 100, OK),
                              (768, 128, ARG), (776, 194 * 4, ARG)):
        assert bwd(dq=q, dk=view(A[11] + 128, 4, row=row, head=head), dv=view(A[13], 4), **kw) == status, (row, head)


@pytest.mark.parametrize("T", [100, 1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_outputs_beside_inputs(layout, T):
    """An output in another part of the tensor that holds the inputs."""
    row, head, part = slices(layout, T, 4, parts=4)
    q, k, v, o = (view(A[1] + 2 * i * part, 4, row=row, head=head) for i in range(4))
    assert fwd(q=q, k=k, v=v, o=o, T_q=T, T_k=T, H_kv=4) == OK
    assert fwd(q=q, k=k, v=v, o=view(A[1] + 2 * (3 * part - 8), 4, row=row, head=head), T_q=T, T_k=T, H_kv=4) == ARG


@pytest.mark.parametrize("T", [30, 3])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_rotated_in_place(layout, T):
    row, head, part = slices(layout, T, 2)
    q, k, v = (view(A[10] + 2 * i * part, 2, row=row, head=head) for i in range(3))
    assert append(k=k, v=v, q=q, q_out=q, k_out=k, H=2, T=T) == OK
    assert append(k=k, v=v, q=q, q_out=q, k_out=v, H=2, T=T) == ARG
    assert append(k=k, v=v, q=q, q_out=k, k_out=k, H=2, T=T) == ARG


def test_views_that_are_taken_share_nothing():
    """Random pairs of views near each other: where the call is taken, no element is in both."""
    import random
    r = random.Random(7)
    taken = 0

    def elements(v, T, H):  # in eights
        return {(v.data + 2 * (t * v.row_stride + h * v.head_stride)) // 16 + i
                for t in range(T) for h in range(H) for i in range(8)}

    for _ in range(4000):
        T, H, H_kv = r.randint(1, 4), r.choice([2, 4]), r.choice([1, 2])
        step = 8 * r.randint(8, 40)
        far = step * r.randint(1, 9) if r.random() < 0.7 else 8 * r.randint(8, 200)
        row, head = (step, far) if r.random() < 0.5 else (far, step)
        row2, head2 = (row, head) if r.random() < 0.7 else (head, row)
        dk = view(A[11] + 1600 * 16, H_kv, row=row, head=head)
        dq = view(A[11] + 1600 * 16 + 16 * r.randint(-300, 300), H, row=row2, head=head2)
        if bwd(dq=dq, dk=dk, T_q=T, T_k=T, H=H, H_kv=H_kv) == OK:
            taken += 1
            assert not elements(dq, T, H) & elements(dk, T, H_kv), (T, H, H_kv, row, head, row2, head2, dq.data - dk.data)
    assert taken > 500


@pytest.mark.parametrize("B,T_q,H,d", [(1, 0, 1, 64), (3, 100, 4, 64), (8, 24000, 16, 128), (4000, 24000, 16, 128), (70, 127, 3, 64)])
def test_size_of_the_gradients_workspace(B, T_q, H, d):
    """What the header says it takes."""
    assert fab.fa_packed_bwd_workspace_size(B, T_q, H, d) == H * (T_q // 128 + B) * (512 * d + 1024) + 128
