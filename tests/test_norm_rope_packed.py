"""Norms and rotation of rows that belong to no sequence or lie past the table: what they hold in
outputs that the call makes."""
import contextlib

import pytest
import torch

from tests.test_paged_edges import ints

gpu = pytest.mark.gpu


def fa_():
    import exact_io_aware_22_gb300 as fa
    return fa


def ok(status=0):
    torch.cuda.synchronize()
    assert fa_().device_status() == status


@contextlib.contextmanager
def nan_in_new_tensors():
    """torch.empty gives NaN: an element that a call does not write shows."""
    was = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    try:
        assert torch.empty(8, device="cuda").isnan().all()
        yield
    finally:
        torch.use_deterministic_algorithms(was[0])
        torch.utils.deterministic.fill_uninitialized_memory = was[1]


# ------------------------------------------------------------------ rows that are left out
@gpu
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("d,T", [(128, 140), (32, 3000)])
def test_rows_left_out_are_zero_in_outputs_that_the_call_makes(norm, d, T):
    """The projection's gradient sums over all rows, those behind the last sequence too: what stands
    there has to be zero, and NaN among the inputs of such rows must not matter."""
    fa, H, Hkv = fa_(), 6, 2
    offsets = [3, 50, 50, T - 9]
    x, dy = (torch.randn(T, H + Hkv, d, device="cuda").bfloat16() for _ in range(2))
    for a in (x, dy):
        a[:3] = float("nan")
        a[T - 9:] = float("inf")
    cs = fa.rope_table(T, d)
    args = dict(cos_sin=cs, cu_seqlens=ints(offsets))
    if norm:
        w = torch.rand(2, d, device="cuda") + 0.5
        args.update(q_weight=w[0], k_weight=w[1], eps=1e-6)
    with nan_in_new_tensors():
        y = fa.norm_rope(x[:, :H], x[:, H:], **args)
        r = fa.norm_rope_bwd(dy[:, :H], dy[:, H:], x[:, :H], x[:, H:], **args)
        one = fa.norm_rope_bwd(dy[:, :H], None, x[:, :H], None, **{k: v for k, v in args.items() if k != "k_weight"})
    ok()
    inside = slice(3, T - 9)
    for a in (*y, r[0], r[1], one[0]):
        assert (a[:3] == 0).all() and (a[T - 9:] == 0).all()
        assert a[inside].isfinite().all() and (a[inside] != 0).any(-1).all()
    assert torch.equal(one[0], r[0]) and one[1] is None
    if norm:
        assert r[2].isfinite().all() and r[3].isfinite().all()
    # the same from outputs that are given, which keep such rows; one of the two given
    full = torch.full((T, H, d), 5.0, device="cuda", dtype=torch.bfloat16)
    with nan_in_new_tensors():
        dq, dk, _, _ = fa.norm_rope_bwd(dy[:, :H], dy[:, H:], x[:, :H], x[:, H:], dq=full, **args)
    ok()
    assert dq is full and (full[:3] == 5).all() and (full[T - 9:] == 5).all()
    assert torch.equal(full[inside], r[0][inside]) and torch.equal(dk, r[1])


@gpu
@pytest.mark.parametrize("norm", [True, False])
def test_positions_outside_the_table_are_zero_in_outputs_that_the_call_makes(norm):
    fa = fa_()
    x = torch.randn(2, 3, 40, 64, device="cuda").half()
    cs = fa.rope_table(30, 32)
    pos = torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1)
    pos[1, 7] = -1
    args = dict(cos_sin=cs, eps=1e-6 if norm else None)
    with nan_in_new_tensors():
        a = fa.norm_rope(x, x, positions=pos, **args)
        b = fa.norm_rope_bwd(x, x, x, x, positions=pos, **args)
        c = fa.norm_rope(x, None, **args)        # by index: rows 30 .. 39 lie past the table
    ok(1)
    for y in (*a, b[0], b[1]):
        left = torch.zeros(2, 40, dtype=torch.bool)
        left[:, 30:], left[1, 7] = True, True
        left = left.cuda()[:, None].expand(2, 3, 40)
        assert (y[left] == 0).all() and y.isfinite().all() and (y[~left] != 0).any(-1).all()
    assert (c[0][:, :, 30:] == 0).all() and c[0].isfinite().all()
