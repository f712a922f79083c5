"""Norms and rotation of packed sequences long enough that a warp goes on from piece to piece, with
rows that belong to no sequence or lie past the table among them, and what such rows hold in outputs
that the call makes.  Against the definitions in 64 bits (tests/norm_rope_util.py, where the tolerances
are derived)."""
import contextlib

import pytest
import torch

from tests import norm_rope_util as nu
from tests import paged_util as pu
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


def packed_rows(lens, first, total, max_pos, bad=()):
    """Rows that a call turns and their positions, for sequences of ``lens`` from row ``first`` on; rows
    of ``bad`` are given a position outside the table of ``max_pos``."""
    rows, at, n = [], [], first
    for m in lens:
        rows += range(n, n + m)
        at += range(m)
        n += m
    assert n <= total
    keep = [i for i, (r, p) in enumerate(zip(rows, at)) if p < max_pos and r not in bad]
    return torch.tensor([rows[i] for i in keep]), torch.tensor([at[i] for i in keep])


# ------------------------------------------------------------------ many pieces to a warp
# d, tokens of whole sequences (about), rotated columns, interleaved, eps, dtype, weights, outputs given
MANY = [
    (128, 5200, 128, False, 1e-6, "bf16", "fp32", True),
    (128, 5200, 64, True, 1e-6, "fp16", "16", False),
    (128, 5200, 128, True, None, "bf16", None, True),
    (128, 5200, 96, False, None, "fp16", None, False),
    (64, 9000, 64, False, 1e-6, "fp16", "16", True),
    (32, 16500, 32, False, 1e-6, "bf16", "16", True),
    (32, 16500, 16, True, 1e-6, "fp16", "fp32", False),
    (32, 16500, 32, True, None, "bf16", None, False),
]


@gpu
@pytest.mark.parametrize("by_position", [False, True])
@pytest.mark.parametrize("case", MANY, ids=["-".join(str(x) for x in c) for c in MANY])
def test_pieces_of_many_packed_sequences(case, by_position):
    """32/8 heads: 16 steps and more to a warp.  Empty sequences, of one token and of many, gaps at both
    ends, a sequence longer than the table, and by positions some outside it in the middle."""
    d, tokens, rot, inter, eps, dtype, wk, given = case
    H, Hkv, t, fa = 32, 8, pu.DT[dtype], fa_()
    g = torch.Generator().manual_seed(d + rot + by_position)
    lens = [0, 1, 1, 0, 700, 1, 33, 0, 0, 2]
    while sum(lens) < tokens:
        lens += [int(torch.randint(1, 900, (), generator=g)), 0, 1]
    first, max_pos = 5, 600
    total = first + sum(lens) + 37
    offsets = [first + sum(lens[:i]) for i in range(len(lens) + 1)]
    bad, pos = (), None
    if by_position:                              # the sequences' indices, some rows' outside the table
        pos = torch.full((total,), 3, dtype=torch.int32)
        for a, m in zip(offsets, lens):
            pos[a:a + m] = torch.arange(m, dtype=torch.int32)
        bad = [first, first + 2, first + 300, first + 301, first + tokens // 2, offsets[-1] - 1]
        pos[bad] = torch.tensor([-1, max_pos, 2 ** 31 - 1, -2 ** 31, max_pos + 5, -7], dtype=torch.int32)
    rows, at = packed_rows(lens, first, total, max_pos, set(bad))
    rest = torch.ones(total, dtype=torch.bool)
    rest[rows] = False
    x = torch.randn((total, H + Hkv, d), generator=g).to(t).cuda()
    dy = (torch.randn((total, H + Hkv, d), generator=g) * 0.7).to(t).cuda()
    w = None if wk is None else (1 + 0.3 * torch.randn((2, d), generator=g)).to(torch.float32 if wk == "fp32" else t).cuda()
    cs = nu.table(max_pos, rot).cuda()
    args = dict(cos_sin=cs, cu_seqlens=ints(offsets), interleaved=inter, eps=eps,
                positions=None if pos is None else pos.cuda())
    if w is not None:
        args.update(q_weight=w[0], k_weight=w[1])
    q, k, gq, gk = x[:, :H], x[:, H:], dy[:, :H], dy[:, H:]
    y, dx = (torch.full_like(x, 7.0) for _ in range(2))
    if given:
        outs, grads = fa.norm_rope(q, k, q_out=y[:, :H], k_out=y[:, H:], **args), \
            fa.norm_rope_bwd(gq, gk, q, k, dq=dx[:, :H], dk=dx[:, H:], **args)
    else:
        with nan_in_new_tensors():
            outs, grads = fa.norm_rope(q, k, **args), fa.norm_rope_bwd(gq, gk, q, k, **args)
    ok(1)                                        # some rows lie outside the table
    rows, rest, rot_rows = rows.cuda(), rest.cuda(), cs[at.cuda()][:, None]
    for i, (v, g_v) in enumerate(((q, gq), (k, gk))):
        assert (outs[i][rest] == (7 if given else 0)).all(), "rows that are left out"
        assert (grads[i][rest] == (7 if given else 0)).all(), "rows that are left out, backward"
        ww = None if w is None else w[i].double()
        if eps is not None and ww is None:
            ww = torch.ones(d, dtype=torch.float64, device="cuda")
        want, tol = nu.forward(v[rows], ww, eps, rot_rows, inter)
        nu.close(outs[i][rows], want.cpu(), tol.cpu(), t, "y")
        want, tol, terms, sizes = nu.backward(g_v[rows], v[rows], ww, eps, rot_rows, inter)
        nu.close(grads[i][rows], want.cpu(), tol.cpu(), t, "dx")
        if w is not None:
            nu.close_dw(grads[2 + i], terms.cpu(), sizes.cpu(), "dw")
    # again, over the same data: bit for bit
    again = fa.norm_rope_bwd(gq, gk, q, k, **args)
    ok(1)
    for a, b in zip(again, grads):
        assert a is None and b is None or torch.equal(a if a.dim() == 1 else a[rows], b if b.dim() == 1 else b[rows])


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
