"""Packed sequences whose offsets overlap (they break the calls' rules): a row goes to the sequence in
which a binary search of the offsets ends, whichever rows the thread has looked up before, so that
the append with norms puts tokens where the plain one does."""
import pytest
import torch

from tests import norm_rope_util as nu
from tests import paged_util as pu
from tests.test_paged_edges import ints

gpu = pytest.mark.gpu


def fa_():
    import exact_io_aware_22_gb300 as fa
    return fa


def ok():
    torch.cuda.synchronize()
    assert fa_().device_status() == 0


def search(offsets, n):
    """The sequence in which a binary search of the offsets ends for row n, or None: it does not hold it."""
    lo, hi = 0, len(offsets) - 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if offsets[mid] <= n else (lo, mid)
    return lo if offsets[lo] <= n < offsets[lo + 1] else None


OVERLAP = (0, 20000, 5001, 30000, 40000)         # rows 5001 .. 19999: of sequences 0 and 2


@gpu
def test_overlapping_sequences_are_searched_alike_by_both_appends():
    fa, T, H, d, page = fa_(), 40000, 2, 32, 64
    lens = [20000, 7, 24999, 10000]
    pool = pu.Pool(lens, 1, d, page, "fp16", fill=3.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H + 2, d), generator=g, device="cuda").half()
    cs = nu.table(25000, d).cuda()
    sides = []
    for eps in (None, 1e-6):
        vc, kc = (torch.full(tuple(pool.kc.shape), 3.0, device="cuda", dtype=torch.float16) for _ in range(2))
        qo = torch.full((T, H, d), 3.0, device="cuda", dtype=torch.float16)
        fa.append_paged(x[:, H:H + 1], x[:, H + 1:], kc, vc, pool.table.cuda(), ints(lens),
                        cu_seqlens=ints(OVERLAP), cos_sin=cs, q=x[:, :H], q_out=qo, eps=eps)
        ok()
        sides.append((vc, (kc != 3).any(-1), (qo != 3).any(-1)))
    assert all(torch.equal(a, b) for a, b in zip(*sides))


@gpu
@pytest.mark.parametrize("norm", [True, False])
def test_overlapping_sequences_do_not_depend_on_the_rows_before(norm):
    fa, T, H, d = fa_(), 40000, 2, 32
    x = torch.randn(T, H, d, device="cuda").half()
    cs = nu.table(25000, d).cuda()
    where = [search(OVERLAP, n) for n in range(T)]
    pos = torch.tensor([n - OVERLAP[b] for n, b in enumerate(where)], dtype=torch.int32, device="cuda")
    args = dict(cos_sin=cs, eps=1e-6 if norm else None)
    want = fa.norm_rope(x, None, positions=pos, **args)[0]
    dwant = fa.norm_rope_bwd(x, None, x, positions=pos, **args)[0]
    got = fa.norm_rope(x, None, cu_seqlens=ints(OVERLAP), **args)[0]
    dgot = fa.norm_rope_bwd(x, None, x, cu_seqlens=ints(OVERLAP), **args)[0]
    ok()
    assert torch.equal(got, want) and torch.equal(dgot, dwant)
