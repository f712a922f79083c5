"""Calls on paged caches at the edges of what they document: offsets that break the rules inside
guarded tensors.  Against the definitions in 64 bits (tests/paged_util.py)."""
import math

import pytest
import torch

from tests import paged_util as pu

gpu = pytest.mark.gpu


def fa_():
    import exact_io_aware_22_gb300 as fa
    return fa


def ok():
    torch.cuda.synchronize()
    assert fa_().device_status() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ offsets that break the rules
def guarded(shape, dtype, fill):
    """A tensor of `fill` inside a larger one of `fill`, and the larger one."""
    n = math.prod(shape)
    whole = torch.full((n + 4096,), fill, dtype=dtype, device="cuda")
    return whole[2048:2048 + n].view(shape), whole


def outside(whole, n):
    return torch.cat([whole[:2048], whole[2048 + n:]])


@gpu
@pytest.mark.parametrize("cu", [(0, 25, 5, 30), (10, 0, 40, 7), (-5, 2, 3, 100), (30, 30, 30, 30),
                                (2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1)])
def test_append_with_broken_offsets_writes_only_places_that_they_name(cu):
    """A token may go where some sequence whose offsets hold it has its position, and nowhere
    else; what a row holds afterwards is what it held, or such a token."""
    fa = fa_()
    T, Hkv, H, d, page, lens = 30, 2, 4, 64, 16, (20, 20, 20)
    pool = pu.Pool(lens, Hkv, d, page, "bf16")
    shape = tuple(pool.kc.shape)
    (kc, kw), (vc, vw) = guarded(shape, torch.bfloat16, 3.0), guarded(shape, torch.bfloat16, 3.0)
    qo, qw = guarded((T, H, d), torch.bfloat16, 3.0)
    k, v, q = (torch.randn(T, n, d, device="cuda").bfloat16() for n in (Hkv, Hkv, H))
    torch.cuda.synchronize()
    fa.device_status()
    fa.append_paged(k, v, kc, vc, pool.table.cuda(), ints(lens), cu_seqlens=ints(cu), q=q, q_out=qo)
    torch.cuda.synchronize()
    fa.device_status()
    places, tokens = {}, set()
    for b in range(3):
        for t in range(max(cu[b], 0), min(cu[b + 1], T)):
            pos = lens[b] - (cu[b + 1] - t)
            if 0 <= pos:
                tokens.add(t)
                if pos < pool.width * page and 0 <= int(pool.table[b, pos // page]) < pool.pages:
                    places[int(pool.table[b, pos // page]), pos % page] = t
    for c, new in ((kc.cpu(), k.cpu()), (vc.cpu(), v.cpu())):
        for p in range(pool.pages):
            for r in range(page):
                row, t = c[p, :, r], places.get((p, r))
                assert (row == 3).all() or (t is not None and torch.equal(row, new[t])), (p, r)
    for t in range(T):
        assert (qo[t] == 3).all() or (t in tokens and torch.equal(qo[t], q[t])), t
    for w, x in ((kw, kc), (vw, vc), (qw, qo)):
        assert (outside(w, x.numel()) == 3).all()


@gpu
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (32, "bf16")])
@pytest.mark.parametrize("cu", [(0, 200, 50), (-7, 50, 100), (60, 20, 90), (100, 100, 100),
                                (2 ** 31 - 1, -2 ** 31, 100), (-2 ** 31, 2 ** 31 - 1, 0)])
def test_fwd_with_broken_offsets_writes_only_rows_that_they_name(cu, d, dtype):
    fa = fa_()
    total, H, most, t = 100, 4, 64, pu.DT[dtype]
    pool = pu.Pool((90, 60), 2, d, 16, dtype)
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(total, H, d, device="cuda").to(t)
    for width in (tb, torch.nn.functional.pad(tb, (0, 4096), value=-1)):   # tiles whole, or maybe cut
        (o, ow), (lse, lw) = guarded((total, H, d), t, 7.0), guarded((H, total), torch.float32, 7.0)
        fa.fwd_paged(q, kc, vc, width, sl, ints(cu), most, out=o, lse=lse)
        ok()
        named = torch.zeros(total, dtype=torch.bool)
        for b in range(2):
            a = min(max(cu[b], 0), total)
            named[a:min(max(cu[b + 1], a), total, a + most)] = True
        assert (o.cpu()[~named] == 7).all() and (lse.cpu()[:, ~named] == 7).all()
        assert not (lse.cpu()[:, named] == 7).any()
        assert (outside(ow, o.numel()) == 7).all() and (outside(lw, lse.numel()) == 7).all()
