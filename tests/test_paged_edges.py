"""Calls on paged caches at the edges of what they document: lengths past the table, rows without
keys beside values that are not finite, the largest queries, sizes past 32 bits, other 1-byte
types, and offsets that break the rules inside guarded tensors.  Against the definitions in 64
bits (tests/paged_util.py)."""
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


# ------------------------------------------------------------------ lengths past the table
@gpu
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("d,dtype,H", [(128, "bf16", 8), (64, "fp16", 8), (32, "bf16", 2)])
def test_lengths_past_the_table_keep_positions(d, dtype, H, window):
    """Sequences of which the table holds only the first keys: the tokens that fit are appended
    at the positions their length gives them, and queries, those of the others among them, see
    the keys that a window and the causal order leave them of those."""
    fa = fa_()
    Hkv, page, room, t = 2, 16, 80, pu.DT[dtype]
    lens, new = [95, 80, 85, 400, 60], [40, 9, 3, 30, 1]
    held = [min(n, room) for n in lens]
    pool = pu.Pool(held, Hkv, d, page, dtype, width=room // page)
    kc, vc, tb, _ = pool.cuda()
    sl, starts = ints(lens), [sum(new[:i]) for i in range(6)]
    cu = ints(starts)
    total = sum(new)
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn((total, n, d), generator=g).to(t).cuda() for n in (H, Hkv, Hkv))
    torch.cuda.synchronize()
    fa.device_status()
    fa.append_paged(k, v, kc, vc, tb, sl, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert fa.device_status() == 1                 # tokens without a place
    pool.kc, pool.vc = kc.cpu(), vc.cpu()
    for b in range(5):
        for i in range(new[b]):
            p = lens[b] - new[b] + i
            if p < room:
                at = int(pool.table[b, p // page])
                assert torch.equal(pool.kc[at, :, p % page], k[starts[b] + i].cpu())
    o, lse = fa.fwd_paged(q, kc, vc, tb, sl, cu, max(new), window=window)
    last = torch.tensor(starts[1:], device="cuda") - 1
    od, ld = fa.decode_paged(q[last], kc, vc, tb, sl, window=window)
    ok()
    for b in range(5):
        c, m = starts[b], new[b]
        at = torch.arange(lens[b] - m, lens[b])
        ref = pu.reference(pool, q[c:c + m].cpu(), b, at, 1 / math.sqrt(d), window=window)
        pu.check_rows(o[c:c + m], lse[:, c:c + m].t(), ref, t, p_half=pu.HALF[t])
        ref = pu.reference(pool, q[c + m - 1:c + m].cpu(), b, at[-1:], 1 / math.sqrt(d), window=window)
        pu.check_rows(od[b:b + 1], ld[b:b + 1], ref, t)


@gpu
@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("width", [4, 400])
def test_decode_windows_past_the_table(cache, width):
    # rows whole and cut; windows that reach back into the table's keys or do not
    fa = fa_()
    page, d, H, Hkv = 16, 128, 8, 2
    room = width * page
    lens = [room + 10, room + 70, room - 3, 2 ** 31 - 1, 0]
    pool = pu.Pool([min(n, room) for n in lens], Hkv, d, page, "e4m3" if cache == "e4m3" else "bf16")
    assert pool.width == width
    kc, vc, tb, _ = pool.cuda()
    q = torch.randn((5, H, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    for window in (40, 70, 2 ** 31 - 1):
        if cache == "e4m3":
            o, lse = fa.decode_paged_fp8(q.cuda(), kc, vc, tb, ints(lens), *pool.scales, window=window)
        else:
            o, lse = fa.decode_paged(q.cuda(), kc, vc, tb, ints(lens), window=window)
        ok()
        for b, n in enumerate(lens):
            ref = pu.reference(pool, q[b:b + 1], b, torch.tensor([n - 1]), 1 / math.sqrt(d), window=window)
            pu.check_rows(o[b:b + 1], lse[b:b + 1], ref, torch.bfloat16)


@gpu
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("window", [0, 1 << 30, 2 ** 31 - 1])
def test_fwd_lengths_near_32_bits(d, dtype, window):
    # every key of the table is earlier than every query; the longest window leaves the first some
    fa = fa_()
    pool = pu.Pool([64, 64, 64], 2, d, 16, dtype)
    kc, vc, tb, _ = pool.cuda()
    lens, new = [2 ** 31 - 1, 2 ** 30 + 40, 64], [200, 70, 5]
    cu = [0, 200, 270, 275]
    q = torch.randn((275, 4, d), generator=torch.Generator().manual_seed(2)).to(pu.DT[dtype])
    o, lse = fa.fwd_paged(q.cuda(), kc, vc, tb, ints(lens), ints(cu), 200, window=window)
    ok()
    for b, (n, m) in enumerate(zip(lens, new)):
        rows = slice(cu[b], cu[b] + m)
        ref = pu.reference(pool, q[rows], b, torch.arange(n - m, n), 1 / math.sqrt(d), window=window)
        pu.check_rows(o[rows], lse[:, rows].t(), ref, pu.DT[dtype], p_half=pu.HALF[pu.DT[dtype]])


# ------------------------------------------------------------------ rows without keys
@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (32, "bf16")])
def test_rows_without_keys_beside_values_that_are_not_finite(d, dtype, bad):
    """More tokens than keys, and windows that end in absent pages: those rows are 0 whatever the
    values of keys that other rows of their tile see; tiles whole, and cut beside a long sequence."""
    fa = fa_()
    for lens, new in (([30, 9], [70, 20]), ([30, 9, 9000], [70, 20, 2])):
        pool = pu.Pool(lens, 2, d, 16, dtype)
        for b in (0, 1):
            pool.vc[int(pool.table[b, 0]), :, 3] = bad
        kc, vc, tb, sl = pool.cuda()
        cu = ints([sum(new[:i]) for i in range(len(new) + 1)])
        q = torch.randn(sum(new), 4, d, device="cuda").to(pu.DT[dtype])
        o, lse = fa.fwd_paged(q, kc, vc, tb, sl, cu, max(new))
        ok()
        for c, n in ((0, 40), (70, 11)):
            assert (o[c:c + n] == 0).all() and (lse[:, c:c + n] == -math.inf).all()
            assert not torch.isfinite(o[c + n + 3:c + (70 if c == 0 else 20)]).any()
    pool = pu.Pool([100], 2, d, 16, dtype)
    pool.vc[int(pool.table[0, 0]), :, 3] = bad      # key 3; keys 16 .. 31 are absent
    pool.table[0, 1] = -1
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(100, 4, d, device="cuda").to(pu.DT[dtype])
    o, lse = fa.fwd_paged(q, kc, vc, tb, sl, ints([0, 100]), 100, window=5)
    ok()
    assert (o[20:32] == 0).all() and (lse[:, 20:32] == -math.inf).all()
    assert torch.isfinite(lse[:, 32:]).all()


# ------------------------------------------------------------------ the largest queries
@gpu
@pytest.mark.parametrize("H", [4, 24])
@pytest.mark.parametrize("e", [125, 126])
def test_decode_fp8_largest_queries(e, H):
    # bf16 queries up to the type's largest against codes and scales so small that scores are not
    pool = pu.Pool((200, 33), 2, 128, 32, "e4m3")
    small = (pu.e4m3(pool.kc) * pool.scales[0] / 16).to(torch.float8_e4m3fn)
    pool.kc.copy_(small.view(torch.uint8))
    pool.scales = (2.0 ** -122, pool.scales[1])
    scale = 2.0 ** (125 - e)
    g = torch.Generator().manual_seed(e)
    top = float(torch.finfo(torch.bfloat16).max)
    q = (torch.randn((2, H, 128), generator=g) * 2.0 ** e).clamp(-top, top).bfloat16()
    assert q.isfinite().all() and q.abs().amax(-1).max() >= 2.0 ** (e + 1)
    kc, vc, tb, sl = pool.cuda()
    o, lse = fa_().decode_paged_fp8(q.cuda(), kc, vc, tb, sl, *pool.scales, scale=scale)
    ok()
    for b, n in enumerate(pool.lens):
        ref = pu.reference(pool, q[b:b + 1], b, torch.tensor([n - 1]), scale)
        pu.check_rows(o[b:b + 1], lse[b:b + 1], ref, torch.bfloat16)


@gpu
def test_decode_fp8_zero_keys_under_the_largest_scale():
    # the scale of the scores overflows, the scores are 0: the mean of the values
    pool = pu.Pool((70,), 2, 128, 32, "e4m3")
    pool.kc.masked_fill_(pool.kc != 0x7F, 0)
    pool.scales = (1.0, pool.scales[1])
    kc, vc, tb, sl = pool.cuda()
    for top, scale in ((2.0 ** 127, 8.0), (2.0 ** 100, 2.0 ** 40)):
        q = torch.full((1, 4, 128), top, dtype=torch.bfloat16)
        o, lse = fa_().decode_paged_fp8(q.cuda(), kc, vc, tb, sl, *pool.scales, scale=scale)
        ok()
        ref = pu.reference(pool, q, 0, torch.tensor([69]), scale)
        pu.check_rows(o, lse, ref, torch.bfloat16)


# ------------------------------------------------------------------ sizes past 32 bits
@gpu
def test_windows_and_bounds_past_32_bits():
    fa = fa_()
    pool = pu.Pool((90, 40), 2, 64, 16, "fp16")
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(2, 8, 64, device="cuda").half()
    cu = ints([0, 1, 2])
    k = torch.randn(1, 2, 40, 64, device="cuda").half()
    want = fa.decode_paged(q, kc, vc, tb, sl), fa.fwd_paged(q, kc, vc, tb, sl, cu, 1), fa.fwd(k, k, k)
    for w in (2 ** 31, 2 ** 32 + 5, 2 ** 40):
        got = (fa.decode_paged(q, kc, vc, tb, sl, window=w),
               fa.fwd_paged(q, kc, vc, tb, sl, cu, 1, window=w), fa.fwd(k, k, k, window=w))
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y)), w
    for w in (-1, -2 ** 31, 5 - 2 ** 32):
        with pytest.raises((ValueError, fa.FAError)):
            fa.decode_paged(q, kc, vc, tb, sl, window=w)
        with pytest.raises((ValueError, fa.FAError)):
            fa.fwd_paged(q, kc, vc, tb, sl, cu, 1, window=w)
    for m in (2 ** 31, 2 ** 32 + 1, 1 - 2 ** 32, 0):
        with pytest.raises((ValueError, fa.FAError)):
            fa.fwd_paged(q, kc, vc, tb, sl, cu, m)
    ok()


# ------------------------------------------------------------------ types of codes
@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool])
def test_python_refuses_other_one_byte_caches(dtype):
    fa = fa_()
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for good in (torch.uint8, torch.float8_e4m3fn):
        c = torch.zeros(4, 2, 16, 128, dtype=torch.uint8).view(good)
        assert fa._paged(c, c.clone(), t, n, None, 2, 128)[1] == 2
    c = torch.zeros(4, 2, 16, 128, dtype=torch.uint8).view(dtype)
    with pytest.raises(TypeError):
        fa._paged(c, c.clone(), t, n, None, 2, 128)
    with pytest.raises(TypeError):                # one cache right, the other not
        fa._paged(c.view(torch.uint8), c, t, n, None, 2, 128)


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
