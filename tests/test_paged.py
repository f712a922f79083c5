"""Paged key/value caches on the GPU: appending with rotation, and decoding, against plain
definitions in 64 bits (tests/paged_util.py, where the tolerances are derived).  Pool rows
that hold no key are NaN, unused table entries out of range."""
import math

import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu


def fa_():
    import exact_io_aware_22_gb300 as fa
    return fa


def ok():
    torch.cuda.synchronize()
    assert fa_().device_status() == 0


# ------------------------------------------------------------------ decoding
def run_decode(lens, H, Hkv, d, dtype, page, cache="16", window=0, layout="hnd", width=None,
               scale=None, seed=0, table=None, qmul=1.0):
    fa = fa_()
    pool = pu.Pool(lens, Hkv, d, page, "e4m3" if cache == "e4m3" else dtype, layout, width, seed=seed)
    if table is not None:
        table(pool)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((len(lens), H, d), generator=g) * qmul).to(pu.DT[dtype])
    scale = 1 / math.sqrt(d) if scale is None else scale
    kc, vc, tb, sl = pool.cuda()
    if cache == "e4m3":
        o, lse = fa.decode_paged_fp8(q.cuda(), kc, vc, tb, sl, *pool.scales, scale=scale, window=window)
    else:
        o, lse = fa.decode_paged(q.cuda(), kc, vc, tb, sl, scale=scale, window=window)
    ok()
    worst = []
    for b, n in enumerate(lens):
        n = min(n, pool.width * page)
        ref = pu.reference(pool, q[b:b + 1], b, torch.tensor([n - 1]), scale, window=window)
        worst.append(pu.check_rows(o[b:b + 1], lse[b:b + 1], ref, pu.DT[dtype]))
    print("worst", max(worst))
    return o, lse


DECODE = [
    # lens, H, Hkv, d, dtype, page, cache, window, layout
    ((777,), 16, 16, 64, "fp16", 16, "16", 0, "hnd"),
    ((1, 2, 15, 16, 17, 0, 63, 64, 65), 8, 2, 128, "bf16", 16, "16", 0, "hnd"),
    ((1, 31, 32, 33, 0, 129), 4, 4, 64, "fp16", 64, "16", 0, "nhd"),
    ((1, 63, 64, 65, 300), 6, 2, 32, "bf16", 32, "16", 0, "pair"),
    ((500, 1000, 3), 20, 1, 128, "bf16", 64, "16", 0, "hnd"),        # 20 heads: two groups, one short
    ((500, 250), 32, 2, 64, "fp16", 128, "16", 0, "nhd"),            # groups of 16
    ((211, 97), 12, 4, 128, "fp16", 1, "16", 0, "hnd"),              # pages of one row
    ((211, 97), 6, 2, 32, "fp16", 2, "16", 0, "nhd"),
    ((333, 40), 5, 1, 64, "bf16", 3, "16", 0, "pair"),
    ((333, 21, 0), 12, 4, 128, "bf16", 20, "16", 0, "hnd"),
    ((1000, 900), 8, 8, 128, "bf16", 100, "16", 0, "nhd"),
    ((700, 5, 0, 64, 129), 12, 4, 128, "bf16", 20, "16", 100, "hnd"),   # windows
    ((700, 5, 64, 129), 8, 2, 64, "fp16", 16, "16", 1, "nhd"),
    ((700, 650, 64), 8, 2, 32, "bf16", 16, "16", 64, "hnd"),
    ((777,), 32, 8, 128, "bf16", 64, "e4m3", 0, "hnd"),
    ((1, 31, 32, 33, 0, 127, 128, 129), 3, 3, 128, "fp16", 16, "e4m3", 0, "nhd"),
    ((300, 7), 16, 1, 128, "bf16", 1, "e4m3", 0, "pair"),
    ((300, 170), 24, 2, 128, "fp16", 24, "e4m3", 50, "hnd"),
    ((900, 33), 100, 1, 64, "fp16", 16, "16", 0, "hnd"),              # 100 heads: seven parts
    ((900, 5000, 33), 70, 2, 128, "bf16", 16, "e4m3", 0, "hnd"),
    ((0, 0, 0), 4, 2, 64, "bf16", 16, "16", 0, "hnd"),                # nothing cached at all
]


@pytest.mark.parametrize("case", DECODE, ids=[f"{c[0][:3]}-{c[1:]}" for c in DECODE])
def test_decode(case):
    lens, H, Hkv, d, dtype, page, cache, window, layout = case
    run_decode(lens, H, Hkv, d, dtype, page, cache, window, layout, seed=len(lens) + page)


@pytest.mark.parametrize("cache,d", [("16", 128), ("e4m3", 128), ("16", 32)])
def test_decode_many_sequences(cache, d):
    # more sequences than threads that scan them, most ranges holding several whole rows
    lens = [int(n) for n in pu.np_rng(5).integers(0, 90, 300)]
    run_decode(lens, 6, 2, d, "bf16", 16, cache)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_decode_long_split(cache):
    # one row over all CTAs, and borders inside rows
    run_decode((20011, 3), 4, 1, 128, "bf16", 64, cache)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("B,n", [(3, 500), (60, 1000), (330, 1500)])
def test_decode_whole_rows(B, n, cache):
    # short rows, and more rows than run at once: a CTA for each; some empty
    lens = [int(x) for x in pu.np_rng(B).integers(0, n, B)]
    lens[B // 2] = 0
    H, Hkv = (12, 3) if B < 300 else (3, 3)
    run_decode(lens, H, Hkv, 128, "bf16", 32, cache, window=0 if B != 60 else 400)


def test_decode_wide_table():
    # a table much wider than the lengths: the split follows the lengths
    run_decode((300, 1000), 8, 2, 128, "bf16", 16, width=4096)


def test_decode_lengths_past_the_table_are_clamped():
    run_decode((64, 40), 8, 2, 64, "fp16", 16, seed=3)
    fa = fa_()
    pool = pu.Pool((64, 40), 2, 64, 16, "fp16", seed=3)
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(2, 8, 64, device="cuda").half()
    o1, l1 = fa.decode_paged(q, kc, vc, tb, sl)
    o2, l2 = fa.decode_paged(q, kc, vc, tb, torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32, device="cuda"))
    o3, l3 = fa.decode_paged(q, kc, vc, tb, torch.tensor([64, -7], dtype=torch.int32, device="cuda"))
    ok()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(o1[0], o3[0]) and (o3[1] == 0).all() and (l3[1] == -math.inf).all()


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("cache,page", [("16", 16), ("16", 4), ("e4m3", 16)])
def test_decode_absent_pages_are_not_attended(bad, cache, page):
    def holes(pool):
        pool.table[0, 1] = bad                   # in the middle
        pool.table[0, 0] = bad                   # and the first
        pool.table[1, :] = bad                   # a row without any page
        pool.table[2, -1] = pool.pages           # just past the pool
    run_decode((10 * page + 3, 5 * page, 12 * page), 8, 2, 128, "bf16", page, cache, table=holes)


def test_decode_large_scores_and_scale():
    # scores far apart: the running maximum moves, late keys dominate
    run_decode((900, 33), 8, 2, 128, "bf16", 32, scale=1.7, qmul=4.0)
    run_decode((900, 33), 8, 2, 128, "bf16", 32, "e4m3", scale=0.9, qmul=4.0)


def test_decode_fp8_tiny_and_huge_queries():
    # bf16 queries outside f16's range
    run_decode((200,), 8, 2, 128, "bf16", 32, "e4m3", scale=2.0 ** -20, qmul=2.0 ** 20)
    run_decode((200,), 8, 2, 128, "bf16", 32, "e4m3", scale=2.0 ** 20, qmul=2.0 ** -20)


def test_decode_fp8_scores_that_underflow():
    # scale * log2(e) times the queries' exponent is below fp32's least number: all scores are 0
    run_decode((70, 33, 500), 8, 2, 128, "bf16", 32, "e4m3", scale=1e-8, qmul=1e-38)


def test_decode_attended_nan_and_inf_propagate():
    fa = fa_()
    pool = pu.Pool((100, 100, 100), 2, 64, 16, "bf16")
    pool.vc[int(pool.table[0, 1]), 0, 3, 5] = float("nan")
    pool.kc[int(pool.table[1, 0]), 1, 0, 0] = float("inf")
    kc, vc, tb, sl = pool.cuda()
    q = torch.ones(3, 4, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = fa.decode_paged(q, kc, vc, tb, sl)
    ok()
    assert o[0, :2, 5].isnan().all() and o[0, :2].isnan().sum() == 2 and not o[0, 2:].isnan().any()
    assert o[1, 2:].isnan().all() and not o[1, :2].isnan().any() and not o[2].isnan().any()


def test_decode_shared_pages():
    # two sequences on the same prefix pages read the same keys
    fa = fa_()
    pool = pu.Pool((96, 96), 2, 64, 16, "fp16")
    pool.table[1] = pool.table[0]
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(1, 8, 64, device="cuda").half().expand(2, 8, 64).contiguous()
    o, lse = fa.decode_paged(q, kc, vc, tb, sl)
    ok()
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_decode_repeats_bit_for_bit_in_any_workspace():
    fa = fa_()
    pool = pu.Pool((5000, 17, 0, 900), 2, 128, 32, "bf16")
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    n = fa.decode_paged_workspace_size(8, 2, 128)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")      # NaN everywhere
    o1, l1 = fa.decode_paged(q, kc, vc, tb, sl)
    for _ in range(20):
        o2, l2 = fa.decode_paged(q, kc, vc, tb, sl, workspace=ws)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    ok()


def test_decode_agrees_with_contiguous_decode():
    fa = fa_()
    B, H, Hkv, d, n = 3, 8, 2, 128, 512
    k, v = (torch.randn(B, Hkv, n, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, H, d, device="cuda").bfloat16()
    sl = torch.tensor([512, 100, 0], dtype=torch.int32, device="cuda")
    o, lse = fa.decode(q, k, v, sl)
    kc, vc = (x.view(B, Hkv, n // 64, 64, d).transpose(1, 2).reshape(-1, Hkv, 64, d) for x in (k, v))
    tb = torch.arange(B * n // 64, dtype=torch.int32, device="cuda").view(B, -1)
    o2, lse2 = fa.decode_paged(q, kc, vc, tb, sl)
    ok()
    assert (o.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * o.float().abs().max()
    assert (lse[:2] - lse2[:2]).abs().max() <= 1e-5


# ------------------------------------------------------------------ appending
def run_append(new, before, H, Hkv, d, dtype, page, rot, interleaved=False, cache="16", layout="hnd",
               pad=(0, 0), fused=False, step=False, positions=False, with_q=True, seed=0):
    """new tokens on top of ``before`` keys; pad: tokens before the first and after the last."""
    fa = fa_()
    lens = [a + b for a, b in zip(new, before)]
    eight = cache == "e4m3"
    pool = pu.Pool(lens, Hkv, d, page, "e4m3" if eight else dtype, layout, seed=seed)
    g = torch.Generator().manual_seed(seed + 7)
    T = sum(new) + sum(pad)
    t = pu.DT[dtype]
    if fused:
        x = torch.randn((T, H + 2 * Hkv, d), generator=g).to(t)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        xc = x.cuda()
        qc, kcu, vcu = xc[:, :H], xc[:, H:H + Hkv], xc[:, H + Hkv:]
    else:
        q, k, v = (torch.randn((T, n, d), generator=g).to(t) for n in (H, Hkv, Hkv))
        qc, kcu, vcu = q.cuda(), k.cuda(), v.cuda()
    cu = torch.tensor([pad[0] + sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    tok = torch.arange(pad[0], pad[0] + sum(new))
    pos = torch.tensor(lens)[seq] - (cu[1:].long()[seq] - tok)
    ang = torch.zeros(T, dtype=torch.int32)
    ang[tok] = pos.int()
    if positions:
        ang = torch.randint(0, max(lens) + 5, (T,), generator=g).to(torch.int32)
    cs = fa.rope_table(max(lens) + 5, rot, device="cpu") if rot else None
    kc, vc, tb, sl = pool.cuda()
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.full((T, H, d), 7.0, dtype=t, device="cuda")
    kw = dict(cu_seqlens=None if step else cu.cuda(), cos_sin=None if cs is None else cs.cuda(),
              interleaved=interleaved, positions=ang.cuda() if positions else None,
              q=qc if with_q else None, q_out=qo if with_q else None)
    if eight:
        r = fa.append_paged_fp8(kcu, vcu, kc, vc, tb, sl, *pool.scales, **kw)
    else:
        r = fa.append_paged(kcu, vcu, kc, vc, tb, sl, **kw)
    ok()
    assert (r is qo) if with_q else (r is None)
    rows = cs[ang[tok].long()] if rot else torch.zeros((len(tok), 0))
    for src, now, old, r_, sc in ((k, kc, k0, rot, pool.scales[0]), (v, vc, v0, 0, pool.scales[1])):
        want, mag = pu.turn(src[tok], rows, r_, interleaved)
        at, row = pool.table[seq, pos // page].long(), (pos % page).long()
        got = now.cpu()[at, :, row]
        if eight:
            pu.check_codes(got, want / sc, mag / sc)
        else:
            pu.check_turned(got, want, mag, t)
        old = old.cpu().clone()
        old[at, :, row] = got                     # every other row keeps its bytes
        i = torch.uint8 if eight else torch.int16
        assert torch.equal(now.cpu().view(i), old.view(i)), "rows that are not new were touched"
    if with_q:
        want, mag = pu.turn(q[tok], rows, rot, interleaved)
        pu.check_turned(qo[tok.cuda()], want, mag, t)
        rest = torch.ones(T, dtype=torch.bool)
        rest[tok] = False
        assert (qo.cpu()[rest] == 7).all(), "rows of no sequence were touched"


APPEND = [
    # new, before, H, Hkv, d, dtype, page, rot, keywords
    ((1,), (0,), 4, 2, 64, "bf16", 16, 64, dict(step=True)),
    ((1, 1, 1), (15, 16, 4000), 32, 8, 128, "bf16", 16, 128, dict(step=True, fused=True)),
    ((1, 1, 1, 1), (0, 1, 63, 64), 8, 1, 128, "fp16", 64, 64, dict(step=True, cache="e4m3", layout="nhd")),
    ((5, 1, 33, 16), (0, 7, 100, 31), 6, 2, 64, "fp16", 16, 32, dict(interleaved=True, layout="nhd")),
    ((5, 0, 33, 0), (0, 7, 100, 0), 6, 2, 64, "bf16", 16, 64, dict(pad=(3, 9), fused=True)),
    ((50, 70), (13, 0), 4, 4, 32, "bf16", 20, 32, dict(layout="pair")),
    ((50, 70), (13, 0), 4, 4, 32, "fp16", 6, 16, dict(interleaved=True, layout="pair", pad=(0, 1))),
    ((130, 3), (1, 900), 12, 4, 128, "bf16", 1, 128, dict(fused=True)),
    ((130, 3), (1, 900), 12, 4, 128, "bf16", 7, 0, dict()),
    ((20, 300), (5, 5), 16, 2, 128, "fp16", 64, 128, dict(cache="e4m3", interleaved=True, positions=True)),
    ((20, 300), (5, 5), 16, 2, 128, "bf16", 64, 96, dict(cache="e4m3", with_q=False)),
    ((20, 31), (5, 5), 2, 2, 64, "bf16", 64, 48, dict(positions=True, with_q=False)),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(c) for c in APPEND])
def test_append(case):
    new, before, H, Hkv, d, dtype, page, rot, kw = case
    run_append(new, before, H, Hkv, d, dtype, page, rot, seed=page, **kw)


def test_append_fp8_saturates_and_keeps_nan():
    fa = fa_()
    pool = pu.Pool((4,), 1, 128, 16, "e4m3")
    kc, vc, tb, sl = pool.cuda()
    k = torch.zeros(4, 1, 128, device="cuda", dtype=torch.bfloat16)
    k[0] = 1e30
    k[1] = -1e30
    k[2] = float("nan")
    k[3, 0, 0] = float("inf")
    fa.append_paged_fp8(k, k, kc, vc, tb, sl, 1.0, 1.0,
                        cu_seqlens=torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    ok()
    got = pu.e4m3(kc[int(pool.table[0, 0]), 0])
    assert (got[0] == 448).all() and (got[1] == -448).all() and got[2].isnan().all()
    assert got[3, 0] == 448 and (got[3, 1:] == 0).all()


def test_append_step_skips_empty_sequences():
    fa = fa_()
    pool = pu.Pool((0, 9, 0), 2, 64, 16, "bf16")
    kc, vc, tb, sl = pool.cuda()
    k0 = kc.clone()
    k, v, q = (torch.randn(3, n, 64, device="cuda").bfloat16() for n in (2, 2, 4))
    qo = torch.full_like(q, 7.0)
    fa.append_paged(k, v, kc, vc, tb, sl, q=q, q_out=qo)
    ok()
    p = int(pool.table[1, 0])
    assert torch.equal(kc[p, :, 8], k[1]) and torch.equal(vc[p, :, 8], v[1])
    k0[p, :, 8] = k[1]
    assert torch.equal(kc.view(torch.int16), k0.view(torch.int16))
    assert torch.equal(qo[1], q[1]) and (qo[0] == 7).all() and (qo[2] == 7).all()


def test_append_reports_tokens_without_a_place():
    fa = fa_()
    torch.cuda.synchronize()
    fa.device_status()
    for how in ("absent page", "past the table", "past the angles"):
        pool = pu.Pool((20, 20), 2, 64, 16, "bf16")
        if how == "absent page":
            pool.table[0, 1] = -1
        kc, vc, tb, sl = pool.cuda()
        if how == "past the table":
            sl = torch.tensor([33, 20], dtype=torch.int32, device="cuda")
        cs = fa.rope_table(19 if how == "past the angles" else 64, 64)
        k, v = (torch.randn(2, 2, 64, device="cuda").bfloat16() for _ in range(2))
        k0 = kc.clone()
        fa.append_paged(k, v, kc, vc, tb, sl, cos_sin=cs)
        torch.cuda.synchronize()
        assert fa.device_status() == 1, how
        assert fa.device_status() == 0
        p = int(pool.table[1, 1])
        if how != "past the angles":              # the other sequence's token is in place
            assert torch.equal(vc[p, :, 3], v[1])
            k0[p, :, 3] = kc[p, :, 3]
        assert torch.equal(kc.view(torch.int16), k0.view(torch.int16)), how


def test_append_offsets_that_do_not_ascend_touch_nothing_outside():
    fa = fa_()
    pool = pu.Pool((20, 20, 20), 2, 64, 16, "bf16")
    kc, vc, tb, sl = pool.cuda()
    k, v = (torch.randn(30, 2, 64, device="cuda").bfloat16() for _ in range(2))
    for cu in ((0, 25, 5, 30), (10, 0, 40, 7), (-5, 2, 3, 100), (30, 30, 30, 30)):
        fa.append_paged(k, v, kc, vc, tb, sl,
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    fa.device_status()


def test_rope_table_of_far_positions():
    fa = fa_()
    t = fa.rope_table(1 << 20, 64, base=500000.0)
    i = torch.arange(0, 64, 2, dtype=torch.float64)
    for p in (0, 1, 777777, (1 << 20) - 1):
        a = p * 500000.0 ** (-i / 64)
        # half an fp32 step, and fp64's own error in an angle of up to 2^20
        assert (t[p].cpu().double() - torch.cat([a.cos(), a.sin()])).abs().max() <= 2.0 ** -24


# ------------------------------------------------------------------ many new tokens
def run_fwd(new, before, H, Hkv, d, dtype, page, causal=True, window=0, layout="hnd", pad=(0, 0),
            scale=None, table=None, lens=None, seed=0, qmul=1.0):
    """new[b] query rows behind before[b] keys (or keys as in ``lens``)."""
    fa = fa_()
    lens = [a + b for a, b in zip(new, before)] if lens is None else lens
    pool = pu.Pool(lens, Hkv, d, page, dtype, layout, seed=seed)
    if table is not None:
        table(pool)
    g = torch.Generator().manual_seed(seed + 3)
    total, t = sum(new) + sum(pad), pu.DT[dtype]
    q = (torch.randn((total, H, d), generator=g) * qmul).to(t)
    scale = 1 / math.sqrt(d) if scale is None else scale
    cu = [pad[0] + sum(new[:i]) for i in range(len(new) + 1)]
    kc, vc, tb, sl = pool.cuda()
    o = torch.full((total, H, d), 7.0, dtype=t, device="cuda")
    lse = torch.full((H, total), 7.0, device="cuda")
    r = fa.fwd_paged(q.cuda(), kc, vc, tb, sl, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                     max(max(new), 1), causal=causal, scale=scale, window=window, out=o, lse=lse)
    ok()
    assert r[0] is o and r[1] is lse
    worst = []
    for b, m in enumerate(new):
        if m == 0:
            continue
        rows = slice(cu[b], cu[b] + m)
        at = torch.arange(lens[b] - m, lens[b])
        ref = pu.reference(pool, q[rows], b, at, scale, causal, window)
        worst.append(pu.check_rows(o[rows], lse[:, rows].t(), ref, t, p_half=pu.HALF[t]))
    print("worst", max(worst))
    rest = torch.ones(total, dtype=torch.bool)
    rest[pad[0]:pad[0] + sum(new)] = False
    assert (o.cpu()[rest] == 7).all() and (lse.cpu()[:, rest] == 7).all(), "rows of no sequence"
    return o, lse


FWD = [
    # new, before, H, Hkv, d, dtype, page, keywords
    ((1,), (0,), 2, 1, 128, "bf16", 16, {}),
    ((5, 5, 5), (100, 300, 0), 8, 2, 128, "bf16", 64, {}),
    ((130, 1, 257, 64), (500, 127, 0, 64), 4, 2, 128, "bf16", 64, {}),
    ((130, 1, 257, 64), (500, 127, 0, 64), 4, 4, 64, "fp16", 16, dict(layout="nhd")),
    ((300, 40), (70, 900), 2, 1, 32, "bf16", 128, dict(layout="pair")),
    ((300, 40), (70, 900), 2, 1, 32, "fp16", 2, dict(pad=(5, 9))),
    ((140, 0, 33), (70, 90, 256), 6, 2, 128, "fp16", 1, dict(pad=(1, 130), layout="nhd")),
    ((140, 0, 33), (70, 90, 256), 6, 2, 64, "bf16", 3, dict(pad=(0, 200))),
    ((200, 300), (900, 15), 4, 2, 128, "bf16", 20, dict(window=100)),
    ((200, 300), (900, 15), 4, 2, 64, "fp16", 48, dict(window=1)),
    ((200, 300), (900, 15), 4, 2, 32, "bf16", 16, dict(window=129)),
    ((200, 300), (900, 15), 4, 2, 128, "fp16", 256, dict(window=5000)),
    ((200, 17), (300, 15), 4, 2, 128, "bf16", 100, dict(causal=False)),
    ((200, 17), (300, 15), 4, 1, 64, "fp16", 8, dict(causal=False, layout="pair")),
    ((700,), (0,), 2, 2, 64, "bf16", 64, dict(qmul=4.0)),
    ((300,), (400,), 2, 2, 128, "bf16", 64, dict(scale=1.3)),
    # keys split over the CTAs, heads packed: 4, 8, 128 and 2 of 6, odd rows
    ((5,), (6000,), 4, 1, 128, "bf16", 64, {}),
    ((5, 70, 1), (3000, 0, 700), 16, 2, 128, "fp16", 16, dict(window=900)),
    ((3, 2), (2500, 300), 128, 1, 64, "bf16", 32, {}),
    ((33, 7), (2000, 100), 6, 1, 64, "fp16", 16, dict(pad=(2, 3))),
    ((9, 130), (3000, 700), 12, 2, 32, "bf16", 16, dict(causal=False)),
    # ranges of several pieces: long and short sequences, some without rows or keys, and tiles
    # for more than one round
    ((5, 1, 0, 64, 3) * 8, (1, 9000, 300, 40, 0) * 8, 8, 2, 128, "bf16", 64, {}),
    ((5, 1, 0, 30, 3) * 13, (1, 7000, 300, 40, 0) * 13, 16, 4, 64, "fp16", 16, dict(window=6000)),
    ((300, 2, 40), (8000, 60, 5), 12, 3, 128, "fp16", 16, dict(pad=(2, 3))),
    ((300, 2, 40), (8000, 60, 5), 12, 3, 32, "bf16", 16, dict(causal=False)),
    ((30, 2, 40), (8000, 60, 5), 12, 3, 128, "bf16", 8, {}),             # several producers
    ((4, 90), (9000, 30), 4, 1, 128, "fp16", 1, dict(layout="nhd")),
]


@pytest.mark.parametrize("case", FWD, ids=[str(c) for c in FWD])
def test_fwd(case):
    new, before, H, Hkv, d, dtype, page, kw = case
    run_fwd(new, before, H, Hkv, d, dtype, page, seed=page, **kw)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (32, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_fwd_more_rows_than_keys(d, dtype, causal):
    # causal rows before the first key see none; a sequence without any key; a tile of them
    run_fwd((300, 10, 140, 600), None, 2, 1, d, dtype, 16, causal=causal, lens=[200, 3, 0, 130])


@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 64), (128, 1), (64, 16), (32, 6), (64, 128)])
def test_fwd_absent_pages_are_not_attended(bad, d, page):
    def holes(pool):
        n = -(-700 // page)
        pool.table[0, n // 2] = bad
        pool.table[0, 0] = bad
        pool.table[1, :] = bad                   # no page at all
        pool.table[2, -(-40 // page) - 1] = pool.pages
    run_fwd((200, 30, 20), (500, 10, 20), 4, 2, d, "bf16", page, table=holes)


def test_fwd_offsets_that_break_the_rules_touch_nothing_outside():
    fa = fa_()
    pool = pu.Pool((90, 60), 2, 64, 16, "bf16")
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(100, 4, 64, device="cuda").bfloat16()
    for cu in ((0, 200, 50), (-7, 50, 100), (60, 20, 90), (100, 100, 100)):
        fa.fwd_paged(q, kc, vc, tb, sl, torch.tensor(cu, dtype=torch.int32, device="cuda"), 64)
    ok()


@pytest.mark.parametrize("d,dtype,H,B", [(128, "bf16", 8, 2), (64, "fp16", 8, 2), (128, "fp16", 8, 80)])
def test_fwd_sequences_longer_than_max_seqlen(d, dtype, H, B):
    # the rows up to max_seqlen get what they would get without it, the others are left alone
    fa = fa_()
    lens, new, most = [500, 90] + [40] * (B - 2), [200, 90] + [30] * (B - 2), 70
    pool = pu.Pool(lens, 2, d, 16, dtype)
    kc, vc, tb, sl = pool.cuda()
    cu = torch.tensor([0] + new).cumsum(0)
    total, t = int(cu[-1]), pu.DT[dtype]
    q = torch.randn((total, H, d), generator=torch.Generator().manual_seed(B)).to(t)
    o = torch.full((total, H, d), 7.0, dtype=t, device="cuda")
    lse = torch.full((H, total), 7.0, device="cuda")
    fa.fwd_paged(q.cuda(), kc, vc, tb, sl, cu.int().cuda(), most, out=o, lse=lse)
    ok()
    for b in range(B):
        m, c = min(new[b], most), int(cu[b])
        at = torch.arange(lens[b] - new[b], lens[b] - new[b] + m)
        ref = pu.reference(pool, q[c:c + m], b, at, 1 / math.sqrt(d))
        pu.check_rows(o[c:c + m], lse[:, c:c + m].t(), ref, t, p_half=pu.HALF[t])
        assert (o[c + m:c + new[b]] == 7).all() and (lse[:, c + m:c + new[b]] == 7).all()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_fwd_ranges_of_rows_without_keys(d, dtype):
    # cut: among long sequences, prompts longer than their keys, and sequences without keys
    lens = [9000, 3, 0, 40, 5000, 0]
    run_fwd((4, 40, 30, 60, 1, 1), None, 8, 2, d, dtype, 16, lens=lens)


def test_fwd_repeats_and_replays_bit_for_bit():
    fa = fa_()
    # 333 rows: tiles enough at 128 heads, keys split at 4
    for d, H in ((128, 4), (64, 4), (128, 128), (64, 128)):
        pool = pu.Pool((700, 400, 33), 2, d, 16, "bf16")
        kc, vc, tb, sl = pool.cuda()
        cu = torch.tensor([0, 300, 310, 333], dtype=torch.int32, device="cuda")
        q = torch.randn(333, H, d, device="cuda").bfloat16()
        assert (fa.fwd_paged_workspace_size(3, 300, H, 2, d) > 0) == (H == 4)
        want = fa.fwd_paged(q, kc, vc, tb, sl, cu, 300)
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            fa.fwd_paged(q, kc, vc, tb, sl, cu, 300, out=o, lse=lse)
        for _ in range(5):
            o.zero_()
            graph.replay()
            again = fa.fwd_paged(q, kc, vc, tb, sl, cu, 300)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
        ok()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_prompt_in_parts_equals_the_whole(d, dtype):
    """Prompts appended and attended in two parts over pages, against fwd_varlen of the whole
    prompts with the same rotated keys; then the last token again as a decoding step."""
    fa = fa_()
    H, Hkv, page, t = 8, 2, 16, pu.DT[dtype]
    first, second = (200, 1, 64), (77, 130, 300)
    lens = [a + b for a, b in zip(first, second)]
    pool = pu.Pool(lens, Hkv, d, page, dtype, fill=float("nan"))
    pool.store.fill_(float("nan"))
    kc, vc, tb, _ = pool.cuda()
    g = torch.Generator().manual_seed(9)
    total = sum(lens)
    q, k, v = (torch.randn((total, n, d), generator=g).to(t).cuda() for n in (H, Hkv, Hkv))
    cs = fa.rope_table(1024, d)
    starts = [sum(lens[:i]) for i in range(4)]

    def cu(x):
        return torch.tensor([sum(x[:i]) for i in range(4)], dtype=torch.int32, device="cuda")

    o = torch.empty_like(q)
    lse = torch.empty(H, total, device="cuda")
    qr = torch.empty_like(q)
    done = [0, 0, 0]
    for part in (first, second):
        rows = torch.cat([torch.arange(s + a, s + a + n) for s, a, n in zip(starts, done, part)]).cuda()
        done = [a + n for a, n in zip(done, part)]
        sl = torch.tensor(done, dtype=torch.int32, device="cuda")
        qp = fa.append_paged(k[rows], v[rows], kc, vc, tb, sl, cu_seqlens=cu(part), cos_sin=cs,
                             q=q[rows])
        op, lp = fa.fwd_paged(qp, kc, vc, tb, sl, cu(part), max(part))
        o[rows], lse[:, rows], qr[rows] = op, lp, qp
    # the whole prompts, their rotated keys read back from the pages
    kr = torch.cat([pool_keys(kc, tb, b, n, page) for b, n in enumerate(lens)])
    want, lw = fa.fwd_varlen(qr, kr, v, cu(lens), max(lens))
    ok()
    assert (o.float() - want.float()).abs().max() <= 4 * pu.HALF[t] * want.float().abs().max()
    assert (lse - lw).abs().max() <= 1e-5
    last = torch.tensor([starts[i + 1] - 1 for i in range(3)], device="cuda")
    od, ld = fa.decode_paged(qr[last], kc, vc, tb, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ok()
    assert (o[last].float() - od.float()).abs().max() <= 4 * pu.HALF[t] * want.float().abs().max()
    assert (lse[:, last].t() - ld).abs().max() <= 1e-5


def pool_keys(kc, tb, b, n, page):
    j = torch.arange(n, device="cuda")
    return kc[tb[b].long()[j // page], :, j % page].contiguous()


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_generation_step_by_step(cache):
    """Prompts appended, then tokens one by one, each attended over what is cached: every step
    against the definition on the cache as it stands, in one captured graph per step."""
    fa = fa_()
    H, Hkv, d, page, dtype = 8, 2, 128, 16, torch.bfloat16
    prompts, steps = (30, 1, 47), 20
    B = len(prompts)
    pool = pu.Pool([n + steps for n in prompts], Hkv, d, page, "e4m3" if cache == "e4m3" else "bf16")
    kc, vc, tb, _ = pool.cuda()
    g = torch.Generator().manual_seed(3)
    cs = fa.rope_table(128, d)
    sl = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 30, 31, 78], dtype=torch.int32, device="cuda")

    def rnd(n, h):
        return torch.randn((n, h, d), generator=g).to(dtype).cuda()

    def append(*a, **kw):
        if cache == "e4m3":
            return fa.append_paged_fp8(*a, *pool.scales, cos_sin=cs, **kw)
        return fa.append_paged(*a, cos_sin=cs, **kw)

    append(rnd(78, Hkv), rnd(78, Hkv), kc, vc, tb, sl, cu_seqlens=cu)
    k, v, q = rnd(B, Hkv), rnd(B, Hkv), rnd(B, H)
    qo, o = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(B, H, device="cuda")
    ws = torch.empty(fa.decode_paged_workspace_size(H, Hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        sl.add_(1)
        append(k, v, kc, vc, tb, sl, q=q, q_out=qo)
        if cache == "e4m3":
            fa.decode_paged_fp8(qo, kc, vc, tb, sl, *pool.scales, out=o, lse=lse, workspace=ws)
        else:
            fa.decode_paged(qo, kc, vc, tb, sl, out=o, lse=lse, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    for i in range(steps):
        for x, h in ((k, Hkv), (v, Hkv), (q, H)):
            x.copy_(rnd(B, h))
        if i == 2:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(graph, stream=side):
                step()
        step() if i < 2 else graph.replay()
        ok()
        pool.kc, pool.vc = kc.cpu(), vc.cpu()
        pool.lens = sl.tolist()
        assert pool.lens == [n + i + 1 for n in prompts]
        for b in range(B):
            ref = pu.reference(pool, qo[b:b + 1].cpu(), b, torch.tensor([pool.lens[b] - 1]),
                               1 / math.sqrt(d))
            pu.check_rows(o[b:b + 1], lse[b:b + 1], ref, dtype)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_pool_past_32_bit_offsets(cache):
    """Pages whose elements lie more than 2^32 from the pool's start: appended to, decoded from
    and attended by many tokens, beside the same work on a small pool."""
    fa = fa_()
    Hkv, page, d, H = 2, 64, 128, 8
    P = (1 << 32) // (Hkv * page * d) + 64
    t = torch.uint8 if cache == "e4m3" else torch.bfloat16
    big = [torch.empty(P, Hkv, page, d, dtype=t, device="cuda") for _ in range(2)]
    small = [torch.zeros(8, Hkv, page, d, dtype=t, device="cuda") for _ in range(2)]
    far = torch.arange(P - 8, P, dtype=torch.int32, device="cuda").flip(0).view(2, 4)
    near = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    sl = torch.tensor([250, 100], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 250, 350], dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn(350, n, d, device="cuda").bfloat16() for n in (Hkv, Hkv, H))
    cs = fa.rope_table(256, d)
    got = []
    for (kc, vc), tb in ((big, far), (small, near)):
        if cache == "e4m3":
            qo = fa.append_paged_fp8(k, v, kc, vc, tb, sl, 0.01, 0.01, cu_seqlens=cu, cos_sin=cs, q=q)
            o = fa.decode_paged_fp8(qo[[249, 349]], kc, vc, tb, sl, 0.01, 0.01)
        else:
            qo = fa.append_paged(k, v, kc, vc, tb, sl, cu_seqlens=cu, cos_sin=cs, q=q)
            o = fa.decode_paged(qo[[249, 349]], kc, vc, tb, sl)
            o += fa.fwd_paged(qo, kc, vc, tb, sl, cu, 250)
        got.append((qo,) + o)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][1].isfinite().all()


def test_tables_and_lengths_seen_through_strides():
    # a table that is a slice of a wider one
    fa = fa_()
    pool = pu.Pool((300, 120, 33), 2, 64, 16, "fp16")
    kc, vc, tb, sl = pool.cuda()
    wide = torch.full((3, tb.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + tb.shape[1]] = tb
    q = torch.randn(3, 8, 64, device="cuda").half()
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    a, b = (fa.decode_paged(q, kc, vc, x, sl) + fa.fwd_paged(q, kc, vc, x, sl, cu, 1)
            for x in (tb, wide[:, 4:4 + tb.shape[1]]))
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_many_small_weights_add_up():
    """One key far above 100000 others whose weights are about 2^-26 each: together 0.2 % of the
    sum, which f16 weights of at most 1 would lose."""
    fa = fa_()
    for cache in ("16", "e4m3"):
        n, d = 100000, 128
        pages = -(-n // 64)
        t = torch.float16
        kc = torch.zeros(pages, 1, 64, d, dtype=t, device="cuda")
        vc = torch.zeros(pages, 1, 64, d, dtype=t, device="cuda")
        kc[0, 0, 0] = 1.0
        vc[1:] = 1.0
        q = torch.full((1, 1, d), 18.0 / d, dtype=t, device="cuda")
        tb = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
        sl = torch.tensor([n], dtype=torch.int32, device="cuda")
        one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        s = float(q.double().sum())
        if cache == "e4m3":
            kc, vc = (x.to(torch.float8_e4m3fn) for x in (kc, vc))
            got = [fa.decode_paged_fp8(q, kc, vc, tb, sl, 1.0, 1.0, scale=1.0)]
        else:
            got = [fa.decode_paged(q, kc, vc, tb, sl, scale=1.0),
                   fa.fwd_paged(q, kc, vc, tb, sl, one, 1, scale=1.0)]
        ok()
        want = (n - 64) / (math.exp(s) + n - 1)
        # the output's rounding, and each weight's: 2^-26 2^7 is f16's 2^-19, a multiple of 2^-24
        for o, lse in got:
            assert abs(float(o[0, 0, 0]) / want - 1) <= 2.0 ** -11 + 2.0 ** -10
            # the sum of 10^5 weights in fp32, and L's own roundings
            assert abs(float(lse.view(-1)[0]) - math.log(math.exp(s) + n - 1)) <= 1e-5


@pytest.mark.parametrize("n", [100, 5000])
def test_c_calls_that_allocate_their_workspace(n):
    """The C entry points with workspace NULL, where rows get a CTA each and where they are cut,
    against the Python calls."""
    fa = fa_()
    lib = fa.load_library()
    pool = pu.Pool((n, n // 2), 2, 64, 16, "fp16")
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(2, 8, 64, device="cuda").half()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    pc, _ = fa._paged(kc, vc, tb, sl, torch.float16, 2, 64)
    o, lse, o2, lse2 = (torch.empty_like(q), torch.empty(2, 8, device="cuda"), torch.empty_like(q),
                        torch.empty(8, 2, device="cuda"))
    st = torch.cuda.current_stream().cuda_stream
    assert lib.fa_decode_paged(q.data_ptr(), pc, o.data_ptr(), lse.data_ptr(), None, 0, 2, 8, 2, 64, 0,
                               0.125, 0, st) == 0
    assert lib.fa_fwd_paged(q.data_ptr(), pc, o2.data_ptr(), lse2.data_ptr(), None, 0, cu.data_ptr(),
                            2, 2, 1, 8, 2, 64, 1, 0, 0.125, 0, st) == 0
    want = fa.decode_paged(q, kc, vc, tb, sl) + fa.fwd_paged(q, kc, vc, tb, sl, cu, 1)
    ok()
    assert all(torch.equal(a, b) for a, b in zip((o, lse, o2, lse2), want))


def test_calls_on_two_streams():
    fa = fa_()
    pool = pu.Pool((3000, 2000), 2, 128, 64, "bf16")
    kc, vc, tb, sl = pool.cuda()
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    q2 = torch.randn(2, 8, 128, device="cuda").bfloat16()
    want, want2 = fa.decode_paged(q, kc, vc, tb, sl), fa.decode_paged(q2, kc, vc, tb, sl)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            a = fa.decode_paged(q, kc, vc, tb, sl)
        with torch.cuda.stream(s2):
            b = fa.decode_paged(q2, kc, vc, tb, sl)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a + b, want + want2))
    ok()
