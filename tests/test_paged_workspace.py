"""fwd_paged's workspace on the GPU: what a call finds in it, what a call before left in it, and
calls whose tiles stay whole although their table would let them be cut, alone and beside other
work.  Every row is compared with the definition in 64 bits (tests/paged_util.py)."""
import math

import pytest
import torch

from tests import paged_util as pu

pytestmark = pytest.mark.gpu

KINDS = [(32, "bf16"), (64, "fp16"), (64, "bf16"), (128, "bf16")]
IDS = [f"d{d}-{t}" for d, t in KINDS]


class Call:
    """fwd_paged of new[b] tokens at the end of lens[b] keys, and its answer by definition."""

    def __init__(self, new, lens, H, Hkv, d, dtype, page=16, width=None, window=0, seed=0):
        import exact_io_aware_22_gb300 as fa
        self.fa, self.new, self.H, self.Hkv, self.d, self.t = fa, list(new), H, Hkv, d, pu.DT[dtype]
        self.window, self.most, self.total = window, max(new), sum(new)
        self.pool = pu.Pool(lens, Hkv, d, page, dtype, width=width, seed=seed)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn((self.total, H, d), generator=g).to(self.t)
        self.starts = [sum(new[:i]) for i in range(len(new) + 1)]
        self.args = (self.q.cuda(), *self.pool.cuda(),
                     torch.tensor(self.starts, dtype=torch.int32, device="cuda"), self.most)
        self.ws_bytes = fa.fwd_paged_workspace_size(len(new), self.most, H, Hkv, d)
        assert self.ws_bytes > 0, "not a call that may be cut"
        self.refs = [pu.reference(self.pool, self.q[c:c + m], b, torch.arange(n - m, n),
                                  1 / math.sqrt(d), window=window)
                     for b, (c, m, n) in enumerate(zip(self.starts, new, lens)) if m]

    def __call__(self, workspace=None):
        o = torch.full((self.total, self.H, self.d), 7.0, dtype=self.t, device="cuda")
        lse = torch.full((self.H, self.total), 7.0, device="cuda")
        return self.fa.fwd_paged(*self.args, window=self.window, out=o, lse=lse, workspace=workspace)

    def check(self, o, lse):
        rows = [(c, m) for c, m in zip(self.starts, self.new) if m]
        for (c, m), ref in zip(rows, self.refs):
            pu.check_rows(o[c:c + m], lse[:, c:c + m].t(), ref, self.t, p_half=pu.HALF[self.t])

    def foreign_workspace(self):
        """A workspace in which every range but the first holds a header of a cut tile that lies
        inside this call's rows, pieces of 9.0 and logsumexps of 0: joined, they would show as
        wrong rows of O, and nothing outside O would be touched."""
        rows, ranges = (256, 152) if self.d == 128 else (128, 304)
        pack = 0
        while pack < 7 and self.H // self.Hkv % (2 << pack) == 0:
            pack += 1
        ws = torch.zeros(self.ws_bytes // 4, dtype=torch.float32, device="cuda")
        parts = 2 * ranges * rows * self.d
        assert ws.numel() == 6 * ranges + parts + 2 * ranges * rows
        ws[6 * ranges:6 * ranges + parts] = 9.0
        have = [(c, m) for c, m in zip(self.starts, self.new) if m]
        head = torch.zeros((ranges, 6), dtype=torch.int32)
        head[0, 0] = 1                             # as of a call that was cut
        for x in range(1, ranges):
            c, m = have[x % len(have)]
            head[x] = torch.tensor([c, 0, 0, min(m << pack, rows), x - 1, x])
        ws[:6 * ranges] = head.flatten().view(torch.float32).cuda()
        return ws


def ok(fa):
    torch.cuda.synchronize()
    assert fa.device_status() == 0


# some sequences without new tokens, one without keys, one with more tokens than keys
NEW, LENS = (5, 0, 33, 1, 0, 4, 20, 64), (37, 90, 33, 200, 0, 0, 12, 300)


@pytest.mark.parametrize("d,dtype", KINDS, ids=IDS)
def test_fwd_with_a_table_much_wider_than_the_lengths(d, dtype):
    c = Call(NEW, LENS, 8, 2, d, dtype, width=4096)
    c.check(*c())
    ok(c.fa)


@pytest.mark.parametrize("d,dtype", KINDS, ids=IDS)
def test_fwd_headers_of_another_call_in_the_workspace(d, dtype):
    c = Call(NEW, LENS, 8, 2, d, dtype, width=4096)
    want = c()
    ws = c.foreign_workspace()
    got = c(ws)
    ok(c.fa)
    c.check(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d,dtype", KINDS, ids=IDS)
def test_fwd_whole_after_cut_in_one_workspace(d, dtype):
    # the long call is cut and leaves its headers; the short ones that follow are not
    cut = Call((5, 3, 1), (9000, 40, 700), 8, 2, d, dtype)
    short = Call(NEW, LENS, 8, 2, d, dtype, width=4096, seed=5)
    ws = torch.full((max(cut.ws_bytes, short.ws_bytes),), 255, dtype=torch.uint8, device="cuda")
    fresh = cut(), short()
    for _ in range(3):
        a, b = cut(ws), short(ws)
        ok(cut.fa)
        for got, want in ((a, fresh[0]), (b, fresh[1])):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    cut.check(*fresh[0])
    short.check(*fresh[1])


@pytest.mark.parametrize("d,dtype", KINDS, ids=IDS)
def test_fwd_beside_decode_on_another_stream(d, dtype):
    """Tiles stay whole, and not all CTAs start at once: decode calls hold part of the SMs.  The
    workspace holds another call's headers before every call."""
    # 9 tokens of 32 heads, 4 to a K/V head, in tiles of their own: more tiles than the 304 CTAs
    many = Call(tuple(0 if i % 5 == 1 else 1 + i % 9 for i in range(48)),
                tuple((37 * i) % 150 for i in range(48)), 32, 8, d, dtype, width=4096)
    few = Call(NEW, LENS, 8, 2, d, dtype, width=4096, seed=5)
    fa = few.fa
    B, H, Hkv, page, n = 32, 32, 8, 64, 4096
    kc, vc = (torch.randn(B * n // page, Hkv, page, 128, device="cuda").bfloat16() for _ in range(2))
    tb = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    sl = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, 128, device="cuda").bfloat16()
    want_d = fa.decode_paged(q, kc, vc, tb, sl)
    calls = [(c, c(), c.foreign_workspace(), torch.empty(c.ws_bytes // 4, device="cuda"))
             for c in (many, few)]
    for c, want, _, _ in calls:
        c.check(*want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            got_d = [fa.decode_paged(q, kc, vc, tb, sl) for _ in range(6)]
        got = []
        for _ in range(3):
            for c, want, foreign, ws in calls:
                ws.copy_(foreign)
                got.append((c(ws), want))
        torch.cuda.synchronize()
        for a, b in got + [(x, want_d) for x in got_d]:
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    ok(fa)
