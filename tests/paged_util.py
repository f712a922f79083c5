"""Paged caches for the tests: pools filled so that a read of anything not attended shows, the
definitions in 64 bits (plain torch on the CPU, one sequence and head at a time), and the
tolerances that the kernels' arithmetic allows.

Tolerances.  With u = 2^-24 (half an fp32 step, relative):
  scores     a product of d terms accumulated in fp32 by tensor-core steps of 16: every partial
             sum is off by at most one step (the units truncate), so a score s is off by at most
             (d / 16 + 16) 2u sum |q k|, and delta is scale times that, plus the roundings of
             the scaled score, 4u max |s|.
  p          relative error expm1(delta) + 2^-15 (the two 16-bit terms of P leave at most 2^-16
             of it, the exponential 2^-21).
  O          |error| <= half a step of the output type + W (2 delta + 2^-15 + (n / 16 + 16) 2u),
             W = sum p |v| / sum p: numerator and denominator share p's relative error at
             worst with opposite signs, and both sums run over n keys in steps of 16.  Where P
             is rounded to 16 bits once (the many-token forward), 2^-15 becomes that half step.
  L          delta + (n / 16 + 16) 2u + 2^-20 + 8u max |s|: the sum's relative error, the
             logarithm's, and the roundings of m and of the final product.
"""
import math

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
U = 2.0 ** -24


def e4m3(codes):
    return codes.cpu().view(torch.uint8).view(torch.float8_e4m3fn).double()


class Pool:
    """A paged cache on the CPU and, through ``cuda``, on the GPU.

    layout: "hnd" (pages, Hkv, page, d), "nhd" (pages, page, Hkv, d) seen transposed,
    "pair" K and V as halves of one (pages, 2, Hkv, page, d) tensor."""

    def __init__(self, lens, Hkv, d, page, dtype, layout="hnd", width=None, extra=3, seed=0,
                 fill=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.d, self.page, self.dtype = list(lens), Hkv, d, page, dtype
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + extra
        self.width = max(max(need), 1) if width is None else width
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), self.width), 2 ** 30, dtype=torch.int32)   # unused: out of range
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        P, eight = self.pages, dtype == "e4m3"
        t = torch.uint8 if eight else DT[dtype]
        shape = (P, 2, Hkv, page, d) if layout == "pair" else \
            (2, P, page, Hkv, d) if layout == "nhd" else (2, P, Hkv, page, d)
        self.store = torch.full(shape, 0x7F if eight else fill, dtype=t)
        self.layout = layout
        self.kc, self.vc = self._views(self.store)
        self.scales = (0.0133, 0.0121) if eight else (1.0, 1.0)
        for b, n in enumerate(lens):
            for j0 in range(0, n, page):
                m, p = min(page, n - j0), int(self.table[b, j0 // page])
                for c, sc in ((self.kc, self.scales[0]), (self.vc, self.scales[1])):
                    x = torch.randn((Hkv, m, d), generator=g)
                    if eight:
                        x = (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    c[p, :, :m] = x.to(t)

    def _views(self, s):
        if self.layout == "pair":
            return s[:, 0], s[:, 1]
        if self.layout == "nhd":
            return s[0].transpose(1, 2), s[1].transpose(1, 2)
        return s[0], s[1]

    def cuda(self):
        s = self.store.cuda()
        k, v = self._views(s)
        return (k, v, self.table.cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def keys(self, b, name, lo, hi, table=None):
        """(Hkv, hi - lo, d) fp64 keys or values and which of them exist."""
        c, t = (self.kc if name == "k" else self.vc), (self.table if table is None else table)[b]
        out = torch.zeros((self.Hkv, hi - lo, self.d), dtype=torch.float64)
        have = torch.zeros(hi - lo, dtype=torch.bool)
        for j in range(lo, hi):
            p = int(t[j // self.page])
            if 0 <= p < self.pages:
                x = c[p, :, j % self.page]
                out[:, j - lo] = (e4m3(x) * self.scales[0 if name == "k" else 1]
                                  if self.dtype == "e4m3" else x.double())
                have[j - lo] = True
        return out, have


def reference(pool, q, b, at, scale, causal=True, window=0, table=None):
    """Attention of queries q (m, H, d) of sequence b at key positions ``at``: O, L (m, H), and
    W, delta, max |s| and the number of keys for the tolerances."""
    n, (m, H, d) = min(pool.lens[b], pool.width * pool.page), q.shape
    k, have = pool.keys(b, "k", 0, n, table)
    v, _ = pool.keys(b, "v", 0, n, table)
    q = q.double()
    j = torch.arange(n)
    allowed = have[None].expand(m, n).clone()
    if causal:
        allowed &= j[None] <= at[:, None]
    if window:
        allowed &= j[None] > at[:, None] - window
    o, lse = torch.zeros((m, H, d), dtype=torch.float64), torch.full((m, H), -math.inf, dtype=torch.float64)
    W, delta, smax = torch.zeros_like(o), torch.zeros_like(lse), torch.zeros_like(lse)
    for h in range(H):
        kh, vh = k[h // (H // pool.Hkv)], v[h // (H // pool.Hkv)]
        s = (q[:, h] @ kh.t()) * scale
        mag = (q[:, h].abs() @ kh.abs().t()) * scale
        s, mag = s.masked_fill(~allowed, -math.inf), mag.masked_fill(~allowed, 0.0)
        some = allowed.any(1)
        if not some.any():
            continue
        top = s[some].amax(1, keepdim=True)
        p = (s[some] - top).exp()
        z = p.sum(1, keepdim=True)
        o[some, h], W[some, h] = (p / z) @ vh, (p / z) @ vh.abs()
        lse[some, h] = (top + z.log())[:, 0]
        smax[some, h] = s[some].abs().masked_fill(~allowed[some], 0.0).amax(1)
        delta[some, h] = mag[some].amax(1) * (d / 16 + 16) * 2 * U + 4 * U * smax[some, h]
    return o, lse, W, delta, smax, n


def check_rows(o, lse, ref, dtype, p_half=2.0 ** -15):
    """Kernel rows o (m, H, d), lse (m, H) against ``reference``'s answer."""
    ro, rl, W, delta, smax, n = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    empty = rl == -math.inf
    assert (lse[empty] == -math.inf).all() and (o[empty] == 0).all(), "a row without keys"
    assert torch.isfinite(o).all(), "non-finite O: something not attended was read"
    assert torch.isfinite(lse[~empty]).all()
    steps = (n / 16 + 16) * 2 * U
    tol = HALF[dtype] * ro.abs() + W * (2 * delta[..., None] + p_half + steps) + TINY[dtype]
    over = ((o - ro).abs() / tol)
    tl = delta + steps + 2.0 ** -20 + 8 * U * smax
    lover = ((lse - rl).abs() / tl)[~empty]
    assert over.max() <= 1, f"O: {float(over.max()):.3g} times the tolerance"
    assert lover.numel() == 0 or lover.max() <= 1, f"L: {float(lover.max()):.3g} times the tolerance"
    return float(over.max()), float(lover.max()) if lover.numel() else 0.0


def turn(x, cs, r, interleaved):
    """Rotation in 64 bits of x (T, heads, d) by table rows cs (T, r), and its terms' magnitude."""
    x = x.double()
    y, mag = x.clone(), x.abs()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = cs[:, i, None].double(), cs[:, r // 2 + i, None].double()
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def check_turned(got, want, mag, dtype):
    """One rounding of fp32 arithmetic: two products and a sum, each half a step off."""
    err = (got.double().cpu() - want).abs()
    tol = HALF[dtype] * want.abs() + 4 * U * mag + TINY[dtype]
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} times the tolerance"


def check_codes(got, want, mag):
    """E4M3: half a step relative, or half the subnormal step, of the value in scale units."""
    want = want.clamp(-448, 448)
    err = (e4m3(got) - want).abs()
    tol = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10)) + 8 * U * mag
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} times the tolerance"


def np_rng(seed):
    return np.random.default_rng(seed)
