"""Scales of E4M3 values at the ends of fp32's range: v_scale is applied to the row's mean of the codes,
which is at most 448, and not to what it is formed from."""
import pytest
import torch

from tests.test_paged_edges import ints


def pools(n, page, key_code, value_codes):
    """K of one code and V of the given values in a pool whose pages lie in order."""
    pages = -(-n // page)
    kc = torch.full((pages * page, 128), float(key_code), device="cuda")
    vc = torch.zeros(pages * page, 128, device="cuda")
    vc[:n] = value_codes[:, None]
    kc, vc = (x.to(torch.float8_e4m3fn).view(pages, 1, page, 128) for x in (kc, vc))
    return kc, vc, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [5, 5000])      # keys split over the CTAs, and tiles whole
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_smallest_value_scale(rows, dtype):
    import exact_io_aware_22_gb300 as fa
    n = 20000
    codes = torch.full((n,), 448.0, device="cuda")
    kc, vc, tb = pools(n, 64, 1.0, codes)
    q = torch.zeros(rows, 8, 128, device="cuda", dtype=dtype)
    for v_scale in (2.0 ** -126, 2.0 ** -122, 2.0 ** -13):
        o, lse = fa.fwd_paged_fp8(q, kc, vc, tb, ints([n]), ints([0, rows]), rows, 1.0, v_scale, causal=False)
        torch.cuda.synchronize()
        assert fa.device_status() == 0
        # equal weights of equal values: the output's rounding alone (fp16: to nothing below 2^-24), and
        # two of fp32
        want = torch.tensor(448.0 * v_scale, dtype=torch.float64)
        half = torch.finfo(dtype).eps / 2
        tol = max(half * float(want), 2.0 ** -25 if dtype == torch.float16 else 0.0) + 2.0 ** -22 * float(want)
        assert float((o.double().cpu() - want).abs().max()) <= tol, v_scale
        assert (lse - torch.tensor(float(n)).log()).abs().max() < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 5000])
def test_values_that_overflow_and_cancel(rows):
    """Keys of +448 and then of -416 times 2^120: parts of the keys have means beyond fp32, all of them
    16 * 2^120."""
    import exact_io_aware_22_gb300 as fa
    n = 40960
    codes = torch.full((n,), 448.0, device="cuda")
    codes[n // 2:] = -416.0
    kc, vc, tb = pools(n, 64, 1.0, codes)
    q = torch.zeros(rows, 8, 128, device="cuda", dtype=torch.bfloat16)
    o, _ = fa.fwd_paged_fp8(q, kc, vc, tb, ints([n]), ints([0, rows]), rows, 1.0, 2.0 ** 120, causal=False)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    # fp32 sums of n terms in tensor-core steps of 16, each off by a step of the largest partial sum (448)
    tol = 2.0 ** 120 * (2.0 ** -8 * 16 + 448 * (n / 16 + 16) * 2.0 ** -23)
    assert o.isfinite().all() and float((o.double() - 2.0 ** 124).abs().max()) <= tol
