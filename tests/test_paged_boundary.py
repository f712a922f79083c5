"""Paged caches on the host: the C entry points and the Python calls refuse invalid arguments
before any CUDA work.  No kernel is launched here."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
M = 0x1000000     # fake buffers 16 MiB apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_22_gb300 import build
    import exact_io_aware_22_gb300 as fa
    return fa.load_library(build.build())


def cache(**kw):
    import exact_io_aware_22_gb300 as fa
    a = dict(K=M, V=2 * M, page_table=3 * M, cache_seqlens=4 * M, page_stride=2 * 16 * 128,
             head_stride=16 * 128, row_stride=128, table_stride=32, pages=100, page_size=16,
             max_pages=32)
    a.update(kw)
    return fa._PagedCache(**a)


def decode(lib, fp8=False, pc=None, **kw):
    a = dict(Q=5 * M, O=6 * M, L=7 * M, ws=0, ws_bytes=0, B=3, H=8, Hkv=2, d=128, window=0,
             scale=0.1, ks=0.01, vs=0.01, dtype=1)
    a.update(kw)
    pc = cache() if pc is None else pc
    head = (a["Q"], ctypes.byref(pc) if pc else None, a["O"], a["L"], a["ws"], a["ws_bytes"], a["B"],
            a["H"], a["Hkv"], a["d"], a["window"], a["scale"])
    if fp8:
        return lib.fa_decode_paged_fp8(*head, a["ks"], a["vs"], a["dtype"], None)
    return lib.fa_decode_paged(*head, a["dtype"], None)


def append(lib, fp8=False, pc=None, **kw):
    a = dict(K=5 * M, ks=256, V=6 * M, vs=256, Q=7 * M, qs=1024, Qo=8 * M, cu=9 * M, pos=0, cs=10 * M,
             max_pos=64, rot=128, inter=0, B=3, T=10, H=8, Hkv=2, d=128, k_scale=0.01, v_scale=0.01,
             dtype=1)
    a.update(kw)
    pc = cache() if pc is None else pc
    head = [ctypes.byref(pc) if pc else None] + [a[n] for n in (
        "K", "ks", "V", "vs", "Q", "qs", "Qo", "cu", "pos", "cs", "max_pos", "rot", "inter", "B", "T",
        "H", "Hkv", "d")]
    if fp8:
        return lib.fa_append_paged_fp8(*head, a["k_scale"], a["v_scale"], a["dtype"], None)
    return lib.fa_append_paged(*head, a["dtype"], None)


CACHE = [
    (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(page_table=0), INVALID),
    (dict(cache_seqlens=0), INVALID), (dict(pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(table_stride=31), INVALID), (dict(max_pages=-1), INVALID),
    (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED),        # 2^31 keys
    (dict(table_stride=1 << 31), UNSUPPORTED),
    (dict(row_stride=64), INVALID), (dict(row_stride=-128), INVALID),
    (dict(row_stride=132), MISALIGNED), (dict(head_stride=16 * 128 + 4), MISALIGNED),
    (dict(page_stride=1 << 40), UNSUPPORTED), (dict(pages=2 ** 31 - 1, page_stride=1 << 38), UNSUPPORTED),
    (dict(head_stride=128), INVALID),                                     # heads over rows
    (dict(page_stride=16 * 128), INVALID),                                # pages over heads
    (dict(V=M), INVALID), (dict(V=M + 4096), INVALID),                    # the pools coincide
    (dict(V=M + 100 * 2 * 16 * 128 * 2 - 256), INVALID),                  # in their last row
    (dict(K=M + 8), MISALIGNED), (dict(V=2 * M + 2), MISALIGNED),
    (dict(page_table=3 * M + 2), MISALIGNED), (dict(cache_seqlens=4 * M + 1), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_rejects(lib, kw, code):
    assert decode(lib, pc=cache(**kw)) == code
    assert append(lib, pc=cache(**kw)) == code


def test_no_cache_rejects(lib):
    assert decode(lib, pc=False) == INVALID and append(lib, pc=False) == INVALID


def test_strides_of_single_entries_do_not_matter(lib):
    # page_size 1, one head: their strides may be anything; the outputs then decide (Q over O)
    pc = cache(page_size=1, row_stride=3, head_stride=0, page_stride=128)
    assert decode(lib, pc=pc, H=4, Hkv=1, O=5 * M) == INVALID
    assert decode(lib, pc=pc, H=4, Hkv=1, Q=5 * M + 8) == MISALIGNED


@pytest.mark.parametrize("kw,code", [
    (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(L=0), INVALID), (dict(B=0), INVALID),
    (dict(H=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(window=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(d=48), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(Q=5 * M + 8), MISALIGNED), (dict(L=7 * M + 2), MISALIGNED),
    (dict(ws=11 * M, ws_bytes=64), INVALID), (dict(ws=11 * M + 4, ws_bytes=1 << 30), MISALIGNED),
    (dict(O=5 * M), INVALID), (dict(O=M + 512), INVALID), (dict(L=2 * M), INVALID),
    (dict(O=3 * M), INVALID), (dict(L=4 * M), INVALID), (dict(L=6 * M + 16), INVALID),
    (dict(ws=6 * M, ws_bytes=1 << 30), INVALID), (dict(ws=2 * M, ws_bytes=1 << 30), INVALID),
    (dict(B=2 ** 31 - 1), UNSUPPORTED), (dict(H=4880, Hkv=1), UNSUPPORTED), (dict(scale=3e38), INVALID),
])
def test_decode_rejects(lib, kw, code):
    assert decode(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d=64), UNSUPPORTED), (dict(ks=0.0), INVALID), (dict(vs=float("inf")), INVALID),
    (dict(ks=-1.0), INVALID), (dict(vs=1e-45), INVALID), (dict(ks=1e-30, scale=1e-20), INVALID),
])
def test_decode_fp8_rejects(lib, kw, code):
    assert decode(lib, fp8=True, **kw) == code


def test_odd_pages_of_32_columns(lib):
    pc = cache(page_size=3, row_stride=32, head_stride=96, page_stride=192)
    assert decode(lib, pc=pc, d=32) == UNSUPPORTED


def test_workspace_size(lib):
    f = lib.fa_decode_paged_workspace_size
    # per CTA (152 x 3; 152 x 2 for groups of more than 8 heads) a header of 12 bytes and two
    # slots of 8 (16) states of d + 4 floats
    assert f(8, 2, 128) == 456 * (12 + 2 * 8 * 132 * 4)
    assert f(64, 4, 32) == 304 * (12 + 2 * 16 * 36 * 4)
    assert f(8, 3, 128) == 0 and f(8, 2, 48) == 0 and f(0, 1, 64) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(Q=0), INVALID), (dict(Qo=0), INVALID),
    (dict(T=0), INVALID), (dict(B=0), INVALID), (dict(Hkv=3), INVALID), (dict(inter=2), INVALID),
    (dict(cu=0), INVALID),                                                # T != B
    (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED),
    (dict(cs=0), INVALID), (dict(max_pos=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(ks=128), INVALID), (dict(vs=255), INVALID),
    (dict(qs=512), INVALID), (dict(ks=260), MISALIGNED), (dict(qs=1 << 31), UNSUPPORTED),
    (dict(K=5 * M + 8), MISALIGNED), (dict(Qo=8 * M + 2), MISALIGNED), (dict(cs=10 * M + 4), MISALIGNED),
    (dict(cu=9 * M + 2), MISALIGNED), (dict(pos=11 * M + 1), MISALIGNED),
    (dict(K=M + 512), INVALID), (dict(V=M), INVALID), (dict(cs=2 * M), INVALID),
    (dict(Qo=7 * M), INVALID), (dict(Qo=5 * M + 1024), INVALID), (dict(Qo=2 * M), INVALID),
    (dict(Qo=3 * M), INVALID), (dict(pos=8 * M + 64), INVALID),
])
def test_append_rejects(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d=64), UNSUPPORTED), (dict(k_scale=0.0), INVALID), (dict(v_scale=float("nan")), INVALID),
    (dict(k_scale=1e-45), INVALID),
])
def test_append_fp8_rejects(lib, kw, code):
    assert append(lib, fp8=True, **kw) == code


def fwd(lib, pc=None, **kw):
    a = dict(Q=5 * M, O=6 * M, L=7 * M, cu=8 * M, ws=0, ws_bytes=0, B=3, total=40, max_len=20, H=8,
             Hkv=2, d=128, causal=1, window=0, scale=0.1, dtype=1)
    a.update(kw)
    pc = cache() if pc is None else pc
    return lib.fa_fwd_paged(a["Q"], ctypes.byref(pc) if pc else None, a["O"], a["L"], a["ws"],
                            a["ws_bytes"], a["cu"], a["B"], a["total"], a["max_len"], a["H"], a["Hkv"], a["d"], a["causal"],
                            a["window"], a["scale"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", CACHE)
def test_fwd_cache_rejects(lib, kw, code):
    assert fwd(lib, pc=cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(L=0), INVALID), (dict(cu=0), INVALID),
    (dict(B=0), INVALID), (dict(total=0), INVALID), (dict(max_len=0), INVALID),
    (dict(max_len=(1 << 29) + 1), UNSUPPORTED), (dict(Hkv=3), INVALID), (dict(window=-1), INVALID),
    (dict(window=5, causal=0), INVALID), (dict(causal=2), INVALID), (dict(scale=-1.0), INVALID),
    (dict(d=16), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(Q=5 * M + 8), MISALIGNED),
    (dict(cu=8 * M + 2), MISALIGNED), (dict(L=7 * M + 1), MISALIGNED), (dict(O=5 * M + 4096), INVALID),
    (dict(O=M), INVALID), (dict(L=2 * M + 64), INVALID), (dict(O=3 * M), INVALID),
    (dict(L=4 * M), INVALID), (dict(L=8 * M), INVALID), (dict(L=6 * M + 64), INVALID),
    (dict(max_len=(1 << 27) + 1), UNSUPPORTED), (dict(B=1 << 30), UNSUPPORTED),
    (dict(scale=3e38), INVALID),
    (dict(ws=11 * M, ws_bytes=64), INVALID), (dict(ws=11 * M + 8, ws_bytes=1 << 30), MISALIGNED),
    (dict(ws=6 * M, ws_bytes=1 << 30), INVALID), (dict(ws=2 * M, ws_bytes=1 << 30), INVALID),
])
def test_fwd_rejects(lib, kw, code):
    assert fwd(lib, **kw) == code


def test_fwd_workspace_size(lib):
    f = lib.fa_fwd_paged_workspace_size
    # a header of 6 ints for each of 152 CTAs, and two tiles of 256 rows of 128 columns and a
    # logsumexp, in fp32; at d = 64 tiles of 128 rows, two CTAs on each SM
    ws = 152 * (24 + 2 * 256 * 129 * 4)
    assert f(3, 20, 8, 2, 128) == ws
    assert f(3, 40, 8, 2, 64) == 304 * (24 + 2 * 128 * 65 * 4)
    assert f(76, 64, 32, 8, 128) == ws and f(77, 64, 32, 8, 128) == 0     # four rounds of tiles
    assert f(1, 1216, 32, 8, 128) == ws and f(1, 1217, 32, 8, 128) == 0   # one, of long prompts
    assert f(3, 20, 8, 3, 128) == 0 and f(3, 0, 8, 2, 128) == 0


def test_fwd_without_cache_rejects(lib):
    assert fwd(lib, pc=False) == INVALID


def test_python_calls_refuse_cpu_tensors(lib):
    import exact_io_aware_22_gb300 as fa
    k = torch.zeros(2, 2, 64, dtype=torch.float16)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.append_paged(k, k, c, c.clone(), t, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_paged(k, c, c.clone(), t, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fwd_paged(k, c, c.clone(), t, n, n, 1)


@pytest.mark.parametrize("kw,what", [
    (dict(kc=torch.zeros(4, 2, 16, 32, dtype=torch.float16)), ValueError),
    (dict(kc=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)), TypeError),
    (dict(kc=torch.zeros(4, 16, 2, 64, dtype=torch.float16).transpose(1, 2)), ValueError),
    (dict(t=torch.zeros(2, 3, dtype=torch.int64)), ValueError),
    (dict(t=torch.zeros(3, 3, dtype=torch.int32)), ValueError),
    (dict(t=torch.zeros(3, 2, dtype=torch.int32).t()), ValueError),
    (dict(n=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(n=torch.zeros(2, dtype=torch.int64)), ValueError),
])
def test_python_cache_checks(kw, what):
    import exact_io_aware_22_gb300 as fa
    a = dict(kc=torch.zeros(4, 2, 16, 64, dtype=torch.float16),
             vc=torch.zeros(4, 2, 16, 64, dtype=torch.float16),
             t=torch.zeros(2, 3, dtype=torch.int32), n=torch.zeros(2, dtype=torch.int32))
    pc, Hkv = fa._paged(a["kc"], a["vc"], a["t"], a["n"], torch.float16, 2, 64)
    assert (Hkv, pc.pages, pc.page_size, pc.max_pages, pc.row_stride) == (2, 4, 16, 3, 64)
    a.update(kw)
    with pytest.raises(what):
        fa._paged(a["kc"], a["vc"], a["t"], a["n"], torch.float16, 2, 64)


@pytest.mark.parametrize("div", [1, 2, 3, 7, 16, 20, 24, 100, 127, 128, 1000, 65535, 2 ** 30])
def test_page_division(div):
    # the kernels' quotient by a page size, in its own arithmetic
    s = 0
    while (1 << s) < div:
        s += 1
    mul = ((1 << 32) * ((1 << s) - div)) // div + 1
    assert mul < 1 << 32
    for x in [0, 1, div - 1, div, div + 1, 2 ** 31 - 1, 2 ** 31 - 2] + \
            [k * div + e for k in (2, 1000, 2 ** 30 // div, (2 ** 31 - 1) // div) for e in (-1, 0, 1)]:
        if 0 <= x < 1 << 31:
            t = (x * mul >> 32) + x
            assert t < 1 << 32 and t >> s == x // div, (x, div)
