"""Largest sizes and strides that the calls with norms and rotation take, and the first that they refuse,
on the host: no kernel is launched here."""
import pytest
import torch

from tests.test_norm_rope_boundary import INVALID, MISALIGNED, UNSUPPORTED, append_norm, call, lib, passes_checks, view  # noqa: F401
from tests.test_paged_boundary import append

D, G = 128, 1 << 44                              # fake buffers 16 TiB apart, never dereferenced


def far(i, heads=8, **kw):
    return view(i * G, heads, **kw)


def heads_of(q, k, N, **kw):
    """Packed (N, heads, d) views of q and k heads, all buffers far apart."""
    row = lambda i, h: far(i, h, row_stride=h * D, batch_stride=0)  # noqa: E731
    a = dict(q=row(1, q), k=row(2, k), qo=row(3, q), ko=row(4, k), gq=row(5, q), gk=row(6, k), B=1, N=N)
    a.update(kw)
    return a


MOST = [
    dict(q=far(9, batch_stride=(1 << 39) - 8)),
    dict(qo=far(9, batch_stride=(1 << 39) - 8), ko=far(10, 2, batch_stride=(1 << 39) - 8)),
    dict(B=128, q=far(9, batch_stride=(1 << 39) - 8)),                       # 127 * 2^39 elements
    dict(pos=14 << 24, pos_stride=(1 << 40) - 1),
    heads_of(2047, 1, 1 << 20), heads_of(1, 2047, 1 << 20), heads_of(1, 1, 2 ** 31 - 1),
]
TOO_MUCH = [
    dict(q=far(9, batch_stride=1 << 39)), dict(qo=far(9, batch_stride=1 << 39)),
    dict(B=130, q=far(9, batch_stride=(1 << 39) - 8)),                       # 129 * 2^39
    dict(heads_of(8, 2, 1 << 26), q=far(9, row_stride=1 << 21)),               # along the rows
    dict(pos=14 << 24, pos_stride=1 << 40),
    heads_of(2048, 1, 1 << 20), heads_of(1, 2048, 1 << 20), heads_of(3, 1, 1 << 30),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers")
@pytest.mark.parametrize("kw", MOST)
def test_largest_sizes_are_taken(lib, kw):  # noqa: F811
    assert passes_checks(call(lib, **kw))
    if "q" not in kw or kw["q"].data != 9 * G:   # the gradient's views are those of the outputs
        assert passes_checks(call(lib, True, **kw))


@pytest.mark.parametrize("kw", TOO_MUCH)
def test_larger_sizes_are_refused(lib, kw):  # noqa: F811
    assert call(lib, **kw) == UNSUPPORTED
    assert call(lib, True, **kw) == UNSUPPORTED


def tokens(T, H, Hkv, **kw):
    a = dict(K=G, ks=Hkv * D, V=2 * G, vs=Hkv * D, Q=3 * G, qs=H * D, Qo=4 * G, T=T, H=H, Hkv=Hkv)
    a.update(kw)
    return a


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers")
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [tokens(1 << 20, 2046, 2), tokens((1 << 30) - 1, 4, 2, Q=0, Qo=0)])
def test_largest_appends_are_taken(lib, fp8, kw):  # noqa: F811
    kw = dict(kw)
    assert passes_checks(append_norm(lib, fp8, **kw)) and passes_checks(append(lib, fp8, **kw))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [tokens(1 << 20, 2048, 2), tokens(1 << 30, 4, 2, Q=0, Qo=0),
                                tokens(1 << 30, 2, 2)])
def test_larger_appends_are_refused(lib, fp8, kw):  # noqa: F811
    assert append_norm(lib, fp8, **dict(kw)) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(dqw=10 << 24 | 2), MISALIGNED), (dict(ws=12 << 24 | 4), MISALIGNED),
    (dict(dkw=12 << 24), INVALID), (dict(ws=3 << 24), INVALID), (dict(dqw=9 << 24), INVALID),
    (dict(dqw=5 << 24), INVALID),
])
def test_gradients_of_weights_and_workspace(lib, kw, code):  # noqa: F811
    assert call(lib, True, **kw) == code
