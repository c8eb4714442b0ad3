"""Refusals of the 8-bit linear-layer entry points: arguments are checked on
the host before any CUDA call, with the position of the first bad one."""
import pytest
import torch

import symmetric_matrix_vector_gb300 as xs
from symmetric_matrix_vector_gb300 import _build

P = 0x1000          # never dereferenced: the checks come first


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_quant(kind):
    f = getattr(xs, "xquant_" + kind)
    assert f(-1, 2, P, 4, P, 4, P, stream=0) == 1
    assert f(4, -1, P, 4, P, 4, P, stream=0) == 2
    assert f(4, 2, P, 3, P, 4, P, stream=0) == 4
    assert f(4, 2, P, 4, P, 3, P, stream=0) == 6
    assert f(0, 2, P, 0, P, 1, P, stream=0) == 4
    assert f(-1, -1, P, 0, P, 0, P, stream=0) == 1
    for a in ((None, 4, P, 4, P), (P, 4, None, 4, P), (P, 4, P, 4, None)):
        assert f(4, 2, *a, stream=0) == -4
    assert f(0, 2, P, 1, P, 1, P, stream=0) == 0
    assert f(4, 0, None, 4, None, 4, None, stream=0) == 0


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_dequant(kind):
    f = getattr(xs, "xdequant_" + kind)
    assert f(-1, 2, P, 4, P, P, 4, stream=0) == 1
    assert f(4, -1, P, 4, P, P, 4, stream=0) == 2
    assert f(4, 2, P, 3, P, P, 4, stream=0) == 4
    assert f(4, 2, P, 4, P, P, 3, stream=0) == 7
    for a in ((None, 4, P, P, 4), (P, 4, None, P, 4), (P, 4, P, None, 4)):
        assert f(4, 2, *a, stream=0) == -4
    assert f(4, 0, None, 4, None, None, 4, stream=0) == 0


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_rmsquant(kind):
    f = getattr(xs, "xrmsquant_" + kind)
    ok = dict(m=4, n=2, X=P, ldx=4, R=P, ldr=4, G=P, eps=1e-5, H=P, ldh=4, Q=P, ldq=4, scale=P,
              rstd=P)

    def call(**kw):
        return f(*{**ok, **kw}.values(), stream=0)

    assert call(m=-1) == 1 and call(n=-1) == 2 and call(ldx=3) == 4 and call(ldr=3) == 6
    assert call(eps=-1e-9) == 8 and call(eps=float("nan")) == 8
    assert call(ldh=3) == 10 and call(ldq=3) == 12
    assert call(ldr=3, ldq=0) == 6
    assert call(X=None) == -4 and call(Q=None) == -4 and call(scale=None) == -4
    # what is optional needs no leading dimension
    assert call(n=0, R=None, ldr=0, G=None, H=None, ldh=0, rstd=None) == 0
    assert call(m=0) == 0


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_rmsgrad(kind):
    f = getattr(xs, "xrmsgrad_" + kind)
    ok = dict(m=4, n=2, dY=P, lddy=4, H=P, ldh=4, G=P, rstd=P, dR=P, lddr=4, dX=P, lddx=4, dG=P)

    def call(**kw):
        return f(*{**ok, **kw}.values(), stream=0)

    assert call(m=-1) == 1 and call(n=-1) == 2 and call(lddy=3) == 4 and call(ldh=3) == 6
    assert call(lddr=3) == 10 and call(lddx=3) == 12
    for name in ("dY", "H", "rstd", "dX"):
        assert call(**{name: None}) == -4
    assert call(n=0, dR=None, lddr=0, dG=None) == 0
    assert call(m=0) == 0


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_gemmq(kind):
    f = getattr(xs, "xgemmq_" + kind)
    ok = dict(m=4, n=2, k=8, alpha=1.0, W=P, ldw=8, sw=P, X=P, ldx=8, sx=P, beta=0.0, Y=P, ldy=4)

    def call(**kw):
        return f(*{**ok, **kw}.values(), stream=0)

    assert call(m=-1) == 1 and call(n=-1) == 2 and call(k=-1) == 3
    assert call(ldw=7) == 6 and call(ldx=7) == 9 and call(ldy=3) == 13
    assert call(k=0, ldw=0) == 6 and call(ldw=0, ldy=0) == 6
    assert call(W=None) == -4 and call(X=None) == -4 and call(Y=None) == -4
    # quick returns touch nothing
    assert call(m=0) == 0 and call(n=0) == 0
    assert call(alpha=0.0, beta=1.0, W=None, X=None) == 0
    assert call(k=0, beta=1.0, W=None, X=None) == 0


def test_status_strings_cover_every_position():
    for st in (1, 2, 3, 4, 6, 7, 8, 9, 10, 12, 13):
        assert xs.xsymv_status_string(st).startswith("invalid argument %d" % st)


def test_kinds_and_tensors():
    with pytest.raises(ValueError):
        xs.quant("d", 4, 2, P, 4, P, 4, P)
    a = torch.zeros(4)
    with pytest.raises(ValueError):
        xs.xquant_s(4, 1, a, 4, P, 4, P, stream=0)


def test_sizes_beyond_the_largest():
    """indexes rounded up to whole blocks stay in 32 bits"""
    big = 0x7fff0001
    assert xs.xquant_b(big, 2, P, big, P, big, P, stream=0) == 1
    assert xs.xquant_b(4, big, P, 4, P, 4, P, stream=0) == 2
    assert xs.xdequant_b(big, 2, P, big, P, P, big, stream=0) == 1
    assert xs.xrmsquant_b(big, 2, P, big, None, 0, None, 0.0, None, 0, P, big, P, None,
                          stream=0) == 1
    assert xs.xrmsgrad_b(big, 2, P, big, P, big, None, P, None, 0, P, big, None, stream=0) == 1
    assert xs.xgemmq_b(big, 2, 4, 1.0, P, 4, None, P, 4, None, 0.0, P, big, stream=0) == 1
    assert xs.xgemmq_b(4, big, 4, 1.0, P, 4, None, P, 4, None, 0.0, P, 4, stream=0) == 2
    assert xs.xgemmq_b(4, 2, big, 1.0, P, big, None, P, big, None, 0.0, P, 4, stream=0) == 3
