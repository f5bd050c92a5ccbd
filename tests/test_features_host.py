"""Operators on feature rows without a GPU: refusals on the host before any
launch, and the 64-bit references' own gradient against differences."""
import ctypes

import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

P = ctypes.c_void_p(4096)  # never read: every call below is refused, or has no rows


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


NORM = dict(x=P, xs=8, r=None, rs=0, w=P, wdt=0, rows=4, c=8, dt=0, eps=1e-6, sum=None, o1=P, o2=P)


def _norm(lib, fn, **kw):
    a = {**NORM, **kw}
    return getattr(lib, fn)(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["wdt"], a["rows"], a["c"], a["dt"], a["eps"],
                            a["sum"], a["o1"], a["o2"], None)


@pytest.mark.parametrize("fn", ["tc_rms_norm", "tc_rms_norm_i8"])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(rows=-1), 1), (dict(c=0), 1), (dict(c=-3), 1), (dict(dt=3), 1), (dict(dt=-1), 1),
    (dict(wdt=2), 1), (dict(dt=1, wdt=2), 1), (dict(xs=-1), 1), (dict(r=P, rs=-8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(o1=None), 1), (dict(c=(1 << 20) + 1), 5),
])
def test_norm_refusals(lib, fn, kw, status):
    assert _norm(lib, fn, **kw) == status
    assert lib.tc_last_error()


def test_norm_i8_needs_its_scale(lib):
    assert _norm(lib, "tc_rms_norm_i8", o2=None) == 1


@pytest.mark.parametrize("fn", ["tc_rms_norm", "tc_rms_norm_i8"])
def test_norm_without_rows_is_nothing(lib, fn):
    assert _norm(lib, fn, rows=0, x=None, o1=None, o2=None) == 0


GRAD = dict(dy=P, dys=8, dh=None, dhs=0, h=P, hs=8, w=P, wdt=0, rstd=P, rows=4, c=8, dt=0, dx=P, dw=P, ws=P, wsb=None)


def _grad(lib, **kw):
    a = {**GRAD, **kw}
    nb = a["wsb"] if a["wsb"] is not None else lib.tc_rms_norm_backward_workspace(max(a["rows"], 0), max(a["c"], 1))
    return lib.tc_rms_norm_backward(a["dy"], a["dys"], a["dh"], a["dhs"], a["h"], a["hs"], a["w"], a["wdt"], a["rstd"],
                                    a["rows"], a["c"], a["dt"], a["dx"], a["dw"], a["ws"], nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(h=None), 1), (dict(rstd=None), 1), (dict(dx=None, dw=None), 1), (dict(dys=-1), 1),
    (dict(hs=-1), 1), (dict(dh=P, dhs=-1), 1), (dict(rows=-1), 1), (dict(c=0), 1), (dict(dt=7), 1), (dict(wdt=1), 1),
    (dict(ws=None), 1), (dict(wsb=0), 1), (dict(wsb=-1), 1), (dict(ws=ctypes.c_void_p(4100)), 1),
    (dict(c=(1 << 20) + 1), 5),
])
def test_norm_grad_refusals(lib, kw, status):
    assert _grad(lib, **kw) == status
    assert lib.tc_last_error()


def test_norm_grad_workspace(lib):
    assert lib.tc_rms_norm_backward_workspace(-1, 8) == 0
    assert lib.tc_rms_norm_backward_workspace(8, 0) == 0
    assert lib.tc_rms_norm_backward_workspace(8, (1 << 20) + 1) == 0
    assert lib.tc_rms_norm_backward_workspace(0, 8) >= 0
    assert lib.tc_rms_norm_backward_workspace(1000, 64) > 0


MM = dict(x=P, xst=8, xs=P, w=P, wst=8, ws=P, b=None, rows=4, n=8, k=8, dt=2, out=P, ost=8)


def _mm(lib, **kw):
    a = {**MM, **kw}
    return lib.tc_matmul_i8(a["x"], a["xst"], a["xs"], a["w"], a["wst"], a["ws"], a["b"], a["rows"], a["n"], a["k"],
                            a["dt"], a["out"], a["ost"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(xs=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(out=None), 1),
    (dict(rows=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(dt=3), 1), (dict(xst=-1), 1), (dict(wst=-1), 1),
    (dict(ost=7), 1), (dict(k=131072), 5), (dict(n=(1 << 20) + 1, ost=1 << 21), 5),
])
def test_matmul_refusals(lib, kw, status):
    assert _mm(lib, **kw) == status
    assert lib.tc_last_error()


def test_matmul_without_rows_is_nothing(lib):
    assert _mm(lib, rows=0, x=None, xs=None, out=None) == 0


CONV = dict(x=P, xst=8, xs=P, nsrc=4, m=P, ndst=4, taps=27, w=P, ws=P, b=None, n=8, k=8, dt=2, out=P, ost=8)


def _conv(lib, **kw):
    a = {**CONV, **kw}
    return lib.tc_sparse_conv_i8(a["x"], a["xst"], a["xs"], a["nsrc"], a["m"], a["ndst"], a["taps"], a["w"], a["ws"],
                                 a["b"], a["n"], a["k"], a["dt"], a["out"], a["ost"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(xs=None), 1), (dict(m=None), 1), (dict(w=None), 1), (dict(ws=None), 1),
    (dict(out=None), 1), (dict(nsrc=-1), 1), (dict(ndst=-1), 1), (dict(taps=0), 1), (dict(taps=513), 1),
    (dict(n=0), 1), (dict(k=0), 1), (dict(dt=9), 1), (dict(xst=-1), 1), (dict(ost=7), 1), (dict(k=131072), 5),
    (dict(nsrc=1 << 31), 5),
])
def test_conv_refusals(lib, kw, status):
    assert _conv(lib, **kw) == status
    assert lib.tc_last_error()


def test_conv_without_rows_is_nothing(lib):
    assert _conv(lib, ndst=0, m=None, out=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: binding.tc_rms_norm(x), lambda: binding.tc_rms_norm_i8(x),
                 lambda: binding.tc_rms_norm_backward(x, x, None, s), lambda: binding.tc_matmul_i8(q, s, q, s),
                 lambda: binding.tc_sparse_conv_i8(q, s, torch.zeros(4, 1, dtype=torch.int32), q[None], s)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("c", [1, 2, 7, 33])
def test_reference_gradient_against_differences(c):
    """Central differences of sum(out * dy) + sum(h * dh) in 64 bits: off by O(step^2) and by 1e-16 / step."""
    gen = torch.Generator().manual_seed(c)
    h = torch.randn(5, c, generator=gen, dtype=torch.float64)
    w, dy, dh = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((c,), (5, c), (5, c)))
    eps = 0.5  # keeps the third derivatives of order one

    def loss(h, w):
        return (ref.rms_norm(h, w, eps)[0] * dy).sum() + (h * dh).sum()

    _, s = ref.rms_norm(h, w, eps)
    dx, dw, _, _ = ref.rms_norm_grad(dy, h, w, s, dh)
    step = 1e-5
    for i in range(5):
        for j in range(c):
            e = torch.zeros_like(h)
            e[i, j] = step
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dx[i, j]) < 1e-7
    for j in range(c):
        e = torch.zeros_like(w)
        e[j] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[j]) < 1e-7
