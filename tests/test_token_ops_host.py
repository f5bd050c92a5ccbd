"""Layer norm, rotary positions and 4-bit rows without a GPU: refusals on the host before any launch, and the 64-bit
references against differences and by themselves."""
import ctypes

import pytest
import torch

from tests import token_ref as ref
from topology_construction_amd import binding

P = ctypes.c_void_p(4096)  # never read: every call below is refused, or has no rows


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


NORM = dict(x=P, xs=8, r=None, rs=0, w=P, wdt=0, b=P, bdt=0, rows=4, c=8, dt=0, eps=1e-5, sum=None, out=P, mean=P, rstd=P)


def _norm(lib, **kw):
    a = {**NORM, **kw}
    return lib.tc_layer_norm(*[a[k] for k in NORM], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(rows=-1), 1), (dict(c=0), 1), (dict(c=-3), 1), (dict(dt=3), 1), (dict(dt=-1), 1),
    (dict(wdt=2), 1), (dict(dt=1, wdt=2), 1), (dict(bdt=1), 1), (dict(dt=2, bdt=1), 1), (dict(xs=-1), 1),
    (dict(r=P, rs=-8), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(out=None), 1), (dict(c=(1 << 20) + 1), 5),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert lib.tc_last_error()


def test_norm_without_rows_is_nothing(lib):
    assert _norm(lib, rows=0, x=None, out=None, mean=None, rstd=None) == 0


GRAD = dict(dy=P, dys=8, dh=None, dhs=0, h=P, hs=8, w=P, wdt=0, mean=P, rstd=P, rows=4, c=8, dt=0, dx=P, dw=P, db=P, ws=P,
            wsb=None)


def _grad(lib, **kw):
    a = {**GRAD, **kw}
    if a["wsb"] is None:
        a["wsb"] = lib.tc_layer_norm_backward_workspace(max(a["rows"], 0), max(a["c"], 1))
    return lib.tc_layer_norm_backward(*[a[k] for k in GRAD], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(h=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dx=None, dw=None, db=None), 1),
    (dict(dys=-1), 1), (dict(hs=-1), 1), (dict(dh=P, dhs=-1), 1), (dict(rows=-1), 1), (dict(c=0), 1), (dict(dt=7), 1),
    (dict(wdt=1), 1), (dict(ws=None), 1), (dict(wsb=0), 1), (dict(wsb=-1), 1), (dict(ws=ctypes.c_void_p(4100)), 1),
    (dict(dw=None, wsb=0), 1), (dict(db=None, ws=None), 1), (dict(c=(1 << 20) + 1), 5),
])
def test_norm_grad_refusals(lib, kw, status):
    assert _grad(lib, **kw) == status
    assert lib.tc_last_error()


def test_norm_grad_workspace(lib):
    f = lib.tc_layer_norm_backward_workspace
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(8, (1 << 20) + 1) == 0
    assert f(0, 8) >= 0 and f(1000, 64) > 0 and f(1000, 20000) > f(1000, 8192)


TURN = dict(x=P, xr=64, xh=16, rows=4, heads=4, dim=16, dt=0, pos=P, ps=3, axes=3, sec=(3, 3, 2), freqs=P, inter=0, inv=0, out=P,
            outr=64, outh=16)


def _turn(lib, **kw):
    a = {**TURN, **kw}
    if a["sec"] is not None:
        a["sec"] = (ctypes.c_int32 * len(a["sec"]))(*a["sec"])
    return lib.tc_rotary(*[a[k] for k in TURN], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(pos=None), 1), (dict(freqs=None), 1), (dict(out=None), 1), (dict(sec=None), 1), (dict(rows=-1), 1),
    (dict(heads=0), 1), (dict(dim=0), 1), (dict(dim=1), 1), (dict(dt=3), 1), (dict(axes=0), 1), (dict(axes=5), 1),
    (dict(sec=(3, 3, 3)), 1), (dict(sec=(0, 0, 0)), 1), (dict(sec=(9, -1, 0)), 1), (dict(sec=(2**31 - 1,) * 3), 1),
    (dict(xr=-1), 1), (dict(xh=-1), 1), (dict(ps=-1), 1), (dict(outr=-64), 1), (dict(outh=-16), 1), (dict(inter=2), 1),
    (dict(inv=-1), 1), (dict(outh=15), 1), (dict(outr=63), 1), (dict(outr=0), 1), (dict(outr=16, outh=63), 1),
    (dict(heads=1, outr=15), 1), (dict(dim=4098, outh=4098, outr=1 << 20), 5), (dict(heads=(1 << 20) + 1), 5),
])
def test_rotary_refusals(lib, kw, status):
    assert _turn(lib, **kw) == status
    assert lib.tc_last_error()


def test_rotary_without_rows_is_nothing(lib):
    assert _turn(lib, rows=0, x=None, pos=None, freqs=None, out=None) == 0


@pytest.mark.parametrize("kw,status", [(dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(xs=-1), 1), (dict(rows=-1), 1),
                                       (dict(c=0), 1), (dict(dt=3), 1), (dict(c=(1 << 20) + 1), 5)])
def test_quantise_refusals(lib, kw, status):
    a = {**dict(x=P, xs=8, rows=4, c=8, dt=0, q=P, s=P), **kw}
    assert lib.tc_quantise_mx4(*a.values(), None) == status
    assert lib.tc_last_error()


@pytest.mark.parametrize("kw,status", [(dict(q=None), 1), (dict(s=None), 1), (dict(out=None), 1), (dict(qs=-1), 1), (dict(ss=-1), 1),
                                       (dict(rows=-1), 1), (dict(c=0), 1), (dict(dt=3), 1), (dict(c=(1 << 20) + 1), 5)])
def test_dequantise_refusals(lib, kw, status):
    a = {**dict(q=P, qs=4, s=P, ss=1, rows=4, c=8, dt=0, out=P), **kw}
    assert lib.tc_dequantise_mx4(*a.values(), None) == status
    assert lib.tc_last_error()


MM = dict(x=P, xst=4, xs=P, xss=1, w=P, wst=4, ws=P, wss=1, b=None, rows=4, n=8, k=8, dt=2, out=P, ost=8)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(xs=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(out=None), 1), (dict(rows=-1), 1),
    (dict(n=0), 1), (dict(k=0), 1), (dict(dt=3), 1), (dict(xst=-1), 1), (dict(wst=-1), 1), (dict(xss=-1), 1), (dict(wss=-1), 1),
    (dict(ost=7), 1), (dict(k=(1 << 20) + 1), 5), (dict(n=(1 << 20) + 1, ost=1 << 21), 5),
])
def test_matmul_refusals(lib, kw, status):
    assert lib.tc_matmul_mx4(*{**MM, **kw}.values(), None) == status
    assert lib.tc_last_error()


def test_without_rows_is_nothing(lib):
    assert lib.tc_quantise_mx4(None, 8, 0, 8, 0, None, None, None) == 0
    assert lib.tc_dequantise_mx4(None, 4, None, 1, 0, 8, 0, None, None) == 0
    assert lib.tc_matmul_mx4(*{**MM, **dict(rows=0, x=None, xs=None, out=None)}.values(), None) == 0


def test_binding_refuses_host_tensors():
    x, s = torch.zeros(4, 8), torch.zeros(4)
    q, e = torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    for call in (lambda: binding.tc_layer_norm(x), lambda: binding.tc_layer_norm_backward(x, x, None, s, s),
                 lambda: binding.tc_rotary(x, torch.zeros(4, 1, dtype=torch.int32), s), lambda: binding.tc_quantise_mx4(x),
                 lambda: binding.tc_dequantise_mx4(q, e), lambda: binding.tc_matmul_mx4(q, e, q, e)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the references


@pytest.mark.parametrize("c", [1, 2, 7, 33])
def test_layer_norm_gradient_against_differences(c):
    """Central differences of sum(out * dy) + sum(h * dh) in 64 bits: off by O(step^2) and by 1e-16 / step."""
    gen = torch.Generator().manual_seed(c)
    h, dy, dh = (torch.randn(5, c, generator=gen, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(c, generator=gen, dtype=torch.float64) for _ in range(2))
    eps = 0.5  # keeps the third derivatives of order one

    def loss(h, w, b):
        return (ref.layer_norm(h, w, b, eps)[0] * dy).sum() + (h * dh).sum()

    _, m, s = ref.layer_norm(h, w, b, eps)
    (dx, dw, db), _ = ref.layer_norm_grad(dy, h, w, m, s, dh, torch.float32)
    step = 1e-5
    for i in range(5):
        for j in range(c):
            e = torch.zeros_like(h)
            e[i, j] = step
            assert abs((loss(h + e, w, b) - loss(h - e, w, b)) / (2 * step) - dx[i, j]) < 1e-7
    for j in range(c):
        e = torch.zeros_like(w)
        e[j] = step
        assert abs((loss(h, w + e, b) - loss(h, w - e, b)) / (2 * step) - dw[j]) < 1e-7
        assert abs((loss(h, w, b + e) - loss(h, w, b - e)) / (2 * step) - db[j]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_against_differences(interleaved):
    """The turn is linear, so differences are its gradient but for their own rounding."""
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(2, 2, 9, generator=gen, dtype=torch.float64) for _ in range(2))
    pos = torch.randint(-50, 50, (2, 3), generator=gen)
    args = pos, torch.rand(4, generator=gen), (2, 0, 2), interleaved
    grad, _ = ref.rotary(dy, *args, True, torch.float32)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = 1.0
        d = (ref.rotary(e.view_as(x), *args, False, torch.float32)[0] * dy).sum()
        assert abs(d - grad.flatten()[i]) < 1e-12


def test_quantised_values_are_the_nearest():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(20, 75, generator=gen) * torch.exp(3 * torch.randn(20, 75, generator=gen))
    codes, scale = ref.quantise_mx4(x)
    back = ref.values(codes, scale)
    assert torch.equal(ref.unpack(ref.pack(codes), 75), codes)
    grid = torch.cat((ref.E2M1, -ref.E2M1))
    unit = torch.ldexp(torch.ones(20, 3, dtype=torch.float64), scale.long() - 127).repeat_interleave(32, 1)[:, :75]
    best = (x.double()[..., None] - grid * unit[..., None]).abs().amin(2)
    assert torch.equal((x.double() - back).abs(), best)
    top = torch.nn.functional.pad(x.abs().double() / unit, (0, 21)).view(20, 3, 32).amax(2)
    assert bool(((top >= 4) & (top < 8)).all())
