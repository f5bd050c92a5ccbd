"""The norm where a workgroup takes its rows in several rounds with a remainder: every number of threads a
row, rows that a workgroup's registers do not hold, rows narrower than a vector; in place too."""
import pytest
import torch

from tests import feature_ref as ref
from tests.feature_bounds import weight_grad_bound
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
IDS = {F32: 0, F16: 1, BF16: 2}
EPS = 1e-6

# on a card of 256 CUs: 2048 workgroups forward, 1024 parts backward
ROUNDS = [(5003, 2056, F16), (5003, 2057, BF16), (4500, 4100, F32),  # a workgroup a row
          (9001, 1000, BF16), (9001, 500, F32),                      # a wave a row
          (40001, 128, BF16), (40001, 61, F32), (140003, 32, F16),   # some lanes a row
          (2500, 3, F32), (2500, 7, F16), (530_001, 3, F32),         # narrower than a vector
          (2100, 16392, F16), (2100, 8200, F32)]                     # not held in registers


def _inputs(rows, c, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, c, generator=g) * torch.exp(torch.randn(1, c, generator=g))).to(dtype)
    r = (2 * torch.randn(rows, c, generator=g)).to(dtype)
    return x, r, (1 + 0.3 * torch.randn(c, generator=g)).to(dtype)


def _within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def _grad_bound(dx, bound, dtype):
    return bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype)


@pytest.mark.parametrize("rows,c,dtype", ROUNDS)
def test_norm_rounds(rows, c, dtype):
    print(f"[norm rounds] {rows} x {c} {dtype}", flush=True)
    x, r, w = _inputs(rows, c, dtype, rows + c)
    h = ref.norm_sum(x, r)
    want, s = ref.rms_norm(h, w, EPS)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    out, got_h, rstd = binding.tc_rms_norm(xd, wd, residual=rd, eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _within(out, want, ref.rms_norm_bound(want, dtype), "out")
    _within(rstd, s, s * ((c + 1) / 2 + 8) * ref.U32, "rstd")
    del out, want
    q, scale, got_h = binding.tc_rms_norm_i8(xd, wd, residual=rd, eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    want_q, want_scale = ref.rms_norm_i8(h, w, s)
    assert torch.equal(q.cpu(), want_q)
    _within(scale, want_scale, want_scale * ((c + 1) / 2 + 10) * ref.U32, "scale")
    del q, want_q
    # gradient: the residual's values as dy, x's as dh
    dx, dw, bound, mag = ref.rms_norm_grad(r, h, w, rstd.cpu(), x)
    gx, gw = binding.tc_rms_norm_backward(rd, got_h, wd, rstd, grad_h=xd)
    _within(gx, dx, _grad_bound(dx, bound, dtype), "grad_x")
    _within(gw, dw, weight_grad_bound(mag, rows), "grad_weight")


@pytest.mark.parametrize("rows,c,dtype", [(5003, 2056, F16), (5003, 2057, BF16), (9001, 1000, BF16), (40001, 61, F32),
                                          (530_001, 3, F32), (2100, 16392, F16)])
def test_norm_rounds_in_place(rows, c, dtype):
    """h over x, h over r, and grad_x over dh, through the C entry points."""
    print(f"[norm in place] {rows} x {c} {dtype}", flush=True)
    lib = binding.load_library()
    x, r, w = _inputs(rows, c, dtype, rows - c)
    h = ref.norm_sum(x, r)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    out0, h0, rstd0 = binding.tc_rms_norm(xd, wd, residual=rd, eps=EPS)
    q0, scale0, _ = binding.tc_rms_norm_i8(xd, wd, residual=rd, eps=EPS)
    assert torch.equal(h0.cpu(), h)
    t, wt = IDS[dtype], IDS[dtype]
    for over in ("x", "r"):
        for i8 in (False, True):
            a, b = xd.clone(), rd.clone()
            to = a if over == "x" else b
            o = torch.empty((rows, c), dtype=torch.int8 if i8 else dtype, device="cuda")
            s = torch.empty(rows, device="cuda")
            call = lib.tc_rms_norm_i8 if i8 else lib.tc_rms_norm
            st = call(a.data_ptr(), c, b.data_ptr(), c, wd.data_ptr(), wt, rows, c, t, EPS, to.data_ptr(), o.data_ptr(),
                      s.data_ptr(), None)
            assert st == 0, lib.tc_last_error()
            torch.cuda.synchronize()
            assert torch.equal(to, h0) and torch.equal(o, q0 if i8 else out0) and torch.equal(s, scale0 if i8 else rstd0)
    gx0, gw0 = binding.tc_rms_norm_backward(rd, h0, wd, rstd0, grad_h=xd)
    dh = xd.clone()
    need = lib.tc_rms_norm_backward_workspace(rows, c)
    work, gw = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(c, device="cuda")
    st = lib.tc_rms_norm_backward(rd.data_ptr(), c, dh.data_ptr(), c, h0.data_ptr(), c, wd.data_ptr(), wt, rstd0.data_ptr(),
                                  rows, c, t, dh.data_ptr(), gw.data_ptr(), work.data_ptr(), need, None)
    assert st == 0, lib.tc_last_error()
    torch.cuda.synchronize()
    assert torch.equal(dh, gx0) and torch.equal(gw, gw0)
