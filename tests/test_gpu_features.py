"""Operators on feature rows on the GPU against their definitions in 64 bits.

Tolerances count roundings (tests/feature_ref.py) and are never fitted. Integers
(the 8-bit rows) have to be equal.
"""
import numpy as np
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding, synth

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _view(t, pad, shift=0):
    """`t` on the GPU as columns [shift, shift + C) of a buffer `pad` + `shift` wider."""
    if not pad and not shift:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + pad + shift), 77, dtype=t.dtype, device="cuda")
    wide[:, shift:shift + t.shape[1]] = t.cuda()
    return wide[:, shift:shift + t.shape[1]]


def _within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                                 f"{got[bad][0]} for {want[bad][0]}, may be {bound[bad][0]} off")


# ------------------------------------------------------------------ norm

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 16), (64, 24), (130, 64), (77, 100), (33, 128), (1, 1024), (9, 1000), (257, 256),
          (4, 2049), (3, 4096), (2, 8192), (2, 8200), (1, 20000)]


def _norm_inputs(rows, c, dtype, seed, wdtype=None):
    g = _gen(seed)
    x = (torch.randn(rows, c, generator=g) * torch.exp(torch.randn(1, c, generator=g))).to(dtype)
    r = (2 * torch.randn(rows, c, generator=g)).to(dtype)
    w = (1 + 0.3 * torch.randn(c, generator=g)).to(wdtype or dtype)
    return x, r, w


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c", SHAPES)
def test_norm(rows, c, dtype):
    print(f"[norm] {rows} x {c} {dtype}", flush=True)
    x, r, w = _norm_inputs(rows, c, dtype, rows * 31 + c)
    h = ref.norm_sum(x, r)
    want, s = ref.rms_norm(h, w, EPS)
    out, got_h, rstd = binding.tc_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _within(out, want, ref.rms_norm_bound(want, dtype), "out")
    _within(rstd, s, s * ((c + 1) / 2 + 8) * ref.U32, "rstd")
    q, scale, got_h = binding.tc_rms_norm_i8(x.cuda(), w.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    want_q, want_scale = ref.rms_norm_i8(h, w, s)
    assert torch.equal(q.cpu(), want_q)
    _within(scale, want_scale, want_scale * ((c + 1) / 2 + 10) * ref.U32, "scale")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 64, 100, 1024])
def test_norm_plain_forms(c, dtype):
    """Without residual, without weight, with a 32-bit weight beside 16-bit rows."""
    for wdtype in (None, F32, dtype):
        x, _, w = _norm_inputs(37, c, dtype, c, wdtype)
        w = w if wdtype is not None else None
        wc = w.cuda() if w is not None else None
        want, s = ref.rms_norm(x, w, EPS)
        xc = x.cuda()
        out, h, _ = binding.tc_rms_norm(xc, wc, eps=EPS)
        assert h is xc
        _within(out, want, ref.rms_norm_bound(want, dtype), f"out {wdtype}")
        q, scale, _ = binding.tc_rms_norm_i8(xc, wc, eps=EPS)
        want_q, want_scale = ref.rms_norm_i8(x, w, s)
        assert torch.equal(q.cpu(), want_q)
        _within(scale, want_scale, want_scale * ((c + 1) / 2 + 10) * ref.U32, f"scale {wdtype}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3), (16, 0)])
def test_norm_strides_and_alignment(pad, shift, dtype):
    for rows, c in [(19, 64), (11, 100), (3, 2048)]:
        x, r, w = _norm_inputs(rows, c, dtype, c + pad)
        h = ref.norm_sum(x, r)
        want, s = ref.rms_norm(h, w, EPS)
        wide_w = torch.zeros(c + 1, dtype=dtype, device="cuda")
        wide_w[1:] = w.cuda()
        out, got_h, rstd = binding.tc_rms_norm(_view(x, pad, shift), wide_w[1:], residual=_view(r, shift, pad), eps=EPS)
        assert torch.equal(got_h.cpu(), h)
        _within(out, want, ref.rms_norm_bound(want, dtype), "out")
        q, _, _ = binding.tc_rms_norm_i8(_view(x, pad, shift), w.cuda(), residual=_view(r, pad, shift), eps=EPS)
        assert torch.equal(q.cpu(), ref.rms_norm_i8(h, w, s)[0])
        dy, dh = _norm_inputs(rows, c, dtype, c + pad + 1)[:2]
        dx, dw, bound, mag = ref.rms_norm_grad(dy, h, w, rstd.cpu(), dh)
        gx, gw = binding.tc_rms_norm_backward(_view(dy, pad, shift), _view(h, shift, pad), wide_w[1:], rstd,
                                              grad_h=_view(dh, pad, shift))
        _within(gx, dx, bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype), "grad_x")
        _within(gw, dw, mag * (rows + 8) * ref.U32, "grad_weight")


def test_norm_broadcast_residual():
    x, r, w = _norm_inputs(40, 96, BF16, 5)
    r = r[:1].expand(40, 96)
    h = ref.norm_sum(x, r)
    want, _ = ref.rms_norm(h, w, EPS)
    out, got_h, _ = binding.tc_rms_norm(x.cuda(), w.cuda(), residual=r[:1].cuda().expand(40, 96), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _within(out, want, ref.rms_norm_bound(want, BF16), "out")


@pytest.mark.parametrize("c", [8, 100, 1024])
def test_norm_sum_in_place(c):
    """h written over the residual (C entry point), and grad_x over dh."""
    lib = binding.load_library()
    x, r, w = _norm_inputs(21, c, BF16, c)
    h = ref.norm_sum(x, r)
    want, _ = ref.rms_norm(h, w, EPS)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    out, rstd = torch.empty_like(xd), torch.empty(21, device="cuda")
    st = lib.tc_rms_norm(xd.data_ptr(), c, rd.data_ptr(), c, wd.data_ptr(), 2, 21, c, 2, EPS, rd.data_ptr(),
                         out.data_ptr(), rstd.data_ptr(), None)
    assert st == 0, lib.tc_last_error()
    torch.cuda.synchronize()
    assert torch.equal(rd.cpu(), h)
    _within(out, want, ref.rms_norm_bound(want, BF16), "out")
    dy, dh = _norm_inputs(21, c, BF16, c + 1)[:2]
    dx, _, bound, _ = ref.rms_norm_grad(dy, h, w, rstd.cpu(), dh)
    dhd, dyd = dh.cuda(), dy.cuda()
    st = lib.tc_rms_norm_backward(dyd.data_ptr(), c, dhd.data_ptr(), c, rd.data_ptr(), c, wd.data_ptr(), 2,
                                  rstd.data_ptr(), 21, c, 2, dhd.data_ptr(), None, None, 0, None)
    assert st == 0, lib.tc_last_error()
    torch.cuda.synchronize()
    _within(dhd, dx, bound + dx.abs() * ref.half_step(BF16) * (1 + 2 ** -6) + ref.tiny(BF16), "grad_x")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("c", [8, 72, 100, 2048])
def test_norm_special_rows(c, dtype):
    """All zeros, one infinity, one NaN, ordinary, tiny values; the rest of the rows stay as they are."""
    x, _, w = _norm_inputs(6, c, dtype, c)
    x[1] = 0
    x[2, c // 2] = float("inf")
    x[3, c - 1] = float("nan")
    x[4] = x[4] * 1e-3
    _, s = ref.rms_norm(x, w, EPS)
    q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), w.cuda(), eps=EPS)
    want_q, want_scale = ref.rms_norm_i8(x, w, s)
    assert torch.equal(q.cpu(), want_q)
    fine = torch.tensor([0, 1, 4, 5])
    _within(scale.cpu()[fine], want_scale[fine], want_scale[fine] * ((c + 1) / 2 + 10) * ref.U32, "scale")
    assert bool(scale[2:4].isnan().all())
    out, _, rstd = binding.tc_rms_norm(x.cuda(), w.cuda(), eps=EPS)
    want, _ = ref.rms_norm(x, w, EPS)
    _within(out.cpu()[fine], want[fine], ref.rms_norm_bound(want, dtype)[fine], "out")
    assert bool(out[3].isnan().all()) and bool(out[2, c // 2].isnan())
    assert float(rstd[2]) == 0.0
    # a zero weight everywhere: p = 0 in every row without a NaN or infinity
    q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), torch.zeros_like(w).cuda(), eps=EPS)
    assert int(q.abs().max()) == 0 and bool((scale[[0, 1, 4, 5]] == 0).all()) and bool(scale[2:4].isnan().all())


def test_norm_rounding_ties():
    """Values that land on half steps go to the even integer."""
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5]])
    q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), eps=0.0)
    assert q.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -2, 64]]


def test_norm_no_rows():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    out, _, rstd = binding.tc_rms_norm(x, w)
    q, scale, _ = binding.tc_rms_norm_i8(x, w)
    assert out.shape == (0, 64) and q.shape == (0, 64) and rstd.shape == scale.shape == (0,)
    gx, gw = binding.tc_rms_norm_backward(x, x, w, rstd)
    assert gx.shape == (0, 64) and bool((gw == 0).all()) and gw.shape == (64,)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c", SHAPES + [(2000, 64), (5000, 12), (700, 512)])
def test_norm_grad(rows, c, dtype):
    print(f"[norm grad] {rows} x {c} {dtype}", flush=True)
    x, r, w = _norm_inputs(rows, c, dtype, rows * 17 + c)
    dy, dh = _norm_inputs(rows, c, dtype, rows * 19 + c)[:2]
    h = ref.norm_sum(x, r)
    _, _, rstd = binding.tc_rms_norm(h.cuda(), w.cuda(), eps=EPS)
    for grad_h in (dh, None):
        dx, dw, bound, mag = ref.rms_norm_grad(dy, h, w, rstd.cpu(), grad_h)
        gx, gw = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd,
                                              grad_h=None if grad_h is None else grad_h.cuda())
        _within(gx, dx, bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype), "grad_x")
        _within(gw, dw, mag * (rows + 8) * ref.U32, "grad_weight")
        again = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd,
                                             grad_h=None if grad_h is None else grad_h.cuda())
        assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])  # a fixed order of every sum
    gx, gw = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), None, rstd)
    dx, _, bound, _ = ref.rms_norm_grad(dy, h, None, rstd.cpu(), None)
    assert gw is None
    _within(gx, dx, bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype), "grad_x without weight")


def test_norm_grad_against_differences():
    """The kernel's gradient (32-bit rows) against central differences of the definition in 64 bits.
    Differences of step 1e-5 are off by about 1e-7 here, the kernel by its bound."""
    rows, c = 3, 20
    x, _, w = _norm_inputs(rows, c, F32, 8)
    dy, dh = _norm_inputs(rows, c, F32, 9)[:2]
    eps = 0.5
    _, h, rstd = binding.tc_rms_norm(x.cuda(), w.cuda(), eps=eps)
    gx, gw = binding.tc_rms_norm_backward(dy.cuda(), h, w.cuda(), rstd, grad_h=dh.cuda())
    _, s = ref.rms_norm(x, w, eps)
    dx, dw, bound, mag = ref.rms_norm_grad(dy, x, w, s, dh)
    # rstd itself is off by (C / 2 + 9) U32; dx depends on it through terms bounded by `bound`'s
    bound = bound * (c + 18) + 1e-6
    step = 1e-5
    xd, wd = x.double(), w.double()

    def loss(h, w):
        return (ref.rms_norm(h, w, eps)[0] * dy.double()).sum() + (h * dh.double()).sum()

    for i in range(rows):
        for j in range(c):
            e = torch.zeros_like(xd)
            e[i, j] = step
            diff = (loss(xd + e, wd) - loss(xd - e, wd)) / (2 * step)
            assert abs(float(gx[i, j]) - float(diff)) <= float(bound[i, j])
    for j in range(c):
        e = torch.zeros_like(wd)
        e[j] = step
        diff = (loss(xd, wd + e) - loss(xd, wd - e)) / (2 * step)
        assert abs(float(gw[j]) - float(diff)) <= float(mag[j]) * (rows + c + 30) * ref.U32 + 1e-6


def test_norm_many_rows():
    """More rows than one resident round of workgroups."""
    rows, c = 300_000, 16
    x, r, w = _norm_inputs(rows, c, F16, 3)
    h = ref.norm_sum(x, r)
    want, s = ref.rms_norm(h, w, EPS)
    out, got_h, rstd = binding.tc_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _within(out, want, ref.rms_norm_bound(want, F16), "out")
    q, _, _ = binding.tc_rms_norm_i8(x.cuda(), w.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(q.cpu(), ref.rms_norm_i8(h, w, s)[0])
    dx, dw, bound, mag = ref.rms_norm_grad(r, h, w, rstd.cpu(), x)
    gx, gw = binding.tc_rms_norm_backward(r.cuda(), h.cuda(), w.cuda(), rstd, grad_h=x.cuda())
    _within(gx, dx, bound + dx.abs() * ref.half_step(F16) * (1 + 2 ** -6) + ref.tiny(F16), "grad_x")
    _within(gw, dw, mag * (rows + 8) * ref.U32, "grad_weight")


# ------------------------------------------------------------------ products


def _rows_i8(rows, c, seed):
    """Rows over the whole int8 range (-128 too), a zero row, scales of several magnitudes."""
    g = _gen(seed)
    q = torch.randint(-128, 128, (rows, c), generator=g, dtype=torch.int8)
    s = torch.exp(torch.randn(rows, generator=g)) * 0.01
    if rows > 2:
        q[rows // 2] = 0
        s[rows // 2] = 0.0
    return q, s


def _check_mm(rows, k, n, dtype, bias, pad=0, shift=0, wpad=0, out_pad=0):
    print(f"[matmul] {rows} x {k} -> {n} {dtype} bias={bias} pad={pad},{shift},{wpad},{out_pad}", flush=True)
    x, xs = _rows_i8(rows, k, rows + 7 * k + n)
    w, ws = _rows_i8(n, k, rows + 5 * k + 3 * n)
    ws = ws / max(1.0, k ** 0.5)
    b = torch.randn(n, generator=_gen(n)) if bias else None
    want, mag = ref.matmul_i8(x, xs, w, ws, b)
    out, base = None, None
    if out_pad:
        base = torch.full((rows, n + out_pad), -5.0, dtype=dtype, device="cuda")
        out = base[:, out_pad // 2:out_pad // 2 + n]
    got = binding.tc_matmul_i8(_view(x, pad, shift), xs.cuda(), _view(w, wpad), ws.cuda(),
                               bias=None if b is None else b.cuda(), out_dtype=dtype, out=out)
    _within(got, want, ref.product_bound(want, mag, dtype), "matmul")
    if base is not None:
        assert bool((base[:, :out_pad // 2] == -5).all()) and bool((base[:, out_pad // 2 + n:] == -5).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 16, 1), (1, 64, 64), (1, 1024, 4096), (2, 100, 33), (5, 4096, 48),
                                      (16, 256, 256), (17, 64, 65), (31, 640, 512), (64, 64, 64), (65, 63, 129),
                                      (100, 1000, 77), (128, 128, 128), (130, 272, 260), (257, 512, 300)])
def test_matmul(rows, k, n, dtype):
    _check_mm(rows, k, n, dtype, bias=(rows + n) % 2 == 0)


@pytest.mark.parametrize("rows,k,n", [(1000, 256, 768), (513, 2048, 640), (2048, 4096, 256), (5000, 64, 64),
                                      (3000, 32, 1000), (300, 8192, 520), (4100, 144, 16), (700, 96, 2050)])
def test_matmul_larger(rows, k, n):
    _check_mm(rows, k, n, BF16, bias=True)


@pytest.mark.parametrize("pad,shift,wpad,out_pad", [(1, 0, 0, 0), (0, 3, 0, 0), (16, 16, 32, 0), (0, 0, 5, 0),
                                                    (0, 0, 0, 2), (0, 0, 0, 16), (4, 8, 12, 6)])
def test_matmul_strides_and_alignment(pad, shift, wpad, out_pad):
    for rows, k, n in [(3, 128, 96), (200, 128, 96), (400, 320, 256), (70, 61, 50)]:
        for dtype in (BF16, F32):
            _check_mm(rows, k, n, dtype, True, pad, shift, wpad, out_pad)


def test_matmul_extremes():
    """The largest sums: -128 * -128 over 131071 channels stays inside int32 and is exact."""
    k = 131071
    x = torch.full((3, k), -128, dtype=torch.int8)
    w = torch.full((17, k), -128, dtype=torch.int8)
    w[1] = 127
    one = torch.ones(17)
    got = binding.tc_matmul_i8(x.cuda(), one[:3].cuda(), w.cuda(), one.cuda(), out_dtype=F32).double().cpu()
    want, mag = ref.matmul_i8(x, one[:3], w, one, None)
    _within(got, want, ref.product_bound(want, mag, F32), "largest sums")


def test_matmul_non_finite_scales():
    """A row whose scale is NaN (the norm had a NaN in it) gives NaN in that row alone."""
    x, xs = _rows_i8(70, 64, 1)
    w, ws = _rows_i8(40, 64, 2)
    xs[7] = float("nan")
    want, mag = ref.matmul_i8(x, xs, w, ws, None)
    got = binding.tc_matmul_i8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out_dtype=F32)
    keep = torch.arange(70) != 7
    assert bool(got[7].isnan().all())
    _within(got.cpu()[keep], want[keep], ref.product_bound(want, mag, F32)[keep], "other rows")


def test_matmul_far_rows():
    """Row offsets beyond 32 bits, in the rows and in the output."""
    stride = 1_500_000_000
    buf = torch.zeros(2 * stride + 256, dtype=torch.int8, device="cuda")
    x, xs = _rows_i8(3, 256, 4)
    xv = buf.as_strided((3, 256), (stride, 1))
    xv.copy_(x.cuda())
    w, ws = _rows_i8(64, 256, 5)
    want, mag = ref.matmul_i8(x, xs, w, ws, None)
    got = binding.tc_matmul_i8(xv, xs.cuda(), w.cuda(), ws.cuda(), out_dtype=BF16)
    _within(got, want, ref.product_bound(want, mag, BF16), "far rows")
    m = torch.tensor([[2], [0], [-1], [1]], dtype=torch.int32)
    want, mag = ref.sparse_conv_i8(x, xs, m, w[None], ws, None)
    got = binding.tc_sparse_conv_i8(xv, xs.cuda(), m.cuda(), w[None].contiguous().cuda(), ws.cuda(), out_dtype=BF16)
    _within(got, want, ref.product_bound(want, mag, BF16), "far rows, mapped")
    far = buf.view(torch.bfloat16).as_strided((3, 64), (stride // 2, 1))
    want, mag = ref.matmul_i8(x, xs, w, ws, None)
    xd = x.cuda()
    binding.tc_matmul_i8(xd, xs.cuda(), w.cuda(), ws.cuda(), out=far)
    _within(far, want, ref.product_bound(want, mag, BF16), "far output rows")


def _random_map(n_dst, taps, n_src, density, seed):
    g = _gen(seed)
    m = torch.randint(0, max(n_src, 1), (n_dst, taps), generator=g, dtype=torch.int32)
    return torch.where(torch.rand(n_dst, taps, generator=g) < density, m, torch.tensor(-1, dtype=torch.int32))


def _check_conv(n_src, m, cin, cout, dtype, bias, pad=0, shift=0):
    print(f"[conv] {n_src} -> {tuple(m.shape)} {cin} -> {cout} {dtype} bias={bias} pad={pad},{shift}", flush=True)
    taps = m.shape[1]
    x, xs = _rows_i8(n_src, cin, n_src + cin)
    w, ws = _rows_i8(cout, taps * cin, n_src + cout)
    w = w.view(cout, taps, cin).transpose(0, 1).contiguous()
    ws = ws / (taps * cin) ** 0.5
    b = torch.randn(cout, generator=_gen(cout)) if bias else None
    want, mag = ref.sparse_conv_i8(x, xs, m, w, ws, b)
    got = binding.tc_sparse_conv_i8(_view(x, pad, shift), xs.cuda(), m.cuda(), w.cuda(), ws.cuda(),
                                    bias=None if b is None else b.cuda(), out_dtype=dtype)
    _within(got, want, ref.product_bound(want, mag, dtype, taps), "conv")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n_dst,taps,cin,cout", [(1, 1, 1, 1), (1, 27, 64, 64), (15, 8, 16, 20), (64, 27, 32, 64),
                                                 (65, 27, 64, 65), (200, 27, 100, 48), (300, 8, 128, 128),
                                                 (129, 125, 24, 40), (500, 27, 192, 96), (70, 512, 8, 9)])
def test_conv(n_dst, taps, cin, cout, dtype):
    n_src = n_dst // 2 + 3
    _check_conv(n_src, _random_map(n_dst, taps, n_src, 0.4, n_dst + taps), cin, cout, dtype, bias=cout % 2 == 0)


@pytest.mark.parametrize("cin,cout", [(256, 256), (64, 512), (512, 64), (1000, 33)])
def test_conv_wide(cin, cout):
    _check_conv(700, _random_map(900, 27, 700, 0.4, cin), cin, cout, BF16, True)


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 3), (16, 16), (4, 8)])
def test_conv_strides_and_alignment(pad, shift):
    for cin, cout in [(64, 64), (52, 45), (128, 32)]:
        _check_conv(90, _random_map(150, 27, 90, 0.4, cin), cin, cout, F16, True, pad, shift)


def test_conv_rows_that_read_nothing():
    m = _random_map(200, 27, 50, 0.3, 1)
    m[3] = -1
    m[64:140] = -1  # whole tiles of a launch among them
    _check_conv(50, m, 64, 64, F32, True)
    _check_conv(50, m, 64, 64, BF16, False)
    _check_conv(50, torch.full((100, 27), -1, dtype=torch.int32), 64, 48, BF16, True)
    _check_conv(50, m[:0], 64, 64, BF16, True)


def test_conv_entries_out_of_range_read_nothing():
    m = _random_map(130, 27, 40, 0.5, 2)
    m[::7, 3] = 40
    m[::5, 9] = 2 ** 31 - 1
    m[::3, 11] = -(2 ** 31)
    m[::4, 26] = -2
    _check_conv(40, m, 64, 80, F32, True)
    _check_conv(40, m, 20, 80, BF16, True)


def test_conv_without_sources():
    m = torch.zeros(33, 8, dtype=torch.int32)
    w = torch.ones(8, 16, 32, dtype=torch.int8, device="cuda")
    b = torch.arange(16.0, device="cuda")
    got = binding.tc_sparse_conv_i8(torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"),
                                    m.cuda(), w, torch.ones(16, device="cuda"), bias=b, out_dtype=F32)
    assert bool((got == b).all())


@pytest.mark.parametrize("op,k,stride,transposed", [(None, 3, 1, False), (("refine", 2), 2, 2, True),
                                                    (("coarsen", 2), 2, 2, False)])
def test_conv_over_built_maps(op, k, stride, transposed):
    """Maps of the library's own topologies, empty members and straddled tiles among them."""
    ijk, off = synth.make_config(3)
    members = [ijk[off[g]:off[g + 1]] for g in (0, 1, 2, 5, 24)]
    ijk, off = synth.concat_members(members)
    src = binding.tc_batch_from_ijk(torch.from_numpy(np.ascontiguousarray(ijk)).cuda(), off)
    dst = src if op is None else binding.tc_build_batched_topology(src, op[0], op[1])
    m = binding.tc_build_kernel_map(src, dst, k, stride, transposed)
    _check_conv(src.voxel_total(), m.cpu(), 32, 24, F16, True)


# ------------------------------------------------------------------ streams, graphs, errors


def _all_ops(t):
    out, h, rstd = binding.tc_rms_norm(t["x"], t["w"], residual=t["r"], stream=t.get("stream"))
    gx, gw = binding.tc_rms_norm_backward(t["dy"], h, t["w"], rstd, grad_h=t["r"], stream=t.get("stream"))
    q, scale, _ = binding.tc_rms_norm_i8(t["x"], t["w"], residual=t["r"], stream=t.get("stream"))
    y = binding.tc_matmul_i8(q, scale, t["w8"], t["ws"], stream=t.get("stream"))
    z = binding.tc_sparse_conv_i8(q, scale, t["map"], t["w27"], t["ws"], out_dtype=F32, stream=t.get("stream"))
    return [out, h, rstd, gx, gw, q, scale, y, z]


def _all_inputs(seed, rows=500, c=64, n=80):
    x, r, w = _norm_inputs(rows, c, BF16, seed)
    dy = _norm_inputs(rows, c, BF16, seed + 1)[0]
    w8, ws = _rows_i8(n, c, seed)
    w27 = _rows_i8(27 * n, c, seed + 2)[0].view(27, n, c)
    t = {"x": x, "r": r, "w": w, "dy": dy, "w8": w8, "ws": ws, "w27": w27, "map": _random_map(rows, 27, rows, 0.4, seed)}
    return {k: v.contiguous().cuda() for k, v in t.items()}


def test_other_stream():
    t = _all_inputs(1)
    want = _all_ops(t)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = _all_ops({**t, "stream": st})
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(st):
        got = _all_ops(t)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays():
    """Captured once, replayed on changed inputs with eager work between, each replay equal to the eager result."""
    t = _all_inputs(3)
    _all_ops(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_ops(t)
    for seed in (10, 11, 12):
        for k, v in _all_inputs(seed).items():
            t[k].copy_(v)
        want = [v.clone() for v in _all_ops(t)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_binding_refusals():
    x, _, w = (v.cuda() for v in _norm_inputs(4, 8, BF16, 0))
    q, s = (v.cuda() for v in _rows_i8(4, 8, 0))
    m = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    rstd = torch.ones(4, device="cuda")
    bad_type = [lambda: binding.tc_rms_norm(x.double()), lambda: binding.tc_rms_norm(x, residual=x.float()),
                lambda: binding.tc_rms_norm_backward(x.float(), x, w, rstd),
                lambda: binding.tc_rms_norm_backward(x, x, w, rstd.half()),
                lambda: binding.tc_matmul_i8(q.int(), s, q, s), lambda: binding.tc_matmul_i8(q, s.half(), q, s),
                lambda: binding.tc_matmul_i8(q, s, q, s, out_dtype=torch.float64),
                lambda: binding.tc_sparse_conv_i8(q, s, m.long(), q[None], s)]
    for call in bad_type:
        with pytest.raises(TypeError):
            call()
    bad_value = [lambda: binding.tc_rms_norm(x, w[:7]), lambda: binding.tc_rms_norm(x, residual=x[:3]),
                 lambda: binding.tc_rms_norm(x.t()), lambda: binding.tc_rms_norm(x[0]),
                 lambda: binding.tc_rms_norm_backward(x, x, w, rstd[:3]),
                 lambda: binding.tc_matmul_i8(q, s, q[:, :7], s), lambda: binding.tc_matmul_i8(q, s[:3], q, s),
                 lambda: binding.tc_matmul_i8(q, s, q, s, bias=s[:2]),
                 lambda: binding.tc_matmul_i8(q, s, q, s, out=torch.empty(3, 4, device="cuda")),
                 lambda: binding.tc_matmul_i8(q, s, q, s, out=torch.empty(1, 4, device="cuda").expand(4, 4)),
                 lambda: binding.tc_sparse_conv_i8(q, s, m, q, s),
                 lambda: binding.tc_sparse_conv_i8(q, s, m, q[None].expand(2, 4, 8), s),
                 lambda: binding.tc_sparse_conv_i8(q, s, m.t().expand(4, 4)[:, 1:], q[None].expand(3, 4, 8), s)]
    for call in bad_value:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.TopoError) as ex:
        binding.tc_rms_norm(x, w.float().half())
    assert ex.value.status == 1
    with pytest.raises(binding.TopoError) as ex:
        binding.tc_rms_norm(x, w, eps=float("nan"))
    assert ex.value.status == 1
    torch.cuda.synchronize()
