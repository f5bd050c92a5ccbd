"""Layer norm, rotary positions and 4-bit rows on the GPU against their definitions in 64 bits (tests/token_ref.py: tolerances
count roundings). What is held in 4 bits has to be equal."""
import pytest
import torch

from tests import feature_ref
from tests import token_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _view(t, pad, shift=0):
    """`t` [rows, ...] on the GPU as a part of each row of a buffer `pad` + `shift` wider."""
    if not pad and not shift:
        return t.cuda()
    each = t[0].numel()
    wide = torch.full((t.shape[0], each + pad + shift), 77, dtype=t.dtype, device="cuda")
    wide[:, shift:shift + each] = t.cuda().flatten(1)
    return wide[:, shift:shift + each].unflatten(1, t.shape[1:])


def _within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                                 f"{got[bad][0]} for {want[bad][0]}, may be {bound[bad][0]} off")


# ------------------------------------------------------------------ layer norm

# narrower than a vector, every number of lanes a row, workgroups, wider than registers hold
SHAPES = [(1, 1), (1, 8), (3, 7), (700, 3), (5, 16), (64, 24), (130, 64), (77, 100), (33, 128), (1, 1024), (9, 1000), (257, 256),
          (4, 2049), (3, 4096), (2, 8192), (2, 8200), (2, 16390), (1, 20000)]


def _norm_inputs(rows, c, dtype, seed, wdtype=None, bdtype=None):
    g = _gen(seed)
    x = (torch.randn(rows, c, generator=g) * torch.exp(torch.randn(1, c, generator=g)) + torch.randn(1, c, generator=g)).to(dtype)
    r = (2 * torch.randn(rows, c, generator=g)).to(dtype)
    w = (1 + 0.3 * torch.randn(c, generator=g)).to(wdtype or dtype)
    b = torch.randn(c, generator=g).to(bdtype or dtype)
    return x, r, w, b


def _check_norm(got, h, w, b, dtype, eps=EPS):
    out, mean, rstd = got
    want, m, s = ref.layer_norm(h, w, b, eps)
    for name, a, v, off in zip(("out", "mean", "rstd"), (out, mean, rstd), (want, m, s), ref.layer_norm_bounds(h, w, b, m, s, dtype)):
        _within(a, v, off, name)


def _check_grad(got, dy, h, w, mean, rstd, dh, dtype):
    gx, gw, gb = got
    (dx, dw, db), (off, mag_w, mag_b, off_w) = ref.layer_norm_grad(dy, h, w, mean.cpu(), rstd.cpu(), dh, dtype)
    _within(gx, dx, off, "grad_x")
    n = ref.layer_norm_sum_roundings(h.shape[0]) * ref.U32 * (1 + 2.0 ** -10)
    if gw is not None:
        _within(gw, dw, mag_w * n + off_w, "grad_weight")
    if gb is not None:
        _within(gb, db, mag_b * n, "grad_bias")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c", SHAPES)
def test_layer_norm(rows, c, dtype):
    print(f"[layer norm] {rows} x {c} {dtype}", flush=True)
    x, r, w, b = _norm_inputs(rows, c, dtype, rows * 31 + c)
    h = feature_ref.norm_sum(x, r)
    out, got_h, mean, rstd = binding.tc_layer_norm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _check_norm((out, mean, rstd), h, w, b, dtype)
    dy, dh, _, _ = _norm_inputs(rows, c, dtype, rows * 31 + c + 1)
    got = binding.tc_layer_norm_backward(dy.cuda(), got_h, w.cuda(), mean, rstd, grad_h=dh.cuda())
    _check_grad(got, dy, h, w, mean, rstd, dh, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 64, 100, 1024, 20000])
def test_layer_norm_plain_forms(c, dtype):
    """Without residual, weight or bias, with 32-bit weights beside 16-bit rows."""
    for wdtype, bdtype in ((None, None), (F32, dtype), (dtype, F32), (None, F32), (F32, None)):
        x, _, w, b = _norm_inputs(37, c, dtype, c, wdtype, bdtype)
        w, b = w if wdtype else None, b if bdtype else None
        wc, bc = (None if t is None else t.cuda() for t in (w, b))
        xc = x.cuda()
        out, h, mean, rstd = binding.tc_layer_norm(xc, wc, bc, eps=EPS)
        assert h is xc
        _check_norm((out, mean, rstd), x, w, b, dtype)
        dy = _norm_inputs(37, c, dtype, c + 1)[0]
        got = binding.tc_layer_norm_backward(dy.cuda(), xc, wc, mean, rstd, with_bias=b is not None)
        assert (got[1] is None) == (w is None) and (got[2] is None) == (b is None)
        _check_grad(got, dy, x, w, mean, rstd, None, dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 3), (16, 0)])
def test_layer_norm_strides_and_alignment(pad, shift, dtype):
    for rows, c in [(19, 64), (11, 100), (3, 2048)]:
        x, r, w, b = _norm_inputs(rows, c, dtype, c + pad)
        h = feature_ref.norm_sum(x, r)
        wide = torch.zeros(2, c + 1, dtype=dtype, device="cuda")
        wide[0, 1:], wide[1, 1:] = w.cuda(), b.cuda()
        out, got_h, mean, rstd = binding.tc_layer_norm(_view(x, pad, shift), wide[0, 1:], wide[1, 1:], residual=_view(r, shift, pad), eps=EPS)
        assert torch.equal(got_h.cpu(), h)
        _check_norm((out, mean, rstd), h, w, b, dtype)
        dy, dh = _norm_inputs(rows, c, dtype, c + pad + 1)[:2]
        got = binding.tc_layer_norm_backward(_view(dy, pad, shift), _view(h, shift, pad), wide[0, 1:], mean, rstd, grad_h=_view(dh, pad, shift))
        _check_grad(got, dy, h, w, mean, rstd, dh, dtype)


# several rounds a workgroup, and a weight gradient of many rows
@pytest.mark.parametrize("rows,c,dtype", [(300_000, 4, F32), (300_000, 5, BF16), (70_000, 8, BF16), (40_000, 24, F32), (20_000, 130, BF16),
                                          (9_000, 300, F32), (5_000, 1030, BF16), (2_500, 2100, BF16), (2_100, 8200, F32)])
def test_layer_norm_rounds(rows, c, dtype):
    print(f"[layer norm rounds] {rows} x {c} {dtype}", flush=True)
    x, r, w, b = _norm_inputs(rows, c, dtype, c, F32, F32)
    h = feature_ref.norm_sum(x, r)
    out, got_h, mean, rstd = binding.tc_layer_norm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got_h.cpu(), h)
    _check_norm((out, mean, rstd), h, w, b, dtype)
    got = binding.tc_layer_norm_backward(r.cuda(), got_h, w.cuda(), mean, rstd, grad_h=x.cuda())
    again = binding.tc_layer_norm_backward(r.cuda(), got_h, w.cuda(), mean, rstd, grad_h=x.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    _check_grad(got, r, h, w, mean, rstd, x, dtype)


@pytest.mark.parametrize("c", [3, 64, 100, 1024, 20000])
def test_layer_norm_far_from_zero(c):
    """Rows whose offset is far above their spread, and constant ones: the spread's digits are kept."""
    g = _gen(c)
    for offset in (1e4, -3e6, 1e8):
        h = (torch.randn(24, c, generator=g) + offset).float()
        h[3] = offset
        w, b = 1 + 0.3 * torch.randn(c, generator=g), torch.randn(c, generator=g)
        out, _, mean, rstd = binding.tc_layer_norm(h.cuda(), w.cuda(), b.cuda(), eps=EPS)
        _check_norm((out, mean, rstd), h, w, b, F32)
        assert torch.equal(out[3].cpu(), b) and float(mean[3]) == float(h[3, 0])
        dy = torch.randn(24, c, generator=g)
        got = binding.tc_layer_norm_backward(dy.cuda(), h.cuda(), w.cuda(), mean, rstd)
        _check_grad(got, dy, h, w, mean, rstd, None, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [4, 100, 1024, 20000])
def test_layer_norm_ends_of_the_range(c, dtype):
    """Spreads from 1e-36 to 1e38: squares and differences that leave 32 bits."""
    g = _gen(c + 7)
    for size, eps in ((1e-36, 0.0), (1e-25, 0.0), (1e-25, 1e-38), (1e-16, 0.0), (1e16, EPS), (1e19, EPS), (1e30, EPS), (6e37, EPS)):
        unit = torch.randn(9, c, generator=g).clamp(-4, 4)
        h = (unit.double() * size).to(dtype)
        w, b = 1 + 0.3 * torch.randn(c, generator=g), torch.randn(c, generator=g)
        out, _, mean, rstd = binding.tc_layer_norm(h.cuda(), w.cuda(), b.cuda(), eps=eps)
        _check_norm((out, mean, rstd), h, w, b, dtype, eps)
        dy = torch.randn(9, c, generator=g).to(dtype)
        got = binding.tc_layer_norm_backward(dy.cuda(), h.cuda(), w.cuda(), mean, rstd)
        _check_grad(got, dy, h, w, mean, rstd, None, dtype)


def test_layer_norm_not_finite():
    """An infinity or NaN makes its own row NaN and no other."""
    x = torch.randn(6, 300, generator=_gen(1))
    x[1, 7], x[3, 299], x[4, 0] = float("inf"), float("nan"), -float("inf")
    out, _, mean, rstd = binding.tc_layer_norm(x.cuda(), eps=EPS)
    bad = torch.tensor([False, True, False, True, True, False])
    assert torch.equal(out.isnan().all(1).cpu(), bad) and torch.equal(out.isnan().any(1).cpu(), bad)
    gx, _, _ = binding.tc_layer_norm_backward(torch.ones(6, 300, device="cuda"), x.cuda(), None, mean, rstd)
    assert torch.equal(gx.isnan().any(1).cpu(), bad)


@pytest.mark.parametrize("c", [5, 100, 1024, 20004])
def test_layer_norm_in_place(c):
    """h written over x or over the residual (C entry point), and grad_x over dh."""
    lib = binding.load_library()
    x, r, w, b = _norm_inputs(21, c, BF16, c)
    h = feature_ref.norm_sum(x, r)
    wd, bd = w.cuda(), b.cuda()
    for over in ("x", "r"):
        xd, rd = x.cuda(), r.cuda()
        to = xd if over == "x" else rd
        out, mean, rstd = torch.empty_like(xd), torch.empty(21, device="cuda"), torch.empty(21, device="cuda")
        st = lib.tc_layer_norm(xd.data_ptr(), c, rd.data_ptr(), c, wd.data_ptr(), 2, bd.data_ptr(), 2, 21, c, 2, EPS, to.data_ptr(),
                               out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), None)
        assert st == 0, lib.tc_last_error()
        torch.cuda.synchronize()
        assert torch.equal(to.cpu(), h)
        _check_norm((out, mean, rstd), h, w, b, BF16)
    dy, dh = _norm_inputs(21, c, BF16, c + 1)[:2]
    dhd, dyd, hd = dh.cuda(), dy.cuda(), h.cuda()
    st = lib.tc_layer_norm_backward(dyd.data_ptr(), c, dhd.data_ptr(), c, hd.data_ptr(), c, wd.data_ptr(), 2, mean.data_ptr(),
                                    rstd.data_ptr(), 21, c, 2, dhd.data_ptr(), None, None, None, 0, None)
    assert st == 0, lib.tc_last_error()
    torch.cuda.synchronize()
    _check_grad((dhd, None, None), dy, h, w, mean, rstd, dh, BF16)


def test_layer_norm_empty():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    out, h, mean, rstd = binding.tc_layer_norm(x, w, w)
    assert out.shape == (0, 64) and h is x and mean.shape == rstd.shape == (0,)
    gx, gw, gb = binding.tc_layer_norm_backward(x, x, w, mean, rstd)
    assert gx.shape == (0, 64) and float(gw.abs().sum() + gb.abs().sum()) == 0


def test_layer_norm_refusals():
    x = torch.zeros(4, 8, device="cuda")
    for bad, kind in ((lambda: binding.tc_layer_norm(x, residual=x.half()), TypeError), (lambda: binding.tc_layer_norm(x, x[0, :7]), ValueError),
                      (lambda: binding.tc_layer_norm(x, None, x[0, :7]), ValueError), (lambda: binding.tc_layer_norm(x[0]), ValueError),
                      (lambda: binding.tc_layer_norm(x.double()), TypeError), (lambda: binding.tc_layer_norm(x.t().contiguous().t()), ValueError),
                      (lambda: binding.tc_layer_norm(x, x[0].half()), binding.TopoError), (lambda: binding.tc_layer_norm(x, eps=-1.0), binding.TopoError),
                      (lambda: binding.tc_layer_norm_backward(x, x, None, x[0, :3], x[0, :4]), ValueError)):
        with pytest.raises(kind):
            bad()


# ------------------------------------------------------------------ rotary positions


def _turn_inputs(rows, heads, dim, sections, dtype, seed, span=1 << 12):
    g = _gen(seed)
    x = torch.randn(rows, heads, dim, generator=g).to(dtype)
    pos = torch.randint(-span, span, (rows, len(sections)), generator=g, dtype=torch.int32)
    freqs = torch.cat([100.0 ** (-torch.arange(n) / max(n, 1)) for n in sections]).float()
    return x, pos, freqs


TURNS = [(1, 1, 2, (1,)), (1, 20, 128, (16, 24, 24)), (5, 3, 16, (2, 3, 3)), (7, 2, 10, (1, 1, 1, 2)), (300, 4, 64, (12, 10, 10)),
         (33, 5, 100, (20, 0, 30)), (3, 7, 75, (10, 3)), (257, 1, 48, (8, 8)), (2, 1, 4096, (2048,)), (1, 3, 4096, (0, 1000, 48)),
         (4, 300, 32, (8, 0, 0, 8)), (2000, 3, 6, (0, 0, 3)), (40, 6, 18, (4, 4))]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,heads,dim,sections", TURNS)
def test_rotary(rows, heads, dim, sections, dtype):
    print(f"[rotary] {rows} x {heads} x {dim} {sections} {dtype}", flush=True)
    x, pos, freqs = _turn_inputs(rows, heads, dim, sections, dtype, rows + dim)
    for interleaved in (False, True):
        for inverse in (False, True):
            out = binding.tc_rotary(x.cuda(), pos.cuda(), freqs.cuda(), sections, interleaved=interleaved, inverse=inverse)
            _within(out, *ref.rotary(x, pos, freqs, sections, interleaved, inverse, dtype), f"out {interleaved} {inverse}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (16, 0)])
def test_rotary_layouts(pad, shift, dtype):
    """Parts of wider rows, heads before rows, one head, in place, positions in a wider table."""
    sections = (5, 6, 7)
    x, pos, freqs = _turn_inputs(50, 4, 42, sections, dtype, 9)
    p = _view(pos, pad, shift)
    f = freqs.cuda()
    for interleaved in (False, True):
        want = ref.rotary(x, pos, freqs, sections, interleaved, False, dtype)
        part = _view(x, pad, shift)
        _within(binding.tc_rotary(part, p, f, sections, interleaved), *want, "part")
        rest = part.clone(memory_format=torch.preserve_format)
        assert binding.tc_rotary(part, p, f, sections, interleaved, out=part) is part
        _within(part, *want, "in place")
        if pad or shift:
            base = part._base
            assert bool((base[:, :shift] == 77).all()) and bool((base[:, shift + 168:] == 77).all())
        heads_first = x.cuda().transpose(0, 1).contiguous().transpose(0, 1)
        to = torch.full((4, 50, 42 + pad), 5.0, dtype=dtype, device="cuda")
        got = binding.tc_rotary(heads_first, p, f, sections, interleaved, out=to.transpose(0, 1)[..., :42])
        _within(got, *want, "heads first")
        assert bool((to[..., 42:] == 5).all())
        one = binding.tc_rotary(rest[:, 2], p, f, sections, interleaved)
        _within(one, want[0][:, 2], want[1][:, 2], "one head")
        same = binding.tc_rotary(x[:1].cuda().expand(50, 4, 42), p, f, sections, interleaved)
        _within(same, *ref.rotary(x[:1].expand(50, 4, 42), pos, freqs, sections, interleaved, False, dtype), "one row for all")
        still = binding.tc_rotary(x.cuda(), p[:1].expand(50, 3), f, sections, interleaved)
        _within(still, *ref.rotary(x, pos[:1].expand(50, 3), freqs, sections, interleaved, False, dtype), "one position for all")


def test_rotary_far_positions():
    """Coordinates over all 32 bits: the angle is exact before it is reduced. Products of 31 and 22 bits are exact in 64."""
    g = _gen(4)
    x = torch.randn(400, 1, 32, generator=g)
    pos = torch.randint(-2 ** 31, 2 ** 31, (400, 2), generator=g).to(torch.int32)
    pos[0], pos[1], pos[2] = -2 ** 31, 2 ** 31 - 1, 0
    freqs = torch.rand(16, generator=g)
    freqs = ((freqs * 2 ** 22).round() / 2 ** 22).float()
    out = binding.tc_rotary(x.cuda(), pos.cuda(), freqs.cuda(), (8, 8))
    _within(out, *ref.rotary(x, pos, freqs, (8, 8), False, False, F32), "out")
    assert torch.equal(out[2].cpu(), x[2])


def test_rotary_turns_back():
    x, pos, freqs = _turn_inputs(100, 4, 64, (10, 10, 12), F32, 3, 1 << 28)
    p, f = pos.cuda(), freqs.cuda()
    there = binding.tc_rotary(x.cuda(), p, f, (10, 10, 12))
    back = binding.tc_rotary(there, p, f, (10, 10, 12), inverse=True)
    # two turns, each off by (|x1| + |x2|) (2^-23 + 4 U32) and a rounding; a turn lengthens neither value beyond the pair's
    size = (x[..., :32].abs() + x[..., 32:].abs()).repeat(1, 1, 2).double()
    _within(back, x.double(), size * 4 * (2.0 ** -23 + 5 * ref.U32), "back")


def test_rotary_empty_and_refusals():
    x, pos, freqs = (t.cuda() for t in _turn_inputs(4, 2, 16, (4, 4), F32, 1))
    assert binding.tc_rotary(x[:0], pos[:0], freqs, (4, 4)).shape == (0, 2, 16)
    assert binding.tc_rotary(x[:, :0], pos, freqs, (4, 4)).shape == (4, 0, 16)
    one = binding.tc_rotary(x, pos[:, :1], freqs)
    assert torch.equal(one, binding.tc_rotary(x, pos[:, :1], freqs, (8,)))
    for bad, kind in ((lambda: binding.tc_rotary(x, pos.long(), freqs, (4, 4)), TypeError), (lambda: binding.tc_rotary(x, pos[:3], freqs, (4, 4)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs.double(), (4, 4)), TypeError), (lambda: binding.tc_rotary(x, pos, freqs, (4, 5)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (8,)), ValueError), (lambda: binding.tc_rotary(x, pos, freqs), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (9, -1)), ValueError), (lambda: binding.tc_rotary(x, pos, freqs, (2 ** 70, 1)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (4.0, 4)), TypeError), (lambda: binding.tc_rotary(x[..., :14], pos, freqs, (4, 4)), binding.TopoError),
                      (lambda: binding.tc_rotary(x[..., ::2], pos, freqs[:4], (2, 2)), ValueError), (lambda: binding.tc_rotary(x[0, 0], pos, freqs, (4, 4)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (4, 4), out=x[:1].clone().expand(4, 2, 16)), binding.TopoError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (4, 4), out=x[:1].expand(4, 2, 16)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (4, 4), out=x[:3]), ValueError), (lambda: binding.tc_rotary(x, pos, freqs, (4, 4), out=x.half()), TypeError),
                      (lambda: binding.tc_rotary(x, pos, freqs.clone().requires_grad_(), (4, 4)), ValueError),
                      (lambda: binding.tc_rotary(x, pos, freqs, (4, 4), out=x.clone().requires_grad_()), ValueError),
                      (lambda: binding.tc_rotary(x.clone().requires_grad_(), pos, freqs, (4, 4), out=x), ValueError)):
        with pytest.raises(kind):
            bad()


# ------------------------------------------------------------------ 4-bit rows


def _wild(rows, c, dtype, seed):
    """Rows with values of all sizes, ties, zeros and blocks of zeros."""
    g = _gen(seed)
    x = torch.randn(rows, c, generator=g) * torch.exp(2 * torch.randn(rows, c, generator=g))
    x = torch.where(torch.rand(rows, c, generator=g) < 0.2, torch.round(x * 4) / 4, x)
    x = torch.where(torch.rand(rows, c, generator=g) < 0.1, torch.zeros_like(x), x)
    x[::5, :32] = 0
    if rows > 2 and c > 40:
        x[1, 33:40] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        x[1, 32] = -7.0
    return x.to(dtype)


def _check_quantised(x, xd):
    q, scale = binding.tc_quantise_mx4(xd)
    codes, want = ref.quantise_mx4(x)
    assert torch.equal(scale.cpu(), want)
    got = ref.unpack(q.cpu(), x.shape[1])
    assert torch.equal(got % 8, codes % 8) and torch.equal(got[codes % 8 != 0], codes[codes % 8 != 0])
    if x.shape[1] % 2:
        assert bool((q[:, -1] < 16).all())
    for dtype in (F32, F16, BF16):
        back = binding.tc_dequantise_mx4(q, scale, channels=x.shape[1], out_dtype=dtype)
        v = ref.values(codes, want).to(dtype)
        assert back.shape == x.shape and torch.equal(back.cpu().nan_to_num(7e7), v.nan_to_num(7e7))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,c", [(1, 1), (1, 2), (3, 31), (2, 32), (5, 33), (40, 8), (7, 64), (9, 75), (130, 100), (1, 1024), (33, 2050), (2, 20001)])
def test_quantise(rows, c, dtype):
    print(f"[mx4 rows] {rows} x {c} {dtype}", flush=True)
    x = _wild(rows, c, dtype, rows + c)
    _check_quantised(x, x.cuda())
    _check_quantised(x, _view(x, 3, 1))
    _check_quantised(x, _view(x, 8, 0))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quantise_ends_of_the_range(dtype):
    g = _gen(2)
    top = 60000.0 if dtype == F16 else 3.3e38
    sizes = (6e-8, 1e-6, 1e-4, top / 8, top) if dtype == F16 else (1e-45, 1e-40, 3e-39, 1e-38, 2.4e-38, 4.8e-38, 1e-37, 1e30, top / 8, top)
    for size in sizes:
        x = ((2 * torch.rand(8, 96, generator=g).double() - 1) * size).to(dtype)
        x[0, 5] = x[0, 40] = -size
        _check_quantised(x, x.cuda())


def test_quantise_not_finite_blocks():
    x = torch.randn(6, 100, generator=_gen(1))
    x[0, 3], x[1, 99], x[2, 40], x[2, 41] = float("inf"), float("nan"), -float("inf"), 3e38
    for dtype in (F32, F16, BF16):
        t = x.to(dtype)
        if dtype == F16:
            t[2, 41] = 1.0
        _check_quantised(t, t.cuda())
        q, scale = binding.tc_quantise_mx4(t.cuda())
        assert int((scale == 255).sum()) == 3 and float(q[0, :16].sum()) == 0


def test_dequantise_every_code():
    """Every code under every scale, in rows of a wider table."""
    q = torch.arange(256, dtype=torch.uint8).view(1, 256).expand(256, 256).contiguous()
    scale = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous()
    want = ref.values(ref.unpack(q, 512), scale)
    for dtype in (F32, F16, BF16):
        out = binding.tc_dequantise_mx4(_view(q, 5, 2), _view(scale, 1, 3), out_dtype=dtype).cpu()
        v = want.to(dtype)  # to 32 bits exactly, or to infinity
        assert torch.equal(out.isnan(), v.isnan()) and torch.equal(out.nan_to_num(0.0), v.nan_to_num(0.0))


# ------------------------------------------------------------------ product of 4-bit rows


def _mx4(rows, k, seed, low=117, high=131):
    g = _gen(seed)
    return (torch.randint(0, 16, (rows, k), generator=g, dtype=torch.uint8),
            torch.randint(low, high, (rows, -(-k // 32)), generator=g, dtype=torch.uint8))


def _product(rows, k, n, dtype, bias, seed, pads=((0, 0), (0, 0), (0, 0), (0, 0)), out=None):
    x, xs = _mx4(rows, k, seed)
    w, ws = _mx4(n, k, seed + 1)
    b = torch.randn(n, generator=_gen(seed + 2)) if bias else None
    packed = [ref.pack(x), xs, ref.pack(w), ws]
    if k % 2:  # beyond an odd number of channels there may be anything
        packed[0][:, -1] |= 0xb0
        packed[2][:, -1] |= 0x70
    got = binding.tc_matmul_mx4(*[_view(t, *p) for t, p in zip(packed, pads)], channels=k, bias=None if b is None else b.cuda(),
                                out_dtype=None if out is not None else dtype, out=out)
    want, mag = ref.matmul_mx4(x, xs, w, ws, b)
    _within(got, want, ref.matmul_mx4_bound(want, mag, k, dtype), f"{rows} x {k} -> {n} {dtype}")
    return got


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 32, 16), (3, 31, 5), (17, 33, 40), (16, 128, 64), (2, 1024, 512), (1, 2000, 33), (40, 601, 77),
                                      (130, 256, 100), (100, 160, 300), (65, 4096, 130), (260, 96, 520), (300, 1056, 48)])
def test_matmul(rows, k, n, dtype):
    print(f"[mx4 matmul] {rows} x {k} -> {n} {dtype}", flush=True)
    _product(rows, k, n, dtype, n % 2 == 0, rows + k + n)


@pytest.mark.parametrize("pads", [((1, 0), (0, 0), (0, 0), (0, 0)), ((0, 0), (1, 1), (0, 0), (0, 3)), ((16, 16), (0, 0), (16, 0), (0, 0)),
                                  ((3, 2), (2, 1), (1, 4), (5, 0)), ((0, 8), (4, 4), (8, 0), (16, 0))])
def test_matmul_strides_and_alignment(pads):
    for rows, k, n in ((70, 256, 48), (150, 544, 130), (9, 101, 20), (300, 128, 600)):
        _product(rows, k, n, BF16, True, k, pads)


def test_matmul_into_a_part():
    for rows, k, n in ((33, 100, 40), (300, 256, 200), (1, 64, 17)):
        wide = torch.full((rows, n + 9), 3.0, device="cuda")
        out = wide[:, 4:4 + n]
        assert _product(rows, k, n, F32, True, 3, out=out) is out
        assert bool((wide[:, :4] == 3).all()) and bool((wide[:, 4 + n:] == 3).all())


def test_matmul_one_weight_or_row_for_all():
    x, xs = _mx4(50, 96, 1)
    w, ws = _mx4(1, 96, 2)
    got = binding.tc_matmul_mx4(ref.pack(x).cuda(), xs.cuda(), ref.pack(w).cuda().expand(70, 48), ws.cuda().expand(70, 3), out_dtype=F32)
    want, mag = ref.matmul_mx4(x, xs, w.expand(70, 96), ws.expand(70, 3), None)
    _within(got, want, ref.matmul_mx4_bound(want, mag, 96, F32), "one weight")


@pytest.mark.parametrize("rows,n", [(4, 20), (200, 150), (300, 520)])
def test_matmul_scales(rows, n):
    """Scales at the ends of the range, and NaN where a block's scale says so: in its row or column alone."""
    k = 200
    x, xs = _mx4(rows, k, 5, 0, 2)
    w, ws = _mx4(n, k, 6, 252, 255)
    xs[2, 3], ws[7, 0] = 255, 255
    x[2, 96:128] = 0  # NaN times zero
    got = binding.tc_matmul_mx4(ref.pack(x).cuda(), xs.cuda(), ref.pack(w).cuda(), ws.cuda(), out_dtype=F32).cpu()
    nan = torch.zeros(rows, n, dtype=torch.bool)
    nan[2], nan[:, 7] = True, True
    assert torch.equal(got.isnan(), nan)
    want, mag = ref.matmul_mx4(x, xs.where(xs < 255, 0), w, ws.where(ws < 255, 0), None)
    _within(got[~nan], want[~nan], ref.matmul_mx4_bound(want, mag, k, F32)[~nan], "finite")


def test_matmul_empty_and_refusals():
    x, xs = (t.cuda() for t in _mx4(4, 64, 1))
    q = x[:, :32].contiguous()
    w, ws = q.clone(), xs.clone()
    assert binding.tc_matmul_mx4(q[:0], xs[:0], w, ws).shape == (0, 4)
    assert binding.tc_quantise_mx4(torch.zeros(0, 64, device="cuda"))[0].shape == (0, 32)
    assert binding.tc_dequantise_mx4(q[:0], xs[:0]).shape == (0, 64)
    f = binding.tc_matmul_mx4
    for bad, kind in ((lambda: f(q, xs, w[:, :31], ws), ValueError), (lambda: f(q, xs[:, :1], w, ws), ValueError), (lambda: f(q, xs[:3], w, ws), ValueError),
                      (lambda: f(q, xs, w, ws, channels=62), ValueError), (lambda: f(q, xs, w, ws, channels=65), ValueError),
                      (lambda: f(q.int(), xs, w, ws), TypeError), (lambda: f(q, xs.float(), w, ws), TypeError), (lambda: f(q, xs, w, ws, bias=xs[0]), TypeError),
                      (lambda: f(q, xs, w, ws, bias=torch.zeros(5, device="cuda")), ValueError), (lambda: f(q, xs, w, ws, out_dtype=torch.int32), TypeError),
                      (lambda: f(q, xs, w, ws, out=torch.zeros(4, 3, device="cuda")), ValueError),
                      (lambda: f(q, xs, w, ws, out=torch.zeros(1, 4, device="cuda").expand(4, 4)), ValueError),
                      (lambda: f(q, xs, w, ws, out_dtype=BF16, out=torch.zeros(4, 4, device="cuda")), ValueError),
                      (lambda: f(q.t().contiguous().t(), xs, w, ws), ValueError), (lambda: f(q[0], xs, w, ws), ValueError),
                      (lambda: binding.tc_dequantise_mx4(q, xs, channels=10), ValueError), (lambda: binding.tc_dequantise_mx4(q, xs, out_dtype=torch.uint8), TypeError),
                      (lambda: binding.tc_quantise_mx4(q), TypeError), (lambda: binding.tc_quantise_mx4(q.float()[0]), ValueError),
                      (lambda: binding.tc_quantise_mx4(torch.zeros(3, 0, device="cuda")), binding.TopoError)):
        with pytest.raises(kind):
            bad()
