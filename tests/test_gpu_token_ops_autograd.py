"""tc_layer_norm and tc_rotary on tensors that require a gradient: graphs whose backward is the operators' own."""
import pytest
import torch

from tests import token_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


def _leaves(rows, c, dtype, wdtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, r = (torch.randn(rows, c, generator=g).to(dtype).cuda().requires_grad_() for _ in range(2))
    w, b = ((1 + 0.3 * torch.randn(c, generator=g)).to(wdtype).cuda().requires_grad_() for _ in range(2))
    dy, dh = (torch.randn(rows, c, generator=g).to(dtype).cuda() for _ in range(2))
    return x, r, w, b, dy, dh


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (F16, F16), (BF16, BF16), (BF16, F32)])
def test_layer_norm_gradients_are_the_operators(dtype, wdtype):
    x, r, w, b, dy, dh = _leaves(130, 72, dtype, wdtype)
    out, h, mean, rstd = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS)
    assert out.requires_grad and h.requires_grad and not mean.requires_grad and not rstd.requires_grad
    with torch.no_grad():
        plain = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS)
    assert not plain[0].requires_grad and all(torch.equal(a, c) for a, c in zip((out, h, mean, rstd), plain))
    gx, gr, gw, gb = torch.autograd.grad([out, h], [x, r, w, b], [dy, dh])
    want = binding.tc_layer_norm_backward(dy, plain[1], w, plain[2], plain[3], grad_h=dh)
    assert torch.equal(gx, want[0]) and torch.equal(gr, want[0])
    assert gw.dtype == gb.dtype == wdtype and torch.equal(gw, want[1].to(wdtype)) and torch.equal(gb, want[2].to(wdtype))
    (dx, _, _), (bound, _, _, _) = ref.layer_norm_grad(dy.cpu(), plain[1].cpu(), w.detach().cpu(), mean.cpu(), rstd.cpu(), dh.cpu(), dtype)
    assert bool(((gx.double().cpu() - dx).abs() <= bound).all())


def test_layer_norm_parts():
    """One output, one leaf, no weight, no bias, no residual."""
    x, r, w, b, dy, dh = _leaves(20, 100, BF16, F32, 1)
    out, h, mean, rstd = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS)
    gx, gb = torch.autograd.grad(out, [x, b], dy, retain_graph=True)
    want = binding.tc_layer_norm_backward(dy, h.detach(), w.detach(), mean, rstd)
    assert torch.equal(gx, want[0]) and torch.equal(gb, want[2])
    gx, gr, gw, gb = torch.autograd.grad(h, [x, r, w, b], dh, allow_unused=True)
    assert torch.equal(gx, dh) and torch.equal(gr, dh) and gw is None and gb is None
    out, h, mean, rstd = binding.tc_layer_norm(x, w, eps=EPS)
    assert h is x
    gx, gw = torch.autograd.grad([out, h * 1.0], [x, w], [dy, dh])  # h's other uses reach x by themselves
    want = binding.tc_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd)
    assert torch.equal(gx, want[0] + dh) and torch.equal(gw, want[1])
    out, _, mean, rstd = binding.tc_layer_norm(x.detach(), None, b, eps=EPS)
    (gb,) = torch.autograd.grad(out, b, dy)
    assert torch.equal(gb, binding.tc_layer_norm_backward(dy, x.detach(), None, mean, rstd)[2])
    out, _, mean, rstd = binding.tc_layer_norm(x, eps=EPS)
    (gx,) = torch.autograd.grad(out, x, dy)
    assert torch.equal(gx, binding.tc_layer_norm_backward(dy, x.detach(), None, mean, rstd, with_bias=False)[0])


def test_layer_norm_gradients_of_any_layout():
    """A sum's gradient is one value with strides 0; a transposed product's has channels apart; broadcast inputs add up."""
    x, r, w, b, dy, _ = _leaves(40, 48, F32, F32, 3)
    out, h, mean, rstd = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS)
    one = torch.ones_like(dy)
    gx, gb = torch.autograd.grad(out.sum() + h.sum(), [x, b], retain_graph=True)
    want = binding.tc_layer_norm_backward(one, h.detach(), w.detach(), mean, rstd, grad_h=one)
    assert torch.equal(gx, want[0]) and torch.equal(gb, want[2])
    across = dy.t().contiguous().t()
    (gx,) = torch.autograd.grad([out, h], [x], [across, across])
    assert torch.equal(gx, binding.tc_layer_norm_backward(dy, h.detach(), w.detach(), mean, rstd, grad_h=dy)[0])
    row = torch.randn(1, 48, generator=torch.Generator().manual_seed(5)).cuda().requires_grad_()
    out, h, mean, rstd = binding.tc_layer_norm(x, w, b, residual=row.expand(40, 48), eps=EPS)
    gx, grow = torch.autograd.grad(out, [x, row], dy)
    want = binding.tc_layer_norm_backward(dy, h.detach(), w.detach(), mean, rstd)[0]
    assert torch.equal(gx, want)
    assert bool(((grow.double() - want.double().sum(0, keepdim=True)).abs() <= want.double().abs().sum(0, keepdim=True) * 41 * ref.U32).all())
    same = x.detach().clone().requires_grad_()
    out, h, mean, rstd = binding.tc_layer_norm(same, w, b, residual=same, eps=EPS)  # the same tensor twice
    (g,) = torch.autograd.grad(out, same, dy)
    assert torch.equal(g, 2 * binding.tc_layer_norm_backward(dy, h.detach(), w.detach(), mean, rstd)[0])


def test_no_rows_and_refusals():
    x, r, w, b, dy, _ = _leaves(8, 16, F32, F32, 8)
    out = binding.tc_layer_norm(x[:0], w, b, eps=EPS)[0]
    gx, gw, gb = torch.autograd.grad(out.sum(), [x, w, b])
    assert float(gx.abs().sum() + gw.abs().sum() + gb.abs().sum()) == 0
    out = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS)[0]
    (gx,) = torch.autograd.grad(out, x, dy, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        binding.tc_layer_norm(fwd.make_dual(x.detach(), dy), w.detach(), eps=EPS)
    with pytest.raises(TypeError):
        binding.tc_layer_norm(x, residual=r.half())
    with pytest.raises(ValueError):
        binding.tc_layer_norm(x, w, b[:7])
    with pytest.raises(binding.TopoError):
        binding.tc_layer_norm(x, w, eps=float("nan"))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_gradient_is_the_turn_back(dtype, interleaved):
    g = torch.Generator().manual_seed(1)
    base = torch.randn(30, 5, 40, generator=g).to(dtype).cuda().requires_grad_()
    pos, freqs = torch.randint(-99, 99, (30, 3), generator=g, dtype=torch.int32).cuda(), torch.rand(18, generator=g).cuda()
    dy = torch.randn(30, 3, 40, generator=g).to(dtype).cuda()
    part = base[:, 1:4]
    out = binding.tc_rotary(part, pos, freqs, (8, 4, 6), interleaved)
    with torch.no_grad():
        assert torch.equal(out, binding.tc_rotary(part, pos, freqs, (8, 4, 6), interleaved))
    (grad,) = torch.autograd.grad(out, base, dy, retain_graph=True)
    want = binding.tc_rotary(dy, pos, freqs, (8, 4, 6), interleaved, inverse=True)
    assert torch.equal(grad[:, 1:4], want) and float(grad[:, 0].abs().sum() + grad[:, 4].abs().sum()) == 0
    exact, bound = ref.rotary(dy.cpu(), pos.cpu(), freqs.cpu(), (8, 4, 6), interleaved, True, dtype)
    assert bool(((want.double().cpu() - exact).abs() <= bound).all())
    for layout in (dy.transpose(0, 1).contiguous().transpose(0, 1), dy.transpose(0, 2).contiguous().transpose(0, 2)):
        assert torch.equal(torch.autograd.grad(out, base, layout, retain_graph=True)[0], grad)
    (grad,) = torch.autograd.grad(out.sum(), base)
    assert torch.equal(grad[:, 1:4], binding.tc_rotary(torch.ones_like(dy), pos, freqs, (8, 4, 6), interleaved, inverse=True))
    back = binding.tc_rotary(out, pos, freqs, (8, 4, 6), interleaved, inverse=True)
    (grad,) = torch.autograd.grad(back, out, dy)
    assert torch.equal(grad, binding.tc_rotary(dy, pos, freqs, (8, 4, 6), interleaved))


def test_rotary_positions_that_change_are_seen():
    x, pos, freqs = torch.randn(4, 1, 8, device="cuda", requires_grad=True), torch.ones(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    out = binding.tc_rotary(x, pos, freqs)
    pos += 1
    with pytest.raises(RuntimeError):
        out.sum().backward()


def test_on_another_stream():
    x, r, w, b, dy, dh = _leaves(64, 32, BF16, BF16, 7)
    pos, freqs = torch.arange(64, dtype=torch.int32, device="cuda")[:, None], torch.rand(8, device="cuda")

    def step(stream=None):
        out, h, _, _ = binding.tc_layer_norm(x, w, b, residual=r, eps=EPS, stream=stream)
        if stream is not None:
            stream.synchronize()
        return torch.autograd.grad([out, h], [x, w, b], [dy, dh])

    want = step()
    turned = binding.tc_rotary(dy.view(64, 2, 16), pos, freqs)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(st)
    again = binding.tc_rotary(dy.view(64, 2, 16), pos, freqs, stream=st)
    q = binding.tc_quantise_mx4(dy, stream=st)
    back = binding.tc_dequantise_mx4(*q, stream=st)
    product = binding.tc_matmul_mx4(*q, *q, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and torch.equal(again, turned)
    q = binding.tc_quantise_mx4(dy)
    assert torch.equal(back, binding.tc_dequantise_mx4(*q)) and torch.equal(product, binding.tc_matmul_mx4(*q, *q))
