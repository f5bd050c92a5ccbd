"""tc_rms_norm on tensors that require a gradient: its outputs carry a graph whose backward is
tc_rms_norm_backward."""
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


def _leaves(rows, c, dtype, wdtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, r = ((torch.randn(rows, c, generator=g)).to(dtype).cuda().requires_grad_() for _ in range(2))
    w = (1 + 0.3 * torch.randn(c, generator=g)).to(wdtype).cuda().requires_grad_()
    dy, dh = (torch.randn(rows, c, generator=g).to(dtype).cuda() for _ in range(2))
    return x, r, w, dy, dh


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (F16, F16), (BF16, BF16), (BF16, F32)])
def test_gradients_are_the_operators(dtype, wdtype):
    x, r, w, dy, dh = _leaves(130, 72, dtype, wdtype)
    out, h, rstd = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    assert out.requires_grad and h.requires_grad and not rstd.requires_grad
    with torch.no_grad():
        plain = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    assert not plain[0].requires_grad and all(torch.equal(a, b) for a, b in zip((out, h, rstd), plain))
    gx, gr, gw = torch.autograd.grad([out, h], [x, r, w], [dy, dh])
    want_x, want_w = binding.tc_rms_norm_backward(dy, plain[1], w, plain[2], grad_h=dh)
    assert torch.equal(gx, want_x) and torch.equal(gr, want_x)
    assert gw.dtype == wdtype and torch.equal(gw, want_w.to(wdtype))
    # against the definition, too
    dx, _, bound, _ = ref.rms_norm_grad(dy.cpu(), plain[1].cpu(), w.detach().cpu(), plain[2].cpu(), dh.cpu())
    bound = bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype)
    assert bool(((gx.double().cpu() - dx).abs() <= bound).all())


def test_only_one_output_used():
    x, r, w, dy, dh = _leaves(20, 100, BF16, F32, 1)
    out, h, rstd = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    gx, gw = torch.autograd.grad(out, [x, w], dy, retain_graph=True)
    want_x, want_w = binding.tc_rms_norm_backward(dy, h.detach(), w.detach(), rstd)
    assert torch.equal(gx, want_x) and torch.equal(gw, want_w)
    gx, gr, gw = torch.autograd.grad(h, [x, r, w], dh, allow_unused=True)
    assert torch.equal(gx, dh) and torch.equal(gr, dh) and gw is None


def test_without_residual_or_weight():
    x, _, w, dy, dh = _leaves(33, 64, F32, F32, 2)
    out, h, rstd = binding.tc_rms_norm(x, w, eps=EPS)
    assert h is x
    gx, gw = torch.autograd.grad([out, h * 1.0], [x, w], [dy, dh])  # h's other uses reach x by themselves
    want_x, want_w = binding.tc_rms_norm_backward(dy, x.detach(), w.detach(), rstd)
    assert torch.equal(gx, want_x + dh) and torch.equal(gw, want_w)
    out, _, rstd = binding.tc_rms_norm(x, eps=EPS)
    (gx,) = torch.autograd.grad(out, x, dy)
    assert torch.equal(gx, binding.tc_rms_norm_backward(dy, x.detach(), None, rstd)[0])
    # a weight alone that requires one
    out, _, rstd = binding.tc_rms_norm(x.detach(), w, eps=EPS)
    (gw,) = torch.autograd.grad(out, w, dy)
    assert torch.equal(gw, want_w)


def test_gradients_of_any_layout():
    """A sum's gradient is one value with strides 0; a transposed product's has channels apart."""
    x, r, w, dy, _ = _leaves(40, 48, F32, F32, 3)
    out, h, rstd = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    one = torch.ones_like(dy)
    gx, gw = torch.autograd.grad(out.sum() + h.sum(), [x, w], retain_graph=True)
    want = binding.tc_rms_norm_backward(one, h.detach(), w.detach(), rstd, grad_h=one)
    assert torch.equal(gx, want[0]) and torch.equal(gw, want[1])
    across = dy.t().contiguous().t()
    gx, gw = torch.autograd.grad([out, h], [x, w], [across, across])
    want = binding.tc_rms_norm_backward(dy, h.detach(), w.detach(), rstd, grad_h=dy)
    assert torch.equal(gx, want[0]) and torch.equal(gw, want[1])


def test_broadcast_residual_and_slices():
    x, _, w, dy, dh = _leaves(40, 48, F32, F32, 4)
    row = torch.randn(1, 48, generator=torch.Generator().manual_seed(5)).cuda().requires_grad_()
    out, h, rstd = binding.tc_rms_norm(x, w, residual=row.expand(40, 48), eps=EPS)
    gx, grow = torch.autograd.grad([out, h], [x, row], [dy, dh])
    want = binding.tc_rms_norm_backward(dy, h.detach(), w.detach(), rstd, grad_h=dh)[0]
    assert torch.equal(gx, want)
    bound = want.double().abs().sum(0, keepdim=True) * 41 * ref.U32
    assert bool(((grow.double() - want.double().sum(0, keepdim=True)).abs() <= bound).all())
    wide = torch.randn(40, 100, generator=torch.Generator().manual_seed(6)).cuda().requires_grad_()
    out, _, rstd = binding.tc_rms_norm(wide[:, 3:51], w, eps=EPS)
    (gwide,) = torch.autograd.grad(out, wide, dy)
    want = binding.tc_rms_norm_backward(dy, wide.detach()[:, 3:51], w.detach(), rstd)[0]
    assert torch.equal(gwide[:, 3:51], want) and float(gwide[:, :3].abs().sum() + gwide[:, 51:].abs().sum()) == 0


def test_other_stream_and_no_rows():
    x, r, w, dy, dh = _leaves(64, 32, BF16, BF16, 7)
    out, h, rstd = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    want = torch.autograd.grad([out, h], [x, w], [dy, dh])
    del out, h  # and with them the nodes of the leaves, which belong to the stream they were made on
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, h, _ = binding.tc_rms_norm(x, w, residual=r, eps=EPS, stream=st)
    st.synchronize()
    got = torch.autograd.grad([out, h], [x, w], [dy, dh])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, _, _ = binding.tc_rms_norm(x[:0], w, eps=EPS)
    gx, gw = torch.autograd.grad(out.sum(), [x, w])
    assert float(gx.abs().sum()) == 0 and float(gw.abs().sum()) == 0


def test_second_derivatives_and_tangents_are_refused():
    x, r, w, dy, _ = _leaves(8, 16, F32, F32, 8)
    out, _, _ = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
    (gx,) = torch.autograd.grad(out, x, dy, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        binding.tc_rms_norm(fwd.make_dual(x.detach(), dy), w.detach(), eps=EPS)


def test_refusals_stay_the_same():
    x, r, w, _, _ = _leaves(4, 8, F32, F32, 9)
    with pytest.raises(TypeError):
        binding.tc_rms_norm(x, residual=r.half())
    with pytest.raises(ValueError):
        binding.tc_rms_norm(x, w[:7])
    with pytest.raises(binding.TopoError):
        binding.tc_rms_norm(x, w, eps=float("nan"))


def test_training_step_captured():
    """Forward and backward in one graph, replayed on changed inputs with eager work between."""
    x, r, w, dy, dh = _leaves(300, 64, BF16, F32, 10)

    def step():
        out, h, _ = binding.tc_rms_norm(x, w, residual=r, eps=EPS)
        return torch.autograd.grad([out, h], [x, r, w], [dy, dh])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12, 13):
        with torch.no_grad():
            for t, v in zip((x, r, w, dy, dh), _leaves(300, 64, BF16, F32, seed)):
                t.copy_(v)
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
