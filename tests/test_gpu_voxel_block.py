"""The example block (examples/voxel_block.py) on the GPU: every step of its serving path
against the step's definition in 64 bits, and its training step's gradients."""
import pytest
import torch

from examples import voxel_block
from tests import feature_ref as ref
from topology_construction_amd import binding, synth

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_serving_path():
    ijk, offsets = synth.make_config(1)
    src, kmap, fine_map = voxel_block.maps_of(ijk, offsets)
    x = torch.randn(src.voxel_total(), 32, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    trace = []
    out, fine = voxel_block.Block(32, 96).serve(x, kmap, fine_map, trace)
    assert out.shape == x.shape and fine.shape == (8 * x.shape[0], 16) and len(trace) == 4
    for op, h, gain, q, s, m, w, ws, bias, y in [[v.cpu() if torch.is_tensor(v) else v for v in t] for t in trace]:
        _, rstd = ref.rms_norm(h, gain, 1e-6)
        want_q, want_s = ref.rms_norm_i8(h, gain, rstd)
        assert torch.equal(q, want_q)
        assert bool(((s.double() - want_s).abs() <= want_s * ((h.shape[1] + 1) / 2 + 10) * ref.U32).all())
        if op == "matmul":
            want, mag = ref.matmul_i8(q, s, w, ws, bias)
            bound = ref.product_bound(want, mag, BF16)
        else:
            want, mag = ref.sparse_conv_i8(q, s, m, w, ws, bias)
            bound = ref.product_bound(want, mag, BF16, m.shape[1])
        assert bool(((y.double() - want).abs() <= bound).all()), op


def test_training_step():
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(300, 48, generator=g).to(BF16).cuda().requires_grad_() for _ in range(2))
    w = torch.rand(48, generator=g).cuda().requires_grad_()
    dy, dh = (torch.randn(300, 48, generator=g).to(BF16).cuda() for _ in range(2))
    out, h = voxel_block.RmsNorm.apply(x, r, w)
    gx, gr, gw = torch.autograd.grad([out, h], [x, r, w], [dy, dh])
    assert torch.equal(gx, gr)
    hc = h.detach().cpu()
    _, _, rstd = binding.tc_rms_norm(h.detach(), w.detach())
    dx, dw, bound, mag = ref.rms_norm_grad(dy.cpu(), hc, w.detach().cpu(), rstd.cpu(), dh.cpu())
    bound = bound + dx.abs() * ref.half_step(BF16) * (1 + 2 ** -6) + ref.tiny(BF16)
    assert bool(((gx.double().cpu() - dx).abs() <= bound).all())
    assert bool(((gw.double().cpu() - dw).abs() <= mag * (300 + 8) * ref.U32).all())
    target = torch.randn(300, 48, generator=g).cuda()
    losses = voxel_block.train(x.detach(), r.detach(), target, 4)
    assert losses[-1] < losses[0]
