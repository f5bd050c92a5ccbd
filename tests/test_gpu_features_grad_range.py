"""The norm's gradient on rows far from magnitude one, against its definition in 64 bits: every factor of
it is in range there (s up to 2^100, g / s as small), so it has to be as near as anywhere else."""
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# one lane a row, some lanes, a wave, a workgroup; fewer channels than a vector, more than registers hold
WIDTHS = [3, 8, 100, 128, 1000, 2056, 8200, 16392]


def _inputs(rows, c, dtype, size, seed):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(rows, c, generator=g) * size).to(dtype)
    w = (1 + 0.3 * torch.randn(c, generator=g)).to(dtype)
    return h, w, torch.randn(rows, c, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size,eps", [(1e14, 1e-6), (1e15, 1e-6), (1e18, 1e-6), (1e30, 1e-6), (1e-14, 0.0), (1e-13, 1e-30),
                                      (1e-30, 0.0)])
def test_norm_grad_range(size, eps, dtype):
    for c in WIDTHS:
        rows = 5
        h, w, dy = _inputs(rows, c, dtype, size, c)
        _, s = ref.rms_norm(h, w, eps)
        rstd = s.float()
        assert bool(torch.isfinite(rstd).all()) and float(rstd.min()) > 1e-37
        dx, dw, bound, mag = ref.rms_norm_grad(dy, h, w, rstd, None)
        bound = bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype)
        gx, gw = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
        bad = ~((gx.double().cpu() - dx).abs() <= bound)
        assert not bool(bad.any()), f"{c} channels: grad_x {int(bad.sum())} of {bad.numel()} off"
        assert bool(((gw.double().cpu() - dw).abs() <= mag * (rows + 8) * ref.U32).all()), f"{c} channels: grad_weight"
        gx, _ = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), None, rstd.cuda())
        dx, _, bound, _ = ref.rms_norm_grad(dy, h, None, rstd, None)
        bound = bound + dx.abs() * ref.half_step(dtype) * (1 + 2 ** -6) + ref.tiny(dtype)
        assert bool(((gx.double().cpu() - dx).abs() <= bound).all()), f"{c} channels: grad_x without weight"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [100, 16392])
def test_norm_weight_grad_range(c, dtype):
    """dy h leaves 32 bits where dy h s does not."""
    h, w, dy = _inputs(3, c, dtype, 1e30, c)
    dy = dy * 1e12
    _, s = ref.rms_norm(h, w, 0.0)
    rstd = s.float()
    _, dw, _, mag = ref.rms_norm_grad(dy, h, w, rstd, None)
    _, gw = binding.tc_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
    assert bool(((gw.double().cpu() - dw).abs() <= mag * 11 * ref.U32).all())
