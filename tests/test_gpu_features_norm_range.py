"""The norm on rows far from magnitude one, against its definition in 64 bits: the squares of finite rows
leave the range of 32 bits on either side, the norm does not."""
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

WIDTHS = [3, 8, 100, 128, 1000, 2056, 8200, 16392]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size,eps", [(1e18, 1e-6), (3e19, 1e-6), (1e25, 0.0), (5e37, 1e-6), (1e-15, 0.0), (8e-16, 0.0), (2e-16, 1e-32),
                                      (1e-18, 0.0), (1e-24, 0.0),
                                      (1e-30, 1e-35), (1e-36, 0.0), (1e-39, 0.0)])
def test_norm_range(size, eps, dtype):
    """5e37: six deviations below the largest value. 1e-39: below the normal range, where s leaves
    32 bits (rstd is infinite) and the outputs do not."""
    for c in WIDTHS:
        g = torch.Generator().manual_seed(c)
        x = (torch.randn(6, c, generator=g, dtype=torch.float64).clamp(-6, 6) * size).to(dtype)
        x[0, 0] = size  # no row of zeros among the narrow ones
        x[1:, 0] = torch.where((x[1:] == 0).all(1), torch.tensor(size, dtype=dtype), x[1:, 0])
        w = (1 + 0.3 * torch.randn(c, generator=g)).to(dtype)
        want, s = ref.rms_norm(x, w, eps)
        out, _, rstd = binding.tc_rms_norm(x.cuda(), w.cuda(), eps=eps)
        bad = ~((out.double().cpu() - want).abs() <= ref.rms_norm_bound(want, dtype))
        assert not bool(bad.any()), f"{c} channels: out {int(bad.sum())} of {bad.numel()} off"
        fits = s < torch.finfo(F32).max
        # s below 2^-126 has fewer bits
        assert bool(((rstd.double().cpu() - s).abs() <= s * ((c + 1) / 2 + 8) * ref.U32 + ref.tiny(F32))[fits].all())
        assert bool(rstd.cpu()[~fits].isinf().all())
        q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), w.cuda(), eps=eps)
        want_q, want_scale = ref.rms_norm_i8(x, w, s)
        assert torch.equal(q.cpu(), want_q), f"{c} channels"
        assert bool(((scale.double().cpu() - want_scale).abs() <= want_scale * ((c + 1) / 2 + 10) * ref.U32).all()), \
            f"{c} channels: scale"


def test_norm_large_weights():
    """h w leaves 32 bits, q and the scale do not."""
    for c in WIDTHS:
        g = torch.Generator().manual_seed(c)
        x = torch.randn(4, c, generator=g).clamp(-6, 6) * 1e30
        w = torch.randn(c, generator=g).clamp(-6, 6) * 1e20
        _, s = ref.rms_norm(x, w, 1e-6)
        q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), w.cuda(), eps=1e-6)
        want_q, want_scale = ref.rms_norm_i8(x, w, s)
        assert torch.equal(q.cpu(), want_q)
        assert bool(((scale.double().cpu() - want_scale).abs() <= want_scale * ((c + 1) / 2 + 10) * ref.U32).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_far_rows_beside_others(dtype):
    """Rows of every size in one call; an infinity, a NaN and a row of zeros keep what they had."""
    sizes = [1.0, 3e19, 1e-20, 5e37, 1e-30, 0.0]
    for c in (8, 100, 2056):
        g = torch.Generator().manual_seed(c)
        x = torch.stack([torch.randn(c, generator=g).clamp(-6, 6) * v for v in sizes] + [torch.ones(c)] * 2).to(dtype)
        x[6, 1], x[7, 2] = float("inf"), float("nan")
        want, s = ref.rms_norm(x, None, 1e-6)
        out, _, rstd = binding.tc_rms_norm(x.cuda(), eps=1e-6)
        assert bool(((out.double().cpu() - want).abs() <= ref.rms_norm_bound(want, dtype))[:6].all())
        assert float(rstd[6]) == 0.0 and bool(rstd[7].isnan())
        q, scale, _ = binding.tc_rms_norm_i8(x.cuda(), eps=1e-6)
        want_q, want_scale = ref.rms_norm_i8(x, None, s)
        assert torch.equal(q.cpu(), want_q) and bool(scale[6:].isnan().all())
        off = (scale.double().cpu() - want_scale).abs()[:6]
        assert bool((off <= want_scale[:6] * ((c + 1) / 2 + 10) * ref.U32 + ref.tiny(F32)).all())
