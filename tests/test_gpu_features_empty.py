"""Matrices without rows have no strides to speak of: a sum's gradient over no rows comes with strides 0."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("strides", [(0, 0), (1, 0), (5, 2)])
def test_no_rows_of_any_strides(strides):
    e = torch.empty(16, device="cuda").as_strided((0, 8), strides)
    q = torch.empty(16, dtype=torch.int8, device="cuda").as_strided((0, 8), strides)
    none, w = torch.empty(0, device="cuda"), torch.ones(8, device="cuda")
    out, h, rstd = binding.tc_rms_norm(e, w, residual=e)
    assert out.shape == h.shape == (0, 8) and rstd.shape == (0,)
    gx, gw = binding.tc_rms_norm_backward(e, h, w, rstd, grad_h=e)
    assert gx.shape == (0, 8) and bool((gw == 0).all())
    w8, ws = torch.ones(4, 8, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    assert binding.tc_matmul_i8(q, none, w8, ws).shape == (0, 4)
    m = torch.full((3, 1), -1, dtype=torch.int32, device="cuda")
    assert bool((binding.tc_sparse_conv_i8(q, none, m, w8[None], ws) == 0).all())


def test_rows_still_need_unit_channel_stride():
    x = torch.ones(8, 4, device="cuda").t()
    with pytest.raises(ValueError):
        binding.tc_rms_norm(x)
