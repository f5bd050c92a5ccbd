"""A type asked for beside `out` has to be its own."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def _product(rows=6, k=32, n=8):
    g = torch.Generator().manual_seed(0)
    q, w = (torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8).cuda() for m in (rows, n))
    s, ws = (torch.rand(m, generator=g).cuda() for m in (rows, n))
    m = torch.arange(rows, dtype=torch.int32).view(-1, 1).cuda()
    return (lambda **kw: binding.tc_matmul_i8(q, s, w, ws, **kw),
            lambda **kw: binding.tc_sparse_conv_i8(q, s, m, w[None].contiguous(), ws, **kw))


def test_out_dtype_beside_out():
    for call in _product():
        out = torch.zeros(6, 8, device="cuda", dtype=torch.float16)
        call(out=out, out_dtype=torch.float16)
        with pytest.raises(ValueError, match="out_dtype"):
            call(out=out, out_dtype=torch.float32)
        with pytest.raises(TypeError, match="out_dtype"):
            call(out=out, out_dtype="float16")
