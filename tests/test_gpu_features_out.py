"""The products' `out`: autograd sees that it was written."""
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


def test_written_out_is_seen():
    for call in _product():
        out = torch.zeros(6, 8, device="cuda")
        scale = torch.ones(8, device="cuda", requires_grad=True)
        y = (out * scale).sum()  # keeps `out` for the backward
        before = out._version
        assert call(out=out) is out
        assert out._version == before + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        part = torch.zeros(6, 20, device="cuda")
        call(out=part[:, 4:12])
        assert part._version == 1 and torch.equal(part[:, 4:12], out)


def test_out_in_inference_mode():
    for call in _product():
        want = call(out_dtype=torch.float32)
        with torch.inference_mode():
            out = torch.zeros(6, 8, device="cuda")
            call(out=out)
            assert torch.equal(out, want)


def test_out_that_requires_a_gradient_is_refused():
    for call in _product():
        out = torch.zeros(6, 8, device="cuda", requires_grad=True)
        with pytest.raises(ValueError, match="gradient"):
            call(out=out)
        with torch.no_grad():
            call(out=out)
        assert float(out.abs().sum()) > 0
