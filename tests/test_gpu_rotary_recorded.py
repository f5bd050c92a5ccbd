"""What autograd may not ask of the rotary positions is refused, not left out without a word."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dx = (torch.randn(9, 2, 24, generator=g, device="cuda") for _ in range(2))
    return x, dx, torch.arange(9, dtype=torch.int32, device="cuda")[:, None], torch.rand(10, generator=g, device="cuda")


def test_tangents_are_refused():
    x, dx, pos, freqs = _inputs()
    with fwd.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            binding.tc_rotary(fwd.make_dual(x, dx), pos, freqs)
        with pytest.raises(ValueError):
            binding.tc_rotary(fwd.make_dual(x, dx), pos, freqs, out=torch.empty_like(x))
        with pytest.raises(ValueError):
            binding.tc_rotary(x, pos, fwd.make_dual(freqs, freqs))


def test_second_derivatives_are_refused():
    x, dx, pos, freqs = _inputs()
    x.requires_grad_()
    dx.requires_grad_()
    (grad,) = torch.autograd.grad(binding.tc_rotary(x, pos, freqs), x, dx, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()


def test_frequencies_that_change_are_seen():
    x, dx, pos, freqs = _inputs()
    x.requires_grad_()
    out = binding.tc_rotary(x, pos, freqs)
    freqs.mul_(2)
    with pytest.raises(RuntimeError):
        out.backward(dx)
