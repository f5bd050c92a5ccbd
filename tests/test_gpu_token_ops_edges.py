"""Calls of the layer norm, the rotary positions and the 4-bit rows that their documentation allows and ordinary use does not
make: large heads, shared tensors, sections of other sequences, tiny eps beside large rows."""
import numpy as np
import pytest
import torch

from tests import token_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# tables of sines as large as a workgroup's part of LDS, with rows enough for every workgroup to want several
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,heads,dim,pairs", [(9000, 1, 4096, 2048), (5000, 2, 4096, 1500), (9000, 1, 4094, 2047), (20_000, 1, 1024, 512)])
def test_rotary_large_heads(rows, heads, dim, pairs, dtype):
    x = torch.randn(rows, heads, dim, generator=_gen(1), device="cuda").to(dtype)
    pos = torch.randint(-500, 500, (rows, 1), generator=_gen(2), device="cuda", dtype=torch.int32)
    freqs = torch.rand(pairs, generator=_gen(3), device="cuda")
    at = torch.tensor([0, 1, 2, 7, 8, 500, rows - 9, rows - 1])
    for interleaved in (False, True):
        out = binding.tc_rotary(x, pos, freqs, interleaved=interleaved)
        want, bound = ref.rotary(x[at.cuda()].cpu(), pos[at.cuda()].cpu(), freqs.cpu(), (pairs,), interleaved, False, dtype)
        assert bool(((out[at.cuda()].double().cpu() - want).abs() <= bound).all())


def test_rotary_out_beside_x():
    """Queries of a packed row turned into the place of its keys; what overlaps x without being x is refused."""
    packed = torch.randn(50, 6, 32, generator=_gen(1), device="cuda")
    pos, freqs = torch.arange(50, dtype=torch.int32, device="cuda")[:, None], torch.rand(16, generator=_gen(2), device="cuda")
    want = binding.tc_rotary(packed[:, :3], pos, freqs)
    before = packed.clone()
    assert torch.equal(binding.tc_rotary(packed[:, :3], pos, freqs, out=packed[:, 3:]), want)
    assert torch.equal(packed[:, :3], before[:, :3])
    flat = torch.randn(51 * 32, device="cuda")
    with pytest.raises(ValueError):
        binding.tc_rotary(flat[:50 * 32].view(50, 1, 32), pos, freqs, out=flat[32:].view(50, 1, 32))
    square = torch.randn(50, 50, 32, device="cuda")
    with pytest.raises(ValueError):
        binding.tc_rotary(square, pos, freqs, out=square.transpose(0, 1))


def test_rotary_sections_of_any_sequence():
    x = torch.randn(9, 2, 24, generator=_gen(1), device="cuda").requires_grad_()
    pos, freqs = torch.randint(0, 9, (9, 3), generator=_gen(2), device="cuda", dtype=torch.int32), torch.rand(12, generator=_gen(3), device="cuda")
    want = binding.tc_rotary(x.detach(), pos, freqs, (3, 4, 5))
    sections = [3, 4, 5]
    out = binding.tc_rotary(x, pos, freqs, sections)
    sections[0] = 99  # the backward has its own
    (grad,) = torch.autograd.grad(out, x, torch.ones_like(x))
    assert torch.equal(out, want) and torch.equal(grad, binding.tc_rotary(torch.ones_like(x), pos, freqs, (3, 4, 5), inverse=True))
    for other in (np.array([3, 4, 5]), torch.tensor([3, 4, 5]), range(3, 6)):
        assert torch.equal(binding.tc_rotary(x.detach(), pos, freqs, other), want)


def test_rotary_frequencies_of_any_size():
    """Zero, huge and negative ones; what is not finite makes its own pairs NaN and no other."""
    x = torch.randn(4, 1, 16, generator=_gen(1), device="cuda")
    pos = torch.tensor([[0], [1], [-7], [3]], dtype=torch.int32, device="cuda")
    freqs = torch.tensor([0.0, -0.5, 1e20, 3e38, 1e-45, float("inf"), float("nan"), 2.0], device="cuda")
    out = binding.tc_rotary(x, pos, freqs)
    size = (x[..., :8].square() + x[..., 8:].square())
    after = (out[..., :8].square() + out[..., 8:].square())
    bad = torch.tensor([5, 6], device="cuda")
    assert bool(out[..., bad].isnan().all()) and bool(out[..., bad + 8].isnan().all())
    fine = torch.tensor([0, 1, 2, 3, 4, 7], device="cuda")
    # a turn keeps a pair's length: cos^2 + sin^2 is off by 4 2^-23, the products and sums by a few roundings
    assert bool(((after - size)[..., fine].abs() <= size[..., fine] * (8 * 2.0 ** -23 + 16 * ref.U32)).all())
    assert torch.equal(out[..., 0], x[..., 0]) and torch.equal(out[0, :, fine], x[0, :, fine])


@pytest.mark.parametrize("c", [3, 100, 1024, 20_000])
def test_layer_norm_tiny_eps_beside_large_rows(c):
    """Constant rows: their units are zero however large s is."""
    for value, eps in ((1e20, 1e-38), (-3e38, 1e-30), (7.0, 1e-38)):
        h = torch.full((5, c), value, device="cuda")
        w, b = torch.rand(c, generator=_gen(1), device="cuda") + 0.5, torch.randn(c, generator=_gen(2), device="cuda")
        out, _, mean, rstd = binding.tc_layer_norm(h, w, b, eps=eps)
        assert torch.equal(out, b.expand(5, c)) and bool((mean == h[0, 0]).all())
        dy = torch.randn(5, c, generator=_gen(3), device="cuda")
        got = binding.tc_layer_norm_backward(dy, h, w, mean, rstd)
        (dx, dw, db), (off, mag_w, mag_b, off_w) = ref.layer_norm_grad(dy.cpu(), h.cpu(), w.cpu(), mean.cpu(), rstd.cpu(), None, F32)
        assert bool(((got[0].double().cpu() - dx).abs() <= off).all())
        assert float(got[1].abs().max()) == 0


def test_layer_norm_of_shared_and_repeated_rows():
    """One row for all, the weight as the bias, x as its own residual and gradient."""
    row = torch.randn(1, 300, generator=_gen(4), device="cuda")
    w = torch.randn(300, generator=_gen(5), device="cuda")
    x = row.expand(70, 300)
    out, h, mean, rstd = binding.tc_layer_norm(x, w, w, residual=x)
    one = binding.tc_layer_norm(row, w, w, residual=row)
    assert all(torch.equal(a, b.expand(a.shape)) for a, b in zip((out, h, mean, rstd), one))
    gx, gw, gb = binding.tc_layer_norm_backward(x, h, w, mean, rstd, grad_h=x)
    first = binding.tc_layer_norm_backward(row, one[1], w, one[2], one[3], grad_h=row)
    assert torch.equal(gx, first[0].expand(70, 300))
    # 70 equal terms in any order
    assert bool(((gb - 70 * row[0]).abs() <= 70 * row[0].abs() * 71 * ref.U32).all())


def test_matmul_of_the_same_rows():
    """x as its own weights: a symmetric product."""
    q, s = binding.tc_quantise_mx4(torch.randn(300, 500, generator=_gen(6), device="cuda"))
    out = binding.tc_matmul_mx4(q, s, q, s, out_dtype=F32)
    codes = ref.unpack(q.cpu(), 500)
    want, mag = ref.matmul_mx4(codes, s.cpu(), codes, s.cpu(), None)
    assert bool(((out.double().cpu() - want).abs() <= ref.matmul_mx4_bound(want, mag, 500, F32)).all())


def test_inference_mode():
    with torch.inference_mode():
        x = torch.randn(20, 64, generator=_gen(1), device="cuda")
        w = torch.nn.Parameter(torch.ones(64, device="cuda"))
        out, h, mean, rstd = binding.tc_layer_norm(x, w)
        q = binding.tc_quantise_mx4(out)
        y = torch.empty(20, 20, device="cuda")
        binding.tc_matmul_mx4(*q, *q, out=y)
        binding.tc_rotary(y, torch.zeros(20, 1, dtype=torch.int32, device="cuda"), torch.ones(10, device="cuda"), out=y)
    assert torch.equal(y, binding.tc_matmul_mx4(*q, *q, out_dtype=F32))
