"""The example transformer block (examples/voxel_tokens.py) on the GPU: every step of its serving path against the step's
definition in 64 bits, and its training path's gradients."""
import pytest
import torch

from examples import voxel_tokens
from tests import token_ref as ref
from topology_construction_amd import binding, synth

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def _voxels(workload=1):
    rows, offsets = synth.make_config(workload)
    src = binding.tc_batch_from_ijk(torch.from_numpy(rows).cuda(), offsets)
    ijk = binding.tc_enumerate_ijk(src)
    return ijk, [int(h["voxel_begin"]) for h in src.headers()] + [ijk.shape[0]]


@pytest.mark.parametrize("channels,heads", [(64, 2), (120, 4)])
def test_serving_path(channels, heads):
    ijk, ends = _voxels()
    x = torch.randn(ijk.shape[0], channels, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    trace = []
    with torch.no_grad():
        out = voxel_tokens.Block(channels, heads, 2 * channels).serve(x, ijk, ends, trace)
    assert out.shape == x.shape and bool(torch.isfinite(out).all())
    assert [t[0] for t in trace] == ["norm", "project", "turn", "turned", "project", "norm", "project", "project"]
    for step in trace:
        t = [v.cpu() if torch.is_tensor(v) else v for v in step[1:]]
        if step[0] == "norm":
            y, residual, gain, shift, h, n = t
            assert torch.equal(h, y if residual is None else (y.float() + residual.float()).to(BF16))
            want, m, s = ref.layer_norm(h, gain, shift, EPS)
            bound = ref.layer_norm_bounds(h, gain, shift, m, s, BF16)[0]
            got = n
        elif step[0] == "turn":
            (before,) = t
            continue
        elif step[0] == "turned":
            at, freqs, sections, got = t
            want, bound = ref.rotary(before, at, freqs, sections, False, False, BF16)
        else:
            a, q, scale, w, w_scale, bias, got = t
            codes, want_scale = ref.quantise_mx4(a)
            mine = ref.unpack(q, a.shape[1])
            assert torch.equal(scale, want_scale) and torch.equal(ref.values(mine, scale), ref.values(codes, want_scale))
            want, mag = ref.matmul_mx4(mine, scale, ref.unpack(w, a.shape[1]), w_scale, bias)
            bound = ref.matmul_mx4_bound(want, mag, a.shape[1], BF16)
        assert bool(((got.double() - want).abs() <= bound).all()), step[0]


def _plain_scores(x, ijk, gain, shift, weight, freqs, sections, heads):
    """The training path's definition in 64 bits, differentiable."""
    n = ref.layer_norm(x, gain, shift, EPS)[0]
    qk = (n @ weight.t()).view(x.shape[0], 2 * heads, -1)
    pairs = freqs.numel()
    angle = ijk.double()[:, ref.axis_of(sections)] * freqs.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = qk[..., :pairs], qk[..., pairs:]
    qk = torch.cat((a * cos - b * sin, a * sin + b * cos), 2)
    return (qk[1:, :heads] * qk[:-1, heads:]).sum(2)


def test_training_gradients():
    """Of the scores along a fixed direction, against the definition's in 64 bits and against a difference of them.

    Every 32-bit step is off by few roundings of its terms: a sum of c terms by (c + 2) U32 of their absolute values. The chain has
    sums over channels (norm, projection, scores) and over voxels (the weights' gradients), at most (4 c + v) U32 of
    the absolute terms' sums in all, which the same expressions over absolute values bound."""
    heads, c = 2, 48
    ijk, _ = _voxels()
    ijk = ijk[:300].contiguous()
    g = torch.Generator().manual_seed(2)
    sections, freqs = voxel_tokens.axes_of(c // heads)
    x, gain, shift = torch.randn(300, c, generator=g), 1 + 0.2 * torch.randn(c, generator=g), 0.2 * torch.randn(c, generator=g)
    weight, dy = torch.randn(2 * c, c, generator=g) / c ** 0.5, torch.randn(299, heads, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, gain, shift, weight)]
    out = voxel_tokens.scores(leaves[0], ijk, *leaves[1:], freqs.cuda(), sections, heads)
    got = torch.autograd.grad(out, leaves, dy.cuda())
    exact = [t.double().requires_grad_() for t in (x, gain, shift, weight)]
    want_out = _plain_scores(exact[0], ijk.cpu(), *exact[1:], freqs, sections, heads)
    want = torch.autograd.grad(want_out, exact, dy.double())
    # absolute terms: |unit| |gain| + |shift| through |weight|, at most sqrt(2) larger by a turn, times the other factor
    with torch.no_grad():
        n = ref.layer_norm(x, gain, shift, EPS)[0].abs()
        qk = (n @ weight.double().abs().t()).view(300, 2 * heads, -1) * 2 ** 0.5
        most = (qk[1:, :heads] * qk[:-1, heads:]).sum(2)
        assert bool(((out.detach().double().cpu() - want_out.detach()).abs() <= most * 4 * (4 * c) * ref.U32).all())
        # gradients: each output's terms once more through the same factors, summed over channels or voxels
        dq = torch.zeros_like(qk)
        dq[1:, :heads] += dy.double().abs()[..., None] * qk[:-1, heads:]
        dq[:-1, heads:] += dy.double().abs()[..., None] * qk[1:, :heads]
        dq = (dq * 2 ** 0.5).view(300, -1)
        dn = dq @ weight.double().abs()
        unit = ref.layer_norm(x, None, None, EPS)[0].abs()
        s = ref.layer_norm(x, None, None, EPS)[2][:, None]
        gy = dn * gain.double().abs()
        mags = (s * (gy + gy.mean(1, keepdim=True) + unit * (gy * unit).mean(1, keepdim=True)), (dn * unit).sum(0), dn.sum(0), dq.t() @ n)
    for a, b, m in zip(got, want, mags):
        assert bool(((a.double().cpu() - b).abs() <= m * 4 * (4 * c + 300) * ref.U32).all())
    # a difference along a direction, of the definition: its gradient is the formula's
    step = 1e-5
    with torch.no_grad():
        ways = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in exact]
        value = lambda sign: (_plain_scores(*(lambda t: (t[0], ijk.cpu(), *t[1:]))([e + sign * step * w for e, w in zip(exact, ways)]), freqs, sections, heads) * dy).sum()
        slope = (value(1) - value(-1)) / (2 * step)
        total = sum((b * w).sum() for b, w in zip(want, ways))
    # the step's third-order term and the 64-bit rounding of a sum of 300 x 48 x 48 terms
    assert abs(slope - total) <= 1e-6 * sum((b * w).abs().sum() for b, w in zip(want, ways))


def test_training_runs():
    ijk, _ = _voxels()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(ijk.shape[0], 64, generator=g).cuda()
    target = torch.randn(ijk.shape[0] - 1, 2, generator=g).cuda()
    losses = voxel_tokens.train(x, ijk, target, 2, 3)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
