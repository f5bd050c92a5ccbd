"""A transformer block over the voxels of a batch, one token a voxel, with the operators on feature rows.

Positions are the voxels' own coordinates in the library's enumeration; a head's pairs of channels are shared out
over x, y and z.

Serving, in 4 bits:   layer norm -> 4-bit rows -> projection to queries, keys and values -> queries and keys turned by
                      their positions -> attention among the voxels of a member (torch) -> 4-bit projection ->
                      layer norm with the residual's addition -> two 4-bit projections with an activation between.
Training:             layer norm, a projection and the turn, recorded by autograd.

Run:  python examples/voxel_tokens.py [--workload 2] [--channels 256] [--heads 4]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from topology_construction_amd import binding, synth  # noqa: E402


def axes_of(dim: int):
    """(pairs of a head for x, y, z; radians a step of each pair): geometric from 1 down to about a hundredth."""
    pairs = dim // 2
    sections = tuple(pairs // 3 + (1 if a < pairs % 3 else 0) for a in range(3))
    freqs = torch.cat([100.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections])
    return sections, freqs.float()


class Block:
    """Random weights of one block, the projections' in 4 bits."""

    def __init__(self, channels: int, heads: int, wide: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.channels, self.heads, self.dim = channels, heads, channels // heads
        self.sections, freqs = axes_of(self.dim)
        self.freqs = freqs.cuda()

        def weights(out, inner):
            return binding.tc_quantise_mx4((torch.randn(out, inner, generator=g) / math.sqrt(inner)).bfloat16().cuda())

        self.qkv, self.out = weights(3 * channels, channels), weights(channels, channels)
        self.up, self.down = weights(wide, channels), weights(channels, wide)
        self.gain1, self.gain2 = ((1 + 0.1 * torch.randn(channels, generator=g)).bfloat16().cuda() for _ in range(2))
        self.shift1, self.shift2 = ((0.1 * torch.randn(channels, generator=g)).bfloat16().cuda() for _ in range(2))
        self.bias = (0.1 * torch.randn(3 * channels, generator=g)).cuda()

    def project(self, x, w, bias=None, keep=lambda step: None):
        q, scale = binding.tc_quantise_mx4(x)
        y = binding.tc_matmul_mx4(q, scale, *w, bias=bias)
        keep(("project", x, q, scale, *w, bias, y))
        return y

    def serve(self, x, ijk, offsets, trace=None):
        """x bfloat16 [voxels, channels], ijk int32 [voxels, 3], offsets of the members -> bfloat16 [voxels, channels]."""
        def keep(step):  # as it is now: queries and keys are turned in place
            if trace is not None:
                trace.append([v.clone() if torch.is_tensor(v) else v for v in step])

        n, _, _, _ = binding.tc_layer_norm(x, self.gain1, self.shift1)
        keep(("norm", x, None, self.gain1, self.shift1, x, n))
        qkv = self.project(n, self.qkv, self.bias, keep).view(-1, 3 * self.heads, self.dim)
        turned = qkv[:, :2 * self.heads]  # queries and keys, turned where they lie
        keep(("turn", turned))
        binding.tc_rotary(turned, ijk, self.freqs, self.sections, out=turned)
        keep(("turned", ijk, self.freqs, self.sections, turned))
        y = torch.empty(x.shape[0], self.heads, self.dim, dtype=x.dtype, device=x.device)
        for a, b in zip(offsets[:-1], offsets[1:]):
            if b > a:
                q, k, v = (t.transpose(0, 1) for t in qkv[a:b].split(self.heads, 1))
                y[a:b] = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None])[0].transpose(0, 1)
        y = self.project(y.view(-1, self.channels), self.out, None, keep)
        n, h, _, _ = binding.tc_layer_norm(y, self.gain2, self.shift2, residual=x)
        keep(("norm", y, x, self.gain2, self.shift2, h, n))
        u = torch.relu(self.project(n, self.up, None, keep))
        return h + self.project(u, self.down, None, keep)


def scores(x, ijk, gain, shift, weight, freqs, sections, heads):
    """Each voxel's query times its neighbour's key in the order of the enumeration, for training: float32 [voxels - 1, heads]."""
    n = binding.tc_layer_norm(x, gain, shift)[0]
    qk = (n @ weight.t()).view(x.shape[0], 2 * heads, -1)
    qk = binding.tc_rotary(qk, ijk, freqs, sections)
    q, k = qk[1:, :heads].float(), qk[:-1, heads:].float()
    return (q * k).sum(2)


def train(x, ijk, target, heads: int, steps: int, rate: float = 1.0):
    """Gradient steps on the norm's and the projection's weights; the losses."""
    c = x.shape[1]
    g = torch.Generator().manual_seed(5)
    sections, freqs = axes_of(c // heads)
    freqs = freqs.cuda()
    gain, shift = (torch.full((c,), v, device="cuda", requires_grad=True) for v in (1.0, 0.0))
    weight = (torch.randn(2 * c, c, generator=g) / math.sqrt(c)).to(x.dtype).cuda().requires_grad_()
    losses = []
    for _ in range(steps):
        loss = (scores(x, ijk, gain, shift, weight, freqs, sections, heads) - target).square().mean()
        grads = torch.autograd.grad(loss, [gain, shift, weight])
        with torch.no_grad():
            for p, d in zip((gain, shift, weight), grads):
                p -= rate / c * d
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", type=int, default=2, help="shells of synth.make_config: 1 two of 16^3, 2 sixteen of 64^3")
    ap.add_argument("--channels", type=int, default=256)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    rows, offsets = synth.make_config(a.workload)
    src = binding.tc_batch_from_ijk(torch.from_numpy(rows).cuda(), offsets)
    ijk = binding.tc_enumerate_ijk(src)
    ends = [int(h["voxel_begin"]) for h in src.headers()] + [ijk.shape[0]]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(ijk.shape[0], a.channels, generator=g).bfloat16().cuda()
    block = Block(a.channels, a.heads, 4 * a.channels)
    out = block.serve(x, ijk, ends)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        out = block.serve(x, ijk, ends)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / a.steps * 1e3
    print(f"serve: {out.shape[0]} voxels x {out.shape[1]}, {ms:.3f} ms a block")
    target = torch.randn(ijk.shape[0] - 1, a.heads, generator=g).cuda()
    print("train: losses " + " ".join(f"{v:.4f}" for v in train(x, ijk, target, a.heads, 5)))


if __name__ == "__main__":
    main()
