"""A residual block of a network on sparse voxels, with the operators on feature rows.

The voxels of a batch of shells are rows of a feature matrix, in the order of the library's
enumeration; a 3x3x3 kernel map of the batch onto itself says what a convolution reads.

Serving, in 8 bits:   norm -> 3x3x3 convolution -> norm with the residual's addition ->
                      widening projection -> activation -> norm -> narrowing projection,
                      then a transposed 2x2x2 convolution onto the refined grids.
Training, one norm:   the norm with the residual's addition, recorded by autograd.

Run:  python examples/voxel_block.py [--workload 2] [--channels 128]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from topology_construction_amd import binding, synth  # noqa: E402


class RmsNorm:
    """The training form: (out, h), recorded by autograd in x, residual and weight."""

    @staticmethod
    def apply(x, residual, weight):
        out, h, _ = binding.tc_rms_norm(x, weight, residual=residual)
        return out, h


def quantise_weights(w):
    """int8 weights and a scale for each output channel (the first axis of `w`, float)."""
    top = w.abs().flatten(1).amax(1).clamp_min(1e-30)
    q = torch.round(w * (127.0 / top).view(-1, *([1] * (w.dim() - 1)))).to(torch.int8)
    return q, top / 127.0


class Block:
    """Random weights of one block, laid out as the operators take them."""

    def __init__(self, channels: int, wide: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def weights(out, *rest):
            w = torch.randn(out, *rest, generator=g) / math.sqrt(math.prod(rest))
            q, scale = quantise_weights(w)
            if len(rest) == 2:  # [out, taps, in] -> [taps, out, in]
                q = q.transpose(0, 1)
            return q.contiguous().cuda(), scale.cuda()

        def gains(n):
            return (1 + 0.1 * torch.randn(n, generator=g)).bfloat16().cuda()

        self.norm1, self.norm2, self.norm3 = gains(channels), gains(channels), gains(wide)
        self.conv, self.conv_scale = weights(channels, 27, channels)
        self.up, self.up_scale = weights(wide, channels)
        self.down, self.down_scale = weights(channels, wide)
        self.bias = (0.1 * torch.randn(channels, generator=g)).cuda()
        self.refine, self.refine_scale = weights(channels // 2, 8, channels)

    def serve(self, x, kmap, fine_map, trace=None):
        """x bfloat16 [voxels, channels] -> (features of the voxels, of the refined voxels)."""
        keep = trace.append if trace is not None else lambda step: None
        q, s, _ = binding.tc_rms_norm_i8(x, self.norm1)
        y = binding.tc_sparse_conv_i8(q, s, kmap, self.conv, self.conv_scale, bias=self.bias)
        keep(("conv", x, self.norm1, q, s, kmap, self.conv, self.conv_scale, self.bias, y))
        q, s, h = binding.tc_rms_norm_i8(y, self.norm2, residual=x)
        u = binding.tc_matmul_i8(q, s, self.up, self.up_scale)
        keep(("matmul", h, self.norm2, q, s, None, self.up, self.up_scale, None, u))
        u = torch.relu(u)
        q, s, _ = binding.tc_rms_norm_i8(u, self.norm3)
        v = binding.tc_matmul_i8(q, s, self.down, self.down_scale)
        keep(("matmul", u, self.norm3, q, s, None, self.down, self.down_scale, None, v))
        q, s, out = binding.tc_rms_norm_i8(v, self.norm1, residual=h)
        fine = binding.tc_sparse_conv_i8(q, s, fine_map, self.refine, self.refine_scale)
        keep(("conv", out, self.norm1, q, s, fine_map, self.refine, self.refine_scale, None, fine))
        return out, fine


def maps_of(ijk, offsets):
    """(batch, 3x3x3 map of the batch onto itself, 2x2x2 transposed map onto its refinement)."""
    src = binding.tc_batch_from_ijk(torch.from_numpy(ijk).cuda(), offsets)
    fine = binding.tc_build_batched_topology(src, "refine", 2)
    return src, binding.tc_build_kernel_map(src, src, 3, 1, False), binding.tc_build_kernel_map(src, fine, 2, 2, True)


def train(x, residual, target, steps: int, rate: float = 0.5):
    """Gradient steps on one norm's weight; the losses."""
    weight = torch.ones(x.shape[1], dtype=torch.float32, device=x.device, requires_grad=True)
    losses = []
    for _ in range(steps):
        out, h = RmsNorm.apply(x, residual, weight)
        loss = (out.float() - target).square().mean()
        (grad,) = torch.autograd.grad(loss, weight)
        with torch.no_grad():
            weight -= rate * x.shape[1] * grad
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", type=int, default=2, help="shells of synth.make_config: 1 two of 16^3, 2 sixteen of 64^3")
    ap.add_argument("--channels", type=int, default=128)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    ijk, offsets = synth.make_config(a.workload)
    src, kmap, fine_map = maps_of(ijk, offsets)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(src.voxel_total(), a.channels, generator=g).bfloat16().cuda()
    block = Block(a.channels, 4 * a.channels)
    out, fine = block.serve(x, kmap, fine_map)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        out, fine = block.serve(x, kmap, fine_map)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / a.steps * 1e3
    print(f"serve: {x.shape[0]} voxels x {a.channels} -> {tuple(fine.shape)} refined, {ms:.3f} ms a block")
    target = torch.randn(x.shape, generator=g).cuda()
    losses = train(x, out, target, 5)
    print("train: losses " + " ".join(f"{v:.4f}" for v in losses))


if __name__ == "__main__":
    main()
