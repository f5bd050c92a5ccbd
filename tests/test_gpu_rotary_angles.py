"""The sines of rotary positions by themselves: the pair (1, 0) turns into (cos, sin), without a rounding of the products. Both
are off by at most 2^-23, over every coordinate."""
import math
import random

import pytest
import torch

from tests import angle_ref
from tests.feature_ref import half_step, tiny
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def _check(low, high, dtype, interleaved, seed):
    """Frequencies of either sign from `low` to `high` in size, over their logarithm."""
    rng = random.Random(seed)
    pairs, rows = 24, 60
    freqs = torch.tensor([rng.choice((-1, 1)) * math.exp(rng.uniform(math.log(low), math.log(high))) for _ in range(pairs)],
                         dtype=torch.float32)
    freqs[0], freqs[1] = low, high
    at = [0, 1, -1, 7, -2 ** 31, 2 ** 31 - 1, 2 ** 30, -2 ** 31 + 1]
    at += [rng.randint(-2 ** 31, 2 ** 31 - 1) for _ in range(30)]
    at += [rng.randint(-2 ** 12, 2 ** 12) for _ in range(rows - len(at))]
    x = torch.zeros(rows, 1, 2 * pairs, dtype=dtype)
    first = torch.arange(pairs) * (2 if interleaved else 1)
    second = first + (1 if interleaved else pairs)
    x[..., first] = 1
    cos, sin = torch.tensor([[angle_ref.cos_sin(p, float(f)) for f in freqs] for p in at], dtype=torch.float64).unbind(2)
    for inverse in (False, True):
        out = binding.tc_rotary(x.cuda(), torch.tensor(at, dtype=torch.int32).cuda()[:, None], freqs.cuda(),
                                interleaved=interleaved, inverse=inverse)[:, 0].double().cpu()
        for got, want in ((out[:, first], cos), (out[:, second], -sin if inverse else sin)):
            off = 2.0 ** -23 if dtype == torch.float32 else 2.0 ** -23 + (want.abs() + 2.0 ** -23) * half_step(dtype) + tiny(dtype)
            worst = ((got - want).abs() - off).max()
            assert float(worst) <= 0, f"{float((got - want).abs().max()):.3g}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("low,high", [(1e-4, 1.0), (0.5, 1.0), (1.0, 10.0), (900.0, 1000.0), (1e5, 1e6), (1e6, 1e12)])
def test_angles(low, high, dtype, interleaved):
    print(f"[angles] {low} to {high} {dtype} interleaved {interleaved}", flush=True)
    _check(low, high, dtype, interleaved, int(high))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("low,high", [(2.0 ** 39, 2.0 ** 41), (2.0 ** 40, 1e18), (1e18, 1e30), (1e30, torch.finfo(torch.float32).max), (1e-45, 1e-30)])
def test_angles_of_any_finite_frequency(low, high, interleaved):
    print(f"[angles] {low} to {high} interleaved {interleaved}", flush=True)
    _check(low, high, torch.float32, interleaved, 5)


def test_frequencies_that_are_not_finite():
    """NaN in their own pairs, and in no other."""
    freqs = torch.tensor([1.0, math.inf, -math.inf, math.nan, 3e38], device="cuda")
    at = torch.tensor([[0], [3], [-2 ** 31]], dtype=torch.int32, device="cuda")
    out = binding.tc_rotary(torch.ones(3, 10, device="cuda"), at, freqs)
    assert out.isnan().tolist() == [[False, True, True, True, False] * 2] * 3
