"""Outputs of the operators on feature rows where a mode answers for torch's dispatcher: it is asked for them, and nothing of it stays."""
import gc
import os
import subprocess
import sys

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu

FIRST_UNDER_A_FAKE_MODE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from topology_construction_amd import binding
x = torch.randn(4, 64, device="cuda")
with FakeTensorMode():
    try:
        binding.tc_layer_norm(x)
    except Exception as e:
        print("fake:", type(e).__name__, flush=True)
    else:
        raise SystemExit("a fake output was written")
out, h, mean, rstd = binding.tc_layer_norm(x)
want = torch.nn.functional.layer_norm(x, (64,))
assert float((out - want).abs().max()) < 1e-5
assert binding.tc_rms_norm(x)[0].shape == (4, 64)
print("real: done", flush=True)
"""


def test_first_call_under_a_fake_mode():
    """The first output of the process is asked for under a mode whose tensors have no memory: later ones have."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_UNDER_A_FAKE_MODE], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "fake: " in r.stdout and "real: done" in r.stdout


class Watched(TorchDispatchMode):
    """Notes the outputs that are asked for, and where they lie."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.made.append(out.data_ptr())
        return out


def _calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(30, 96, generator=g, device="cuda").bfloat16()
    w = torch.randn(96, generator=g, device="cuda")
    q, scale = binding.tc_quantise_mx4(x)
    x8, s8 = binding.tc_rms_norm_i8(x)[:2]
    at, freqs = torch.arange(30, dtype=torch.int32, device="cuda")[:, None], torch.rand(48, generator=g, device="cuda")
    _, h, mean, rstd = binding.tc_layer_norm(x, w)
    return [lambda: binding.tc_rms_norm(x, w, residual=x), lambda: binding.tc_layer_norm(x, w, w, residual=x),
            lambda: binding.tc_layer_norm_backward(x, h, w, mean, rstd), lambda: binding.tc_rotary(x, at, freqs),
            lambda: binding.tc_quantise_mx4(x), lambda: binding.tc_dequantise_mx4(q, scale), lambda: binding.tc_matmul_mx4(q, scale, q, scale)]


def test_a_mode_sees_every_output():
    for call in _calls():
        want = call()
        with Watched() as mode:
            got = call()
        for a, b in zip(*((r if isinstance(r, tuple) else (r,)) for r in (got, want))):
            assert torch.equal(a, b) and a.data_ptr() in mode.made
        again = call()
        for a, b in zip(*((r if isinstance(r, tuple) else (r,)) for r in (again, want))):
            assert torch.equal(a, b)


def test_outputs_are_of_torchs_allocator():
    x = torch.randn(1000, 1024, device="cuda")
    gc.collect()  # what earlier tests left
    before = torch.cuda.memory_allocated()
    out = binding.tc_layer_norm(x)[0]
    assert torch.cuda.memory_allocated() - before >= out.numel() * 4
    del out
    assert torch.cuda.memory_allocated() == before
