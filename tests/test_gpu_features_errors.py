"""Outputs that torch's allocator refuses: its own error, as from torch's operators, and work goes on."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def test_no_memory_for_an_output():
    rows, n = 1 << 21, 1 << 12  # an output of 32 GiB, with a limit of 2 % of the card: refused before the driver is asked
    x = torch.zeros(1, 16, dtype=torch.int8, device="cuda").expand(rows, 16)
    xs = torch.ones(rows, device="cuda")
    w, ws = torch.zeros(n, 16, dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda")
    wide = torch.zeros(1, n, device="cuda").expand(rows, n)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.02)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            binding.tc_matmul_i8(x, xs, w, ws, out_dtype=torch.float32)
        with pytest.raises(torch.OutOfMemoryError):
            binding.tc_rms_norm(wide)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    out = binding.tc_matmul_i8(x[:4], xs[:4], w, ws)
    assert float(out.abs().sum()) == 0
