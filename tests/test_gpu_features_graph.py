"""The larger variants of the 8-bit products in a captured graph, replayed on changed inputs with eager work
between the replays (tests/test_gpu_features.py has the small ones)."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu


def _inputs(seed, n_dst, taps, cin, cout, pad):
    g = torch.Generator().manual_seed(seed)
    n_src = n_dst // 2
    x = torch.randint(-128, 128, (n_src, cin + pad), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (taps, cout, cin), generator=g, dtype=torch.int8)
    m = torch.randint(-n_src, n_src, (n_dst, taps), generator=g, dtype=torch.int32)
    return [t.cuda() for t in (x, torch.rand(n_src, generator=g), m, w, torch.rand(cout, generator=g))]


def _run(t, cin):
    x, xs, m, w, ws = t
    y = binding.tc_sparse_conv_i8(x[:, :cin], xs, m, w, ws, out_dtype=torch.float32)
    z = binding.tc_matmul_i8(x[:, :cin], xs, w[0], ws)
    return [y, z]


# weights of all taps in LDS (more than the 60 KiB that need no asking), tiles of 256 rows through registers
# and straight into LDS, tiles of 64 rows
@pytest.mark.parametrize("n_dst,taps,cin,cout,pad", [(98_500, 8, 120, 64, 3), (98_500, 27, 60, 60, 1), (33_000, 27, 128, 96, 0),
                                                     (33_000, 4, 200, 70, 0), (8_300, 27, 64, 64, 0)])
def test_graph_replays(n_dst, taps, cin, cout, pad):
    print(f"[graph] {n_dst} x {taps} {cin} -> {cout} pad={pad}", flush=True)
    t = _inputs(1, n_dst, taps, cin, cout, pad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # nothing ran before: the first call of a variant may be a captured one
        got = _run(t, cin)
    for seed in (2, 3, 4):
        for a, b in zip(t, _inputs(seed, n_dst, taps, cin, cout, pad)):
            a.copy_(b)
        want = [v.clone() for v in _run(t, cin)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
