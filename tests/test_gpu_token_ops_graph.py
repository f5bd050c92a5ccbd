"""Layer norm, rotary positions and 4-bit rows in captured graphs, replayed on changed inputs with eager work between, two
graphs and two streams side by side."""
import pytest
import torch

from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _inputs(seed, rows, c):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, dy = (torch.randn(rows, c, generator=g, device="cuda").to(BF16) for _ in range(3))
    w, b = (torch.randn(c, generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(-500, 500, (rows, 3), generator=g, device="cuda", dtype=torch.int32)
    wide = (torch.randn(3 * c, c, generator=g, device="cuda") / c ** 0.5).to(BF16)
    return [x, r, dy, w, b, pos, wide]


def _run(t, freqs, sections):
    """A block's path: norm, 4-bit projection, turn in place, and the norm's gradient."""
    x, r, dy, w, b, pos, wide = t
    out, h, mean, rstd = binding.tc_layer_norm(x, w, b, residual=r)
    qkv = binding.tc_matmul_mx4(*binding.tc_quantise_mx4(out), *binding.tc_quantise_mx4(wide))
    heads = qkv.view(x.shape[0], 6, -1)
    turned = binding.tc_rotary(heads[:, :4], pos, freqs, sections, out=heads[:, :4])
    back = binding.tc_dequantise_mx4(*binding.tc_quantise_mx4(turned.reshape(x.shape[0], -1)))
    return [out, h, qkv, back, *binding.tc_layer_norm_backward(dy, h, w, mean, rstd, grad_h=x)]


# each tile of the product: few rows, 64 x 64, 128 x 128, 256 x 256, all steps at once; wide rows of the norm
@pytest.mark.parametrize("rows,c", [(1, 256), (300, 64), (700, 640), (1200, 2560), (70_000, 128), (2_000, 5000)])
def test_graph_replays(rows, c):
    print(f"[graph] {rows} x {c}", flush=True)
    pairs = c // 4
    freqs, sections = torch.rand(pairs, device="cuda"), (pairs // 2, pairs // 4, pairs - pairs // 2 - pairs // 4)
    t = _inputs(1, rows, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # nothing ran before: the first call of a variant may be a captured one
        got = _run(t, freqs, sections)
    for seed in (2, 3, 4):
        for a, b in zip(t, _inputs(seed, rows, c)):
            a.copy_(b)
        want = [v.clone() for v in _run(t, freqs, sections)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_two_graphs_on_two_streams():
    """Each graph has its own outputs and workspaces: replayed at once they do not meet."""
    freqs, sections = torch.rand(64, device="cuda"), (30, 20, 14)
    sets = [_inputs(s, 3000, 256) for s in (1, 2)]
    want = [[v.clone() for v in _run(t, freqs, sections)] for t in sets]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in sets], []
    for graph, t in zip(graphs, sets):
        with torch.cuda.graph(graph):
            got.append(_run(t, freqs, sections))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_calls_at_once():
    """Eager calls on two streams."""
    freqs, sections = torch.rand(64, device="cuda"), (30, 20, 14)
    sets = [_inputs(s, 3000, 256) for s in (3, 4)]
    want = [[v.clone() for v in _run(t, freqs, sections)] for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, t in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(_run(t, freqs, sections))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_training_step_captured():
    """Forward and backward of the norm and the turn in one graph, with torch.autograd.grad."""
    leaves = [t.requires_grad_() for t in _inputs(5, 300, 64)[:2]]
    w, b = (torch.randn(64, device="cuda", requires_grad=True) for _ in range(2))
    pos, freqs = torch.arange(300, dtype=torch.int32, device="cuda")[:, None], torch.rand(8, device="cuda")
    dy = torch.randn(300, 4, 16, device="cuda").to(BF16)

    def step():
        out, h, _, _ = binding.tc_layer_norm(leaves[0], w, b, residual=leaves[1])
        y = binding.tc_rotary(out.view(300, 4, 16), pos, freqs)
        return torch.autograd.grad([y, h], [*leaves, w, b], [dy, dy.view(300, 64)])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12, 13):
        with torch.no_grad():
            for t, v in zip(leaves, _inputs(seed, 300, 64)):
                t.copy_(v)
            dy.copy_(_inputs(seed, 300, 64)[2].view(300, 4, 16))
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
