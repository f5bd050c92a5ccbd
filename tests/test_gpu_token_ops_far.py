"""Layer norm, rotary positions and 4-bit rows where an offset passes 32 bits, looked at on the rows at both ends and around the
place where 2^31 elements or bytes are passed."""
import pytest
import torch

from tests import feature_ref, token_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _places(rows, per_row):
    near = (1 << 31) // per_row
    at = torch.cat([torch.arange(3), torch.arange(near - 3, near + 4), torch.arange(rows - 3, rows)])
    return at[(at >= 0) & (at < rows)].unique()


def _within(got, want, bound, what):
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("rows,c", [(270_000, 8192), (132_000, 16392)])
def test_layer_norm(rows, c):
    print(f"[far norm] {rows} x {c}", flush=True)
    x = torch.randn(rows, c, generator=_gen(c), device="cuda", dtype=BF16)
    w, b = ((1 + 0.3 * torch.randn(c, generator=_gen(i), device="cuda")).to(BF16) for i in (1, 2))
    at = _places(rows, c).cuda()
    h = feature_ref.norm_sum(x[at].cpu(), x[at].cpu())
    out, h2, mean, rstd = binding.tc_layer_norm(x, w, b, residual=x, eps=EPS)
    assert torch.equal(h2[at].cpu(), h)
    want, m, s = ref.layer_norm(h, w.cpu(), b.cpu(), EPS)
    _within(out[at], want, ref.layer_norm_bounds(h, w.cpu(), b.cpu(), m, s, BF16)[0], "out")
    gx, _, _ = binding.tc_layer_norm_backward(x, h2, w, mean, rstd, grad_h=out)
    (dx, _, _), (bound, _, _, _) = ref.layer_norm_grad(x[at].cpu(), h, w.cpu(), mean[at].cpu(), rstd[at].cpu(), out[at].cpu(), BF16)
    _within(gx[at], dx, bound, "grad_x")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(interleaved):
    rows, heads, dim = 140_000, 128, 128
    x = torch.randn(rows, heads, dim, generator=_gen(1), device="cuda", dtype=BF16)
    pos = torch.randint(-5000, 5000, (rows, 2), generator=_gen(2), device="cuda", dtype=torch.int32)
    freqs = torch.rand(64, generator=_gen(3), device="cuda")
    at = _places(rows, heads * dim).cuda()
    want, bound = ref.rotary(x[at].cpu(), pos[at].cpu(), freqs.cpu(), (40, 24), interleaved, False, BF16)
    out = binding.tc_rotary(x, pos, freqs, (40, 24), interleaved)
    _within(out[at], want, bound, "rows first")
    # heads 2^24 elements apart and more
    across = x.view(heads, rows, dim).transpose(0, 1)
    want, bound = ref.rotary(across[at].cpu(), pos[at].cpu(), freqs.cpu(), (40, 24), interleaved, False, BF16)
    to = out.view(heads, rows, dim).transpose(0, 1)
    binding.tc_rotary(across, pos, freqs, (40, 24), interleaved, out=to)
    _within(to[at], want, bound, "heads first")


def test_mx4_rows():
    rows, c = 1_060_000, 4096  # 4.3e9 values, 2.2e9 bytes of them
    x = torch.randn(rows, c, generator=_gen(4), device="cuda", dtype=BF16)
    at = torch.cat([_places(rows, c), _places(rows, c // 2)]).unique().cuda()
    codes, scale = ref.quantise_mx4(x[at].cpu())
    q, s = binding.tc_quantise_mx4(x)
    del x
    assert torch.equal(s[at].cpu(), scale) and torch.equal(ref.values(ref.unpack(q[at].cpu(), c), scale), ref.values(codes, scale))
    back = binding.tc_dequantise_mx4(q, s)
    assert torch.equal(back[at].cpu().double(), ref.values(codes, scale))
    del back
    # rows from beyond 2^31 bytes on, and an output of more than 2^31 elements
    w, ws = torch.randint(0, 256, (2064, c // 2), generator=_gen(5), device="cuda", dtype=torch.uint8), torch.full((2064, c // 32), 124, dtype=torch.uint8, device="cuda")
    out = binding.tc_matmul_mx4(q, s, w, ws)
    at = torch.cat([at.cpu(), _places(rows, 2064)]).unique().cuda()
    want, mag = ref.matmul_mx4(ref.unpack(q[at].cpu(), c), s[at].cpu(), ref.unpack(w.cpu(), c), ws.cpu(), None)
    _within(out[at], want, ref.matmul_mx4_bound(want, mag, c, BF16), "product")


@pytest.mark.parametrize("k,n", [(64, 40), (288, 40)])
def test_mx4_rows_far_apart(k, n):
    """Strides beyond what a tile's 32-bit offsets reach: a row every 2^25 bytes."""
    rows = 200
    wide = torch.randint(0, 256, (rows, 1 << 25), generator=_gen(6), device="cuda", dtype=torch.uint8)
    x, xs = wide[:, 7:7 + k // 2], wide[:, 1000:1000 + -(-k // 32)]
    xs.copy_(torch.randint(117, 131, xs.shape, device="cuda", dtype=torch.uint8))
    w, ws = torch.randint(0, 256, (n, k // 2), generator=_gen(7), device="cuda", dtype=torch.uint8), torch.full((n, -(-k // 32)), 125, dtype=torch.uint8, device="cuda")
    for many in (1, 100):  # few tiles, and many
        w_, ws_ = w.repeat(many, 1), ws.repeat(many, 1)
        out = binding.tc_matmul_mx4(x, xs, w_, ws_)
        want, mag = ref.matmul_mx4(ref.unpack(x.cpu(), k), xs.cpu(), ref.unpack(w_.cpu(), k), ws_.cpu(), None)
        _within(out, want, ref.matmul_mx4_bound(want, mag, k, BF16), f"{many}")
