"""The operators on feature rows where an offset passes 32 bits: in the rows, the outputs, the map. Looked at
on the rows at both ends and around the place where 2^31 elements are passed."""
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


def _cuda_gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _places(rows, per_row):
    near = (1 << 31) // per_row
    at = torch.cat([torch.arange(3), torch.arange(near - 3, near + 4), torch.arange(rows - 3, rows)])
    return at[(at >= 0) & (at < rows)].unique()


def _within(got, want, bound, what):
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("rows,c", [(270_000, 8192), (132_000, 16392)])
def test_norm(rows, c):
    print(f"[far norm] {rows} x {c}", flush=True)
    x = torch.randn(rows, c, generator=_cuda_gen(c), device="cuda", dtype=BF16)
    w = (1 + 0.3 * torch.randn(c, generator=_cuda_gen(1), device="cuda")).to(BF16)
    at = _places(rows, c).cuda()
    h, wc = x[at].cpu(), w.cpu()
    want, s = ref.rms_norm(h, wc, EPS)
    out, _, rstd = binding.tc_rms_norm(x, w, eps=EPS)
    _within(out[at], want, ref.rms_norm_bound(want, BF16), "out")
    gx, _ = binding.tc_rms_norm_backward(x, x, w, rstd, grad_h=out)
    dx, _, bound, _ = ref.rms_norm_grad(h, h, wc, rstd[at].cpu(), out[at].cpu())
    _within(gx[at], dx, bound + dx.abs() * ref.half_step(BF16) * (1 + 2 ** -6) + ref.tiny(BF16), "grad_x")
    del out, gx
    q, scale, h2 = binding.tc_rms_norm_i8(x, w, residual=x, eps=EPS)
    hc = ref.norm_sum(h, h)
    assert torch.equal(h2[at].cpu(), hc)
    want_q, want_scale = ref.rms_norm_i8(hc, wc, ref.rms_norm(hc, wc, EPS)[1])
    assert torch.equal(q[at].cpu(), want_q)
    _within(scale[at], want_scale, want_scale * ((c + 1) / 2 + 10) * ref.U32, "scale")


def _i8(shape, seed):
    q = torch.randint(-128, 128, shape, generator=_cuda_gen(seed), device="cuda", dtype=torch.int8)
    return q, torch.rand(shape[0], generator=_cuda_gen(seed + 1), device="cuda") + 0.5


def test_matmul_output():
    rows, k, n = 34_000_000, 16, 64
    x, xs = _i8((rows, k), 1)
    w, ws = _i8((n, k), 3)
    out = binding.tc_matmul_i8(x, xs, w, ws)
    at = _places(rows, n).cuda()
    want, mag = ref.matmul_i8(x[at].cpu(), xs[at].cpu(), w.cpu(), ws.cpu(), None)
    _within(out[at], want, ref.product_bound(want, mag, BF16), "matmul")


# map of more than 2^31 entries, output of more than 2^31 elements; then sources of just under and more than
# 2^31 bytes (rows by 31-bit offsets, and not) for each number of output rows
@pytest.mark.parametrize("n_src,n_dst,taps,cin,cout", [(1000, 80_000_000, 27, 16, 16), (1000, 34_000_000, 2, 16, 64),
                                                       (16_777_214, 100_000, 8, 128, 64), (20_000_000, 100_000, 8, 128, 64),
                                                       (16_777_214, 40_000, 8, 128, 96), (20_000_000, 40_000, 8, 128, 96),
                                                       (20_000_000, 9_000, 8, 128, 40), (20_000_000, 50, 8, 128, 40)])
def test_conv(n_src, n_dst, taps, cin, cout):
    print(f"[far conv] {n_src} -> {n_dst} x {taps} {cin} -> {cout}", flush=True)
    x, xs = _i8((n_src, cin), 1)
    w, ws = _i8((taps * cout, cin), 3)
    w, ws = w.view(taps, cout, cin), ws[:cout]
    m = torch.randint(-n_src // 2, n_src, (n_dst, taps), generator=_cuda_gen(5), device="cuda", dtype=torch.int32)
    at = torch.cat([_places(n_dst, taps), _places(n_dst, cout)]).unique().cuda()
    m[at[0], 0] = m[at[-1], 1] = n_src - 1
    out = binding.tc_sparse_conv_i8(x, xs, m, w, ws)
    mc = m[at].cpu()
    rows = mc.clamp_min(0).flatten().unique()  # the sources that these rows read, numbered anew
    mine = torch.where(mc < 0, mc.long(), torch.searchsorted(rows, mc.clamp_min(0)))
    rows = rows.long().cuda()
    want, mag = ref.sparse_conv_i8(x[rows].cpu(), xs[rows].cpu(), mine, w.cpu(), ws.cpu(), None)
    _within(out[at], want, ref.product_bound(want, mag, BF16, taps), "conv")
