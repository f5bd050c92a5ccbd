"""The 8-bit products at sizes that take their larger tiles, on the GPU, against their
definitions in 64 bits: on the first and last rows, on rows around tile borders, and on some between."""
import pytest
import torch

from tests import feature_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows_i8(rows, c, seed):
    g = _gen(seed)
    q = torch.randint(-128, 128, (rows, c), generator=g, dtype=torch.int8)
    return q, torch.exp(torch.randn(rows, generator=g)) * 0.01


def _some(n, seed):
    """Rows to look at: both ends, the borders of tiles of 256, 64 and 16, and 200 others."""
    near = torch.tensor([i * s + d for s in (256, 64, 16) for i in (1, 2, 7) for d in (-1, 0, 1)])
    rows = torch.cat([torch.arange(300), torch.arange(n - 300, n), near + n // 512 * 256,
                      torch.randint(0, n, (200,), generator=_gen(seed))])
    return rows[(rows >= 0) & (rows < n)].unique()


def _pad(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), 99, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def _within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("rows,k,n,dtype,pad", [
    (33000, 96, 256, BF16, 0), (33000, 100, 250, F16, 0), (33001, 64, 256, F32, 3), (33000, 13, 256, BF16, 16),
    (24600, 1024, 1024, BF16, 0), (24600, 1031, 1010, F32, 0), (24600, 1040, 1024, F16, 16)])
def test_matmul_large_tiles(rows, k, n, dtype, pad):
    print(f"[matmul large] {rows} x {k} -> {n} {dtype} pad={pad}", flush=True)
    x, xs = _rows_i8(rows, k, rows + k)
    w, ws = _rows_i8(n, k, k + n)
    b = torch.randn(n, generator=_gen(n))
    xs[rows // 2] = float("nan")
    got = binding.tc_matmul_i8(_pad(x, pad), xs.cuda(), w.cuda(), ws.cuda(), bias=b.cuda(), out_dtype=dtype).cpu()
    assert bool(got[rows // 2].isnan().all()) and int(got.isnan().any(1).sum()) == 1
    at = _some(rows, k)
    at = at[at != rows // 2]
    want, mag = ref.matmul_i8(x[at], xs[at], w, ws, b)
    _within(got[at], want, ref.product_bound(want, mag, dtype), "matmul")


CONV = [  # tiles of 256 rows: many rows, or more than 64 output channels
    (98500, 3, 64, 33, F16, 0), (98500, 2, 16, 16, BF16, 0), (98500, 3, 13, 24, F32, 0), (98500, 8, 100, 20, BF16, 0),
    (98500, 1, 7, 9, BF16, 0), (98500, 9, 48, 64, F32, 16), (98500, 2, 200, 48, BF16, 0),
    (33000, 27, 128, 96, BF16, 0), (33000, 5, 100, 128, BF16, 0), (33000, 5, 128, 128, F32, 5), (33000, 4, 200, 70, F16, 0),
    (33000, 3, 256, 72, BF16, 0), (33000, 40, 32, 65, BF16, 0), (33000, 6, 60, 100, F32, 0), (17000, 3, 64, 200, BF16, 0),
    # tiles of 256 rows from any address, with the weights of all taps in LDS and without
    (98500, 8, 120, 64, F32, 3), (98500, 8, 52, 45, F16, 4), (98500, 27, 60, 60, F16, 0), (98500, 27, 52, 20, BF16, 0),
    (98500, 9, 100, 60, BF16, 0), (98500, 27, 100, 12, F32, 0), (98500, 32, 10, 16, BF16, 0),
    # tiles of 64 rows
    (8300, 27, 64, 64, BF16, 0), (8300, 8, 100, 33, F16, 0), (8300, 33, 12, 16, F32, 0), (8300, 3, 200, 40, BF16, 0),
    (8300, 2, 5, 7, BF16, 0), (4200, 27, 96, 100, BF16, 0), (8300, 1, 128, 20, F32, 3), (8300, 5, 8, 32, BF16, 0)]


@pytest.mark.parametrize("n_dst,taps,cin,cout,dtype,pad", CONV)
def test_conv_large_tiles(n_dst, taps, cin, cout, dtype, pad):
    print(f"[conv large] {n_dst} x {taps} {cin} -> {cout} {dtype} pad={pad}", flush=True)
    n_src, g = n_dst // 3, _gen(taps + cin)
    # neighbours in runs, as surfaces have them; a stretch of rows without any, whole tiles of it
    base = torch.arange(n_dst).view(-1, 1) // 3 + torch.randint(-40, 40, (1, taps), generator=g)
    keep = (torch.rand(n_dst // 16 + 1, taps, generator=g) < 0.5).repeat_interleave(16, 0)[:n_dst]
    keep &= torch.rand(n_dst, taps, generator=g) < 0.8
    m = torch.where(keep, base, torch.tensor(-1)).to(torch.int32)
    m[2000:2700] = -1
    m[5, :] = n_src + 7
    m[6, 0] = 2 ** 31 - 1
    x, xs = _rows_i8(n_src, cin, n_src)
    w, ws = _rows_i8(cout, taps * cin, cout)
    w = w.view(cout, taps, cin).transpose(0, 1).contiguous()
    b = torch.randn(cout, generator=g)
    xs[n_src // 2] = float("nan")
    got = binding.tc_sparse_conv_i8(_pad(x, pad), xs.cuda(), m.cuda(), w.cuda(), ws.cuda(), bias=b.cuda(),
                                    out_dtype=dtype).cpu()
    reads_nan = (m == n_src // 2).any(1)
    assert torch.equal(got.isnan().all(1), reads_nan) and torch.equal(got.isnan().any(1), reads_nan)
    at = _some(n_dst, cin)
    at = torch.cat([at, torch.arange(1990, 2720)]).unique()
    at = at[~reads_nan[at]]
    want, mag = ref.sparse_conv_i8(x, xs, m[at], w, ws, b)
    _within(got[at], want, ref.product_bound(want, mag, dtype, taps), "conv")


@pytest.mark.parametrize("rows,cin,cout", [(99000, 32, 48), (40000, 128, 96), (9000, 52, 45)])
def test_conv_same_result_again(rows, cin, cout):
    """The order of every sum is fixed: two calls, bit for bit, also on rows moved by one (unaligned)."""
    x, xs = _rows_i8(rows, cin, 1)
    w, ws = _rows_i8(4 * cout, cin, 2)
    m = torch.randint(-rows // 2, rows, (rows, 4), generator=_gen(3), dtype=torch.int32).clamp_min(-1).cuda()
    w, ws = w.view(4, cout, cin).cuda(), ws[:cout].cuda()
    a = binding.tc_sparse_conv_i8(x.cuda(), xs.cuda(), m, w, ws, out_dtype=F32)
    assert torch.equal(a, binding.tc_sparse_conv_i8(x.cuda(), xs.cuda(), m, w, ws, out_dtype=F32))
    assert torch.equal(a, binding.tc_sparse_conv_i8(_pad(x, 3), xs.cuda(), m, w, ws, out_dtype=F32))
