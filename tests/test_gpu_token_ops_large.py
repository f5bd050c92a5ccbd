"""The product of 4-bit rows at the sizes of its larger tiles, and the operators' other variants at sizes of many workgroups,
against the definitions in 64 bits, computed on the GPU."""
import pytest
import torch

from tests import token_ref as ref
from topology_construction_amd import binding

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _mx4(rows, k, seed, pad=0):
    """Packed rows in a buffer `pad` bytes wider, scales, and the values in 64 bits."""
    g = _gen(seed)
    q = torch.randint(0, 256, (rows, (k + 1) // 2 + pad), generator=g, device="cuda", dtype=torch.uint8)[:, pad // 2:][:, :(k + 1) // 2]
    s = torch.randint(117, 131, (rows, -(-k // 32) + pad), generator=g, device="cuda", dtype=torch.uint8)[:, :-(-k // 32)]
    table = torch.cat((ref.E2M1, -ref.E2M1)).cuda()
    v = table[ref.unpack(q, k).long()] * torch.exp2(s.double() - 127).repeat_interleave(32, 1)[:, :k]
    return q, s, v


def _check(rows, k, n, dtype, bias, pad=0):
    print(f"[mx4 large] {rows} x {k} -> {n} {dtype} pad={pad}", flush=True)
    x, xs, a = _mx4(rows, k, rows + k, pad)
    w, ws, b = _mx4(n, k, n + 1, pad)
    plus = torch.randn(n, generator=_gen(3), device="cuda") if bias else None
    got = binding.tc_matmul_mx4(x, xs, w, ws, channels=k, bias=plus, out_dtype=dtype)
    bt = b.t().contiguous()
    want = a @ bt
    mag = a.abs() @ bt.abs()
    if bias:
        want, mag = want + plus.double(), mag + plus.double().abs()
    bad = ~((got.double() - want).abs() <= ref.matmul_mx4_bound(want, mag, k, dtype))
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"
    again = binding.tc_matmul_mx4(x, xs, w, ws, channels=k, bias=plus, out_dtype=dtype)
    assert torch.equal(got, again)


# tiles of 256 x 256; numbers of steps on both sides of those that exponents are loaded for
@pytest.mark.parametrize("rows,k,n,dtype,pad", [(3500, 288, 3590, BF16, 0), (3500, 384, 3590, F32, 0), (3585, 1024, 3700, F16, 0), (3584, 1152, 3584, BF16, 32),
                                                (3500, 2176, 3600, BF16, 0), (3500, 601, 3590, BF16, 0), (3590, 1055, 3501, F32, 3), (3500, 384, 3590, F16, 5)])
def test_largest_tiles(rows, k, n, dtype, pad):
    _check(rows, k, n, dtype, rows % 2 == 0, pad)


# 128 x 128
@pytest.mark.parametrize("rows,k,n,dtype,pad", [(2100, 288, 2000, F32, 0), (2048, 640, 2048, BF16, 0), (2000, 1025, 2111, BF16, 0), (2100, 4096, 2000, F16, 0),
                                                (2100, 700, 2000, F32, 1), (130, 1056, 20000, BF16, 16)])
def test_middle_tiles(rows, k, n, dtype, pad):
    _check(rows, k, n, dtype, rows % 4 == 0, pad)


# 64 x 64
@pytest.mark.parametrize("rows,k,n,dtype,pad", [(1003, 601, 523, F32, 0), (1000, 32, 600, BF16, 0), (700, 2304, 1000, F16, 0), (900, 1000, 700, BF16, 2), (64, 256, 8192, F32, 0),
                                                (20, 77, 9000, F16, 0)])
def test_small_tiles(rows, k, n, dtype, pad):
    _check(rows, k, n, dtype, True, pad)


# all steps at once
@pytest.mark.parametrize("rows,k,n,dtype,pad", [(70_001, 256, 250, BF16, 0), (66_000, 64, 300, F32, 0), (140_000, 128, 66, F16, 0), (66_000, 160, 257, BF16, 48),
                                                (66_000, 255, 130, F32, 0), (140_000, 33, 40, BF16, 0)])
def test_short_rows(rows, k, n, dtype, pad):
    _check(rows, k, n, dtype, n % 2 == 0, pad)


# input channels split over waves
@pytest.mark.parametrize("rows,k,n,dtype,pad", [(1, 4096, 5000, BF16, 0), (8, 8192, 1000, F32, 0), (50, 4096, 4100, F16, 0), (64, 1000, 4096, BF16, 1), (16, 5000, 4000, BF16, 0),
                                                (30, 1023, 999, F32, 4), (3, 20000, 70, BF16, 0)])
def test_few_rows(rows, k, n, dtype, pad):
    _check(rows, k, n, dtype, True, pad)


def test_out_of_every_alignment():
    """Rows of outputs whose ends meet other columns, for each tile."""
    for rows, k, n in ((3500, 288, 3590), (2100, 288, 2001), (1003, 96, 523), (66_000, 96, 133)):
        x, xs, a = _mx4(rows, k, 1)
        w, ws, b = _mx4(n, k, 2)
        want, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
        for dtype, shift in ((BF16, 1), (F32, 3), (BF16, 8)):
            wide = torch.full((rows, n + shift + 6), 9.0, device="cuda", dtype=dtype)
            out = wide[:, shift:shift + n]
            binding.tc_matmul_mx4(x, xs, w, ws, out=out)
            assert bool(((out.double() - want).abs() <= ref.matmul_mx4_bound(want, mag, k, dtype)).all())
            assert bool((wide[:, :shift] == 9).all()) and bool((wide[:, shift + n:] == 9).all())


@pytest.mark.parametrize("k", [96, 640])
def test_nan_scales_stay_in_their_rows_and_columns(k):
    for rows, n in ((3500, 3590), (2100, 2000), (1003, 523), (66_000, 130), (20, 700)):
        x, xs, _ = _mx4(rows, k, 1)
        w, ws, _ = _mx4(n, k, 2)
        xs, ws = xs.clone(), ws.clone()
        xs[rows - 1, -1], ws[n // 2, 0] = 255, 255
        nan = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
        nan[rows - 1], nan[:, n // 2] = True, True
        assert torch.equal(binding.tc_matmul_mx4(x, xs, w, ws).isnan(), nan)


@pytest.mark.parametrize("rows,c,dtype", [(50_000, 300, BF16), (100_003, 33, F32), (3, 300_001, F16)])
def test_quantise_many(rows, c, dtype):
    """Equal to the values' own rows taken in parts, and back."""
    x = torch.randn(rows, c, generator=_gen(c), device="cuda").to(dtype)
    q, scale = binding.tc_quantise_mx4(x)
    at = torch.randperm(rows, generator=_gen(1), device="cuda")[:200]
    codes, want = ref.quantise_mx4(x[at].cpu())
    assert torch.equal(scale[at].cpu(), want)
    back = binding.tc_dequantise_mx4(q, scale, channels=c, out_dtype=F32)
    assert torch.equal(back[at].cpu().double(), ref.values(codes, want))
    again = binding.tc_quantise_mx4(back)  # what is representable stays
    assert torch.equal(binding.tc_dequantise_mx4(*again, channels=c, out_dtype=F32), back)


@pytest.mark.parametrize("rows,heads,dim,sections,dtype", [(30_000, 16, 64, (12, 10, 10), BF16), (9_001, 5, 100, (17, 17, 16), F32), (700, 40, 128, (16, 24, 24), F16),
                                                           (64, 1, 2048, (1024,), BF16)])
def test_rotary_many(rows, heads, dim, sections, dtype):
    x = torch.randn(rows, heads, dim, generator=_gen(dim), device="cuda").to(dtype)
    pos = torch.randint(-5000, 5000, (rows, len(sections)), generator=_gen(2), device="cuda", dtype=torch.int32)
    freqs = torch.cat([100.0 ** (-torch.arange(n) / n) for n in sections]).float()
    at = torch.randperm(rows, generator=_gen(1), device="cuda")[:300].cpu()
    for interleaved in (False, True):
        out = binding.tc_rotary(x, pos, freqs.cuda(), sections, interleaved)
        want, bound = ref.rotary(x.cpu()[at], pos.cpu()[at], freqs, sections, interleaved, False, dtype)
        assert bool(((out.cpu()[at].double() - want).abs() <= bound).all())
        assert torch.equal(binding.tc_rotary(x, pos, freqs.cuda(), sections, interleaved, out=x.clone()), out)
