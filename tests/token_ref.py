"""Layer norm, rotary positions and microscaled 4-bit rows in 64 bits, from their definitions, with the error bounds that
the 32-bit kernels are held to (U32 and half_step as in tests/feature_ref.py)."""
import torch

from tests.feature_ref import U32, half_step, tiny

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _or(w, value, c):
    return torch.full((c,), value, dtype=torch.float64) if w is None else w.double()


# ------------------------------------------------------------------ layer norm


def layer_norm(h, weight, bias, eps):
    """(out, mean, s) from the stored h."""
    hd = h.double()
    m = hd.mean(1)
    u = hd - m[:, None]
    s = 1.0 / torch.sqrt((u * u).mean(1) + float(torch.tensor(eps, dtype=torch.float32)))
    c = h.shape[1]
    return u * s[:, None] * _or(weight, 1.0, c) + _or(bias, 0.0, c), m, s


def layer_norm_bounds(h, weight, bias, m, s, dtype):
    """|errors| of (out, mean, s). The 64-bit sum of the mean is off by (C + 2) 2^-53 of the sum of |h|; a difference
    (h - hi) - lo by two roundings of itself, that, and the rounding of lo, at most 2^-48 |m| = `shift` in all. The
    mean of C squares is then off by (C + 6) U32 of itself and 2 shift of its root; s by half of that
    (relative), and by the root, the quotient and the additions."""
    c = h.shape[1]
    hd, w, b = h.double(), _or(weight, 1.0, c), _or(bias, 0.0, c)
    shift = 2.0 ** -48 * m.abs() + (c + 2) * 2.0 ** -53 * hd.abs().mean(1)
    rel = ((c + 6) / 2 + 4) * U32 + shift * s
    uw = (hd - m[:, None]) * s[:, None] * w
    inner = uw.abs() * (rel[:, None] + 6 * U32) + (shift * s)[:, None] * w.abs() + U32 * (uw.abs() + b.abs())
    out = inner * (1 + 2 ** -6) + (uw + b).abs() * half_step(dtype) * (1 + 2 ** -6) + tiny(dtype)
    return out, m.abs() * U32 + shift + 2.0 ** -149, s * rel * (1 + 2 ** -6) + 2.0 ** -149


def layer_norm_grad(grad_out, h, weight, mean, rstd, grad_h, dtype):
    """((grad_x, grad_weight, grad_bias), (bound of grad_x, sum of |terms| of grad_weight, of grad_bias, what the
    units' errors add to grad_weight)), from the stored 32-bit mean and s.

    v = (h - mean) s is rounded once, mean(v) is off by (C + 2) U32 of mean |v|, u = v - mean(v) by two more roundings."""
    dy, hd, s = grad_out.double(), h.double(), rstd.double()[:, None]
    c = h.shape[1]
    g = dy * _or(weight, 1.0, c)
    u = (hd - hd.mean(1, keepdim=True)) * s
    mg, mgu = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    dh = torch.zeros_like(dy) if grad_h is None else grad_h.double()
    dx = s * (g - mg - u * mgu) + dh
    v = ((hd - mean.double()[:, None]) * s).abs()
    mv = v.mean(1, keepdim=True)
    off_u = U32 * (3 * v + (c + 4) * mv + u.abs())
    off_mg = (c + 3) * U32 * g.abs().mean(1, keepdim=True)
    off_mgu = (c + 8) * U32 * ((g.abs() * v).mean(1, keepdim=True) + 2 * mv * g.abs().mean(1, keepdim=True))
    inner = off_mg + u.abs() * off_mgu + mgu.abs() * off_u + 6 * U32 * (g.abs() + mg.abs() + (u * mgu).abs())
    bound = (s * inner + 4 * U32 * (dx.abs() + dh.abs())) * (1 + 2 ** -6) + dx.abs() * half_step(dtype) * (1 + 2 ** -6) + tiny(dtype)
    return (dx, (dy * u).sum(0), dy.sum(0)), (bound, (dy * u).abs().sum(0), dy.abs().sum(0), (dy.abs() * off_u).sum(0))


def layer_norm_sum_roundings(rows: int) -> int:
    """Roundings of a term of the weight's or bias's gradient: its two products; the rows of one thread (the rows in at
    least min(rows, 256) parts); six doublings over a wave, three over its workgroup; 32 slices of at most 1024 parts (32
    each), by eights, and the eights."""
    return 2 + -(-rows // 256) + 6 + 3 + 32 + 7 + 3


# ------------------------------------------------------------------ rotary positions


def axis_of(sections):
    return torch.cat([torch.full((n,), a, dtype=torch.int64) for a, n in enumerate(sections)])


def rotary(x, positions, freqs, sections, interleaved, inverse, dtype):
    """(out, bound) for x [rows, heads, dim]. Angles: |position| < 2^29 and a 24-bit frequency make an exact product. cos and sin
    are off by 2^-23 at most, each product and the sum by one rounding."""
    pairs = freqs.numel()
    angle = positions.double()[:, axis_of(sections)] * freqs.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None] * (-1.0 if inverse else 1.0)
    xd = x.double()
    first = torch.arange(pairs) * (2 if interleaved else 1)
    second = first + (1 if interleaved else pairs)
    a, b = xd[..., first], xd[..., second]
    out, bound = xd.clone(), torch.zeros_like(xd)
    out[..., first], out[..., second] = a * cos - b * sin, a * sin + b * cos
    off = (a.abs() + b.abs()) * (2.0 ** -23 + 4 * U32)
    for at in (first, second):
        bound[..., at] = off + out[..., at].abs() * half_step(dtype) * (1 + 2 ** -6) + tiny(dtype)
    return out, bound


# ------------------------------------------------------------------ microscaled 4-bit rows


def quantise_mx4(x):
    """(codes uint8 [rows, channels], scale uint8 [rows, blocks])."""
    rows, c = x.shape
    t = torch.nn.functional.pad(x.double(), (0, -c % 32)).view(rows, -1, 32)
    fine = torch.isfinite(t).all(2)
    t = torch.where(fine[..., None], t, torch.zeros_like(t))
    top = t.abs().amax(2)
    # floor(log2): frexp's mantissa lies in [1/2, 1)
    e = torch.where(top > 0, torch.frexp(top)[1].long() - 3, torch.full_like(top, -127).long()).clamp(min=-127)
    y = torch.ldexp(t.abs(), -e[..., None])
    borders = (E2M1[1:] + E2M1[:-1]) / 2
    code = torch.zeros_like(y, dtype=torch.int64)
    for i in range(7):  # a tie goes to the even code
        code += (y >= borders[i]) if i % 2 else (y > borders[i])
    code += 8 * torch.signbit(t)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255))
    return code.view(rows, -1)[:, :c].to(torch.uint8), scale.to(torch.uint8)


def pack(codes):
    codes = torch.nn.functional.pad(codes, (0, codes.shape[1] % 2))
    return codes[:, ::2] | (codes[:, 1::2] << 4)


def unpack(q, channels):
    return torch.stack((q & 15, q >> 4), 2).flatten(1)[:, :channels]


def values(codes, scale):
    """What codes [rows, channels] under scales stand for, in 64 bits."""
    v = torch.cat((E2M1, -E2M1))[codes.long()]
    unit = torch.ldexp(torch.ones(scale.shape, dtype=torch.float64), scale.long() - 127)
    unit = torch.where(scale == 255, torch.full_like(unit, float("nan")), unit)
    return v * unit.repeat_interleave(32, 1)[:, :codes.shape[1]]


def matmul_mx4(x, x_scale, w, w_scale, bias):
    """(out, sum of |terms|) of codes and scales."""
    a, b = values(x, x_scale), values(w, w_scale)
    plus = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else bias.double()
    return a @ b.t() + plus, a.abs() @ b.abs().t() + plus.abs()


def matmul_mx4_bound(out, mag, k, dtype):
    """A sum of k products in floats, in any order, the parts of the waves and the bias; one rounding to the output's type."""
    return out.abs() * half_step(dtype) * (1 + 2 ** -6) + (k + 12) * U32 * mag + tiny(dtype)
