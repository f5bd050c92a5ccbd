"""The operators on feature rows in 64 bits, from their definitions, with the
error bounds that the 32-bit kernels are held to.

U32 = 2^-24 is half a step of a float, half_step(t) that of an output type. A sum
of n products held in floats, in any order, is off by at most (n + 1) U32 times
the sum of the terms' absolute values.
"""
import torch

U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Absolute rounding of results below the normal range."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def norm_sum(x, residual):
    """h, in the rows' type: the 32-bit sum, rounded once."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def rms_norm(h, weight, eps):
    """(out, s) in 64 bits from the stored h."""
    hd = h.double()
    s = 1.0 / torch.sqrt((hd * hd).mean(1) + float(torch.tensor(eps, dtype=torch.float32)))
    w = torch.ones(h.shape[1], dtype=torch.float64) if weight is None else weight.double()
    return hd * s[:, None] * w, s


def rms_norm_bound(out, dtype):
    """|error| of out: the mean of C squares is off by (C + 1) U32 of itself, s by half
    of that, and the root, the quotient and the products by one rounding each."""
    c = out.shape[1]
    return out.abs() * (half_step(dtype) + ((c + 1) / 2 + 8) * U32) * (1 + 2 ** -6) + tiny(dtype)


def rms_norm_i8(h, weight, s):
    """(q, scale) from the stored h; s as rms_norm gives it."""
    p = h.double() if weight is None else h.double() * weight.double()
    a = p.abs().amax(1)
    fine = torch.isfinite(p).all(1)
    # a quotient, rounded once: torch takes `127.0 / a` as 127 times the rounded reciprocal
    factor = torch.where(fine & (a > 0), torch.full_like(a, 127.0) / a, torch.zeros_like(a))
    q = torch.round(torch.nan_to_num(p, nan=0.0, posinf=0.0, neginf=0.0) * factor[:, None]).to(torch.int8)
    scale = torch.where(a > 0, a * s / 127.0, torch.zeros_like(a))
    return q, torch.where(fine, scale, torch.full_like(a, float("nan")))


def rms_norm_grad(grad_out, h, weight, rstd, grad_h):
    """(grad_x, grad_weight, bound of grad_x without the output's rounding, sum of |terms| of grad_weight)."""
    dy, hd, s = grad_out.double(), h.double(), rstd.double()[:, None]
    w = torch.ones(h.shape[1], dtype=torch.float64) if weight is None else weight.double()
    c = h.shape[1]
    g = dy * w
    dh = torch.zeros_like(dy) if grad_h is None else grad_h.double()
    dx = s * g - hd * s ** 3 * (g * hd).mean(1, keepdim=True) + dh
    # the dot product: (C + 2) U32 of its terms (each a product of three); the rest: a few roundings of each term
    bound = U32 * (hd.abs() * s ** 3 * (g * hd).abs().mean(1, keepdim=True) * (c + 12) + 8 * (s * g).abs() + 4 * dh.abs())
    terms = dy * hd * s
    return dx, terms.sum(0), bound, terms.abs().sum(0)


def matmul_i8(x, xs, w, ws, bias):
    """(out, sum of |terms|) in 64 bits; integer sums are exact there."""
    prod = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    b = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else bias.double()
    return prod + b, prod.abs() + b.abs()


def sparse_conv_i8(x, xs, kmap, w, ws, bias):
    """(out, sum of |terms| over the taps) in 64 bits."""
    n_dst, taps = kmap.shape
    out = torch.zeros((n_dst, w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    m = kmap.long()
    for t in range(taps):
        j = ((m[:, t] >= 0) & (m[:, t] < x.shape[0])).nonzero().flatten()
        i = m[j, t]
        v = (x[i].double() @ w[t].double().t()) * xs[i].double()[:, None] * ws.double()
        out.index_add_(0, j, v)
        mag.index_add_(0, j, v.abs())
    b = torch.zeros(w.shape[1], dtype=torch.float64) if bias is None else bias.double()
    return out + b, mag + b.abs()


def product_bound(out, mag, dtype, taps=1):
    """One rounding of each integer sum, its two scales and the bias, one for each tap's addition, one to the output's type."""
    return out.abs() * half_step(dtype) * (1 + 2 ** -6) + (taps + 6) * U32 * mag + tiny(dtype)
