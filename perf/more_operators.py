"""The operators of a token model on voxel rows, in their plain forms and as calls of the library, with the cases they are timed at.

A voxel (or a token) is one row of a feature matrix. The layer norm with the residual's addition is trained (forward and
backward) and served; rotary positions turn a row's heads by the voxel's three coordinates (or a token's time, height and
width); microscaled 4-bit rows (blocks of 32 values of e2m1 under one power of two) are what projections are served in.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a single token's norm, served: latency
        {"name": "layer_norm_one_row", "op": "norm", "rows": 1, "channels": 1024, "dtype": "bf16", "pad": 0},
        # a training step on two res-16 shells, 32-bit, an odd width in a wider buffer
        {"name": "layer_norm_train_small_f32", "op": "norm_train", "rows": 997, "channels": 100, "dtype": "f32", "pad": 3},
        # a training step on the voxels of 16 res-64 shells
        {"name": "layer_norm_train_16_shells", "op": "norm_train", "rows": 124800, "channels": 128, "dtype": "bf16", "pad": 0},
        # wide rows: a coarse level, or a token model over its voxels
        {"name": "layer_norm_train_wide", "op": "norm_train", "rows": 16384, "channels": 4096, "dtype": "f16", "pad": 0},
        # queries and keys of a single token with time, height and width: latency
        {"name": "rotary_one_token", "op": "rotary", "rows": 1, "heads": 20, "dim": 128, "sections": "16 24 24", "interleaved": False, "train": False,
         "far": False, "dtype": "bf16", "pad": 0},
        # heads of the voxels of 16 res-64 shells in one step of training, turned by their coordinates, and the gradient turned back
        {"name": "rotary_16_shells", "op": "rotary", "rows": 124800, "heads": 16, "dim": 64, "sections": "12 10 10", "interleaved": True, "train": True,
         "far": True, "dtype": "bf16", "pad": 1024},
        # a single token in front of a 4-bit projection
        {"name": "mx4_rows_one_row", "op": "mx4", "rows": 1, "channels": 1024, "dtype": "bf16", "pad": 0},
        # the voxels of 16 res-64 shells in front of a 4-bit projection
        {"name": "mx4_rows_16_shells", "op": "mx4", "rows": 124800, "channels": 256, "dtype": "bf16", "pad": 0},
        # a projection of a single token: latency and the weights' bytes
        {"name": "mx4_matmul_one_row", "op": "matmul", "rows": 1, "k": 1024, "n": 4096, "dtype": "bf16", "bias": False, "pad": 0},
        # odd sizes in every direction, 32-bit output with a bias
        {"name": "mx4_matmul_odd", "op": "matmul", "rows": 1003, "k": 601, "n": 523, "dtype": "f32", "bias": True, "pad": 5},
        # the widening projection on the voxels of 16 res-64 shells
        {"name": "mx4_matmul_16_shells", "op": "matmul", "rows": 124800, "k": 256, "n": 768, "dtype": "bf16", "bias": True, "pad": 0},
        # a product that the matrix units bound
        {"name": "mx4_matmul_large", "op": "matmul", "rows": 16384, "k": 4096, "n": 4096, "dtype": "bf16", "bias": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "rotary", "mx4", "matmul", "matmul"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    pad = rng.choice([0, 0, 3, 16])
    most = (1 << 27) // BYTES[dtype]  # elements
    if op in ("norm", "norm_train", "mx4"):
        channels = _log(rng, 8, 8192)
        return {"op": op, "rows": _log(rng, 1, min(130000, most // channels)), "channels": channels, "dtype": dtype, "pad": pad}
    if op == "rotary":
        heads, axes = rng.randint(1, 32), rng.randint(1, 4)
        pairs = _log(rng, 8, 128)
        cuts = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
        sections = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        dim = 2 * pairs + rng.choice([0, 0, 0, 1, 32])
        return {"op": op, "rows": _log(rng, 1, min(130000, most // (heads * dim))), "heads": heads, "dim": dim, "sections": sections,
                "interleaved": rng.random() < 0.5, "train": rng.random() < 0.5, "far": rng.random() < 0.5, "dtype": dtype, "pad": pad}
    k, n = _log(rng, 16, 4096), _log(rng, 16, 4096)
    return {"op": op, "rows": _log(rng, 1, min(130000, (1 << 38) // (k * n))), "k": k, "n": n, "dtype": dtype, "bias": rng.random() < 0.5, "pad": pad}


def _sections(case):
    """Pairs of a head turned by each axis."""
    return tuple(int(n) for n in case["sections"].split())


# ------------------------------------------------------------------ inputs


def _in_buffer(t, pad):
    """`t` [rows, ...] as the front of each row of a wider buffer, as a slice of concatenated features (or of q, k and v) is."""
    if not pad:
        return t.contiguous()
    rows, each = t.shape[0], t[0].numel()
    wide = torch.zeros((rows, each + pad), dtype=t.dtype, device=t.device)
    wide[:, :each] = t.reshape(rows, each)
    return wide[:, :each].unflatten(1, t.shape[1:])


def _features(shape, gen):
    """Rows whose channels differ in size and offset; one in a hundred is all zero."""
    t = torch.randn(shape, generator=gen, device="cuda")
    t *= torch.exp(0.5 * torch.randn((1, shape[1]), generator=gen, device="cuda"))
    t += 0.5 * torch.randn((1, shape[1]), generator=gen, device="cuda")
    return t * (torch.rand((shape[0], 1), generator=gen, device="cuda") > 0.01)


def _mx4_rows(shape, gen):
    """(uint8 [rows, ceil(k / 2)], uint8 [rows, ceil(k / 32)]): rows held in 4 bits, the even channel in the low half of its
    byte, with the scale exponents of their blocks, biased by 127."""
    rows, k = shape
    t = torch.zeros((rows, -(-k // 32) * 32), device="cuda")
    t[:, :k] = _features(shape, gen)
    t = t.view(rows, -1, 32)
    e = torch.frexp(t.abs().amax(2, keepdim=True))[1] - 3
    grid = torch.tensor(E2M1, device="cuda")
    code = torch.bucketize(torch.ldexp(t.abs(), -e), (grid[1:] + grid[:-1]) / 2) + 8 * (t < 0)
    code = code.view(rows, -1).to(torch.uint8)[:, :k + k % 2]
    scale = (e.squeeze(2) + 127).clamp(0, 254).to(torch.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    t = DTYPES[case["dtype"]]
    if case["op"].startswith("norm"):
        shape = (case["rows"], case["channels"])
        s["x"] = _in_buffer(_features(shape, gen).to(t), case["pad"])
        s["residual"] = (2.0 * torch.randn(shape, generator=gen, device="cuda")).to(t)
        s["weight"] = (1.0 + 0.2 * torch.randn(shape[1], generator=gen, device="cuda")).to(t)
        s["bias"] = (0.2 * torch.randn(shape[1], generator=gen, device="cuda")).to(t)
        if case["op"] == "norm_train":
            s["grad_out"] = torch.randn(shape, generator=gen, device="cuda").to(t)
            s["grad_h"] = torch.randn(shape, generator=gen, device="cuda").to(t)
    elif case["op"] == "rotary":
        shape = (case["rows"], case["heads"], case["dim"])
        s["x"] = _in_buffer(torch.randn(shape, generator=gen, device="cuda").to(t), case["pad"])
        if case["train"]:
            s["grad_out"] = torch.randn(shape, generator=gen, device="cuda").to(t)
        sections = _sections(case)
        # voxel coordinates of a batch's members, or grids far from the origin
        s["positions"] = torch.randint(0, 64, (case["rows"], len(sections)), generator=gen, device="cuda", dtype=torch.int32)
        if case["far"]:
            s["positions"] += torch.randint(-(1 << 28), 1 << 28, (1, len(sections)), generator=gen, device="cuda", dtype=torch.int32)
        s["freqs"] = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections]).float().cuda()
    elif case["op"] == "mx4":
        s["x"] = _in_buffer(_features((case["rows"], case["channels"]), gen).to(t), case["pad"])
    else:
        q, s["x_scale"] = _mx4_rows((case["rows"], case["k"]), gen)
        s["x"] = _in_buffer(q, case["pad"])
        s["w"], s["w_scale"] = _mx4_rows((case["n"], case["k"]), gen)
        s["w_scale"] = (s["w_scale"].int() - int(math.log2(case["k"]) / 2)).clamp(0, 254).to(torch.uint8)
        s["bias"] = torch.randn(case["n"], generator=gen, device="cuda") if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass


def _norm_plain(s):
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    u = hf - hf.mean(-1, keepdim=True)
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    u = u * rstd
    w = s["weight"].float()
    out = {"out": (u * w + s["bias"].float()).to(h.dtype), "h": h}
    if "grad_out" not in s:
        return out
    dy = s["grad_out"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - u * (g * u).mean(-1, keepdim=True)) + s["grad_h"].float()
    return {**out, "grad_x": dx.to(h.dtype), "grad_weight": (dy * u).sum(0), "grad_bias": dy.sum(0)}


def _rotate_plain(x, cos, sin, interleaved):
    pairs = cos.shape[-1]
    xf = x.float()
    a, b = (xf[..., 0:2 * pairs:2], xf[..., 1:2 * pairs:2]) if interleaved else (xf[..., :pairs], xf[..., pairs:2 * pairs])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, xf[..., 2 * pairs:]), -1).to(x.dtype)


def _rotary_plain(s):
    case = s["case"]
    axis = torch.cat([torch.full((n,), a, dtype=torch.int64) for a, n in enumerate(_sections(case))]).to(s["x"].device)
    angle = (s["positions"].double()[:, axis] * s["freqs"].double()).unsqueeze(1)  # far positions' angles need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {"out": _rotate_plain(s["x"], cos, sin, case["interleaved"])}
    if case["train"]:
        out["grad_x"] = _rotate_plain(s["grad_out"], cos, -sin, case["interleaved"])
    return out


def _mx4_plain(s):
    x = s["x"].float()
    rows, k = x.shape
    t = torch.nn.functional.pad(x, (0, -k % 32)).view(rows, -1, 32)
    e = (torch.frexp(t.abs().amax(2, keepdim=True))[1] - 3).clamp(-127, 127)
    a = torch.ldexp(t.abs().double(), -e)
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6.0)
    return torch.ldexp(a, e).copysign(t.double()).view(rows, -1)[:, :k].to(s["x"].dtype)


def _unpack_plain(q, scale, k):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    v = table[torch.stack((q & 15, q >> 4), 2).flatten(1)[:, :k].int()]
    return v * torch.ldexp(torch.ones_like(v[:, :1]), scale.int() - 127).repeat_interleave(32, 1)[:, :k]


def _matmul_plain(s):
    k = s["case"]["k"]
    out = _unpack_plain(s["x"], s["x_scale"], k) @ _unpack_plain(s["w"], s["w_scale"], k).t()
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(DTYPES[s["case"]["dtype"]])


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"norm": _norm_plain, "norm_train": _norm_plain, "rotary": _rotary_plain, "mx4": _mx4_plain, "matmul": _matmul_plain}[op](s)
    from topology_construction_amd import binding
    if op.startswith("norm"):
        out, h, mean, rstd = binding.tc_layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        if op == "norm":
            return {"out": out, "h": h}
        grad_x, grad_weight, grad_bias = binding.tc_layer_norm_backward(s["grad_out"], h, s["weight"], mean, rstd, grad_h=s["grad_h"])
        return {"out": out, "h": h, "grad_x": grad_x, "grad_weight": grad_weight, "grad_bias": grad_bias}
    if op == "rotary":
        out = {"out": binding.tc_rotary(s["x"], s["positions"], s["freqs"], _sections(case), interleaved=case["interleaved"])}
        if case["train"]:
            out["grad_x"] = binding.tc_rotary(s["grad_out"], s["positions"], s["freqs"], _sections(case), interleaved=case["interleaved"], inverse=True)
        return out
    if op == "mx4":
        q, scale = binding.tc_quantise_mx4(s["x"])
        return binding.tc_dequantise_mx4(q, scale, channels=case["channels"], out_dtype=s["x"].dtype)
    return binding.tc_matmul_mx4(s["x"], s["x_scale"], s["w"], s["w_scale"], channels=case["k"], bias=s["bias"], out_dtype=DTYPES[case["dtype"]])


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    t = BYTES[case["dtype"]]
    if case["op"].startswith("norm"):
        n = case["rows"] * case["channels"]
        if case["op"] == "norm":  # x and residual in, out and h out
            return {"bytes": 4 * n * t + 2 * t * case["channels"], "flops": 9 * n}
        # both gradients in and one out besides (h is read by the backward too)
        return {"bytes": 8 * n * t + (2 * t + 8) * case["channels"] + 16 * case["rows"], "flops": 24 * n}
    if case["op"] == "rotary":
        n, passes = case["rows"] * case["heads"] * case["dim"], 2 if case["train"] else 1
        pairs = sum(_sections(case))
        return {"bytes": passes * (2 * n * t + 4 * case["rows"] * len(_sections(case)) + 4 * pairs), "flops": passes * 6 * case["rows"] * case["heads"] * pairs}
    if case["op"] == "mx4":  # the rows in, the values that their 4 bits stand for out
        n = case["rows"] * case["channels"]
        return {"bytes": 2 * n * t, "flops": 4 * n}
    m, k, n = case["rows"], case["k"], case["n"]
    return {"bytes": (m + n) * (-(-k // 2) + -(-k // 32)) + t * m * n + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_norm(s):
    # the sum is held in the inputs' type: the norm is the norm of what is held
    h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    n = h.shape[1]
    w, b = s["weight"].double(), s["bias"].double()
    centre = h.sum(1, keepdim=True) / n
    length = ((h - centre).pow(2).sum(1, keepdim=True) / n + EPS).sqrt()
    unit = (h - centre) / length
    out = {"out": torch.addcmul(b, unit, w), "h": h}
    if "grad_out" not in s:
        return out
    gy = s["grad_out"].double()
    gu = gy * w
    # across the unit row and the row of ones
    gu = gu - gu.sum(1, keepdim=True) / n - unit * ((gu * unit).sum(1, keepdim=True) / n)
    return {**out, "grad_x": gu / length + s["grad_h"].double(), "grad_weight": torch.einsum("rc,rc->c", gy, unit), "grad_bias": gy.sum(0)}


def _exact_turn(x, turn, interleaved):
    pairs = turn.shape[-1]
    front = x.double()[..., :2 * pairs]
    front = front.unflatten(-1, (pairs, 2)) if interleaved else front.unflatten(-1, (2, pairs)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(front.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, x.double()[..., 2 * pairs:]), -1)


def _exact_rotary(s):
    case = s["case"]
    columns, at = [], 0
    for axis, count in enumerate(_sections(case)):
        # 29 bits times 24: exact
        columns.append(torch.outer(s["positions"][:, axis].double(), s["freqs"][at:at + count].double()))
        at += count
    angle = torch.cat(columns, 1).unsqueeze(1)
    turn = torch.polar(torch.ones_like(angle), angle)
    out = {"out": _exact_turn(s["x"], turn, case["interleaved"])}
    if case["train"]:
        out["grad_x"] = _exact_turn(s["grad_out"], turn.conj(), case["interleaved"])
    return out


def _exact_mx4(s):
    x = s["x"].double()
    out = torch.empty_like(x)
    for at in range(0, x.shape[1], 32):
        block = x[:, at:at + 32]
        top = block.abs().amax(1, keepdim=True)
        # top is in [4, 8) units: the exponent of a 64-bit number, from its bits
        unit = torch.ldexp(torch.ones_like(top), (((top.view(torch.int64) >> 52) & 2047) - 1023 - 2).clamp(min=-127))
        y = block.abs() / unit
        code = torch.zeros_like(y, dtype=torch.int64)
        for i in range(7):  # a border goes to the even code
            border = (E2M1[i] + E2M1[i + 1]) / 2
            code += (y >= border) if i % 2 else (y > border)
        out[:, at:at + 32] = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[code] * unit * block.sign()
    return out


def _exact_matmul(s):
    k = s["case"]["k"]

    def values(q, scale):
        low, high = (q & 15).double(), (q >> 4).double()
        code = torch.stack((low, high), 2).flatten(1)[:, :k]
        sign, code = torch.where(code >= 8, -1.0, 1.0), code % 8
        half = torch.floor(code / 2)  # the exponent's two bits; below 1 there is no leading one
        v = torch.where(half == 0, code / 2, torch.exp2(half - 1) * (1 + 0.5 * (code % 2))) * sign
        block = torch.arange(k, device=q.device) // 32
        return v * torch.exp2(scale.double() - 127)[:, block]

    out = values(s["x"], s["x_scale"]) @ values(s["w"], s["w_scale"]).t().contiguous()
    return out if s["bias"] is None else out + s["bias"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    return {"rotary": _exact_rotary, "mx4": _exact_mx4, "matmul": _exact_matmul}[case["op"]](s)
