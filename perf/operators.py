"""The feature operators on voxel rows, in their plain forms and as calls of the library, with the cases they are timed at.

A voxel of a batch is one row of a feature matrix, in the order of the enumeration. Three groups of operators work on
such rows: the root-mean-square norm with the residual's addition (trained: forward and backward; served: with an 8-bit
output), the product of 8-bit rows with 8-bit weights (a projection), and the same product over a kernel map (a sparse
convolution).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # a single token (or one global feature row) in front of a projection, served: latency
        {"name": "norm_i8_one_row", "op": "norm_i8", "rows": 1, "channels": 1024, "dtype": "bf16", "pad": 0},
        # the voxels of 16 res-64 shells at a network's first level, served
        {"name": "norm_i8_16_shells_c64", "op": "norm_i8", "rows": 124800, "channels": 64, "dtype": "bf16", "pad": 0},
        # a training step of the norm on two res-16 shells, 32-bit, an odd width in a wider buffer
        {"name": "norm_train_small_f32", "op": "norm_train", "rows": 997, "channels": 100, "dtype": "f32", "pad": 3},
        # a training step on the voxels of 16 res-64 shells
        {"name": "norm_train_16_shells", "op": "norm_train", "rows": 124800, "channels": 128, "dtype": "bf16", "pad": 0},
        # wide rows: a coarse level, or a token model over its voxels
        {"name": "norm_train_wide", "op": "norm_train", "rows": 16384, "channels": 4096, "dtype": "f16", "pad": 0},
        # a projection of a single token: latency and the weights' bytes
        {"name": "matmul_one_row", "op": "matmul", "rows": 1, "k": 1024, "n": 4096, "dtype": "bf16", "bias": False, "pad": 0},
        # odd sizes in every direction, 32-bit output with a bias
        {"name": "matmul_odd", "op": "matmul", "rows": 1003, "k": 601, "n": 523, "dtype": "f32", "bias": True, "pad": 5},
        # the widening projection on the voxels of 16 res-64 shells
        {"name": "matmul_16_shells", "op": "matmul", "rows": 124800, "k": 256, "n": 768, "dtype": "bf16", "bias": True, "pad": 0},
        # a product that the matrix units bound
        {"name": "matmul_large", "op": "matmul", "rows": 16384, "k": 4096, "n": 4096, "dtype": "bf16", "bias": False, "pad": 0},
        # a 3x3x3 convolution on two res-16 shells: latency
        {"name": "conv_small", "op": "conv", "kind": "k3s1", "members": 2, "res": 16, "cin": 64, "cout": 64, "dtype": "bf16", "bias": True, "pad": 0},
        # a 3x3x3 convolution on 16 res-64 shells
        {"name": "conv_16_shells", "op": "conv", "kind": "k3s1", "members": 16, "res": 64, "cin": 128, "cout": 128, "dtype": "bf16", "bias": True, "pad": 0},
        # a transposed 2x2x2 convolution of stride 2 onto the refined grids, odd widths
        {"name": "conv_up_odd", "op": "conv", "kind": "up2", "members": 8, "res": 32, "cin": 52, "cout": 45, "dtype": "f16", "bias": False, "pad": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_i8", "norm_train", "matmul", "conv"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    pad = rng.choice([0, 0, 3, 16])
    if op.startswith("norm"):
        channels = _log(rng, 8, 8192)
        return {"op": op, "rows": _log(rng, 1, min(130000, (1 << 26) // channels // BYTES[dtype] * 2)), "channels": channels, "dtype": dtype, "pad": pad}
    if op == "matmul":
        k, n = _log(rng, 16, 4096), _log(rng, 16, 4096)
        return {"op": op, "rows": _log(rng, 1, min(130000, (1 << 38) // (k * n))), "k": k, "n": n, "dtype": dtype, "bias": rng.random() < 0.5, "pad": pad}
    # cost counted in members * res^2 voxels (a surface), times the weights' size
    cin, cout = _log(rng, 8, 128), _log(rng, 8, 128)
    return {"op": op, "kind": rng.choice(["k3s1", "k3s1", "down2", "up2"]), "members": rng.randint(1, 16), "res": _log(rng, 12, 48), "cin": cin, "cout": cout,
            "dtype": dtype, "bias": rng.random() < 0.5, "pad": pad}


# ------------------------------------------------------------------ inputs


def _shells(case, seed, device):
    """Voxels int64 [V, 4] (member, x, y, z) of ellipsoid shells, one voxel thick, radii U[0.3, 0.45] of the resolution.
    The radii go with the case, so the number of voxels does too; the seed moves each member by an even offset."""
    members, res = case["members"], case["res"]
    radii = random.Random(members * 1000 + res)
    r = torch.tensor([[radii.uniform(0.3, 0.45) * res for _ in range(3)] for _ in range(members)], dtype=torch.float64, device=device)
    g = torch.arange(res, dtype=torch.float64, device=device) + 0.5 - 0.5 * res
    q = [g.view(1, -1, 1, 1), g.view(1, 1, -1, 1), g.view(1, 1, 1, -1)]
    a = [q[d] / r[:, d].view(-1, 1, 1, 1) for d in range(3)]
    b = [a[d] / r[:, d].view(-1, 1, 1, 1) for d in range(3)]
    rho = (a[0] ** 2 + a[1] ** 2 + a[2] ** 2).sqrt()
    grad = (b[0] ** 2 + b[1] ** 2 + b[2] ** 2).sqrt() / rho
    v = ((rho - 1).abs() < 0.5 * grad).nonzero()
    moves = random.Random(seed)
    move = torch.tensor([[0] + [2 * moves.randint(0, 5) for _ in range(3)] for _ in range(members)], device=device)
    return v + move[v[:, 0]]


def _ordered(v):
    """The voxels in canonical order: member, then x-major blocks of 128, of 8, and voxels."""
    key = v[:, 0]
    for shift, mask in ((7, 1023), (3, 15), (0, 7)):
        for d in (1, 2, 3):
            key = key * (mask + 1) + ((v[:, d] >> shift) & mask)
    return v[key.argsort()]


def _kernel_map(case, seed, device):
    """(number of source voxels, int32 [V_dst, taps]): the source row each target row reads at each kernel offset, or -1."""
    src = _ordered(_shells(case, seed, device))
    dst = src
    scale, lo, hi = 1, -1, 1
    if case["kind"] == "down2":
        dst = _ordered(torch.cat([src[:, :1], src[:, 1:] >> 1], 1).unique(dim=0))
        scale, lo, hi = 2, 0, 1
    elif case["kind"] == "up2":
        corner = torch.cartesian_prod(*([torch.arange(2, device=device)] * 3))
        corner = torch.cat([torch.zeros_like(corner[:, :1]), corner], 1)
        dst = _ordered((src * torch.tensor([1, 2, 2, 2], device=device)).unsqueeze(1).add(corner).view(-1, 4))
        lo, hi = 0, 1
    side = case["res"] + 16
    table = torch.full((case["members"], side, side, side), -1, dtype=torch.int32, device=device)
    at = src + torch.tensor([0, 2, 2, 2], device=device)
    table[at[:, 0], at[:, 1], at[:, 2], at[:, 3]] = torch.arange(src.shape[0], dtype=torch.int32, device=device)
    span = torch.arange(lo, hi + 1, device=device)
    columns = []
    for d in torch.cartesian_prod(span, span, span):
        if case["kind"] == "up2":
            o = dst[:, 1:] - d
            here = (o & 1).eq(0).all(1)
            o = (o >> 1) + 2
        else:
            o = dst[:, 1:] * scale + d + 2
            here = torch.ones_like(o[:, 0], dtype=torch.bool)
        columns.append(torch.where(here, table[dst[:, 0], o[:, 0], o[:, 1], o[:, 2]], -1))
    return src.shape[0], torch.stack(columns, 1).to(torch.int32).contiguous()


def _in_buffer(t, pad):
    """`t` as the first columns of a wider buffer, as a slice of concatenated features is."""
    if not pad:
        return t.contiguous()
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _rows_i8(shape, gen, spread):
    """8-bit rows with one scale each, as a quantised layer holds them; `spread` of the channels' sizes. Some rows are all zero."""
    t = torch.randn(shape, generator=gen, device="cuda")
    if spread:
        t *= torch.exp(0.5 * torch.randn((1, shape[-1]), generator=gen, device="cuda"))
        t *= (torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") > 0.01)
    a = t.abs().amax(-1, keepdim=True)
    q = torch.round(t * torch.where(a > 0, 127.0 / a, torch.zeros_like(a))).to(torch.int8)
    return q, (a / 127.0).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    t = DTYPES[case["dtype"]]
    if case["op"].startswith("norm"):
        shape = (case["rows"], case["channels"])
        gain = torch.exp(0.5 * torch.randn((1, shape[1]), generator=gen, device="cuda"))
        s["x"] = _in_buffer((torch.randn(shape, generator=gen, device="cuda") * gain).to(t), case["pad"])
        s["residual"] = (2.0 * torch.randn(shape, generator=gen, device="cuda")).to(t)
        s["weight"] = (1.0 + 0.2 * torch.randn(shape[1], generator=gen, device="cuda")).to(t)
        if case["op"] == "norm_train":
            s["grad_out"] = torch.randn(shape, generator=gen, device="cuda").to(t)
            s["grad_h"] = torch.randn(shape, generator=gen, device="cuda").to(t)
        return s
    if case["op"] == "matmul":
        rows, cin, cout = case["rows"], case["k"], case["n"]
        w, ws = _rows_i8((cout, cin), gen, False)
    else:
        rows, s["map"] = _kernel_map(case, seed, "cuda")
        cin, cout = case["cin"], case["cout"]
        taps = s["map"].shape[1]
        w, ws = _rows_i8((cout, taps * cin), gen, False)
        w = w.view(cout, taps, cin).transpose(0, 1).contiguous()
    x, s["x_scale"] = _rows_i8((rows, cin), gen, True)
    s["x"] = _in_buffer(x, case["pad"])
    s["w"], s["w_scale"] = w, ws / math.sqrt(cin)
    s["bias"] = torch.randn(cout, generator=gen, device="cuda") if case["bias"] else None
    s["out_dtype"] = t
    return s


# ------------------------------------------------------------------ one pass


def _norm_plain(s):
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    return h, hf, torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS)


def _train_plain(s):
    h, hf, rstd = _norm_plain(s)
    w = s["weight"].float()
    out = (hf * rstd * w).to(h.dtype)
    dy = s["grad_out"].float()
    g = dy * w
    dx = rstd * g - hf * rstd.pow(3) * (g * hf).mean(-1, keepdim=True) + s["grad_h"].float()
    return {"out": out, "h": h, "grad_x": dx.to(h.dtype), "grad_weight": (dy * hf * rstd).sum(0)}


def _norm_i8_plain(s):
    h, hf, rstd = _norm_plain(s)
    # products in 64 bits, where they are exact: the integers next to a rounding border come out the same everywhere
    p = h.double() * s["weight"].double()
    a = p.abs().amax(-1, keepdim=True)
    q = torch.round(p * torch.where(a > 0, torch.full_like(a, 127.0) / a, torch.zeros_like(a)))
    scale = a.float() * rstd / 127.0
    return {"h": h, "values": q.float() * scale}


def _matmul_plain(s):
    out = (s["x"].float() @ s["w"].float().t()) * s["x_scale"].unsqueeze(1) * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(s["out_dtype"])


def _conv_plain(s):
    x = s["x"].float() * s["x_scale"].unsqueeze(1)
    x = torch.cat([x, torch.zeros_like(x[:1])])  # what absent neighbours read
    m = s["map"].long()
    rows = x[torch.where(m < 0, x.shape[0] - 1, m)]  # [V_dst, taps, cin]
    w = s["w"].float().transpose(1, 2).reshape(-1, s["w"].shape[1])
    out = (rows.view(m.shape[0], -1) @ w) * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(s["out_dtype"])


def run(s):
    op = s["case"]["op"]
    if own:
        from topology_construction_amd import binding
        if op == "norm_train":
            out, h, rstd = binding.tc_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            grad_x, grad_weight = binding.tc_rms_norm_backward(s["grad_out"], h, s["weight"], rstd, grad_h=s["grad_h"])
            return {"out": out, "h": h, "grad_x": grad_x, "grad_weight": grad_weight}
        if op == "norm_i8":
            q, scale, h = binding.tc_rms_norm_i8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return {"h": h, "values": q * scale.unsqueeze(1)}
        if op == "matmul":
            return binding.tc_matmul_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=s["out_dtype"])
        return binding.tc_sparse_conv_i8(s["x"], s["x_scale"], s["map"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=s["out_dtype"])
    if op == "norm_train":
        return _train_plain(s)
    if op == "norm_i8":
        return _norm_i8_plain(s)
    return _matmul_plain(s) if op == "matmul" else _conv_plain(s)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    t = BYTES[case["dtype"]]
    if case["op"].startswith("norm"):
        n = case["rows"] * case["channels"]
        if case["op"] == "norm_i8":  # x, residual and h; the 8-bit rows as 32-bit values
            return {"bytes": n * (3 * t + 4) + t * case["channels"], "flops": 8 * n}
        # x, residual, out and h; both gradients in and one out (h is read by the backward too)
        return {"bytes": n * 8 * t + (t + 4) * case["channels"] + 8 * case["rows"], "flops": 17 * n}
    bias = 4 if case["bias"] else 0
    if case["op"] == "matmul":
        m, k, n = case["rows"], case["k"], case["n"]
        return {"bytes": m * (k + 4) + n * (k + 4 + bias) + t * m * n, "flops": 2 * m * n * k}
    src, m = _kernel_map(case, 0, "cpu")
    cin, cout = case["cin"], case["cout"]
    return {"bytes": 4 * m.numel() + src * (cin + 4) + m.shape[1] * cin * cout + cout * (4 + bias) + t * m.shape[0] * cout,
            "flops": 2 * int((m >= 0).sum()) * cin * cout}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        out = torch.matmul(s["x"].double(), s["w"].double().t())
        out = torch.einsum("mn,m,n->mn", out, s["x_scale"].double(), s["w_scale"].double())
        return out if s["bias"] is None else out + s["bias"].double()
    if case["op"] == "conv":
        m = s["map"].long()
        out = torch.zeros((m.shape[0], case["cout"]), dtype=torch.float64, device=m.device)
        for k in range(m.shape[1]):
            j = (m[:, k] >= 0).nonzero().squeeze(1)
            i = m[j, k]
            out.index_add_(0, j, (s["x"][i].double() @ s["w"][k].double().t()) * s["x_scale"][i].double().unsqueeze(1))
        out = out * s["w_scale"].double()
        return out if s["bias"] is None else out + s["bias"].double()
    # the sum is held in the inputs' type: the norm is the norm of what is held
    h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    w = s["weight"].double()
    unit = h / (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).sqrt()
    if case["op"] == "norm_i8":
        y = unit * w
        step = y.abs().amax(1, keepdim=True) / 127.0
        p = h * w
        top = p.abs().amax(1, keepdim=True)
        q = torch.where(top > 0, torch.round(p * (torch.full_like(top, 127.0) / top)), torch.zeros_like(p))
        return {"h": h, "values": q * step}
    gy = s["grad_out"].double()
    along = (gy * w * unit).sum(1, keepdim=True) / h.shape[1]
    length = (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).sqrt()
    grad_x = (gy * w - unit * along) / length + s["grad_h"].double()
    return {"out": unit * w, "h": h, "grad_x": grad_x, "grad_weight": (gy * unit).sum(0)}
