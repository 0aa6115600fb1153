"""The operators around a feed-forward block, as cases to be timed.

  ffn   the gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T: `forward`, and `step`, a training step's forward
        and backward (y, dx and the three weight gradients)
  norm  the norm after a block, its gate, the scaled residual and the norm before the next block: `forward` (the new
        residual and the normed rows), and `step`, forward and backward (all gradients)
  w4    products with 4-bit weights that have a scale, and perhaps a zero point, per group: `matmul`, and `gated`, the
        first half of the gated block in that form

Sizes: dim 5120 and inter 2304 are the layer that this repository benchmarks, 8192 x 2048 the widest that it tests; the
others are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    ffn = dict(op="ffn", dim=5120, inter=2304, dtype="bf16", act="silu", limit=10.0)
    norm = dict(op="norm", dim=5120, dtype="bf16", gate="channel", res_scale=1.0)
    return [
        # one token while serving: bound by reading the weights
        dict(ffn, name="ffn one token", dir="forward", m=1),
        # a small ragged batch while serving, the widest layer, the other activation and type
        dict(ffn, name="ffn 47 tokens", dir="forward", m=47, dim=8192, inter=2048, dtype="f16", act="gelu", limit=0.0),
        # a prompt: bound by the matrix cores
        dict(ffn, name="ffn prompt", dir="forward", m=2048),
        # a training step of a short ragged batch, sizes that no tile divides
        dict(ffn, name="ffn ragged step", dir="step", m=1013, dim=1544, inter=4104, dtype="f16", act="gelu", limit=0.0),
        # a training step of a full batch
        dict(ffn, name="ffn step", dir="step", m=8192),
        # one token while serving: latency
        dict(norm, name="norm one token", dir="forward", m=1),
        # a prompt, with a gate of its own for each token
        dict(norm, name="norm prompt", dir="forward", m=2048, gate="token", res_scale=0.5),
        # a training step of 32-bit rows of odd length with a gate for every value
        dict(norm, name="norm ragged step", dir="step", m=1003, dim=1111, dtype="f32", gate="full", res_scale=0.7),
        # a training step of a full batch
        dict(norm, name="norm step", dir="step", m=8192),
        # one token's down projection while serving, codes around 8
        dict(op="w4", name="w4 one token", kind="matmul", m=1, rows=5120, cols=2304, group=128, zeros=False, dtype="bf16"),
        # eight sequences' gate and up projections, small groups with zero points
        dict(op="w4", name="w4 gated 8 tokens", kind="gated", m=8, rows=2304, cols=5120, group=32, zeros=True, dtype="bf16"),
        # a vocabulary-sized product for a small ragged batch
        dict(op="w4", name="w4 wide output", kind="matmul", m=19, rows=32768, cols=8192, group=64, zeros=True, dtype="f16"),
    ]


def draw(rng):
    def log(lo, hi, step=1):  # a multiple of `step`, of no one model's width
        v = step * max(1, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))
        return v + step if v == 3 * 1024 else v

    kind = rng.choice(["ffn forward", "ffn step", "norm forward", "norm step", "matmul", "gated"])
    op, dir_ = kind.split() if " " in kind else ("w4", kind)
    if op == "ffn":
        dim, inter = log(256, 8192, 8), log(256, 8192, 8)
        m = min(log(1, 8192), 8192 * 5120 * 2304 // (dim * inter))
        return dict(op="ffn", dir=dir_, m=m, dim=dim, inter=inter, dtype=rng.choice(["bf16", "f16"]),
                    act=rng.choice(["silu", "gelu"]), limit=rng.choice([0.0, 2.0, 10.0]))
    if op == "norm":
        dim = log(64, 8192)
        return dict(op="norm", dir=dir_, m=min(log(1, 16384), 8192 * 2560 // dim), dim=dim,
                    dtype=rng.choice(["bf16", "f16", "f32"]), gate=rng.choice(["none", "channel", "token", "full"]),
                    res_scale=rng.choice([1.0, 0.5, 0.7]))
    group = rng.choice([32, 64, 128])
    return dict(op="w4", kind=dir_, m=log(1, 64), rows=log(64, 16384), cols=log(256, 8192, group),
                group=group, zeros=rng.choice([False, True]), dtype=rng.choice(["bf16", "f16"]))


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, dtype, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale + mean).to(dtype)


def rows_in(g, m, dim, dtype):
    """Normed rows, a few of whose channels are much larger than the others, as in a trained model."""
    loud = 1 + 7 * (torch.rand(dim, generator=g, device="cuda") < 0.005)
    return (torch.randn((m, dim), generator=g, device="cuda") * loud).to(dtype)


def quantised(g, rows, cols, group, zeros, dtype):
    """Codes [rows, cols / 2] (the even column in the low four bits), scales [rows, cols / group], and zero points
    [rows, cols / group] in bytes, or None."""
    q = torch.randn((rows, cols), generator=g, device="cuda").mul_(2.6).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
    s = normal(g, (rows, cols // group), torch.float32, 0.2, 1.0).clamp_min_(0.3).mul_(0.02 / 2.6).to(dtype)
    z = torch.randint(5, 11, (rows, cols // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return {"codes": q[:, 0::2] | (q[:, 1::2] << 4), "scales": s, "zeros": z}


def prepare(case, seed):
    g, dtype, m = generator(seed), DTYPES[case["dtype"]], case["m"]
    s = {"case": case}
    if case["op"] == "ffn":
        d, i = case["dim"], case["inter"]
        s["x"] = rows_in(g, m, d, dtype)
        s["wg"], s["wu"] = (normal(g, (i, d), dtype, 1.2 / math.sqrt(d)) for _ in range(2))
        s["wd"] = normal(g, (d, i), dtype, 1 / math.sqrt(i))
        s["y"] = torch.empty_like(s["x"])
        if case["dir"] == "step":
            s["dy"] = normal(g, (m, d), dtype, 0.1)
            s["dx"], s["dwg"], s["dwu"], s["dwd"] = (torch.empty_like(s[k]) for k in ("x", "wg", "wu", "wd"))
        if own:  # the block's description, and the memory that its calls work in
            import mixture_experts_ffn_gemv_amd as moe

            s["ffn"] = moe.make_ffn(s["wg"], s["wu"], s["wd"], act=case["act"], limit=case["limit"])
            forward, saved, backward = moe.moe_ffn_workspace(s["ffn"], m)
            step = case["dir"] == "step"
            s["work"] = torch.empty(max(forward, backward if step else 0), dtype=torch.uint8, device="cuda")
            s["saved"] = torch.empty(saved, dtype=torch.uint8, device="cuda") if step else None
    elif case["op"] == "norm":
        d = case["dim"]
        s["r"] = rows_in(g, m, d, dtype).mul_(2)
        s["y"] = rows_in(g, m, d, dtype)
        s["w_post"], s["w_pre"] = (normal(g, (d,), dtype, 0.2, 1.0) for _ in range(2))
        shape = {"none": None, "channel": (d,), "token": (m, 1), "full": (m, d)}[case["gate"]]
        s["gate"] = None if shape is None else normal(g, shape, dtype, 0.3, 0.5)
        s["r_out"], s["n"] = torch.empty_like(s["r"]), torch.empty_like(s["r"])
        if case["dir"] == "step":
            s["dr_out"], s["dn"] = normal(g, (m, d), dtype, 0.1), normal(g, (m, d), dtype, 0.1)
            s["stats"] = torch.empty((m, 2), dtype=torch.float32, device="cuda")
            for k in ("r", "y", "w_post", "w_pre", "gate"):
                s["d_" + k] = None if s[k] is None else torch.empty_like(s[k])
        if own:  # the norms' description, and the memory that the backward pass works in
            import mixture_experts_ffn_gemv_amd as moe

            s["norm"] = moe.make_norm(d, dtype, w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, res_scale=case["res_scale"])
            if case["dir"] == "step":
                s["work"] = torch.empty(moe.moe_norm_workspace(s["norm"], m), dtype=torch.uint8, device="cuda")
    else:
        s["x"] = rows_in(g, m, case["cols"], dtype)
        s["w"] = [quantised(g, case["rows"], case["cols"], case["group"], case["zeros"], dtype)
                  for _ in range(2 if case["kind"] == "gated" else 1)]
        s["out"] = torch.empty((m, case["rows"]), dtype=dtype, device="cuda")
        if own:  # the matrices' descriptions: their codes stay as they are
            import mixture_experts_ffn_gemv_amd as moe

            s["w4"] = [moe.make_w4(w["codes"], w["scales"], w["zeros"], group=case["group"]) for w in s["w"]]
    return s


def act_plain(v, act):
    """act(v) and act'(v)."""
    if act == "silu":
        t = 1 / (1 + torch.exp(-v))
        return v * t, t * (1 + v * (1 - t))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def gated_plain(g, u, act, limit):
    """h = act(g) u of the clamped g and u, with act and its derivative there."""
    if limit > 0:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    a, da = act_plain(g, act)
    return a * u, a, da, u


def ffn_plain(s):
    c = s["case"]
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.t(), x @ wu.t()
    h, a, da, uc = gated_plain(g, u, c["act"], c["limit"])
    dtype = s["x"].dtype
    y = (h @ wd.t()).to(dtype)
    if c["dir"] == "forward":
        return {"y": y}
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * uc * da, dh * a
    if c["limit"] > 0:
        dg, du = dg * (g <= c["limit"]), du * (u.abs() <= c["limit"])
    return {"y": y, "dx": (dg @ wg + du @ wu).to(dtype), "dwg": (dg.t() @ x).to(dtype), "dwu": (du.t() @ x).to(dtype),
            "dwd": (dy.t() @ h).to(dtype)}


def norm_plain(s):
    c = s["case"]
    r, y, w_post, w_pre = (s[k].float() for k in ("r", "y", "w_post", "w_pre"))
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    rs1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    p = y * rs1 * w_post
    t = c["res_scale"] * r + gate * p
    rs2 = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    out = {"r_out": t.to(s["r"].dtype), "n": (t * rs2 * w_pre).to(s["r"].dtype)}
    if c["dir"] == "forward":
        return out
    dn = s["dn"].float()
    a = w_pre * dn
    e = s["dr_out"].float() + rs2 * (a - t * rs2 * rs2 * (t * a).mean(1, keepdim=True))
    dp = gate * e
    b = w_post * dp
    grads = {"r": c["res_scale"] * e, "y": rs1 * (b - y * rs1 * rs1 * (y * b).mean(1, keepdim=True)),
             "w_post": (dp * y * rs1).sum(0), "w_pre": (dn * t * rs2).sum(0)}
    if c["gate"] != "none":
        grads["gate"] = {"channel": lambda v: v.sum(0), "token": lambda v: v.sum(1, keepdim=True), "full": lambda v: v}[c["gate"]](e * p)
    return out | {"d_" + k: v.to(s[k].dtype) for k, v in grads.items()}


def dequantised(w, group):
    q = torch.stack((w["codes"] & 15, w["codes"] >> 4), 2).flatten(1).float()
    z = 8.0 if w["zeros"] is None else w["zeros"].float()[:, :, None]
    return ((q.view(q.shape[0], -1, group) - z) * w["scales"].float()[:, :, None]).flatten(1)


def w4_plain(s):
    x, group = s["x"].float(), s["case"]["group"]
    first = x @ dequantised(s["w"][0], group).t()
    if s["case"]["kind"] == "gated":
        first = gated_plain(first, x @ dequantised(s["w"][1], group).t(), "silu", 10.0)[0]
    return {"out": first.to(s["x"].dtype)}


def run(s):
    c = s["case"]
    if not own:
        return {"ffn": ffn_plain, "norm": norm_plain, "w4": w4_plain}[c["op"]](s)
    import mixture_experts_ffn_gemv_amd as moe

    if c["op"] == "ffn":
        if c["dir"] == "forward":
            moe.moe_ffn_forward(s["ffn"], s["x"], s["y"], s["work"])
            return {"y": s["y"]}
        moe.moe_ffn_forward(s["ffn"], s["x"], s["y"], s["work"], saved=s["saved"])
        moe.moe_ffn_backward(s["ffn"], s["x"], s["dy"], s["saved"], s["work"], dx=s["dx"], dw_gate=s["dwg"],
                             dw_up=s["dwu"], dw_down=s["dwd"])
        return {k: s[k] for k in ("y", "dx", "dwg", "dwu", "dwd")}
    if c["op"] == "norm":
        out = {"r_out": s["r_out"], "n": s["n"]}
        if c["dir"] == "forward":
            moe.moe_norm_forward(s["norm"], s["r"], s["y"], s["r_out"], s["n"], gate=s["gate"])
            return out
        moe.moe_norm_forward(s["norm"], s["r"], s["y"], s["r_out"], s["n"], gate=s["gate"], stats=s["stats"])
        moe.moe_norm_backward(s["norm"], s["r"], s["y"], s["stats"], s["dr_out"], s["dn"], s["work"], gate=s["gate"],
                              dr=s["d_r"], dy=s["d_y"], dgate=s["d_gate"], dw_post=s["d_w_post"], dw_pre=s["d_w_pre"])
        return out | {"d_" + k: s["d_" + k] for k in ("r", "y", "w_post", "w_pre", "gate") if s["d_" + k] is not None}
    if c["kind"] == "gated":
        moe.moe_w4_gated(s["w4"][0], s["w4"][1], s["x"], s["out"], act="silu", limit=10.0)
    else:
        moe.moe_w4_matmul(s["w4"][0], s["x"], s["out"])
    return {"out": s["out"]}


def work(case):
    m, size = case["m"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ffn":
        d, i = case["dim"], case["inter"]
        if case["dir"] == "forward":
            return {"bytes": 2 * (3 * d * i + 2 * m * d), "flops": 6 * m * d * i}
        return {"bytes": 2 * (6 * d * i + 4 * m * d), "flops": 18 * m * d * i}
    if case["op"] == "norm":
        d = case["dim"]
        gate = {"none": 0, "channel": d, "token": m, "full": m * d}[case["gate"]]
        if case["dir"] == "forward":
            return {"bytes": size * (4 * m * d + 2 * d + gate), "flops": 10 * m * d}
        return {"bytes": size * (8 * m * d + 4 * d + 2 * gate), "flops": 40 * m * d}
    n, k = case["rows"], case["cols"]
    each = n * k // 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2)
    matrices = 2 if case["kind"] == "gated" else 1
    return {"bytes": matrices * each + 2 * m * (n + k), "flops": matrices * 2 * m * n * k}


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating the forward definition."""
    s = prepare(case, seed)

    def leaf(t):
        return None if t is None else t.double().requires_grad_(case.get("dir") == "step")

    def block(gate, up, act, limit):
        if limit > 0:
            gate, up = torch.clamp(gate, max=limit), torch.clamp(up, min=-limit, max=limit)
        if act == "silu":
            return gate * torch.sigmoid(gate) * up
        return torch.nn.functional.gelu(gate, approximate="tanh") * up

    if case["op"] == "ffn":
        x, wg, wu, wd = leaves = [leaf(s[k]) for k in ("x", "wg", "wu", "wd")]
        lin = torch.nn.functional.linear
        y = lin(block(lin(x, wg), lin(x, wu), case["act"], case["limit"]), wd)
        out = {"y": y.detach()}
        if case["dir"] == "step":
            out |= dict(zip(("dx", "dwg", "dwu", "dwd"), torch.autograd.grad(y, leaves, s["dy"].double())))
        return out
    if case["op"] == "norm":
        names = [k for k in ("r", "y", "w_post", "w_pre", "gate") if s[k] is not None]
        v = {k: leaf(s[k]) for k in names}

        def rms(t):
            return t / (t.square().sum(-1, keepdim=True) / t.shape[-1] + EPS).sqrt()

        branch = rms(v["y"]) * v["w_post"]
        if "gate" in v:
            branch = branch * v["gate"]
        r_out = v["r"] * case["res_scale"] + branch
        n = rms(r_out) * v["w_pre"]
        out = {"r_out": r_out.detach(), "n": n.detach()}
        if case["dir"] == "step":
            grads = torch.autograd.grad([r_out, n], [v[k] for k in names], [s["dr_out"].double(), s["dn"].double()])
            out |= {"d_" + k: t for k, t in zip(names, grads)}
        return out
    products = []
    for w in s["w"]:
        wide = torch.empty((case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
        wide[:, 0::2], wide[:, 1::2] = w["codes"] % 16, w["codes"] // 16
        zero = torch.full_like(w["scales"], 8).double() if w["zeros"] is None else w["zeros"].double()
        wide -= zero.repeat_interleave(case["group"], 1)
        wide *= w["scales"].double().repeat_interleave(case["group"], 1)
        products.append(s["x"].double() @ wide.t())
    return {"out": block(products[0], products[1], "silu", 10.0) if case["kind"] == "gated" else products[0]}
