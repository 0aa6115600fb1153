"""Float64 references of the operators around the layer, from their definitions,
and the errors that the kernels' roundings allow.

u(dtype): the largest relative error of rounding to a type. A sum whose operands
were rounded independently is off by about u / sqrt(3) times the root of the sum of
its terms' squares; 8 times that is allowed, plus the rounding of the result itself
(u |result|, and half the smallest step for f16), plus 2^-18 times the sum of the
terms' magnitudes for f32 accumulation.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the smallest step of f16; below 2^-120 f32 itself ends (exp(88.7) overflows, and 88.7 e^-88.7 < 2^-120)
TINY = {torch.bfloat16: 2.0 ** -120, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -120}
ACC = 2.0 ** -18


def generator(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + mean).to(dtype)


def act_both(v, act):
    """act(v), act'(v) in float64."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return v * s, s + v * s * (1 - s)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v ** 3))
    return v * (1 + t) / 2, (1 + t) / 2 + v / 2 * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def gated(g, u, act, limit):
    """act(gc), act'(gc), uc"""
    gc, uc = (g.clamp(max=limit), u.clamp(-limit, limit)) if limit > 0 else (g, u)
    a, da = act_both(gc, act)
    return a, da, uc


def rounded_sum(values, squares, magnitudes, dtype):
    """Allowed error of a stored sum: of its rounded operands, the accumulation, and the store."""
    u = U[dtype]
    return 8 * u / math.sqrt(3) * squares.sqrt() + ACC * magnitudes + u * (1 + ACC) * values.abs() + TINY[dtype]


def ffn(x, wg, wu, wd, act, limit, dy=None):
    """-> {name: (value, allowed error)} of y, and with dy of the gradients."""
    dt = x.dtype
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    a, da, uc = gated(g, u, act, limit)
    h = a * uc
    # what f32 accumulation of g and u may move, as an error of the operands built from them
    eg, eu = ACC * (x.abs() @ wg.abs().t()), ACC * (x.abs() @ wu.abs().t())
    eh = (da * uc).abs() * eg + a.abs() * eu + ACC * h.abs() + TINY[dt]
    y = h @ wd.t()
    out = {"y": (y, rounded_sum(y, h ** 2 @ (wd ** 2).t(), h.abs() @ wd.abs().t(), dt) + eh @ wd.abs().t())}
    if dy is None:
        return out
    dy = dy.double()
    dh = dy @ wd
    edh = ACC * (dy.abs() @ wd.abs())
    dg, du = dh * uc * da, dh * a
    # act'' is at most 1.2 in either form
    edg = (uc * da).abs() * edh + (dh * da).abs() * eu + 1.2 * (dh * uc).abs() * eg + ACC * dg.abs() + TINY[dt]
    edu = a.abs() * edh + (dh * da).abs() * eg + ACC * du.abs() + TINY[dt]
    if limit > 0:
        dg, du = dg * (g <= limit), du * (u.abs() <= limit)
        # within g's or u's own error of a clamp the gradient may fall on either side of it
        edg = edg + (dh * uc * da).abs() * ((g - limit).abs() <= eg)
        edu = edu + (dh * a).abs() * ((u.abs() - limit).abs() <= eu)
    dx = dg @ wg + du @ wu
    out["dx"] = (dx, rounded_sum(dx, dg ** 2 @ wg ** 2 + du ** 2 @ wu ** 2, dg.abs() @ wg.abs() + du.abs() @ wu.abs(), dt)
                 + edg @ wg.abs() + edu @ wu.abs())
    for name, left, right, e in (("dw_gate", dg, x, edg), ("dw_up", du, x, edu)):
        v = left.t() @ right
        out[name] = (v, rounded_sum(v, (left ** 2).t() @ right ** 2, left.abs().t() @ right.abs(), dt) + e.t() @ right.abs())
    v = dy.t() @ h
    out["dw_down"] = (v, rounded_sum(v, (dy ** 2).t() @ h ** 2, dy.abs().t() @ h.abs(), dt) + dy.abs().t() @ eh)
    return out


def norm(r, y, w_post, w_pre, gate, eps, scale, dr_out=None, dn=None):
    """-> {name: (value, allowed error)}; gate broadcasts against [m, dim]. Everything is f32 until stored."""
    dt = r.dtype
    dim, m = r.shape[1], r.shape[0]
    r = r.double()
    y = torch.zeros_like(r) if y is None else y.double()
    wp, wn = (torch.ones(dim, dtype=torch.float64) if w is None else w.double() for w in (w_post, w_pre))
    gt = torch.ones(1, 1, dtype=torch.float64) if gate is None else gate.double()
    one = torch.ones(m, 1, dtype=torch.float64)
    rs1 = one if w_post is None else 1 / ((y * y).mean(1, keepdim=True) + eps).sqrt()
    p = y * rs1 * wp
    t = scale * r + gt * p
    f32 = 2.0 ** -20   # a few f32 operations and a sum of squares, relative
    et = f32 * ((scale * r).abs() + (gt * p).abs())

    def stored(v, e):
        return v, e + U[dt] * (v.abs() + e) + TINY[dt]

    out = {"r_out": stored(t, et)}
    rs2 = one if w_pre is None else 1 / ((t * t).mean(1, keepdim=True) + eps).sqrt()
    # rs2 moves by at most what its terms move, relative to the row's norm
    ers2 = rs2 * (f32 + (t.abs() * et).mean(1, keepdim=True) * rs2 ** 2)
    if w_pre is not None:
        out["n"] = stored(t * rs2 * wn, (et * rs2 + t.abs() * ers2) * wn.abs() + f32 * (t * rs2 * wn).abs())
    if dr_out is None and dn is None:
        return out
    do = torch.zeros_like(r) if dr_out is None else dr_out.double()
    d = torch.zeros_like(r) if dn is None else dn.double()
    a = wn * d
    e = do + (rs2 * (a - t * rs2 ** 2 * (t * a).mean(1, keepdim=True)) if dn is not None else 0)
    # every term of e, with the f32 sums' errors: magnitudes times a few f32 roundings
    ta = (t * a).abs().mean(1, keepdim=True)
    mag = do.abs() + (rs2 * (a.abs() + t.abs() * rs2 ** 2 * ta) if dn is not None else 0)
    grow = 1 + rs2 ** 2 * (t.abs() * (scale * r).abs() + t.abs() * (gt * p).abs()).mean(1, keepdim=True)
    ee = 8 * f32 * grow * mag + (rs2 ** 3 * et * ta if dn is not None else 0)
    out["dr"] = stored(scale * e, abs(scale) * ee)
    dp, edp = gt * e, gt.abs() * (ee + f32 * e.abs())
    if w_post is None:
        out["dy"] = stored(dp, edp)
    else:
        b, eb = wp * dp, wp.abs() * edp
        v = rs1 * (b - y * rs1 ** 2 * (y * b).mean(1, keepdim=True))
        mags = rs1 * (b.abs() + y.abs() * rs1 ** 2 * (y * b).abs().mean(1, keepdim=True))
        out["dy"] = stored(v, 8 * f32 * mags + rs1 * (eb + y.abs() * rs1 ** 2 * (y.abs() * eb).mean(1, keepdim=True)))
        v = dp * y * rs1
        out["dw_post"] = stored(v.sum(0), ((edp * (y * rs1).abs()) + 4 * f32 * v.abs()).sum(0))
    if w_pre is not None:
        v = d * t * rs2
        out["dw_pre"] = stored(v.sum(0), (d.abs() * (et * rs2 + t.abs() * ers2) + 4 * f32 * v.abs()).sum(0))
    if gate is not None:
        v, ev = e * p, ee * p.abs() + 4 * f32 * (e * p).abs()
        if gate.dim() == 1:
            out["dgate"] = stored(v.sum(0), ev.sum(0))
        elif gate.shape[1] == 1 and dim != 1:
            out["dgate"] = stored(v.sum(1, keepdim=True), ev.sum(1, keepdim=True))
        else:
            out["dgate"] = stored(v, ev)
    return out


def w4_values(codes, scales, zeros, group):
    """The matrix in float64."""
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double()
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 1)
    return (q - z) * scales.double().repeat_interleave(group, 1)


def w4_product(x, codes, scales, zeros, group):
    """-> (x W^T, error of the f32 sums): per group the terms are as large as (c + 15) s |x| before the
    zero point's part is taken off, c = 128 for bf16 and 64 for f16."""
    c = 128 if x.dtype == torch.bfloat16 else 64
    big = (c + 15) * scales.double().abs().repeat_interleave(group, 1)
    return x.double() @ w4_values(codes, scales, zeros, group).t(), 2.0 ** -21 * (x.double().abs() @ big.t())


def check(got, value, allowed, what):
    """Every value within its allowed error; the worst share of it is returned."""
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    assert torch.isfinite(got).all(), what
    share = ((got - value).abs() / allowed.clamp(min=1e-300)).max().item() if got.numel() else 0.0
    assert share <= 1.0, f"{what}: {share:.3g} times the allowed error"
    return share
