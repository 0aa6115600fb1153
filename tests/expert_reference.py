"""Float64 references of sorting by expert, of products with bias, activation and residual, and of dropout, from
their definitions, and the errors that the kernels' roundings allow (the rules are block_reference's)."""
import numpy
import torch

import block_reference as ref

F32 = 2.0 ** -24


def stored(v, e, dtype):
    return v, e + ref.U[dtype] * (v.abs() + e) + ref.TINY[dtype]


def sort(idx, n_experts):
    """-> row_of, pick_of, offsets, counted pick by pick"""
    flat = idx.flatten().tolist()
    lists = [[] for _ in range(n_experts)]
    for i, e in enumerate(flat):
        if 0 <= e < n_experts:
            lists[e].append(i)
    row_of, pick_of, offsets = [-1] * len(flat), [-1] * len(flat), [0]
    row = 0
    for picks in lists:
        for i in picks:
            row_of[i], pick_of[row] = row, i
            row += 1
        offsets.append(row)
    t = lambda v, shape: torch.tensor(v, dtype=torch.int32).reshape(shape)   # noqa: E731
    return t(row_of, idx.shape), t(pick_of, (len(flat),)), t(offsets, (n_experts + 1,))


def rows_at(rows, row_of):
    """[m, topk, dim] in float64; zeros where a pick has no row (whatever any row holds)"""
    there = (row_of >= 0) & (row_of < rows.shape[0])
    at = torch.zeros((*row_of.shape, rows.shape[1]), dtype=torch.float64)
    at[there] = rows.double()[row_of[there].long()]
    return at, there


def combine(e, weights, row_of, dtype):
    """-> (value, allowed error) of the weighted sum (weights None: of the sum)"""
    at, there = rows_at(e, row_of)
    w = there.double() if weights is None else torch.where(there, weights.double(), 0.0)
    terms = w[:, :, None] * at
    return stored(terms.sum(1), (row_of.shape[1] + 1) * F32 * terms.abs().sum(1), dtype)


def combine_backward(dy, e, weights, row_of, rows):
    """-> {name: (value, allowed)} with de NaN where no pick has the row"""
    at, there = rows_at(e, row_of)
    d = dy.double()
    terms = at * torch.where(there[:, :, None], d[:, None, :], 0.0)
    # a sum of dim products in f32, whichever order: dim + 1 roundings at most
    dw = terms.sum(2), (dy.shape[1] + 2) * F32 * terms.abs().sum(2) + ref.TINY[torch.float32]
    de = torch.full((rows, dy.shape[1]), float("nan"), dtype=torch.float64)
    for t, j in there.nonzero().tolist():
        de[row_of[t, j]] = weights[t, j].double() * d[t]
    return {"dweights": dw, "de": stored(de, F32 * de.abs(), dy.dtype)}


def act_both(z, act):
    return (z, torch.ones_like(z)) if act == "none" else ref.act_both(z, act)


def linear(x, w, bias, residual, act, dy=None):
    """-> {name: (value, allowed)} of one matrix"""
    dt = x.dtype
    x, w = x.double(), w.double()
    b = 0.0 if bias is None else bias.double()
    z = x @ w.t() + b
    ez = ref.ACC * (x.abs() @ w.abs().t() + (0.0 if bias is None else b.abs()))
    a, da = act_both(z, act)
    r = torch.zeros_like(z) if residual is None else residual.double()
    # act' and act'' are at most 1.2 in size; a few f32 roundings of the activation and the sum
    out = {"y": stored(a + r, (da.abs() + 1.2 * ez) * ez + ref.ACC * (a.abs() + r.abs()) + ref.TINY[dt], dt)}
    if dy is None:
        return out
    d = dy.double()
    dz = d * da
    edz = 1.2 * d.abs() * ez + ref.ACC * dz.abs() + ref.TINY[dt] if act != "none" else torch.zeros_like(dz)
    once = 0.0 if act == "none" else 1.0   # dz is rounded as an operand only where it is not dy itself
    dx, dw = dz @ w, dz.t() @ x
    out["dx"] = (dx, ref.rounded_sum(dx, once * (dz ** 2 @ w ** 2), dz.abs() @ w.abs(), dt) + edz @ w.abs())
    out["dw"] = (dw, ref.rounded_sum(dw, once * ((dz ** 2).t() @ x ** 2), dz.abs().t() @ x.abs(), dt) + edz.t() @ x.abs())
    out["dbias"] = stored(dz.sum(0), edz.sum(0) + ref.ACC * dz.abs().sum(0), dt)
    return out


def experts(x, w, bias, residual, act, offsets, dy=None):
    """The same for a matrix per expert; rows behind the last are NaN (left as they are)."""
    m, (n_experts, n, k) = x.shape[0], w.shape
    shapes = {"y": (m, n), "dx": (m, k), "dw": w.shape, "dbias": w.shape[:2]}
    names = shapes if dy is not None else ("y",)
    out = {name: [torch.full(shapes[name], float("nan") if name in ("y", "dx") else 0.0, dtype=torch.float64), torch.zeros(shapes[name], dtype=torch.float64)]
           for name in names}
    for e in range(n_experts):
        part = slice(int(offsets[e]), int(offsets[e + 1]))
        if part.start == part.stop:
            continue
        one = linear(x[part], w[e], None if bias is None else bias[e], None if residual is None else residual[part], act,
                     None if dy is None else dy[part])
        for name in names:
            for i in (0, 1):
                out[name][i][part if name in ("y", "dx") else e] = one[name][i]
    return out


def philox(counter, key):
    """Philox-4x32-10 of four arrays of 32-bit words and two words"""
    x, k = [c.astype(numpy.uint64) for c in counter], [int(v) for v in key]
    low, s = numpy.uint64(0xFFFFFFFF), numpy.uint64(32)
    for _ in range(10):
        p0, p1 = x[0] * numpy.uint64(0xD2511F53), x[2] * numpy.uint64(0xCD9E8D57)
        x = [(p1 >> s) ^ x[1] ^ numpy.uint64(k[0]), p1 & low, (p0 >> s) ^ x[3] ^ numpy.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return x


def keep(seed, use, m, dim, p):
    """bool [m, dim]"""
    c = numpy.arange((dim + 7) // 8)[None, :] + numpy.zeros((m, 1), dtype=numpy.int64)
    r = numpy.arange(m)[:, None] + numpy.zeros_like(c)
    words = philox([c, r, numpy.full_like(c, use % 2 ** 32), numpy.full_like(c, (use >> 32) % 2 ** 32)],
                   [seed % 2 ** 32, (seed >> 32) % 2 ** 32])
    bits = numpy.empty((m, c.shape[1], 8), dtype=numpy.int64)
    for i, w in enumerate(words):
        bits[:, :, 2 * i], bits[:, :, 2 * i + 1] = w & numpy.uint64(0xFFFF), w >> numpy.uint64(16)
    return torch.from_numpy(bits.reshape(m, -1)[:, :dim] >= round(p * 65536))


def dropout(x, residual, mask, p):
    t = round(p * 65536)
    v = torch.where(mask, x.double() * (65536 / (65536 - t) if t < 65536 else 0.0), 0.0)
    e = 3 * F32 * v.abs()
    if residual is not None:
        v, e = v + residual.double(), e + F32 * (v.abs() + residual.double().abs())
    return stored(v, e, x.dtype)
