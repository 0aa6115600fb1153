"""The steps of a mixture-of-experts block with 16-bit experts, and of a dense one with biases, as cases to be timed.

  sort     tokens sorted by the experts they picked and back: `forward` (positions, sorted rows, weighted sums), and
           `step`, a training step's forward and backward (the gradients of the sorted rows, of the experts' results
           and of the routing weights)
  linear   act(x W^T + bias) + residual: `forward`, and `step`, forward and backward (y, dx, dW and dbias)
  experts  the same product with a matrix per expert, of rows sorted by expert
  dropout  residual + dropout(x) with a mask that is made anew in the backward pass: `step`, y and dx

Sizes: dim 5120, inter 2304, 384 experts and 6 picks are the layer that this repository benchmarks, 8192 x 2048 the
widest that it tests; the others are generic.
"""
import math

import numpy
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    sort = dict(op="sort", dim=5120, experts=384, topk=6, dtype="bf16", padded=0)
    linear = dict(op="linear", dtype="bf16", bias=True, residual=True)
    experts = dict(op="experts", dtype="bf16", bias=False, padded=0)
    return [
        # one token while serving: latency
        dict(sort, name="sort one token", dir="forward", m=1),
        # a ragged prompt, whose last tokens are padding without a pick
        dict(sort, name="sort prompt", dir="forward", m=1999, dtype="f16", padded=37),
        # a training step of a full batch
        dict(sort, name="sort step", dir="step", m=8192),
        # one token's projection back to the residual while serving: bound by reading the weights
        dict(linear, name="linear one token", dir="forward", m=1, cols=2304, rows=5120, act="none"),
        # a small ragged batch while serving, the widest layer, the other activation and type
        dict(linear, name="linear 23 tokens", dir="forward", m=23, cols=8192, rows=2048, act="gelu", dtype="f16", residual=False),
        # a training step of a short ragged batch, sizes that no tile divides, an odd number of outputs
        dict(linear, name="linear ragged step", dir="step", m=1013, cols=1544, rows=4101, act="gelu", dtype="f16"),
        # a training step of a full batch: bound by the matrix cores
        dict(linear, name="linear step", dir="step", m=8192, cols=5120, rows=2304, act="silu"),
        # one token's six experts while serving: their weights
        dict(experts, name="experts one token", dir="forward", tokens=1, experts=384, topk=6, cols=5120, rows=2304, act="silu"),
        # a prompt over every expert, some tens of rows each: their weights, read once
        dict(experts, name="experts prompt", dir="forward", tokens=500, experts=64, topk=6, cols=2048, rows=1408, act="gelu",
             dtype="f16", bias=True),
        # a training step of a batch whose last tokens are padding
        dict(experts, name="experts step", dir="step", tokens=4096, experts=32, topk=4, cols=2048, rows=1408, act="silu", padded=50),
        # a training step of 32-bit rows of odd length: latency
        dict(op="dropout", name="dropout ragged step", m=1003, dim=1111, dtype="f32", p=0.2, residual=True),
        # a training step of a full batch: memory
        dict(op="dropout", name="dropout step", m=8192, dim=5120, dtype="bf16", p=0.1, residual=True),
    ]


def draw(rng):
    def log(lo, hi, step=1):   # a multiple of `step`
        return step * max(1, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))

    kind = rng.choice(["sort forward", "sort step", "linear forward", "linear step", "experts forward", "experts step", "dropout"])
    op, dir_ = kind.split() if " " in kind else (kind, "step")
    if op == "sort":
        dim, topk = log(64, 8192), rng.choice([1, 2, 4, 6, 8])
        m = min(log(1, 8192), 8192 * 6 * 5120 // (dim * topk * 2))
        return dict(op="sort", dir=dir_, m=m, dim=dim, topk=topk, experts=log(8, 512), dtype=rng.choice(["bf16", "f16", "f32"]),
                    padded=rng.choice([0, m // 7]))
    if op == "dropout":
        dim = log(64, 8192)
        return dict(op="dropout", m=min(log(1, 16384), 8192 * 2560 // dim), dim=dim, dtype=rng.choice(["bf16", "f16", "f32"]),
                    p=rng.choice([0.1, 0.2, 0.5]), residual=rng.choice([False, True]))
    cols, rows = log(256, 8192, 8), log(64, 8192)
    case = dict(op=op, dir=dir_, cols=cols, rows=rows, dtype=rng.choice(["bf16", "f16"]), act=rng.choice(["none", "silu", "gelu"]),
                bias=rng.choice([False, True]))
    if op == "linear":
        return dict(case, m=min(log(1, 8192), 8192 * 5120 * 2304 // (cols * rows)), residual=rng.choice([False, True]))
    topk = rng.choice([1, 2, 4, 6])
    experts = max(topk, min(log(4, 128), 12 * 10 ** 8 // (cols * rows)))
    tokens = max(1, min(log(1, 8192), 4 * 10 ** 10 // (cols * rows * topk)))
    return dict(case, experts=experts, topk=topk, tokens=tokens, padded=rng.choice([0, tokens // 7]))


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


def picks(g, m, topk, experts, padded):
    """Each token's experts, some more popular than others; -1 where a token is padding."""
    keys = torch.randn(experts, generator=g, device="cuda") + 1.5 * torch.randn((m, experts), generator=g, device="cuda")
    idx = keys.topk(topk, dim=1).indices.int()
    idx[m - padded:] = -1
    return idx.contiguous()


def prepare(case, seed):
    g, dtype, op = generator(seed), DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if own:
        import mixture_experts_ffn_gemv_amd as moe
    if op == "sort":
        m, dim, topk, experts = case["m"], case["dim"], case["topk"], case["experts"]
        n = m * topk
        s["idx"] = picks(g, m, topk, experts, case["padded"])
        weights = torch.rand((m, topk), generator=g, device="cuda") + 0.1
        s["weights"] = weights / weights.sum(1, keepdim=True) * 1.5
        s["x"], s["e"] = rows_in(g, m, dim, dtype), rows_in(g, n, dim, dtype)
        s["row_of"] = torch.zeros((m, topk), dtype=torch.int32, device="cuda")
        s["pick_of"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        s["xs"], s["y"] = torch.zeros_like(s["e"]), torch.empty_like(s["x"])
        if case["dir"] == "step":
            s["dy"], s["dxs"] = normal(g, (m, dim), dtype, 0.1), normal(g, (n, dim), dtype, 0.1)
            s["de"], s["dweights"], s["dx"] = torch.zeros_like(s["e"]), torch.empty_like(s["weights"]), torch.empty_like(s["x"])
        if own:   # the memory that the sort works in
            s["work"] = torch.empty(moe.moe_sort_workspace(m, topk, experts), dtype=torch.uint8, device="cuda")
    elif op == "dropout":
        m, dim = case["m"], case["dim"]
        s["x"], s["dy"] = rows_in(g, m, dim, dtype), normal(g, (m, dim), dtype, 0.1)
        s["residual"] = rows_in(g, m, dim, dtype).mul_(2) if case["residual"] else None
        # the generator's key and the number of this use of it
        s["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device="cuda")
        s["y"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        if own:
            s["dropout"] = moe.make_dropout(dim, dtype, case["p"])
    else:
        k, n = case["cols"], case["rows"]
        if op == "linear":
            m, shape = case["m"], (n, k)
            s["offsets"] = None
        else:   # rows sorted by expert; behind the last expert's are those of padding, which are left as they are
            m, shape = case["tokens"] * case["topk"], (case["experts"], n, k)
            idx = picks(g, case["tokens"], case["topk"], case["experts"], case["padded"])
            count = torch.bincount(idx.flatten() + 1, minlength=case["experts"] + 1)
            count[0] = 0
            s["offsets"] = count.cumsum(0).int()
        s["x"] = rows_in(g, m, k, dtype)
        s["w"] = torch.empty(shape, dtype=dtype, device="cuda").normal_(0, 1.2 / math.sqrt(k), generator=g)
        s["bias"] = normal(g, shape[:-1], dtype, 0.3) if case["bias"] else None
        s["residual"] = rows_in(g, m, n, dtype).mul_(2) if case.get("residual") else None
        s["y"] = torch.zeros((m, n), dtype=dtype, device="cuda")
        if case["dir"] == "step":
            s["dy"], s["dx"], s["dw"] = normal(g, (m, n), dtype, 0.1), torch.zeros_like(s["x"]), torch.empty_like(s["w"])
            s["dbias"] = torch.empty_like(s["bias"]) if case["bias"] else None
        if own:   # the matrices' description, and the memory that its calls work in
            s["linear"] = moe.make_linear(s["w"], s["bias"], act=case["act"])
            forward, saved, backward = moe.moe_linear_workspace(s["linear"], m)
            step = case["dir"] == "step"
            s["work"] = torch.empty(max(forward, backward if step else 0), dtype=torch.uint8, device="cuda")
            s["saved"] = torch.empty(saved, dtype=torch.uint8, device="cuda") if step else None
    return s


def sort_plain(s):
    c = s["case"]
    m, topk, experts, dtype = c["m"], c["topk"], c["experts"], s["x"].dtype
    flat = s["idx"].flatten().long()
    valid = flat >= 0
    order = torch.argsort(torch.where(valid, flat, experts), stable=True)
    rows = torch.arange(m * topk, device="cuda")
    offsets = torch.cat((rows[:1] * 0, (flat[:, None] == torch.arange(experts, device="cuda")).sum(0).cumsum(0)))
    pick_of = torch.where(rows < offsets[-1], order, -1)
    row_of = torch.empty_like(order)
    row_of[order] = rows
    row_of = torch.where(valid, row_of, -1).view(m, topk)
    there = (row_of >= 0)[:, :, None]
    xs = torch.where((pick_of >= 0)[:, None], s["x"][order // topk], torch.zeros_like(s["e"]))

    def at(rows):   # [m, topk, dim] in 32 bits, zeros for picks without a row
        return torch.where(there, rows[row_of.clamp(min=0)].float(), 0.0)

    out = {"row_of": row_of.int(), "pick_of": pick_of.int(), "offsets": offsets.int(), "xs": xs,
           "y": (s["weights"][:, :, None] * at(s["e"])).sum(1).to(dtype)}
    if c["dir"] == "step":
        dy = s["dy"].float()
        de = s["weights"].flatten()[order][:, None] * dy[order // topk]
        out["de"] = torch.where((pick_of >= 0)[:, None], de, 0.0).to(dtype)
        out["dweights"] = (at(s["e"]) * dy[:, None, :]).sum(2)
        out["dx"] = at(s["dxs"]).sum(1).to(dtype)
    return out


def act_plain(v, act):
    """act(v) and act'(v)."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "silu":
        t = 1 / (1 + torch.exp(-v))
        return v * t, t * (1 + v * (1 - t))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def linear_plain(s):
    c, dtype = s["case"], s["x"].dtype
    step = c["dir"] == "step"
    one = s["offsets"] is None
    w, bias = (s["w"][None], s["bias"] if s["bias"] is None else s["bias"][None]) if one else (s["w"], s["bias"])
    ends = [0, s["x"].shape[0]] if one else s["offsets"].tolist()
    out = {"y": torch.zeros_like(s["y"])}
    if step:
        out["dx"], out["dw"] = torch.zeros_like(s["x"]), torch.zeros_like(w)
        if bias is not None:
            out["dbias"] = torch.zeros_like(bias)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            continue
        x, we = s["x"][a:b].float(), w[e].float()
        z = x @ we.t()
        if bias is not None:
            z = z + bias[e].float()
        y, da = act_plain(z, c["act"])
        out["y"][a:b] = y if s["residual"] is None else y + s["residual"][a:b].float()
        if step:
            dz = s["dy"][a:b].float() * da
            out["dx"][a:b] = dz @ we
            out["dw"][e] = dz.t() @ x
            if bias is not None:
                out["dbias"][e] = dz.sum(0)
    if step and one:
        out = {k: v[0] if k in ("dw", "dbias") else v for k, v in out.items()}
    return {k: v.to(dtype) for k, v in out.items()}


MULTIPLIERS, WEYL, LOW = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85), 0xFFFFFFFF


def keep_plain(rng, m, dim, p):
    """The values that are kept, [m, dim]: those whose 16 random bits are at least p 2^16. A row's eight values 8 c .. 8 c + 7
    share the 128 bits of Philox-4x32-10 (Salmon et al., 2011) at the counter (c, row, use's low word, its high word)."""
    key = [rng[0] & LOW, (rng[0] >> 32) & LOW]
    c = torch.arange((dim + 7) // 8, device="cuda")[None, :].expand(m, -1)
    r = torch.arange(m, device="cuda")[:, None].expand_as(c)
    ctr = [c, r, (rng[1] & LOW).expand_as(c), ((rng[1] >> 32) & LOW).expand_as(c)]
    for _ in range(10):
        a, b = ctr[0] * MULTIPLIERS[0], ctr[2] * MULTIPLIERS[1]   # 64 bits, whose top one may be a sign
        ctr = [((b >> 32) & LOW) ^ ctr[1] ^ key[0], b & LOW, ((a >> 32) & LOW) ^ ctr[3] ^ key[1], a & LOW]
        key = [(k + d) & LOW for k, d in zip(key, WEYL)]
    bits = torch.stack([h for w in ctr for h in (w & 0xFFFF, w >> 16)], 2).flatten(1)[:, :dim]
    return bits >= round(p * 65536)


def dropout_plain(s):
    c, dtype = s["case"], s["x"].dtype
    keep, scale = keep_plain(s["rng"], c["m"], c["dim"], c["p"]), 65536 / (65536 - round(c["p"] * 65536))
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(dtype), "dx": torch.where(keep, s["dy"].float() * scale, 0.0).to(dtype)}


def run(s):
    c = s["case"]
    step = c.get("dir") == "step"
    if not own:
        return {"sort": sort_plain, "linear": linear_plain, "experts": linear_plain, "dropout": dropout_plain}[c["op"]](s)
    import mixture_experts_ffn_gemv_amd as moe

    if c["op"] == "sort":
        moe.moe_sort(s["idx"], c["experts"], s["row_of"], s["pick_of"], s["offsets"], s["work"])
        moe.moe_dispatch_forward(s["x"], s["row_of"], s["xs"])
        moe.moe_combine_forward(s["e"], s["weights"], s["row_of"], s["y"])
        if step:
            moe.moe_combine_backward(s["dy"], s["e"], s["weights"], s["row_of"], s["de"], s["dweights"])
            moe.moe_dispatch_backward(s["dxs"], s["row_of"], s["dx"])
        return {k: s[k] for k in ("row_of", "pick_of", "offsets", "xs", "y") + (("de", "dweights", "dx") if step else ())}
    if c["op"] == "dropout":
        moe.moe_dropout_forward(s["dropout"], s["rng"], s["x"], s["y"], residual=s["residual"])
        moe.moe_dropout_backward(s["dropout"], s["rng"], s["dy"], s["dx"])
        return {"y": s["y"], "dx": s["dx"]}
    moe.moe_linear_forward(s["linear"], s["x"], s["y"], s["work"], offsets=s["offsets"], residual=s["residual"], saved=s["saved"])
    if not step:
        return {"y": s["y"]}
    moe.moe_linear_backward(s["linear"], s["x"], s["dy"], s["saved"], s["work"], offsets=s["offsets"], dx=s["dx"], dw=s["dw"],
                            dbias=s["dbias"])
    return {k: s[k] for k in ("y", "dx", "dw") + (("dbias",) if s["dbias"] is not None else ())}


def work(case):
    size, step = 4 if case["dtype"] == "f32" else 2, case.get("dir") == "step"
    if case["op"] == "sort":
        m, n, dim = case["m"], (case["m"] - case["padded"]) * case["topk"], case["dim"]
        moved = size * dim * (2 * m + 2 * n) + 4 * (4 * case["m"] * case["topk"] + case["experts"])
        if step:   # e is read once, for both of its uses
            moved += size * dim * (2 * m + 2 * n) + 4 * case["m"] * case["topk"]
        return {"bytes": moved, "flops": 2 * n * dim * (4 if step else 1)}
    if case["op"] == "dropout":
        values = case["m"] * case["dim"]
        return {"bytes": size * values * (5 if case["residual"] else 4), "flops": 4 * values}
    k, n = case["cols"], case["rows"]
    if case["op"] == "linear":
        m, matrices, used = case["m"], 1, 1
    else:   # a matrix without rows is not read; its gradient is written
        m, matrices = (case["tokens"] - case["padded"]) * case["topk"], case["experts"]
        used = min(matrices, m)
    moved = 2 * (used * n * k + m * (k + n) + (used * n if case["bias"] else 0) + (m * n if case.get("residual") else 0))
    if step:
        moved += 2 * (matrices * n * k + m * (k + n) + (matrices * n if case["bias"] else 0))
    return {"bytes": moved, "flops": 2 * m * n * k * (3 if step else 1)}


def exact_keep(rng, m, dim, p):
    """Which values are kept, in NumPy's unsigned words, a column of blocks at a time."""
    seed, use = (int(v) % 2 ** 64 for v in rng.tolist())
    u = numpy.uint64
    keep = numpy.empty((m, (dim + 7) // 8 * 8), dtype=bool)
    blocks = numpy.arange((dim + 7) // 8, dtype=u)
    for first in range(0, m, 1024):
        row = numpy.arange(first, min(m, first + 1024), dtype=u)
        x0, x1 = numpy.broadcast_arrays(blocks[None, :], row[:, None])
        x2, x3 = numpy.full(x0.shape, use % 2 ** 32, dtype=u), numpy.full(x0.shape, use >> 32, dtype=u)
        for i in range(10):
            k0, k1 = u((seed + i * 0x9E3779B9) % 2 ** 32), u(((seed >> 32) + i * 0xBB67AE85) % 2 ** 32)
            p0, p1 = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
            x0, x1, x2, x3 = (p1 >> u(32)) ^ x1 ^ k0, p1 & u(LOW), (p0 >> u(32)) ^ x3 ^ k1, p0 & u(LOW)
        words = numpy.stack((x0, x1, x2, x3), axis=2).astype("<u4").view("<u2").reshape(len(row), -1)
        keep[first:first + 1024] = words >= round(p * 65536)
    return torch.from_numpy(keep[:, :dim]).cuda()


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating the forward definition."""
    s = prepare(case, seed)
    step = case.get("dir") == "step"
    if case["op"] == "sort":
        m, topk, experts = case["m"], case["topk"], case["experts"]
        idx = s["idx"].cpu().numpy().reshape(-1)
        lists = [numpy.flatnonzero(idx == e) for e in range(experts)]   # picks in their order
        sorted_picks = numpy.concatenate(lists)
        pick_of = numpy.full(m * topk, -1)
        pick_of[:len(sorted_picks)] = sorted_picks
        row_of = numpy.full(m * topk, -1)
        row_of[sorted_picks] = numpy.arange(len(sorted_picks))
        offsets = numpy.cumsum([0] + [len(v) for v in lists])
        out = {k: torch.from_numpy(v).int().cuda() for k, v in (("row_of", row_of.reshape(m, topk)), ("pick_of", pick_of),
                                                                ("offsets", offsets))}
        rows, chosen = torch.arange(len(sorted_picks), device="cuda"), torch.from_numpy(sorted_picks).cuda()
        xs = torch.zeros(s["e"].shape, dtype=torch.float64, device="cuda")
        xs[rows] = s["x"].double()[chosen // topk]
        w = s["weights"].double().flatten()
        y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        y.index_add_(0, chosen // topk, w[chosen, None] * s["e"].double()[rows])
        out |= {"xs": xs, "y": y}
        if step:
            dy = s["dy"].double()
            de, dw, dx = torch.zeros_like(xs), torch.zeros_like(w), torch.zeros_like(y)
            de[rows] = w[chosen, None] * dy[chosen // topk]
            dw[chosen] = (s["e"].double()[rows] * dy[chosen // topk]).sum(1)
            dx.index_add_(0, chosen // topk, s["dxs"].double()[rows])
            out |= {"de": de, "dweights": dw.view(m, topk), "dx": dx}
        return out
    if case["op"] == "dropout":
        p = round(case["p"] * 65536) / 65536
        factor = exact_keep(s["rng"], case["m"], case["dim"], case["p"]).double() / (1 - p)
        y = factor * s["x"].double()
        return {"y": y if s["residual"] is None else y + s["residual"].double(), "dx": factor * s["dy"].double()}

    def forward(x, w, b, r):
        z = torch.nn.functional.linear(x, w, b)
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = torch.nn.functional.gelu(z, approximate="tanh")
        return z if r is None else z + r

    n = s["x"].shape[0]
    ends = [0, n] if case["op"] == "linear" else s["offsets"].tolist()
    names = ("y", "dx", "dw") + (("dbias",) if case["bias"] else ()) if step else ("y",)
    out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in names}
    for e in range(len(ends) - 1):
        part = slice(ends[e], ends[e + 1])
        if part.start == part.stop:
            continue

        def of(t):
            return t if t is None or case["op"] == "linear" else t[e]

        leaves = [None if t is None else t.double().requires_grad_(step) for t in (s["x"][part], of(s["w"]), of(s["bias"]))]
        r = None if s["residual"] is None else s["residual"][part].double()
        y = forward(*leaves, r)
        out["y"][part] = y.detach()
        if step:
            grads = torch.autograd.grad(y, [t for t in leaves if t is not None], s["dy"][part].double())
            out["dx"][part] = grads[0]
            for k, v in zip(("dw", "dbias"), grads[1:]):
                of(out[k]).copy_(v)
    return out
