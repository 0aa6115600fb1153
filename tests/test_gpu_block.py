"""GPU: the operators around the layer against float64, at the sizes, strides and
values where they can go wrong."""
import pytest
import torch

import block_reference as ref
import mixture_experts_ffn_gemv_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def strided(t, extra):
    """The same rows on the device, `extra` values (NaN) after each, and a NaN row before and after."""
    m, n = t.shape
    wide = torch.full((m + 2, n + extra), float("nan"), dtype=t.dtype, device=DEV)
    wide[1:m + 1, :n] = t.to(DEV)
    return wide[1:m + 1, :n]


def untouched(view):
    """The values around a strided result are still NaN."""
    base = view._base if view._base is not None else view
    inner = base.clone()
    inner[1:-1, :view.shape[1]] = float("nan")
    return bool(torch.isnan(inner).all())


def empty(m, n, dtype, extra=0):
    return strided(torch.full((m, n), float("nan"), dtype=dtype), extra)


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # what a call reads before writing it is NaN


# ------------------------------------------------------------------ gated feed-forward block

def ffn_case(m, dim, inter, dtype, act, limit, seed):
    g = ref.generator(seed)
    x, dy = ref.normal(g, (m, dim), dtype), ref.normal(g, (m, dim), dtype)
    wg, wu = (ref.normal(g, (inter, dim), dtype, 1.2 / dim ** 0.5) for _ in range(2))
    return x, dy, wg, wu, ref.normal(g, (dim, inter), dtype, 1 / inter ** 0.5), act, limit


def ffn_run(c, extra=0, backward=True, stream=None, want=("dx", "dw_gate", "dw_up", "dw_down")):
    x, dy, wg, wu, wd, act, limit = c
    (m, dim), inter, dt = x.shape, wg.shape[0], x.dtype
    f = moe.make_ffn(wg.to(DEV), wu.to(DEV), wd.to(DEV), act=act, limit=limit)
    nf, ns, nb = moe.moe_ffn_workspace(f, m)
    dx_, ddy, y = strided(x, extra), strided(dy, extra), empty(m, dim, dt, extra)
    saved, work_f, work_b = workspace(ns) if backward else None, workspace(nf), workspace(nb)
    out = {"y": y}
    if backward:
        shapes = {"dw_gate": (inter, dim), "dw_up": (inter, dim), "dw_down": (dim, inter)}
        grads = {k: empty(m, dim, dt, extra) if k == "dx" else torch.full(shapes[k], float("nan"), dtype=dt, device=DEV)
                 for k in want}
    torch.cuda.synchronize()
    moe.moe_ffn_forward(f, dx_, y, work_f, saved=saved, stream=stream)
    if backward:
        moe.moe_ffn_backward(f, dx_, ddy, saved, work_b, stream=stream, **grads)
        out.update(grads)
    torch.cuda.synchronize()
    return out


FFN = [(1, 256, 256, BF16, "silu", 0.0), (2, 8, 8, F16, "gelu", 0.0), (3, 264, 136, BF16, "silu", 1.0),
       (15, 64, 1040, F16, "silu", 0.0), (16, 520, 72, BF16, "gelu", 2.0), (17, 512, 512, F16, "gelu", 0.0),
       (33, 136, 264, BF16, "silu", 10.0), (64, 256, 768, F16, "silu", 1.5), (65, 768, 256, BF16, "gelu", 0.0),
       (127, 72, 200, BF16, "silu", 0.0), (130, 1024, 520, F16, "gelu", 0.0), (257, 392, 648, BF16, "silu", 0.0),
       (300, 264, 264, F16, "silu", 10.0)]


@pytest.mark.parametrize("m,dim,inter,dtype,act,limit", FFN)
def test_ffn_against_float64(m, dim, inter, dtype, act, limit):
    c = ffn_case(m, dim, inter, dtype, act, limit, seed=m)
    want = ref.ffn(c[0], c[2], c[3], c[4], act, limit, dy=c[1])
    got = ffn_run(c, extra=0 if m % 2 else 24)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, f"{k} of m={m}")
    for k in ("y", "dx"):
        assert untouched(got[k]), k


@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("gelu", 2.0)])
@pytest.mark.parametrize("m,dim,inter,dtype", [(1, 256, 264, BF16), (2, 72, 1544, F16), (5, 1032, 2312, BF16), (16, 264, 520, F16),
                                               (16, 264, 1024, BF16), (1, 72, 16384, BF16), (3, 264, 4104, F16), (6, 136, 2560, BF16)])
def test_ffn_of_few_rows_rounds_once(m, dim, inter, dtype, act, limit):
    # h in two parts of 16 bits, where it fits into LDS twice, is off by u^2 of itself (in f16 by half its smallest
    # step at least): what is left of y's error is its own rounding and f32's sums
    c = ffn_case(m, dim, inter, dtype, act, limit, seed=inter)
    x, _, wg, wu, wd = (t.double() for t in c[:5])
    g, u = x @ wg.t(), x @ wu.t()
    a, da, uc = ref.gated(g, u, act, limit)
    eg, eu = ref.ACC * (x.abs() @ wg.abs().t()), ref.ACC * (x.abs() @ wu.abs().t())
    eh = (da * uc).abs() * eg + a.abs() * eu + (ref.ACC + ref.U[dtype] ** 2) * (a * uc).abs() + ref.TINY[dtype]
    y = (a * uc) @ wd.t()
    e = eh @ wd.abs().t() + ref.ACC * ((a * uc).abs() @ wd.abs().t())
    got = ffn_run(c, extra=8, backward=False)["y"]
    ref.check(got, y, e + ref.U[dtype] * (y.abs() + e) + ref.TINY[dtype], f"m={m} of {dim} x {inter}")
    assert untouched(got)


def test_ffn_of_infinite_weights_and_h():
    # the second part of h adds nothing to what is infinite
    for m, inter in ((2, 136), (14, 4104)):
        c = list(ffn_case(m, 40, inter, F16, "silu", 0.0, seed=m))
        c[2], c[3] = c[2].abs() + 0.01, c[3].abs() + 0.01
        c[0] = c[0].abs() + 0.01
        c[4] = c[4].clone()
        clean = ffn_run(c, backward=False)["y"]
        c[4][3, 5], c[4][7, inter - 1] = float("inf"), float("-inf")
        y = ffn_run(c, backward=False)["y"]
        assert (y[:, 3] == float("inf")).all() and (y[:, 7] == float("-inf")).all()
        rest = torch.tensor([i not in (3, 7) for i in range(40)], device=DEV)
        assert torch.equal(y[:, rest], clean[:, rest])
        c[0], c[4] = c[0].clone(), c[4].abs() + 0.01
        c[0][1] = 3e4   # h past f16's largest value
        y = ffn_run(c, backward=False)["y"]
        assert torch.isfinite(y[0, rest]).all() and (y[1] == float("inf")).all()


def test_ffn_large_tiles_against_float64():
    # enough output tiles for the largest tiles in every product, none of them whole
    m, dim, inter = 2100, 4360, 2312
    g = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g, device=DEV) * k).to(BF16)   # noqa: E731
    c = (rnd(m, dim), rnd(m, dim), rnd(inter, dim, k=0.02), rnd(inter, dim, k=0.02), rnd(dim, inter, k=0.02), "silu", 0.0)
    got = ffn_run(c)
    want = ref.ffn(c[0], c[2], c[3], c[4], "silu", 0.0, dy=c[1])   # float64 on the device
    for k, (v, e) in want.items():
        ref.check(got[k], v.cpu(), e.cpu(), k)


def test_ffn_same_bits_with_and_without_saving_and_again():
    c = ffn_case(70, 512, 384, BF16, "silu", 10.0, seed=3)
    a, b, n = ffn_run(c), ffn_run(c), ffn_run(c, backward=False)
    assert torch.equal(a["y"], n["y"])
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("m,dim,inter", [(17, 2056, 520), (24, 520, 2056), (33, 1544, 264), (40, 264, 1544), (41, 520, 776)])
def test_ffn_few_rows_by_weight_rows_against_float64(m, dim, inter):
    # the edges of what a workgroup has room for, k past the last whole slab
    test_ffn_few_rows_in_tiles_against_float64(m, dim, inter)


@pytest.mark.parametrize("m,dim,inter", [(50, 4136, 72), (35, 4072, 2064), (64, 4104, 2088)])
def test_ffn_few_rows_in_tiles_against_float64(m, dim, inter):
    # more workgroups than CUs if split by weight rows: the second product, the first, both in tiles
    c = ffn_case(m, dim, inter, BF16 if m % 2 else F16, "silu", 10.0, seed=m)
    want, got = ref.ffn(c[0], c[2], c[3], c[4], "silu", 10.0, dy=c[1]), ffn_run(c, extra=8)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, f"{k} of m={m}")
    assert untouched(got["y"])


@pytest.mark.parametrize("want", [("dx",), ("dw_gate",), ("dw_up", "dw_down"), ("dw_down",), ("dw_gate", "dw_down")])
def test_ffn_backward_of_some_outputs(want):
    c = ffn_case(40, 264, 392, F16, "gelu", 0.0, seed=9)
    a, b = ffn_run(c), ffn_run(c, want=want)
    for k in want:
        assert torch.equal(a[k], b[k]), k


def test_ffn_of_no_rows():
    c = ffn_case(0, 64, 128, BF16, "silu", 0.0, seed=1)
    out = ffn_run(c)
    assert out["y"].shape == (0, 64)
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert not out[k].any(), k


def test_ffn_on_another_stream_and_in_a_graph():
    c = ffn_case(20, 512, 768, BF16, "silu", 10.0, seed=4)
    want = ffn_run(c)
    side = torch.cuda.Stream()
    got = ffn_run(c, stream=side)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    x, dy, wg, wu, wd = (t.to(DEV) for t in c[:5])
    f = moe.make_ffn(wg, wu, wd, act="silu", limit=10.0)
    nf, ns, nb = moe.moe_ffn_workspace(f, 20)
    work, saved = workspace(max(nf, nb)), workspace(ns)
    y, dx, dwg, dwu, dwd = (torch.empty_like(t) for t in (x, x, wg, wu, wd))

    def step():
        moe.moe_ffn_forward(f, x, y, work, saved=saved)
        moe.moe_ffn_backward(f, x, dy, saved, work, dx=dx, dw_gate=dwg, dw_up=dwu, dw_down=dwd)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (y, dx, dwg, dwu, dwd):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k, t in (("y", y), ("dx", dx), ("dw_gate", dwg), ("dw_up", dwu), ("dw_down", dwd)):
            assert torch.equal(t, want[k]), k


def test_ffn_workspace_of_a_larger_batch():
    # one workspace, sized for the most rows, in calls of fewer; nothing past what moe_ffn_workspace says is written
    dim, inter, most = 520, 264, 1536
    c = ffn_case(most, dim, inter, BF16, "silu", 10.0, seed=1)
    w = [t.to(DEV) for t in c[2:5]]
    f = moe.make_ffn(*w, act="silu", limit=10.0)
    sizes = [moe.moe_ffn_workspace(f, most)[i] for i in range(3)]
    kept = [workspace(n + 256) for n in sizes]
    forward, saved, backward = (k[:n] for k, n in zip(kept, sizes))
    for m in (most, 1000, 300, 129, 128, 65, 40, 20, 3):
        x, dy = (t[:m].to(DEV) for t in c[:2])
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw = [torch.empty_like(t) for t in w]
        moe.moe_ffn_forward(f, x, y, forward, saved=saved)
        moe.moe_ffn_backward(f, x, dy, saved, backward, dx=dx, dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2])
        want = ffn_run((c[0][:m], c[1][:m], *c[2:]))
        for k, t in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y, dx, *dw)):
            assert torch.equal(t, want[k]), (m, k)
    assert all(bool((k[n:] == 0xFF).all()) for k, n in zip(kept, sizes))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_saturated_activations(act):
    # gate values from -1e4 to 1e4: the activation is 0 or its argument, and its derivative 0 or 1
    dim = inter = 64
    x = torch.eye(dim, dtype=F32).mul(100).to(BF16)
    wg = torch.diag(torch.linspace(-100, 100, dim)).to(BF16)
    c = (x, torch.ones(dim, dim).to(BF16), wg, torch.diag(torch.full((dim,), 0.01)).to(BF16),
         torch.eye(dim).to(BF16), act, 0.0)
    want, got = ref.ffn(c[0], c[2], c[3], c[4], act, 0.0, dy=c[1]), ffn_run(c)
    for k, (v, e) in want.items():
        ref.check(got[k], torch.nan_to_num(v), torch.nan_to_num(e), k)


def test_ffn_keeps_a_nan_in_its_row():
    c = list(ffn_case(35, 128, 192, BF16, "silu", 1.0, seed=2))
    clean = ffn_run(c, backward=False)["y"]
    c[0][17, 5] = float("nan")
    y = ffn_run(c, backward=False)["y"]
    assert torch.isnan(y[17]).all()
    rest = torch.arange(35, device=DEV) != 17
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("m", [5, 70])
@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("gelu", 0.0), ("gelu", 1.0)])
def test_ffn_backward_keeps_a_nan_of_one_gate(act, limit, m):
    # one row of Wg is NaN: g is NaN in that column alone, and so are dg and du
    c = list(ffn_case(m, 72, 136, F16, act, limit, seed=m))
    clean = ffn_run(c)
    c[2] = c[2].clone()
    c[2][37] = float("nan")
    got = ffn_run(c)
    rest = torch.arange(136, device=DEV) != 37
    for k in ("dw_gate", "dw_up"):
        assert torch.isnan(got[k][37]).all(), k
        assert torch.equal(got[k][rest], clean[k][rest]), k
    assert torch.isnan(got["dw_down"][:, 37]).all() and torch.isnan(got["dx"]).all()


@pytest.mark.parametrize("m,dim,inter", [(1, 264, 264), (3, 40, 1040), (6, 1544, 520), (16, 512, 264), (20, 520, 264), (70, 264, 136)])
def test_ffn_of_infinite_values(m, dim, inter):
    # an infinity of x under positive weights: g and u are clamped, as they are with a large x. Without clamps h is
    # infinite, and so is y under positive weights
    for at in (0, dim // 2, dim - 1):
        c = list(ffn_case(m, dim, inter, BF16, "silu", 10.0, seed=m))
        c[2], c[3], c[4] = (t.abs() + 0.01 for t in c[2:5])
        clean, row = ffn_run(c, backward=False)["y"], m // 2
        c[0] = c[0].clone()
        c[0][row, at] = 1e6
        large = ffn_run(c, backward=False)["y"]
        c[0][row, at] = float("inf")
        y = ffn_run(c, backward=False)["y"]
        assert torch.isfinite(y).all() and torch.equal(y, large), at
        c[6] = 0.0
        assert (ffn_run(c, backward=False)["y"][row] == float("inf")).all(), at
        rest = torch.arange(m, device=DEV) != row
        assert torch.equal(y[rest], clean[rest]), at


def test_ffn_gradient_against_differences():
    # (loss(x + e v) - loss(x - e v)) / 2e for loss = <dy, y>, along v = the gradient's own direction, at e = 1/16 and
    # 1/32 of |x|, joined so that the cubic term cancels: y's rounding (2^-11, independent) is far below the difference
    c = ffn_case(24, 128, 256, F16, "gelu", 0.0, seed=8)
    got = ffn_run(c)
    for at, name in ((0, "dx"), (2, "dw_gate"), (3, "dw_up"), (4, "dw_down")):
        grad = got[name].double().cpu()
        v = grad / grad.norm()

        def slope(step):
            loss = []
            for sign in (1, -1):
                moved = list(c)
                moved[at] = (c[at].double() + sign * step * v).to(F16)
                loss.append((ffn_run(moved, backward=False)["y"].double().cpu() * c[1].double()).sum().item())
            return (loss[0] - loss[1]) / (2 * step)

        step = c[at].double().norm().item() / 16
        joined = (4 * slope(step / 2) - slope(step)) / 3
        assert abs(joined / grad.norm().item() - 1) < 0.03, (name, joined, grad.norm().item())


# ------------------------------------------------------------------ norms around a block

def norm_case(m, dim, dtype, gate, seed, post=True, pre=True):
    g = ref.generator(seed)
    c = dict(r=ref.normal(g, (m, dim), dtype, 2.0), y=ref.normal(g, (m, dim), dtype), dr_out=ref.normal(g, (m, dim), dtype),
             dn=ref.normal(g, (m, dim), dtype) if pre else None)
    c["w_post"] = ref.normal(g, (dim,), dtype, 0.2, 1.0) if post else None
    c["w_pre"] = ref.normal(g, (dim,), dtype, 0.2, 1.0) if pre else None
    shape = {"none": None, "channel": (dim,), "token": (m, 1), "full": (m, dim)}[gate]
    c["gate"] = None if shape is None else ref.normal(g, shape, dtype, 0.3, 0.5)
    return c


def norm_run(c, scale, extra=0, eps=1e-6, backward=True, stream=None):
    dev = {k: None if v is None else strided(v, extra) if v.dim() == 2 and k != "gate" else v.to(DEV) for k, v in c.items()}
    (m, dim), dt = c["r"].shape, c["r"].dtype
    f = moe.make_norm(dim, dt, w_post=dev["w_post"], w_pre=dev["w_pre"], eps=eps, res_scale=scale)
    out = {"r_out": empty(m, dim, dt, extra)}
    if c["w_pre"] is not None:
        out["n"] = empty(m, dim, dt, extra)
    stats = torch.full((m, 2), float("nan"), dtype=F32, device=DEV)
    work = workspace(moe.moe_norm_workspace(f, m))
    if backward:
        grads = {"dr": empty(m, dim, dt, extra)}
        if c["y"] is not None:
            grads["dy"] = empty(m, dim, dt, extra)
        for k, v in (("dgate", c["gate"]), ("dw_post", c["w_post"]), ("dw_pre", c["w_pre"])):
            if v is not None:
                grads[k] = torch.full(v.shape, float("nan"), dtype=dt, device=DEV)
    torch.cuda.synchronize()
    moe.moe_norm_forward(f, dev["r"], dev["y"], out["r_out"], out.get("n"), gate=dev["gate"], stats=stats, stream=stream)
    if backward:
        moe.moe_norm_backward(f, dev["r"], dev["y"], stats, dev["dr_out"], dev["dn"], work, gate=dev["gate"], stream=stream,
                              **grads)
        out.update(grads)
    torch.cuda.synchronize()
    return out


NORM = [(1, 1, F32, "none"), (5, 1, F16, "channel"), (3, 7, BF16, "token"), (33, 8, F32, "full"), (70, 64, BF16, "channel"),
        (9, 100, F16, "full"), (31, 257, F32, "token"), (12, 512, BF16, "none"), (64, 520, F16, "channel"),
        (7, 1111, F32, "full"), (5, 2304, BF16, "token"), (600, 136, BF16, "channel"), (3, 5120, F16, "full"),
        (2, 8192, F32, "channel"), (3, 8193, BF16, "channel"), (2, 16384, F16, "token"), (1, 16384, F32, "full"),
        (2, 16383, F32, "none")]


@pytest.mark.parametrize("m,dim,dtype,gate", NORM)
def test_norm_against_float64(m, dim, dtype, gate):
    c = norm_case(m, dim, dtype, gate, seed=dim)
    scale = 0.7 if m % 2 else 1.0
    want = ref.norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], 1e-6, scale, c["dr_out"], c["dn"])
    for extra in (0, 8, 3):   # whole rows, rows on 16-byte boundaries, rows on none
        got = norm_run(c, scale, extra=extra)
        assert set(got) == set(want)
        for k, (v, e) in want.items():
            ref.check(got[k], v, e, f"{k} of [{m}, {dim}] + {extra}")
        for k in ("r_out", "n", "dr", "dy"):
            assert untouched(got[k]), k


@pytest.mark.parametrize("post,pre,gate", [(True, False, "channel"), (False, True, "full"), (False, False, "token"),
                                           (False, True, "none"), (True, False, "none")])
def test_norm_without_one_of_the_norms(post, pre, gate):
    c = norm_case(21, 328, BF16, gate, seed=6, post=post, pre=pre)
    want = ref.norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], 1e-5, 0.5, c["dr_out"], c["dn"])
    got = norm_run(c, 0.5, eps=1e-5)
    assert set(got) == set(want)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, k)


@pytest.mark.parametrize("keep", ["dr_out", "dn"])
def test_norm_with_one_incoming_gradient(keep):
    c = norm_case(10, 264, F32, "channel", seed=7)
    c["dn" if keep == "dr_out" else "dr_out"] = None
    want = ref.norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], 1e-6, 1.0, c["dr_out"], c["dn"])
    got = norm_run(c, 1.0)
    if keep == "dr_out":   # nothing reaches the norm before the next block
        assert not got.pop("dw_pre").any()
        want.pop("dw_pre")
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, k)


def test_norm_before_the_first_block():
    c = norm_case(9, 520, BF16, "none", seed=8, post=False)
    c["y"] = None
    want = ref.norm(c["r"], None, None, c["w_pre"], None, 1e-6, 1.0, c["dr_out"], c["dn"])
    want.pop("dy")
    got = norm_run(c, 1.0)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, k)
    r = c["r"].to(DEV)   # n alone
    f, n = moe.make_norm(520, BF16, w_pre=c["w_pre"].to(DEV)), torch.empty_like(r)
    moe.moe_norm_forward(f, r, None, None, n)
    assert torch.equal(n, got["n"].contiguous())


@pytest.mark.parametrize("dim", [264, 2048])
def test_norm_in_place(dim):
    c = norm_case(50, dim, BF16, "channel", seed=3)
    want = norm_run(c, 0.5)
    d = {k: v.to(DEV) for k, v in c.items()}
    f = moe.make_norm(dim, BF16, w_post=d["w_post"], w_pre=d["w_pre"], res_scale=0.5)
    r, y = d["r"].clone(), d["y"].clone()
    stats = torch.empty(50, 2, device=DEV)
    moe.moe_norm_forward(f, r, y, r, y, gate=d["gate"], stats=stats)
    assert torch.equal(r, want["r_out"]) and torch.equal(y, want["n"])
    work = workspace(moe.moe_norm_workspace(f, 50))
    moe.moe_norm_backward(f, d["r"], d["y"], stats, d["dr_out"], d["dn"], work, gate=d["gate"], dr=d["dr_out"], dy=d["dn"])
    assert torch.equal(d["dr_out"], want["dr"]) and torch.equal(d["dn"], want["dy"])


def test_norm_rows_of_zeros_and_of_the_largest_values():
    c = norm_case(6, 96, F32, "none", seed=5)
    c["r"][1], c["y"][1] = 0, 0
    c["r"][2], c["y"][2] = 0, 1e15
    c["r"][3], c["y"][3] = 1e15, 0
    c["r"][4], c["y"][4] = 1e-18, 1e-18
    want = ref.norm(c["r"], c["y"], c["w_post"], c["w_pre"], None, 1e-6, 1.0, c["dr_out"], c["dn"])
    got = norm_run(c, 1.0)
    for k, (v, e) in want.items():
        ref.check(got[k], v, e, k)
    assert not got["n"][1].any()


def test_norm_keeps_what_is_not_finite_in_its_row():
    c = norm_case(8, 200, BF16, "channel", seed=4)
    clean = norm_run(c, 1.0, backward=False)
    c["y"][2, 3], c["r"][5, 199] = float("nan"), float("inf")
    got = norm_run(c, 1.0, backward=False)
    rest = [0, 1, 3, 4, 6, 7]
    for k in ("r_out", "n"):
        assert torch.equal(got[k][rest], clean[k][rest]), k
        assert torch.isnan(got[k][2]).all(), k
    assert got["r_out"][5, 199] == float("inf") and torch.isnan(got["n"][5, 199])


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("m,dim,dtype", [(8, 7, BF16), (8, 200, BF16), (9, 1111, F32), (8, 5120, F16), (8, 8200, BF16)])
@pytest.mark.parametrize("without", ["w_pre", "dn"])
def test_norm_backward_with_nothing_after_the_residual_does_not_read_it(without, m, dim, dtype, gate):
    # e = dr_out there: no gradient depends on r, whatever r holds
    c = norm_case(m, dim, dtype, gate, seed=dim, pre=without == "dn")
    c["dn"] = None
    clean = norm_run(c, 0.5)
    c["r"][0, 3], c["r"][0, dim - 1], c["r"][5, 2], c["r"][7, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    got = norm_run(c, 0.5)
    for k in set(got) - {"r_out", "n"}:
        assert torch.isfinite(got[k]).all(), k
        assert torch.equal(got[k], clean[k]), k


def test_norm_of_no_rows():
    c = norm_case(0, 72, F16, "channel", seed=1)
    got = norm_run(c, 1.0)
    for k in ("dgate", "dw_post", "dw_pre"):
        assert not got[k].any(), k


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_norm_of_no_rows_with_weights_that_are_not_finite(value):
    c = norm_case(0, 72, F32, "channel", seed=1)
    c["gate"][3], c["w_post"][5] = value, value
    got = norm_run(c, 1.0)
    for k in ("dgate", "dw_post", "dw_pre"):
        assert torch.isfinite(got[k]).all() and not got[k].any(), k


def test_norm_same_bits_again_on_a_stream_and_in_a_graph():
    c = norm_case(700, 1024, BF16, "channel", seed=2)
    want = norm_run(c, 1.0)
    for stream in (None, torch.cuda.Stream()):
        got = norm_run(c, 1.0, stream=stream)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    d = {k: v.to(DEV) for k, v in c.items()}
    f = moe.make_norm(1024, BF16, w_post=d["w_post"], w_pre=d["w_pre"])
    out = {k: torch.empty_like(want[k]) for k in want}
    stats, work = torch.empty(700, 2, device=DEV), workspace(moe.moe_norm_workspace(f, 700))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_norm_forward(f, d["r"], d["y"], out["r_out"], out["n"], gate=d["gate"], stats=stats)
        moe.moe_norm_backward(f, d["r"], d["y"], stats, d["dr_out"], d["dn"], work, gate=d["gate"], dr=out["dr"], dy=out["dy"],
                              dgate=out["dgate"], dw_post=out["dw_post"], dw_pre=out["dw_pre"])
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), k


def test_norm_gradient_against_differences():
    # f32 rows: central differences of loss = <dr_out, r'> + <dn, n> with a step of 1/64 of each input's size leave
    # rounding below 1e-4 of the slope and the cubic term below 1e-3
    c = norm_case(6, 65, F32, "channel", seed=12)
    got = norm_run(c, 0.7)

    def loss(case):
        o = norm_run(case, 0.7, backward=False)
        return ((o["r_out"].double().cpu() * c["dr_out"].double()).sum() + (o["n"].double().cpu() * c["dn"].double()).sum()).item()

    for name, k in (("dr", "r"), ("dy", "y"), ("dgate", "gate"), ("dw_post", "w_post"), ("dw_pre", "w_pre")):
        grad = got[name].double().cpu()
        step, v = c[k].double().norm().item() / 64, grad / grad.norm()
        hi, lo = (loss({**c, k: (c[k].double() + s * step * v).float()}) for s in (1, -1))
        slope = (hi - lo) / (2 * step)
        assert abs(slope / grad.norm().item() - 1) < 2e-3, (name, slope, grad.norm().item())


# ------------------------------------------------------------------ 4-bit weights

def w4_case(rows, cols, group, zeros, dtype, seed):
    g = ref.generator(seed)
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand((rows, cols // group), generator=g, dtype=torch.float64) * 0.02 + 0.001).to(dtype)
    z = torch.randint(0, 16, (rows, cols // group), generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def w4_make(c, group):
    return moe.make_w4(c[0].to(DEV), c[1].to(DEV), None if c[2] is None else c[2].to(DEV), group=group)


W4 = [(1, 16, 32, 32, True, BF16), (1, 1, 128, 128, False, F16), (2, 33, 96, 32, True, F16), (4, 100, 640, 64, True, BF16),
      (5, 48, 1024, 128, False, BF16), (8, 17, 160, 32, False, F16), (9, 64, 2304, 128, True, F16),
      (16, 31, 320, 64, True, BF16), (17, 80, 4096, 32, True, BF16), (32, 47, 192, 64, False, F16),
      (33, 16, 1280, 128, True, BF16), (64, 65, 256, 32, True, F16), (65, 40, 512, 64, True, BF16),
      (150, 24, 1152, 128, False, BF16), (1, 50, 65536, 64, True, BF16),
      (24, 33, 640, 32, True, F16), (20, 48, 896, 128, False, BF16)]


@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", W4)
def test_w4_matmul_against_float64(m, rows, cols, group, zeros, dtype):
    c = w4_case(rows, cols, group, zeros, dtype, seed=rows + cols)
    x = ref.normal(ref.generator(m), (m, cols), dtype)
    v, e = ref.w4_product(x, *c, group)
    for extra in (0, 8):
        y = empty(m, rows, dtype, extra + rows % 2)
        moe.moe_w4_matmul(w4_make(c, group), strided(x, extra), y)
        ref.check(y, v, e + ref.U[dtype] * (v.abs() + e) + ref.TINY[dtype], f"[{m}, {cols}] x [{rows}]")
        assert untouched(y)


W4_MANY = [(17, 8225, 160, 32, True, BF16), (24, 8196, 192, 64, True, BF16), (27, 8210, 96, 32, False, BF16), (70, 2740, 256, 64, False, F16), (32, 8200, 384, 128, True, F16)]


@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", W4_MANY)
def test_w4_matmul_of_many_workgroups_against_float64(m, rows, cols, group, zeros, dtype):
    test_w4_matmul_against_float64(m, rows, cols, group, zeros, dtype)


@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", [(m, rows // 2 + 1, *rest) for m, rows, *rest in W4_MANY])
def test_w4_gated_of_many_workgroups_against_float64(m, rows, cols, group, zeros, dtype):
    test_w4_gated_against_float64(m, rows, cols, group, zeros, dtype, "silu", 0.5)


@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("silu", 0.5), ("gelu", 0.0)])
@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", [W4[i] for i in (0, 3, 6, 8, 11, 12, 15, 16)])
def test_w4_gated_against_float64(m, rows, cols, group, zeros, dtype, act, limit):
    cg, cu = (w4_case(rows, cols, group, zeros, dtype, seed=s) for s in (rows, cols + 1))
    x = ref.normal(ref.generator(m), (m, cols), dtype)
    (g, eg), (u, eu) = ref.w4_product(x, *cg, group), ref.w4_product(x, *cu, group)
    a, da, uc = ref.gated(g, u, act, limit)
    v = a * uc
    e = (da * uc).abs() * eg + a.abs() * eu + 2 * eg * eu + ref.ACC * v.abs()
    h = empty(m, rows, dtype)
    moe.moe_w4_gated(w4_make(cg, group), w4_make(cu, group), x.to(DEV), h, act=act, limit=limit)
    ref.check(h, v, e + ref.U[dtype] * (v.abs() + e) + ref.TINY[dtype], f"gated [{m}, {cols}] x [{rows}]")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_w4_each_code_and_column(group, dtype):
    # unit rows of x pick single columns: the result is the weight itself, rounded once. Column k of row n has the
    # code (n + 3 k) % 16, its group the scale 2^-(group % 4) and the zero point (n + group) % 16
    cols, rows = 256, 16
    k, n = torch.arange(cols), torch.arange(rows)[:, None]
    q = ((n + 3 * k) % 16).to(torch.uint8)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    gi = torch.arange(cols // group)
    scales = (0.5 ** (gi % 4)).to(dtype).expand(rows, -1).contiguous()
    zeros = ((n + gi) % 16).to(torch.uint8)
    w = moe.make_w4(codes.to(DEV), scales.to(DEV), zeros.to(DEV), group=group)
    want = ref.w4_values(codes, scales, zeros, group).t()
    x = torch.eye(cols).to(dtype).to(DEV)
    for t0 in range(0, cols, 5):   # five rows at a time: another place of the tile for each column
        y = torch.empty(min(5, cols - t0), rows, dtype=dtype, device=DEV)
        moe.moe_w4_matmul(w, x[t0:t0 + 5], y)
        assert torch.equal(y.cpu().double(), want[t0:t0 + 5])


def test_w4_rows_keep_to_themselves():
    # a row that is not finite leaves the others' bits alone; the same bits again, on a stream, and in a graph
    c = w4_case(70, 384, 64, True, BF16, seed=1)
    w, x = w4_make(c, 64), ref.normal(ref.generator(3), (11, 384), BF16).to(DEV)
    y = torch.empty(11, 70, dtype=BF16, device=DEV)
    moe.moe_w4_matmul(w, x, y)
    bad, z = x.clone(), torch.empty_like(y)
    bad[4, 100], bad[7, 3] = float("nan"), float("inf")
    moe.moe_w4_matmul(w, bad, z)
    rest = torch.tensor([i not in (4, 7) for i in range(11)], device=DEV)
    assert torch.equal(y[rest], z[rest]) and torch.isnan(z[4]).all() and torch.isnan(z[7]).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_w4_matmul(w, x, z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w4_matmul(w, x, z)
    for _ in range(3):
        z.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_w4_scales_at_any_place():
    # scales and zero points that start in the middle of a word
    c = w4_case(20, 256, 32, True, F16, seed=2)
    x = ref.normal(ref.generator(1), (3, 256), F16).to(DEV)
    y, z = torch.empty(3, 20, dtype=F16, device=DEV), torch.empty(3, 20, dtype=F16, device=DEV)
    moe.moe_w4_matmul(w4_make(c, 32), x, y)
    s = torch.zeros(161, dtype=F16, device=DEV)[1:].view(20, 8).copy_(c[1])
    zp = torch.zeros(163, dtype=torch.uint8, device=DEV)[3:].view(20, 8).copy_(c[2])
    moe.moe_w4_matmul(moe.make_w4(c[0].to(DEV), s, zp, group=32), x, z)
    assert torch.equal(y, z)


# ------------------------------------------------------------------ rows of a larger tensor

def test_one_row_of_any_stride():
    # the last token of a sequence, [1, dim] out of [1, tokens, dim]: no second row lies anywhere
    dim, inter, tokens = 64, 128, 70001
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)   # noqa: E731
    last = rnd(1, tokens, dim)[:, -1]
    odd = rnd(1, 2, 264)[:, 1, :dim].as_strided((1, dim), (1, 1))
    assert last.stride(0) > 1 << 22 and odd.stride(0) < dim
    f = moe.make_ffn(rnd(inter, dim), rnd(inter, dim), rnd(dim, inter))
    nf, ns, nb = moe.moe_ffn_workspace(f, 1)
    n = moe.make_norm(dim, BF16, w_post=rnd(dim), w_pre=rnd(dim))
    c = w4_case(48, dim, 32, True, BF16, seed=1)
    w = w4_make(c, 32)

    def outputs(x):
        y, dx, r, v, q, h = (torch.full((1, k), float("nan"), dtype=BF16, device=DEV) for k in (dim, dim, dim, dim, 48, 48))
        saved = workspace(ns)
        moe.moe_ffn_forward(f, x, y, workspace(nf), saved=saved)
        moe.moe_ffn_backward(f, x, x, saved, workspace(nb), dx=dx)
        moe.moe_norm_forward(n, x, x, r, v)
        moe.moe_w4_matmul(w, x, q)
        moe.moe_w4_gated(w, w, x, h)
        return y, dx, r, v, q, h

    for x in (last, odd):
        for a, b in zip(outputs(x), outputs(x.clone().contiguous())):
            assert torch.isfinite(a).all() and torch.equal(a, b)
