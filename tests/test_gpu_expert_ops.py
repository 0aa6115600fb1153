"""GPU: tokens sorted by expert and back, products with bias, activation and residual (one matrix, or one per expert) and
dropout against float64, at the sizes, strides, masks and values where they can go wrong."""
import math

import pytest
import torch

import block_reference as base
import expert_reference as ref
import mixture_experts_ffn_gemv_amd as moe
import synthetic as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


def strided(t, extra):
    """The same rows on the device, `extra` values (NaN) after each, and a NaN row before and after."""
    m, n = t.shape
    wide = torch.full((m + 2, n + extra), NAN, dtype=t.dtype, device=DEV)
    wide[1:m + 1, :n] = t.to(DEV)
    return wide[1:m + 1, :n]


def untouched(view):
    inner = view._base.clone()
    inner[1:-1, :view.shape[1]] = NAN
    return bool(torch.isnan(inner).all())


def empty(m, n, dtype, extra=0):
    return strided(torch.full((m, n), NAN, dtype=dtype), extra)


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # what a call reads before writing it is NaN


def guarded(n, value=-77):
    """n int32 between two guard words -> (view, the guards are whole)"""
    wide = torch.full((n + 2,), value, dtype=torch.int32, device=DEV)
    return wide[1:-1], lambda: bool((wide[[0, -1]] == value).all())


def check(got, value, allowed, what):
    """Like block_reference's, but a NaN of the reference stands for a value that has to be NaN still."""
    got = got.detach().cpu().double()
    left = torch.isnan(value)
    assert torch.isnan(got[left]).all(), f"{what}: written where nothing belongs"
    base.check(got[~left], value[~left], allowed[~left], what)


# ------------------------------------------------------------------ sort

def picks(m, topk, n_experts, seed, bad=0.0):
    g = base.generator(seed)
    idx = (torch.rand(m, topk, generator=g) ** 2 * n_experts).int().clamp(max=n_experts - 1)   # popular ones first; repeats
    out = torch.tensor([-1, n_experts, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.randint(4, (m, topk), generator=g)]
    return torch.where(torch.rand(m, topk, generator=g) < bad, out, idx).contiguous()


def sort_run(idx, n_experts, stream=None, want_picks=True):
    m, topk = idx.shape
    idx_d = idx.to(DEV)
    (row_of, g0), (pick_of, g1), (offsets, g2) = guarded(m * topk), guarded(m * topk), guarded(n_experts + 1)
    work = workspace(moe.moe_sort_workspace(m, topk, n_experts))
    torch.cuda.synchronize()
    moe.moe_sort(idx_d, n_experts, row_of.view(m, topk), pick_of if want_picks else None, offsets, work, stream=stream)
    torch.cuda.synchronize()
    assert g0() and g1() and g2()
    return row_of.view(m, topk).cpu(), pick_of.cpu(), offsets.cpu()


@pytest.mark.parametrize("m,topk,n_experts,bad", [
    (0, 6, 384, 0), (1, 1, 1, 0), (1, 6, 384, 0), (2, 3, 5, 1.0), (7, 64, 1024, 0.1), (64, 1, 1, 0), (1000, 8, 3, 0.3), (1023, 1, 1024, 0),
    (1025, 8, 65, 0.05), (1365, 6, 384, 0), (1366, 6, 384, 0.02), (8191, 6, 384, 0.01), (9001, 7, 129, 1.0), (70001, 8, 64, 0.1),
    (4100, 64, 1000, 0)])
def test_sort_is_the_stable_order(m, topk, n_experts, bad):
    idx = picks(m, topk, n_experts, m, bad)
    for got, want in zip(sort_run(idx, n_experts), ref.sort(idx, n_experts)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("n", [24 * 1024, 24 * 1024 + 1, 48 * 1024 - 5, 48 * 1024, 48 * 1024 + 1, 60000])
def test_sort_of_as_many_picks_as_one_launch_takes_and_one_more(n):
    idx = picks(n, 1, 1024, n, bad=0.03)
    for got, want in zip(sort_run(idx, 1024), ref.sort(idx, 1024)):
        assert torch.equal(got, want)


def test_sort_without_picks_and_on_another_stream():
    idx = picks(3000, 6, 100, 5)
    want = ref.sort(idx, 100)
    got = sort_run(idx, 100, stream=torch.cuda.Stream(), want_picks=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and (got[1] == -77).all()


# ------------------------------------------------------------------ rows to experts and back

MOVES = [(1, 1, 1, BF16), (5, 3, 2, F16), (4, 7, 3, BF16), (9, 8, 6, F16), (33, 9, 8, BF16), (17, 64, 9, F32), (31, 3, 4, F32), (3, 5, 2, F32),
         (70, 130, 5, F16), (41, 1111, 6, BF16), (23, 1111, 6, F32), (40, 1032, 1, BF16), (37, 5120, 6, F16), (11, 2056, 64, BF16),
         (300, 257, 7, F32), (1, 5120, 6, BF16)]


def move_case(m, dim, topk, dtype, seed, bad=0.15):
    g = base.generator(seed)
    n_experts = 5
    idx = picks(m, topk, n_experts, seed, bad)
    if m > 2:
        idx[-1] = -1   # a padded token
    row_of, _, offsets = ref.sort(idx, n_experts)
    w = torch.rand(m, topk, generator=g) * 2 - 0.5
    w[row_of < 0] = NAN   # the weight of no row takes no part
    n = m * topk
    return dict(row_of=row_of, w=w, n=n, used=int(offsets[-1]), x=base.normal(g, (m, dim), dtype), e=base.normal(g, (n, dim), dtype),
                dy=base.normal(g, (m, dim), dtype))


@pytest.mark.parametrize("m,dim,topk,dtype", MOVES)
def test_rows_to_experts_and_back(m, dim, topk, dtype):
    c = move_case(m, dim, topk, dtype, seed=dim + topk)
    extra = 0 if m % 2 else 5
    row_of, w = c["row_of"].to(DEV), c["w"].to(DEV)
    c["e"][c["used"]:] = NAN   # rows that no pick has may hold anything
    e = strided(c["e"], extra)
    for rows in {c["n"], max(1, c["used"] - 2)}:   # all, and room for fewer than there are: the others take no part
        there = torch.where(c["row_of"] < rows, c["row_of"], -1)
        xs, y, de, dx = empty(rows, dim, dtype, extra), empty(m, dim, dtype, extra), empty(rows, dim, dtype, extra), empty(m, dim, dtype, extra)
        dw = torch.full((m, topk), NAN, device=DEV)
        moe.moe_dispatch_forward(strided(c["x"], extra), row_of, xs)
        moe.moe_combine_forward(e[:rows], w, row_of, y)
        moe.moe_combine_backward(strided(c["dy"], extra), e[:rows], w, row_of, de, dw)
        moe.moe_dispatch_backward(e[:rows], row_of, dx)
        torch.cuda.synchronize()
        want = torch.full((rows, dim), NAN, dtype=dtype)
        for t, j in (there >= 0).nonzero().tolist():
            want[there[t, j]] = c["x"][t]
        assert torch.equal(torch.nan_to_num(xs.cpu(), nan=-99.0), torch.nan_to_num(want, nan=-99.0))
        check(y, *ref.combine(c["e"][:rows], c["w"], there, dtype), "y")
        check(dx, *ref.combine(c["e"][:rows], None, there, dtype), "dx")
        back = ref.combine_backward(c["dy"], c["e"][:rows], c["w"], there, rows)
        check(de, *back["de"], "de")
        check(dw, *back["dweights"], "dweights")
        for t in (xs, y, de, dx):
            assert untouched(t)
        only = torch.full((m, topk), NAN, device=DEV)
        de2 = torch.full_like(de.contiguous(), NAN)
        moe.moe_combine_backward(c["dy"].to(DEV), e[:rows], w, row_of, None, only)
        moe.moe_combine_backward(c["dy"].to(DEV), e[:rows], w, row_of, de2, None)
        assert torch.equal(only, dw) and torch.equal(torch.nan_to_num(de2, nan=-99.0), torch.nan_to_num(de.contiguous(), nan=-99.0))


def test_tokens_without_rows_give_zeros():
    row_of = torch.full((5, 3), -1, dtype=torch.int32, device=DEV)
    w, nothing = torch.full((5, 3), NAN, device=DEV), torch.empty(0, 40, dtype=BF16, device=DEV)
    dy = torch.full((5, 40), NAN, dtype=BF16, device=DEV)
    for e in (nothing, torch.full((15, 40), NAN, dtype=BF16, device=DEV)):
        y, dx, dw = torch.full_like(dy, 7), torch.full_like(dy, 7), torch.full((5, 3), 7.0, device=DEV)
        xs = torch.full_like(e, 3)
        moe.moe_dispatch_forward(dy, row_of, xs)
        moe.moe_combine_forward(e, w, row_of, y)
        moe.moe_dispatch_backward(e, row_of, dx)
        moe.moe_combine_backward(dy, e, w, row_of, torch.empty_like(e), dw)
        assert not y.any() and not dx.any() and not dw.any() and (xs == 3).all()


def test_infinities_stay_with_their_tokens():
    c = move_case(40, 264, 4, BF16, seed=3, bad=0.0)
    bad = int(c["row_of"][7, 2])
    c["e"][bad, 5], c["e"][bad, 6] = INF, NAN
    y = torch.empty(40, 264, dtype=BF16, device=DEV)
    c["w"] = c["w"].nan_to_num(1.0).abs() + 0.1
    moe.moe_combine_forward(c["e"].to(DEV), c["w"].to(DEV), c["row_of"].to(DEV), y)
    odd = ~torch.isfinite(y.cpu())
    assert odd[7, 5] and odd[7, 6] and odd.sum() == 2


def test_long_rows_and_many():
    # past what the grid holds at once, and outputs larger than the L2s
    m, dim, topk = 4001, 2568, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, dim, generator=g, device=DEV).to(BF16)
    idx = torch.randint(0, 40, (m, topk), generator=g, device=DEV, dtype=torch.int32)
    row_of, pick_of, offsets = torch.empty_like(idx), torch.empty(m * topk, dtype=torch.int32, device=DEV), torch.empty(41, dtype=torch.int32, device=DEV)
    moe.moe_sort(idx, 40, row_of, pick_of, offsets, workspace(moe.moe_sort_workspace(m, topk, 40)))
    xs = torch.empty(m * topk, dim, dtype=BF16, device=DEV)
    moe.moe_dispatch_forward(x, row_of, xs)
    assert torch.equal(xs, x[pick_of.long() // topk])
    w = torch.rand(m, topk, generator=g, device=DEV)
    y = torch.empty_like(x)
    moe.moe_combine_forward(xs, w, row_of, y)
    at = xs.double()[row_of.long()] * w.double()[:, :, None]
    base.check(y, *[t.cpu() for t in ref.stored(at.sum(1), 4 * ref.F32 * at.abs().sum(1), BF16)], "y")
    dy, de, dw = torch.randn(m, dim, generator=g, device=DEV).to(BF16), torch.empty_like(xs), torch.empty_like(w)
    moe.moe_combine_backward(dy, xs, w, row_of, de, dw)
    terms = xs.double()[row_of.long()] * dy.double()[:, None, :]
    base.check(dw, terms.sum(2).cpu(), ((dim + 2) * ref.F32 * terms.abs().sum(2)).cpu(), "dweights")
    v = (w.double().flatten()[pick_of.long()][:, None] * dy.double()[pick_of.long() // topk])
    base.check(de, *[t.cpu() for t in ref.stored(v, ref.F32 * v.abs(), BF16)], "de")


# ------------------------------------------------------------------ products with bias, activation and residual

def linear_case(m, k, n, dtype, seed, n_experts=0):
    g = base.generator(seed)
    shape = (n_experts, n, k) if n_experts else (n, k)
    return dict(x=base.normal(g, (m, k), dtype), dy=base.normal(g, (m, n), dtype), w=base.normal(g, shape, dtype, 1.2 / k ** 0.5),
                bias=base.normal(g, shape[:-1], dtype, 0.5), residual=base.normal(g, (m, n), dtype))


def linear_run(c, act, bias=True, residual=True, offsets=None, extra=0, step=True, stream=None, want=("dx", "dw", "dbias")):
    (m, k), n, dt = c["x"].shape, c["w"].shape[-2], c["x"].dtype
    f = moe.make_linear(c["w"].to(DEV), c["bias"].to(DEV) if bias else None, act=act)
    nf, ns, nb = moe.moe_linear_workspace(f, m)
    wide = (extra + 7) // 8 * 8
    x, dy, y, r = strided(c["x"], wide), strided(c["dy"], extra), empty(m, n, dt, extra), strided(c["residual"], extra) if residual else None
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    saved, work_f, work_b = workspace(ns) if step else None, workspace(nf), workspace(nb)
    grads = {"dx": empty(m, k, dt, wide), "dw": torch.full_like(f.tensors[0], NAN), "dbias": torch.full_like(f.tensors[1], NAN) if bias else None}
    grads = {name: t if name in want else None for name, t in grads.items()}
    torch.cuda.synchronize()
    moe.moe_linear_forward(f, x, y, work_f, offsets=off, residual=r, saved=saved, stream=stream)
    if step:
        moe.moe_linear_backward(f, x, dy, saved, work_b, offsets=off, stream=stream, **grads)
    torch.cuda.synchronize()
    return {"y": y, **({name: t for name, t in grads.items() if t is not None} if step else {})}


LINEAR = [(1, 8, 1, BF16, "none"), (1, 256, 264, F16, "silu"), (2, 64, 37, BF16, "gelu"), (3, 4104, 40, F16, "none"), (15, 72, 130, BF16, "silu"),
          (16, 2312, 19, F16, "gelu"), (16, 520, 4099, BF16, "none"), (17, 264, 72, F16, "silu"), (23, 1032, 257, BF16, "gelu"),
          (33, 136, 264, F16, "none"), (64, 256, 771, BF16, "silu"), (65, 776, 256, F16, "gelu"), (127, 72, 201, BF16, "none"),
          (130, 1024, 520, BF16, "silu"), (257, 392, 646, F16, "gelu"), (300, 264, 264, BF16, "none"), (40, 4104, 72, BF16, "silu"), (3, 72, 33001, F16, "gelu"), (12, 520, 40000, BF16, "none")]


@pytest.mark.parametrize("m,k,n,dtype,act", LINEAR)
def test_linear_against_float64(m, k, n, dtype, act):
    c = linear_case(m, k, n, dtype, seed=m + n)
    bias, residual, extra = m % 3 != 0, m % 4 != 1, 0 if m % 2 else 24 + n % 2
    got = linear_run(c, act, bias, residual, extra=extra)
    want = ref.linear(c["x"], c["w"], c["bias"] if bias else None, c["residual"] if residual else None, act, dy=c["dy"])
    for name, t in got.items():
        base.check(t, *want[name], f"{name} of m={m}")
    for name in ("y", "dx"):
        assert untouched(got[name]), name


FEW = [(1, 952, 364, BF16, "silu"), (5, 1544, 4101, F16, "gelu"), (8, 520, 70, BF16, "none"), (7, 8, 3, F16, "silu"), (6, 5128, 1030, BF16, "gelu"),
       (2, 8, 33001, F16, "silu"), (8, 512, 64, BF16, "gelu"), (4, 1032, 16, F16, "none"), (3, 520, 17, BF16, "silu"), (9, 520, 70, BF16, "silu")]


@pytest.mark.parametrize("m,k,n,dtype,act", FEW)
def test_gradients_of_few_rows_against_float64(m, k, n, dtype, act):
    c = linear_case(m, k, n, dtype, seed=k + n)
    want = ref.linear(c["x"], c["w"], c["bias"], c["residual"], act, dy=c["dy"])
    got = linear_run(c, act, extra=5 * (m % 2))
    for name, t in got.items():
        check(t, *want[name], name)
    assert untouched(got["dx"])
    for only in ("dx", "dw", "dbias"):   # each by itself: the same bits
        alone = linear_run(c, act, extra=5 * (m % 2), want=(only,))
        assert torch.equal(alone[only], got[only]), only


def test_few_rows_round_their_gradients_once():
    # dW of one row is dz x: off by half a step of bf16 (2^-8), and by what z and the slope are off in f32. 64 terms of z are off by
    # 64 2^-24 sum |x w| < 2e-4, and the slope, whose derivative is at most 1/2, by half of that: less than 2^-12
    c = linear_case(1, 64, 4096, BF16, seed=11)
    got = linear_run(c, "silu", residual=False)["dw"].cpu().double()
    x, w, dy = (c[name].double() for name in ("x", "w", "dy"))
    assert (x.abs() @ w.abs().T).max() < 50
    z = x @ w.T + c["bias"].double()
    s = torch.sigmoid(z)
    slope = s * (1 + z * (1 - s))
    value, most = (dy * slope).T * x, dy.T.abs() * x.abs() * 2.0 ** -12
    assert ((got - value).abs() <= value.abs() * 2.0 ** -8 + most * 1.01).all()


def test_linear_large_tiles_against_float64():
    # enough output tiles for the largest tiles in every product, none of them whole
    m, k, n = 2100, 4360, 2309
    g = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=DEV) * scale).to(BF16)   # noqa: E731
    c = dict(x=rnd(m, k), dy=rnd(m, n), w=rnd(n, k, scale=0.02), bias=rnd(n), residual=rnd(m, n))
    got = linear_run(c, "silu")
    want = ref.linear(c["x"], c["w"], c["bias"], c["residual"], "silu", dy=c["dy"])   # float64 on the device
    for name, (v, e) in want.items():
        base.check(got[name], v.cpu(), e.cpu(), name)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dw", "dbias"), ()])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_backward_of_some_outputs(want, act):
    c = linear_case(70, 264, 392, F16, seed=9)
    a, b = linear_run(c, act), linear_run(c, act, want=want)
    for name in want:
        assert torch.equal(a[name], b[name]), name


def test_linear_same_bits_with_and_without_saving_and_again():
    c = linear_case(70, 512, 384, BF16, seed=3)
    a, b, n = linear_run(c, "silu"), linear_run(c, "silu"), linear_run(c, "silu", step=False)
    assert torch.equal(a["y"], n["y"])
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_linear_onto_its_residual():
    for m in (5, 150):
        c = linear_case(m, 264, 390, BF16, seed=m)
        want = linear_run(c, "gelu", step=False)["y"]
        f = moe.make_linear(c["w"].to(DEV), c["bias"].to(DEV), act="gelu")
        r = c["residual"].to(DEV)
        moe.moe_linear_forward(f, c["x"].to(DEV), r, workspace(moe.moe_linear_workspace(f, m)[0]), residual=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("n_experts", [0, 4])
def test_linear_of_no_rows(n_experts):
    c = linear_case(0, 64, 130, BF16, seed=1, n_experts=n_experts)
    out = linear_run(c, "silu", offsets=[0] * (n_experts + 1) if n_experts else None)
    assert out["y"].shape == (0, 130) and not out["dw"].any() and not out["dbias"].any()


@pytest.mark.parametrize("m", [3, 200])
def test_linear_infinities_stay_in_their_rows_and_columns(m):
    c = linear_case(m, 136, 90, BF16, seed=8)
    clean = linear_run(c, "silu", step=False)
    c["x"][1, 3] = INF
    c["w"][5, 7] = NAN
    got = linear_run(c, "silu", step=False)
    rows, cols = torch.arange(m, device=DEV) != 1, torch.arange(90, device=DEV) != 5
    assert torch.equal(got["y"][rows][:, cols], clean["y"][rows][:, cols])
    assert torch.isnan(got["y"][:, 5]).all() and not torch.isfinite(got["y"][1]).any()


# ------------------------------------------------------------------ a matrix per expert

EXPERTS = [  # rows of each expert (and rows behind the last), K, N
    ([1, 0, 0, 1, 1], 0, 264, 130, BF16, "silu"),            # a token's picks
    ([0, 0, 3], 2, 72, 19, F16, "none"),                     # the first ones without rows
    ([0, 0], 5, 64, 40, BF16, "gelu"),                       # no rows at all
    ([17, 0, 1, 40, 0], 0, 520, 72, F16, "gelu"),            # more of one expert than a workgroup's rows
    ([16, 15, 33, 1], 9, 2056, 137, BF16, "silu"),
    ([60] * 3 + [0] + [31], 3, 136, 264, F16, "silu"),
    ([130, 0, 127, 1, 300], 11, 264, 200, BF16, "gelu"),
    ([700, 1, 0, 300], 0, 72, 264, BF16, "none"),
    ([5] * 70 + [0] * 30 + [70], 0, 40, 24, F16, "silu"),    # more experts than a wavefront's lanes
    ([1, 0, 2] * 30, 4, 72, 1401, BF16, "gelu"),             # a wavefront's own weight rows, past the last of them
    ([3] + [1] * 60, 0, 520, 712, F16, "none"),
]


@pytest.mark.parametrize("counts,behind,k,n,dtype,act", EXPERTS)
def test_experts_against_float64(counts, behind, k, n, dtype, act):
    offsets = [0]
    for v in counts:
        offsets.append(offsets[-1] + v)
    m = offsets[-1] + behind
    c = linear_case(m, k, n, dtype, seed=m + k, n_experts=len(counts))
    for name in ("x", "dy", "residual"):
        c[name][offsets[-1]:] = NAN   # rows behind the last are not read
    bias, residual = m % 3 != 0, m % 2 == 0
    got = linear_run(c, act, bias, residual, offsets=offsets, extra=8 * (m % 2))
    want = ref.experts(c["x"], c["w"], c["bias"] if bias else None, c["residual"] if residual else None, act, offsets, dy=c["dy"])
    for name, t in got.items():
        check(t, *want[name], name)
    for name in ("y", "dx"):
        assert untouched(got[name]), name


def test_experts_large_tiles_against_float64():
    counts, k, n = [1900, 0, 2500, 300, 257], 1040, 1032
    offsets = [0]
    for v in counts:
        offsets.append(offsets[-1] + v)
    m = offsets[-1] + 5
    g = torch.Generator(device=DEV).manual_seed(6)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=DEV) * scale).to(F16)   # noqa: E731
    c = dict(x=rnd(m, k), dy=rnd(m, n), w=rnd(5, n, k, scale=0.03), bias=rnd(5, n), residual=rnd(m, n))
    got = linear_run(c, "gelu", offsets=offsets)
    for e in range(5):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            assert not got["dw"][e].any() and not got["dbias"][e].any()
            continue
        want = ref.linear(c["x"][a:b], c["w"][e], c["bias"][e], c["residual"][a:b], "gelu", dy=c["dy"][a:b])
        for name, (v, allowed) in want.items():
            base.check(got[name][a:b] if name in ("y", "dx") else got[name][e], v.cpu(), allowed.cpu(), name)
    assert torch.isnan(got["y"][offsets[-1]:]).all() and torch.isnan(got["dx"][offsets[-1]:]).all()


def test_one_matrix_with_offsets_is_the_product_of_its_rows():
    for m, act in ((7, "silu"), (400, "none"), (400, "gelu")):
        c = linear_case(m, 264, 136, BF16, seed=m)
        c["w"], c["bias"] = c["w"][None], c["bias"][None]
        got = linear_run(c, act, offsets=[0, m - 3])
        one = {k: v[0] if k in ("w", "bias") else v[:m - 3] for k, v in c.items()}
        want = ref.linear(one["x"], one["w"], one["bias"], one["residual"], act, dy=one["dy"])
        for name, t in got.items():
            base.check(t[:m - 3] if name in ("y", "dx") else t[0], *want[name], name)
        assert torch.isnan(got["y"][m - 3:]).all() and torch.isnan(got["dx"][m - 3:]).all()


# ------------------------------------------------------------------ dropout

DROPS = [(1, 1, BF16, 0.5), (3, 7, F16, 0.1), (2, 8, BF16, 0.1), (5, 9, F32, 0.3), (4, 3, F32, 0.5), (7, 12, F32, 0.2), (33, 64, F16, 0.9),
         (41, 1111, BF16, 0.1), (29, 1111, F32, 0.2), (70, 5120, F16, 0.1), (9, 260, BF16, 0.0), (9, 260, F32, 1.0), (600, 4104, BF16, 0.5),
         (3, 20, F16, 1e-6), (5, 13, F32, 0.99999)]


@pytest.mark.parametrize("m,dim,dtype,p", DROPS)
def test_dropout_against_the_generator(m, dim, dtype, p):
    g = base.generator(dim)
    seed, use = (0x1234567890ABCDEF, -5) if m % 2 else (-(2 ** 63), 2 ** 40 + 3)
    x, r, dy = (base.normal(g, (m, dim), dtype) for _ in range(3))
    extra = 0 if m % 2 else 3
    mask = ref.keep(seed, use, m, dim, p)
    v = x.clone()
    v[~mask] = torch.tensor([NAN, INF], dtype=dtype).repeat(v[~mask].numel())[:v[~mask].numel()]   # what is dropped may hold anything
    f, rng = moe.make_dropout(dim, dtype, p), torch.tensor([seed, use], device=DEV)
    y, plain, dx = (empty(m, dim, dtype, extra) for _ in range(3))
    moe.moe_dropout_forward(f, rng, strided(v, extra), y, residual=strided(r, extra + 1))
    moe.moe_dropout_forward(f, rng, strided(v, extra), plain)
    moe.moe_dropout_backward(f, rng, strided(dy, extra), dx)
    torch.cuda.synchronize()
    base.check(y, *ref.dropout(x, r, mask, p), "y")
    base.check(plain, *ref.dropout(x, None, mask, p), "y without a residual")
    base.check(dx, *ref.dropout(dy, None, mask, p), "dx")
    assert all(untouched(t) for t in (y, plain, dx))
    on_r, on_x = r.to(DEV), v.to(DEV)
    moe.moe_dropout_forward(f, rng, v.to(DEV), on_r, residual=on_r)
    moe.moe_dropout_forward(f, rng, on_x, on_x, residual=r.to(DEV))
    assert torch.equal(on_r, y) and torch.equal(on_x, y)


def test_dropout_share_and_uses():
    m, dim, p = 400, 1000, 0.3
    f, x = moe.make_dropout(dim, F32, p), torch.ones(m, dim, device=DEV)
    kept = []
    for use in range(3):
        y = torch.empty_like(x)
        moe.moe_dropout_forward(f, torch.tensor([7, use], device=DEV), x, y)
        kept.append((y != 0).double())
    n = m * dim
    for i, a in enumerate(kept):   # 5 sigma of a binomial share, and of two independent ones
        assert abs(a.mean().item() - 0.7) < 5 * math.sqrt(0.21 / n)
        for b in kept[:i]:
            assert abs((a * b).mean().item() - 0.49) < 5 * math.sqrt(0.49 * 0.51 / n)


# ------------------------------------------------------------------ together

def chain_tensors(m, topk, n_experts, dim, inter, dtype, seed):
    """A block's forward and backward pass: sorted, two products per expert, combined, dropped, added."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s, scale=1.0, dt=dtype: (torch.randn(*s, generator=g, device=DEV) * scale).to(dt)   # noqa: E731
    t = dict(x=rnd(m, dim), r=rnd(m, dim), dout=rnd(m, dim), w1=rnd(n_experts, inter, dim, scale=dim ** -0.5), b1=rnd(n_experts, inter, scale=0.3),
             w2=rnd(n_experts, dim, inter, scale=inter ** -0.5), b2=rnd(n_experts, dim, scale=0.3),
             weights=torch.rand(m, topk, generator=g, device=DEV) + 0.2,
             idx=torch.randint(0, n_experts, (m, topk), generator=g, device=DEV, dtype=torch.int32))
    t["idx"][-2:] = -1   # padding
    n = m * topk
    new = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device=DEV)   # noqa: E731
    t |= dict(row_of=new(m, topk, dt=torch.int32), pick_of=new(n, dt=torch.int32), offsets=new(n_experts + 1, dt=torch.int32), xs=new(n, dim),
              h=new(n, inter), e=new(n, dim), y=new(m, dim), out=new(m, dim), dy=new(m, dim), de=new(n, dim), dh=new(n, inter), dxs=new(n, dim),
              dx=new(m, dim), dweights=new(m, topk, dt=F32), rng=torch.tensor([99, 0], device=DEV))
    t |= {"d" + k: torch.empty_like(t[k]) for k in ("w1", "b1", "w2", "b2")}
    t["up"], t["down"] = moe.make_linear(t["w1"], t["b1"], act="gelu"), moe.make_linear(t["w2"], t["b2"])
    t["drop"] = moe.make_dropout(dim, dtype, 0.25)
    s1, s2 = moe.moe_linear_workspace(t["up"], n), moe.moe_linear_workspace(t["down"], n)
    t["work"] = workspace(max(s1[0], s1[2], s2[0], s2[2], moe.moe_sort_workspace(m, topk, n_experts)))
    t["s1"], t["s2"] = workspace(s1[1]), workspace(s2[1])
    return t


OUTPUTS = ("out", "dx", "dweights", "dw1", "db1", "dw2", "db2")


def chain_step(t, stream=None):
    n_experts = t["w1"].shape[0]
    kw = dict(stream=stream)
    moe.moe_sort(t["idx"], n_experts, t["row_of"], t["pick_of"], t["offsets"], t["work"], **kw)
    moe.moe_dispatch_forward(t["x"], t["row_of"], t["xs"], **kw)
    moe.moe_linear_forward(t["up"], t["xs"], t["h"], t["work"], offsets=t["offsets"], saved=t["s1"], **kw)
    moe.moe_linear_forward(t["down"], t["h"], t["e"], t["work"], offsets=t["offsets"], saved=t["s2"], **kw)
    moe.moe_combine_forward(t["e"], t["weights"], t["row_of"], t["y"], **kw)
    moe.moe_dropout_forward(t["drop"], t["rng"], t["y"], t["out"], residual=t["r"], **kw)
    moe.moe_dropout_backward(t["drop"], t["rng"], t["dout"], t["dy"], **kw)
    moe.moe_combine_backward(t["dy"], t["e"], t["weights"], t["row_of"], t["de"], t["dweights"], **kw)
    moe.moe_linear_backward(t["down"], t["h"], t["de"], t["s2"], t["work"], offsets=t["offsets"], dx=t["dh"], dw=t["dw2"], dbias=t["db2"], **kw)
    moe.moe_linear_backward(t["up"], t["xs"], t["dh"], t["s1"], t["work"], offsets=t["offsets"], dx=t["dxs"], dw=t["dw1"], dbias=t["db1"], **kw)
    moe.moe_dispatch_backward(t["dxs"], t["row_of"], t["dx"], **kw)


def chain_loss(t, values, mask):
    """The block in float64 from its definition, as a function of the tensors it learns: sum(out * dout)."""
    x, weights, w1, b1, w2, b2 = values
    out = t["r"].double()
    for j in range(t["idx"].shape[1]):
        for e in range(t["w1"].shape[0]):
            on = (t["idx"][:, j] == e).nonzero().flatten()
            h = torch.nn.functional.gelu(x[on] @ w1[e].t() + b1[e], approximate="tanh")
            y = weights[on, j, None] * (h @ w2[e].t() + b2[e])
            out = out.index_add(0, on, y * mask[on].double() / 0.75)
    return out, (out * t["dout"].double()).sum()


@pytest.mark.parametrize("m,dtype", [(5, BF16), (90, F16), (600, BF16)])
def test_a_block_of_them_and_its_gradients(m, dtype):
    t = chain_tensors(m, 2, 6, 136, 264, dtype, seed=m)
    chain_step(t)
    mask = ref.keep(99, 0, m, 136, 0.25).to(DEV)
    values = [t[k].double().requires_grad_() for k in ("x", "weights", "w1", "b1", "w2", "b2")]
    out, loss = chain_loss(t, values, mask)
    want = dict(zip(("out", "dx", "dweights", "dw1", "db1", "dw2", "db2"), [out.detach(), *torch.autograd.grad(loss, values)]))
    # at most five roundings of independent values lie one after another between inputs and results, each off by u / sqrt(3)
    # of its value on average at most: sqrt(5 / 3) u of the norm, and twice that is allowed
    for k in OUTPUTS:
        off = ((t[k].double() - want[k]).norm() / want[k].norm()).item()
        assert off < 2 * math.sqrt(5 / 3) * base.U[dtype], (k, off)
    assert not t["dx"][-2:].any() and torch.equal(t["out"][-2:], t["r"][-2:])
    # against differences: the loss along a direction, a step of h either way (its error is h^2 of the third derivative)
    g = torch.Generator(device=DEV).manual_seed(1)
    with torch.no_grad():
        for i, k in enumerate(("dx", "dweights", "dw1", "db1", "dw2", "db2")):
            d, h = torch.randn(values[i].shape, generator=g, device=DEV, dtype=torch.float64), 1e-4
            ends = [chain_loss(t, [v + s * h * d if i == n else v for n, v in enumerate(values)], mask)[1].item() for s in (1, -1)]
            slope, got = (ends[0] - ends[1]) / (2 * h), (t[k].double() * d).sum().item()
            # each value of the gradient is off as above, in an independent direction
            assert abs(slope - got) < 6 * math.sqrt(5 / 3) * base.U[dtype] * t[k].double().norm().item() + 1e-6 * abs(slope), k


def test_a_block_of_them_captured_with_new_masks():
    t = chain_tensors(70, 2, 6, 136, 264, BF16, seed=2)
    want = []
    for use in range(4):
        t["rng"][1] = use
        chain_step(t)
        want.append([t[k].clone() for k in OUTPUTS])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain_step(t)
    for use in (2, 0, 3, 1, 2):
        t["rng"][1] = use
        for k in OUTPUTS:
            t[k].fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for k, w in zip(OUTPUTS, want[use]):
            assert torch.equal(t[k], w), (use, k)
        chain_loss(t, [t[k].double() for k in ("x", "weights", "w1", "b1", "w2", "b2")], torch.ones(70, 136, dtype=torch.bool, device=DEV))


def test_a_block_of_them_on_another_stream():
    a, b = (chain_tensors(200, 2, 6, 136, 264, F16, seed=4) for _ in range(2))
    chain_step(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    chain_step(b, stream=side)
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(a[k], b[k]), k


def test_two_blocks_of_them_at_once():
    # each with its own buffers, workspaces and stream
    a, b, c, d = (chain_tensors(300, 2, 6, 136, 264, F16, seed=s) for s in (4, 5, 4, 5))
    chain_step(a)
    chain_step(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for t, s in zip((c, d), streams):
            chain_step(t, stream=s)
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(a[k], c[k]) and torch.equal(b[k], d[k]), k


def test_with_the_routing_of_the_layer():
    # the picks and weights that moe_route writes are what moe_sort and moe_combine_forward take
    shape, m = S.TINY, 50
    cfg = moe.make_cfg(shape.dim, shape.inter, shape.n_routed, shape.topk, max_tokens=m)
    ctx = moe.moe_create(cfg)
    wr, bias = (v.to(DEV) for v in S.make_router(shape, 0, 0.05, (-0.1, 0.1)))
    x = S.make_tokens(m, shape.dim, 0).to(DEV)
    weights, idx = torch.empty(m, shape.topk, device=DEV), torch.empty(m, shape.topk, dtype=torch.int32, device=DEV)
    moe.moe_route(ctx, moe.make_weights(wr, bias), x, m, weights, idx)
    torch.cuda.synchronize()
    n = m * shape.topk
    row_of, pick_of, offsets = torch.empty_like(idx), torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(shape.n_routed + 1, dtype=torch.int32, device=DEV)
    moe.moe_sort(idx, shape.n_routed, row_of, pick_of, offsets, None)
    for got, want in zip((row_of, pick_of, offsets), ref.sort(idx.cpu(), shape.n_routed)):
        assert torch.equal(got.cpu(), want)
    xs, y = torch.empty(n, shape.dim, dtype=BF16, device=DEV), torch.empty_like(x)
    moe.moe_dispatch_forward(x, row_of, xs)
    moe.moe_combine_forward(xs, weights, row_of, y)
    total = weights.double().sum(1, keepdim=True).cpu()
    v = total * x.double().cpu()
    base.check(y, *ref.stored(v, (shape.topk + 1) * ref.F32 * v.abs(), BF16), "y")
    moe.moe_destroy(ctx)


def test_tensors_of_another_device_are_refused(monkeypatch):
    # (as it looks where these tensors' device is not the current one)
    t = dict(x=torch.zeros(3, 64, dtype=BF16, device=DEV), row_of=torch.zeros(3, 1, dtype=torch.int32, device=DEV), w=torch.zeros(3, 1, device=DEV),
             offsets=torch.zeros(2, dtype=torch.int32, device=DEV), rng=torch.zeros(2, dtype=torch.int64, device=DEV),
             work=torch.empty(1 << 22, dtype=torch.uint8, device=DEV))
    x, row_of, w = t["x"], t["row_of"], t["w"]
    y = torch.full_like(x, 7)
    f, drop = moe.make_linear(torch.zeros(64, 64, dtype=BF16, device=DEV)), moe.make_dropout(64, BF16, 0.5)
    calls = [lambda: moe.moe_sort(row_of, 1, row_of, None, t["offsets"], None), lambda: moe.moe_dispatch_forward(x, row_of, y),
             lambda: moe.moe_dispatch_backward(x, row_of, y), lambda: moe.moe_combine_forward(x, w, row_of, y),
             lambda: moe.moe_combine_backward(x, x, w, row_of, y, w), lambda: moe.moe_linear_forward(f, x, y, t["work"]),
             lambda: moe.moe_linear_backward(f, x, x, None, t["work"], dx=y), lambda: moe.moe_dropout_forward(drop, t["rng"], x, y),
             lambda: moe.moe_dropout_backward(drop, t["rng"], x, y)]
    monkeypatch.setattr(moe, "_several", True)
    here = torch.cuda.current_device()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here + 1)
    for call in calls:
        with pytest.raises(moe.MoeError):
            call()
    monkeypatch.undo()
    monkeypatch.setattr(moe, "_several", True)
    assert (y == 7).all() and not row_of.any()
    moe.moe_linear_forward(f, x, y, t["work"])
    assert not y.any()
