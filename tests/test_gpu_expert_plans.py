"""GPU: products with a matrix per expert, by the kernels and tiles that the library's own rules choose for them, against
float64 on the device."""
import pytest
import torch

import block_reference as base
import expert_reference as ref
import mixture_experts_ffn_gemv_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16
NAN = float("nan")


def tensors(m, k, n, dtype, seed, n_experts=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=DEV) * scale).to(dtype)   # noqa: E731
    shape = (n_experts, n, k) if n_experts else (n, k)
    return dict(x=rnd(m, k), dy=rnd(m, n), w=rnd(*shape, scale=1.2 / k ** 0.5), bias=rnd(*shape[:-1], scale=0.5), residual=rnd(m, n))


def ends(counts):
    offsets = [0]
    for v in counts:
        offsets.append(offsets[-1] + v)
    return offsets


def backward(c, act, offsets, saved, want):
    f = moe.make_linear(c["w"], c["bias"], act=act)
    work = torch.full((moe.moe_linear_workspace(f, c["x"].shape[0])[2],), 0xFF, dtype=torch.uint8, device=DEV)
    out = {"dx": torch.full_like(c["x"], NAN), "dw": torch.full_like(c["w"], NAN), "dbias": torch.full_like(c["bias"], NAN)}
    out = {name: out[name] for name in want}
    moe.moe_linear_backward(f, c["x"], c["dy"], saved, work, offsets=offsets, **out)
    torch.cuda.synchronize()
    return out


def forward(c, act, offsets):
    f = moe.make_linear(c["w"], c["bias"], act=act)
    work, saved = (torch.full((v,), 0xFF, dtype=torch.uint8, device=DEV) for v in moe.moe_linear_workspace(f, c["x"].shape[0])[:2])
    y = torch.full_like(c["dy"], NAN)
    moe.moe_linear_forward(f, c["x"], y, work, offsets=offsets, residual=c["residual"], saved=saved)
    torch.cuda.synchronize()
    return y, saved


def check(got, want, what):
    base.check(got, want[0].cpu(), want[1].cpu(), what)


@pytest.mark.parametrize("counts,k,n,dtype,act", [([3, 0, 70, 130, 1], 264, 392, BF16, "silu"), ([1900, 0, 2500, 300, 257], 1040, 1032, F16, "gelu"),
                                                  ([20] * 90 + [0] * 40, 136, 264, BF16, "none")])
def test_gradients_of_experts_each_by_itself(counts, k, n, dtype, act):
    offsets = ends(counts)
    c = tensors(offsets[-1], k, n, dtype, seed=k, n_experts=len(counts))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    _, saved = forward(c, act, off)
    together = backward(c, act, off, saved, ("dx", "dw", "dbias"))
    for name, t in together.items():
        assert torch.isfinite(t).all()
        assert torch.equal(backward(c, act, off, saved, (name,))[name], t), name


@pytest.mark.parametrize("n_experts", [64, 65, 200])
def test_gradients_of_many_experts_with_few_rows_and_many(n_experts):
    # (those with few rows are launched apart: more rows on average than that, in an order that their number decides)
    counts = [(200, 3, 0, 65, 64, 128, 1)[e * 5 % 7] for e in range(n_experts)]
    offsets = ends(counts)
    used, m = offsets[-1], offsets[-1] + 9
    assert used > 64 * n_experts
    c = tensors(m, 72, 136, F16, seed=n_experts, n_experts=n_experts)
    for name in ("x", "dy", "residual"):
        c[name][used:] = NAN
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y, saved = forward(c, "silu", off)
    got = {"y": y, **backward(c, "silu", off, saved, ("dx", "dw", "dbias"))}
    assert torch.isnan(got["y"][used:]).all() and torch.isnan(got["dx"][used:]).all()
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a == b:
            assert not got["dw"][e].any() and not got["dbias"][e].any(), e
            continue
        want = ref.linear(c["x"][a:b], c["w"][e], c["bias"][e], c["residual"][a:b], "silu", dy=c["dy"][a:b])
        for name, t in got.items():
            check(t[a:b] if name in ("y", "dx") else t[e], want[name], f"{name} of expert {e}")


def experts_against_float64(counts, behind, k, n, dtype, act, seed):
    offsets = ends(counts)
    used, m = offsets[-1], offsets[-1] + behind
    c = tensors(m, k, n, dtype, seed=seed, n_experts=len(counts))
    for name in ("x", "dy", "residual"):
        c[name][used:] = NAN   # rows behind the last are not read
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y, saved = forward(c, act, off)
    got = {"y": y, **backward(c, act, off, saved, ("dx", "dw", "dbias"))}
    assert torch.isnan(got["y"][used:]).all() and torch.isnan(got["dx"][used:]).all()
    idle = [e for e, v in enumerate(counts) if v == 0]
    assert not got["dw"][idle].any() and not got["dbias"][idle].any()
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a == b:
            continue
        want = ref.linear(c["x"][a:b], c["w"][e], c["bias"][e], c["residual"][a:b], act, dy=c["dy"][a:b])
        for name, t in got.items():
            check(t[a:b] if name in ("y", "dx") else t[e], want[name], f"{name} of expert {e}")


def picked(n_experts, at):
    counts = [0] * n_experts
    for e in at:
        counts[e] += 1
    return counts


@pytest.mark.parametrize("counts,behind,k,n,dtype,act", [
    # so few rows that each goes by the weights of its expert: experts past those whose offsets are read at a time (64 and 256),
    # rows of x of many steps, outputs that sixteen do not divide
    (picked(300, (3, 70, 130, 256, 299, 299)), 0, 5128, 1030, BF16, "silu"),
    (picked(384, (0, 63, 64, 255, 320, 383)), 0, 5120, 2304, BF16, "none"),
    (picked(280, (279, 257, 257, 5)), 1, 2568, 1000, F16, "gelu"),
    # an expert with more rows than a workgroup has room for
    (picked(300, (290,) * 5 + (17, 100, 299)), 0, 2056, 2309, F16, "silu"),
    ([9, 0, 1, 0, 2, 0, 0, 0], 0, 2056, 1033, BF16, "gelu"),
    ([0, 1, 11, 0, 0, 0, 0, 1, 0, 0], 1, 5120, 1030, F16, "none")])
def test_few_rows_of_many_experts(counts, behind, k, n, dtype, act):
    experts_against_float64(counts, behind, k, n, dtype, act, seed=k + n)


@pytest.mark.parametrize("counts,k,n,dtype,act", [
    # the largest tiles in y, dx and dW, none of them whole
    ([700, 0, 33, 1500, 64, 65, 900, 257] * 4, 2056, 1544, BF16, "silu"),
    ([1801, 300, 3000, 0, 1, 2000, 800, 400, 600, 700, 398, 0], 2568, 2309, F16, "gelu")])
def test_experts_by_the_largest_tiles(counts, k, n, dtype, act):
    experts_against_float64(counts, 5, k, n, dtype, act, seed=k)


def test_one_matrix_by_the_largest_tiles():
    m, k, n = 5000, 2600, 2309   # 200 of them in y, 220 in dx, 110 in dW, none of the last ones whole
    c = tensors(m, k, n, BF16, seed=5)
    want = ref.linear(c["x"], c["w"], c["bias"], c["residual"], "silu", dy=c["dy"])
    y, saved = forward(c, "silu", None)
    got = {"y": y, **backward(c, "silu", None, saved, ("dx", "dw", "dbias"))}
    for name, t in got.items():
        check(t, want[name], name)
    for name in ("dx", "dw", "dbias"):   # each by itself: against the same reference, since it may be cut up otherwise
        check(backward(c, "silu", None, saved, (name,))[name], want[name], f"{name} by itself")
