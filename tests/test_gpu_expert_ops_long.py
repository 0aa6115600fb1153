"""GPU: products with bias, activation and residual where workgroups take many tiles one after another, where tiles are
split along k and joined, and where the longer of dx's and dW's tiles is either one's; against float64 on the device."""
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


def run(c, act, bias=True, offsets=None, want=("dx", "dw", "dbias")):
    f = moe.make_linear(c["w"], c["bias"] if bias else None, act=act)
    m = c["x"].shape[0]
    forward, saved, backward = (torch.full((v,), 0xFF, dtype=torch.uint8, device=DEV) for v in moe.moe_linear_workspace(f, m))
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    out = {"y": torch.full_like(c["dy"], NAN), "dx": torch.full_like(c["x"], NAN), "dw": torch.full_like(c["w"], NAN),
           "dbias": torch.full_like(c["bias"], NAN)}
    grads = {k: out[k] if k in want and (bias or k != "dbias") else None for k in ("dx", "dw", "dbias")}
    moe.moe_linear_forward(f, c["x"], out["y"], forward, offsets=off, residual=c["residual"], saved=saved)
    moe.moe_linear_backward(f, c["x"], c["dy"], saved, backward, offsets=off, **grads)
    torch.cuda.synchronize()
    return {"y": out["y"], **{k: v for k, v in grads.items() if v is not None}}


def check(got, want, what):
    v, e = want
    share = ((got.double() - v).abs() / e).max().item()
    assert torch.isfinite(got).all() and share <= 1.0, (what, share)


DENSE = [(8200, 1288, 2309, BF16, "silu"),    # a round of the largest tiles and a part of one; dW's tiles are the longer
         (8192, 2568, 2304, F16, "gelu"),     # the tiles past a whole round in pieces along k
         (4100, 2056, 2048, BF16, "gelu"),    # whole rounds
         (700, 4104, 6152, F16, "silu"),      # dx's tiles are the longer, several a workgroup
         (3000, 520, 8200, BF16, "none"),     # many short tiles
         (5000, 8200, 136, F16, "none"),      # dW in pieces along k
         (20000, 264, 72, BF16, "gelu")]


@pytest.mark.parametrize("m,k,n,dtype,act", DENSE)
def test_linear_of_many_tiles_against_float64(m, k, n, dtype, act):
    c = tensors(m, k, n, dtype, seed=m)
    got = run(c, act)
    want = ref.linear(c["x"], c["w"], c["bias"], c["residual"], act, dy=c["dy"])
    for name, t in got.items():
        check(t, want[name], f"{name} of {m} x {k} x {n}")
    # each by itself, and again: the same bits, whatever the tiles and their order
    again = run(c, act)
    for name, t in again.items():
        assert torch.equal(t, got[name]), name


@pytest.mark.parametrize("want", [("dx",), ("dw",)])
def test_one_gradient_of_many_tiles(want):
    m, k, n = 4000, 1544, 2056
    c = tensors(m, k, n, BF16, seed=3)
    got = run(c, "silu", want=want)
    check(got[want[0]], ref.linear(c["x"], c["w"], c["bias"], c["residual"], "silu", dy=c["dy"])[want[0]], want[0])


def counts_of(n_experts, rows, seed):
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(n_experts, generator=g) ** 3
    share[::7] = 0
    return (share / share.sum() * rows).int().tolist()


@pytest.mark.parametrize("n_experts,rows,k,n,dtype,act", [
    (40, 12000, 1032, 1544, BF16, "silu"),     # the largest tiles, several of an expert and of a workgroup
    (6, 9000, 2056, 520, F16, "none"),
    (300, 4000, 136, 264, BF16, "gelu"),       # more experts than their offsets are read at a time
    (1024, 2500, 72, 40, F16, "silu"),
    (1000, 700, 264, 130, BF16, "none"),       # few rows, most experts without any
    (64, 3000, 2056, 1033, F16, "gelu")])
def test_experts_of_many_tiles_against_float64(n_experts, rows, k, n, dtype, act):
    counts = counts_of(n_experts, rows, seed=n_experts)
    offsets = [0]
    for v in counts:
        offsets.append(offsets[-1] + v)
    used, m = offsets[-1], offsets[-1] + 13
    c = tensors(m, k, n, dtype, seed=rows, n_experts=n_experts)
    for name in ("x", "dy", "residual"):
        c[name][used:] = NAN   # rows behind the last are not read
    for bias in (True, False):
        got = run(c, act, bias=bias, offsets=offsets)
        assert torch.isnan(got["y"][used:]).all() and torch.isnan(got["dx"][used:]).all()
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if a == b:
                assert not got["dw"][e].any() and not (bias and got["dbias"][e].any()), e
                continue
            want = ref.linear(c["x"][a:b], c["w"][e], c["bias"][e] if bias else None, c["residual"][a:b], act, dy=c["dy"][a:b])
            for name, t in got.items():
                check(t[a:b] if name in ("y", "dx") else t[e], want[name], f"{name} of expert {e}")


def test_gradients_of_more_workgroups_than_a_grid_holds_along_one_axis():
    # (a workgroup a token: 2^24 of 256 threads; tokens without rows but for the last)
    m, dim = 1 << 24, 1032
    dy = torch.empty(m, dim, dtype=BF16, device=DEV)
    dy[-1] = 2
    e = torch.full((1, dim), 3.0, dtype=BF16, device=DEV)
    row_of = torch.full((m, 1), -1, dtype=torch.int32, device=DEV)
    row_of[-1] = 0
    weights, dweights, de = torch.full((m, 1), 0.5, device=DEV), torch.full((m, 1), NAN, device=DEV), torch.full_like(e, NAN)
    moe.moe_combine_backward(dy, e, weights, row_of, de, dweights)
    torch.cuda.synchronize()
    assert not dweights[:-1].any() and dweights[-1].item() == 6.0 * dim and (de == 1).all()
