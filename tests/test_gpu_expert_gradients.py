"""GPU: gradients of products with few rows of a matrix, against float64: what is held in fewer bits before the result is
must not show in it."""
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
    g = base.generator(seed)
    shape = (n_experts, n, k) if n_experts else (n, k)
    return dict(x=base.normal(g, (m, k), dtype), dy=base.normal(g, (m, n), dtype), w=base.normal(g, shape, dtype, 1.2 / k ** 0.5),
                bias=base.normal(g, shape[:-1], dtype, 0.5))


def gradients(c, act, offsets=None):
    c = {name: t.to(DEV) for name, t in c.items()}
    f, m = moe.make_linear(c["w"], c["bias"], act=act), c["x"].shape[0]
    forward, saved, backward = (torch.full((v,), 0xFF, dtype=torch.uint8, device=DEV) for v in moe.moe_linear_workspace(f, m))
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    out = {"dx": torch.full_like(c["x"], NAN), "dw": torch.full_like(c["w"], NAN), "dbias": torch.full_like(c["bias"], NAN)}
    moe.moe_linear_forward(f, c["x"], torch.full_like(c["dy"], NAN), forward, offsets=off, saved=saved)
    moe.moe_linear_backward(f, c["x"], c["dy"], saved, backward, offsets=off, **out)
    torch.cuda.synchronize()
    return out


def once_rounded(x, w, bias, act, dy):
    """-> {name: (value, allowed)}: the sums' own rounding, and what keeping dz in two parts of the type leaves: each is off by
    half a step of what it stands for, so that dz is off by u^2 (2^-16 and 2^-22 of it), and in f16 by half the smallest step."""
    dt = x.dtype
    x, w, d = x.double(), w.double(), dy.double()
    z = x @ w.t() + bias.double()
    _, da = ref.act_both(z, act)
    dz = d * da
    # as in expert_reference: the second derivative is at most 1.2 in size
    edz = 1.2 * d.abs() * base.ACC * (x.abs() @ w.abs().t() + bias.double().abs()) + base.ACC * dz.abs() + base.TINY[dt]
    two = edz + base.U[dt] ** 2 * (dz.abs() + edz) + base.TINY[dt]
    dx, dw = dz @ w, dz.t() @ x
    return {"dx": ref.stored(dx, two @ w.abs() + base.ACC * (dz.abs() @ w.abs()), dt),
            "dw": ref.stored(dw, two.t() @ x.abs() + base.ACC * (dz.abs().t() @ x.abs()), dt),
            "dbias": ref.stored(dz.sum(0), edz.sum(0) + base.ACC * dz.abs().sum(0), dt)}


@pytest.mark.parametrize("m,k,n,dtype,act", [(9, 264, 64, BF16, "silu"), (9, 952, 100, F16, "gelu"), (16, 520, 4101, F16, "silu"),
                                             (23, 2056, 130, BF16, "gelu"), (33, 72, 1033, BF16, "silu"), (63, 1288, 257, F16, "gelu"),
                                             (64, 264, 2309, BF16, "silu"), (40, 72, 33001, BF16, "gelu"), (12, 16392, 72, F16, "silu")])
def test_gradients_of_some_rows_are_rounded_once(m, k, n, dtype, act):
    c = tensors(m, k, n, dtype, seed=m + k + n)
    got = gradients(c, act)
    for name, want in once_rounded(c["x"], c["w"], c["bias"], act, c["dy"]).items():
        base.check(got[name], *want, f"{name} of {m} rows")


@pytest.mark.parametrize("counts,behind,k,n,dtype,act", [
    ([1], 0, 264, 64, BF16, "silu"),                          # one token's only pick
    ([1], 90, 264, 100, F16, "gelu"),                         # the same with many rows of padding behind it
    ([0, 1, 0, 8, 2], 3, 520, 100, F16, "gelu"),
    ([64, 65, 3, 0, 200, 1], 5, 136, 264, BF16, "gelu"),      # experts with few rows beside others with many
    ([2, 0, 1] * 60, 0, 72, 130, F16, "silu"),                # several experts in every chunk of rows, more than a wavefront's lanes
    ([60, 0, 33, 64, 1, 90, 32, 7] * 3, 2, 1032, 2056, F16, "silu"),   # dW by the largest tiles
    ([300, 0, 17, 31, 64, 900], 11, 392, 520, BF16, "silu")])
def test_gradients_of_experts_with_few_rows_are_rounded_once(counts, behind, k, n, dtype, act):
    offsets = [0]
    for v in counts:
        offsets.append(offsets[-1] + v)
    m = offsets[-1] + behind
    c = tensors(m, k, n, dtype, seed=m + k, n_experts=len(counts))
    for name in ("x", "dy"):
        c[name][offsets[-1]:] = NAN
    got = gradients(c, act, offsets)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        one = c["x"][a:b], c["w"][e], c["bias"][e], act, c["dy"][a:b]
        want = once_rounded(*one) if b - a <= 64 else ref.linear(one[0], one[1], one[2], None, act, dy=one[4])
        for name in got:
            base.check(got[name][a:b] if name == "dx" else got[name][e], *want[name], f"{name} of expert {e}, {b - a} rows")
    assert torch.isnan(got["dx"][offsets[-1]:]).all()


def test_infinite_and_missing_gradients_of_few_rows():
    # dz past f16 is infinite, and NaN is NaN: what is kept beside it must not make another of it
    m, k, n = 20, 136, 90
    c = tensors(m, k, n, F16, seed=3)
    for row, col in ((3, 5), (7, 11)):   # z is 2.4 there, where the slope is 1.0998
        c["bias"][col] = (2.4 - c["x"][row].double() @ c["w"][col].double()).to(F16)
    clean = gradients(c, "silu")
    c["dy"][3, 5], c["dy"][7, 11], c["dy"][9, 13] = -65504.0, float("inf"), NAN
    got = gradients(c, "silu")
    rows, cols = [r for r in range(m) if r not in (3, 7, 9)], [v for v in range(n) if v not in (5, 11, 13)]
    for name, part in (("dx", rows), ("dw", cols), ("dbias", cols)):
        assert torch.equal(got[name][part], clean[name][part]), name
    assert torch.isnan(got["dx"][9]).all() and torch.isnan(got["dw"][13]).all() and torch.isnan(got["dbias"][13])
    inf = float("inf")
    for row, col, dz in ((3, 5, -inf), (7, 11, inf)):
        assert torch.equal(got["dx"][row].cpu().double(), torch.sign(c["w"][col].double()) * dz)
        assert torch.equal(got["dw"][col].cpu().double(), torch.sign(c["x"][row].double()) * dz)
        assert got["dbias"][col] == dz
