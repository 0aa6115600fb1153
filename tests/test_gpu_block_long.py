"""GPU: the operators around the layer where a workgroup takes many steps: rows after rows, rings of
buffers that come round again, the largest tiles and their joins. Against float64, on the device."""
import pytest
import torch

import block_reference as ref
import mixture_experts_ffn_gemv_amd as moe
from test_gpu_block import BF16, DEV, F16, F32, empty, ffn_run, norm_run, strided, untouched, w4_case, w4_make, workspace

pytestmark = pytest.mark.gpu


def normal(g, shape, dtype, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale + mean).to(dtype)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def agree(got, want, what):
    assert set(got) == set(want)
    for k, (v, e) in want.items():
        ref.check(got[k], v.cpu(), e.cpu(), f"{k} of {what}")


# ------------------------------------------------------------------ gated feed-forward block

def ffn_against_float64(m, dim, inter, dtype, act, limit, extra=0):
    g = generator(m + dim)
    x, dy = normal(g, (m, dim), dtype), normal(g, (m, dim), dtype)
    wg, wu = (normal(g, (inter, dim), dtype, 1.2 / dim ** 0.5) for _ in range(2))
    wd = normal(g, (dim, inter), dtype, 1 / inter ** 0.5)
    got = ffn_run((x, dy, wg, wu, wd, act, limit), extra=extra)
    agree(got, ref.ffn(x, wg, wu, wd, act, limit, dy=dy), f"m={m} of {dim} x {inter}")
    for k in ("y", "dx"):
        assert untouched(got[k]), k


# Tiles of 256 where these numbers of them and of K steps make them the shorter: for g and u with a join and
# for dh without; dh with one; dx with one; y with one; the weights' gradients with one; g, u, dh and dx with one each
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,dim,inter", [(3340, 520, 2376), (4740, 520, 3432), (3480, 4744, 264), (3340, 4744, 528),
                                         (3900, 784, 1584), (4799, 1032, 3344)])
def test_ffn_in_the_largest_tiles(m, dim, inter, dtype):
    ffn_against_float64(m, dim, inter, dtype, "silu" if dtype is BF16 else "gelu", 2.0 if m % 2 else 0.0, extra=8)


# One token and a few that fit into LDS whole, with 5 chunks of weights in flight, fewer, and several times as many
@pytest.mark.parametrize("m,dim,inter", [(1, 5128, 2312), (3, 5128, 2312), (2, 16384, 264), (1, 264, 16376), (4, 1288, 1536),
                                         (16, 1544, 2040)])
def test_ffn_few_rows_many_chunks(m, dim, inter):
    ffn_against_float64(m, dim, inter, BF16 if m % 2 else F16, "silu", 10.0, extra=24)


# 6 to 16 rows that do not: slabs of 512, five in flight: 5, 6, 9, 10, 11, 15, 16 and 32 of them
@pytest.mark.parametrize("m,dim,inter", [(7, 5128, 2568), (13, 2568, 5128), (16, 5128, 2568), (16, 5120, 2560), (9, 8192, 4104),
                                         (14, 4608, 5640), (12, 7680, 3080), (16, 16384, 136), (6, 16384, 7688)])
def test_ffn_few_rows_in_slabs(m, dim, inter):
    ffn_against_float64(m, dim, inter, BF16 if m % 2 else F16, "silu", 10.0, extra=24)


# 17 to 64 rows: slabs of 256, eight in flight, up to eight rounds of them, room for 24, 32, 40, 48 and 64 rows. Above 32
# rows a product goes by weight rows or in tiles, by its K and its weights: of the last six one goes by weight rows in both,
# in two rounds of workgroups in the second, the others in one of the two
@pytest.mark.parametrize("m,dim,inter", [(17, 4360, 520), (24, 520, 4360), (32, 8200, 264), (26, 136, 8200), (33, 4104, 264),
                                         (40, 264, 4232), (48, 4360, 136), (43, 136, 4104), (64, 136, 8200), (49, 8200, 72),
                                         (20, 16384, 16), (31, 16, 16384), (33, 264, 10248),
                                         (40, 5128, 2312), (40, 8200, 2040), (48, 6152, 2040), (41, 4088, 4104), (56, 4088, 4104),
                                         (64, 6152, 2040)])
def test_ffn_more_rows_in_slabs(m, dim, inter):
    ffn_against_float64(m, dim, inter, BF16 if m % 2 else F16, "gelu", 0.0, extra=16)


# ------------------------------------------------------------------ norms around a block

def norm_case(m, dim, dtype, gate, seed):
    g = generator(seed)
    c = {k: normal(g, (m, dim), dtype, s) for k, s in (("r", 2.0), ("y", 1.0), ("dr_out", 1.0), ("dn", 1.0))}
    c["w_post"], c["w_pre"] = (normal(g, (dim,), dtype, 0.2, 1.0) for _ in range(2))
    shape = {"none": None, "channel": (dim,), "token": (m, 1), "full": (m, dim)}[gate]
    c["gate"] = None if shape is None else normal(g, shape, dtype, 0.3, 0.5)
    return c


# At least three rows, one after another, for a thread: single values; several rows per wavefront, whole and with a shifted
# last chunk; a wavefront per row; a workgroup per row with one, two and four chunks per thread, whole and shifted.
# Past 32 MB an output is stored past the L2s: the last four
NORM = [(1000003, 7, BF16, "token"), (130001, 64, BF16, "channel"), (61445, 100, F16, "full"), (80003, 257, F16, "channel"),
        (16001, 512, BF16, "token"), (1601, 5120, BF16, "channel"), (1601, 8192, BF16, "token"), (1601, 5119, F16, "full"),
        (4003, 1111, F32, "token"), (900, 16384, F16, "channel"),
        (1601, 8193, F32, "channel"), (900, 16383, F32, "full"), (1100, 16384, BF16, "none"), (130001, 136, BF16, "channel")]


@pytest.mark.parametrize("m,dim,dtype,gate", NORM)
def test_norm_of_many_rows(m, dim, dtype, gate):
    c, scale = norm_case(m, dim, dtype, gate, seed=dim), 0.7 if m % 2 else 1.0
    with torch.device(DEV):
        want = ref.norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], 1e-6, scale, c["dr_out"], c["dn"])
    for extra in (0, 3) if dim % 8 else (0, 8):
        got = norm_run(c, scale, extra=extra)
        agree(got, want, f"[{m}, {dim}] + {extra}")
        for k in ("r_out", "n", "dr", "dy"):
            assert untouched(got[k]), k


@pytest.mark.parametrize("m,dim,dtype,gate", [NORM[i] for i in (1, 2, 4, 5, 7, 10, 13)])
def test_norm_of_many_rows_in_place(m, dim, dtype, gate):
    c = norm_case(m, dim, dtype, gate, seed=dim)
    want = norm_run(c, 0.5)
    f = moe.make_norm(dim, dtype, w_post=c["w_post"], w_pre=c["w_pre"], res_scale=0.5)
    r, y, dr, dy = (c[k].clone() for k in ("r", "y", "dr_out", "dn"))
    stats, work = torch.empty(m, 2, device=DEV), workspace(moe.moe_norm_workspace(f, m))
    moe.moe_norm_forward(f, r, y, r, y, gate=c["gate"], stats=stats)
    moe.moe_norm_backward(f, c["r"], c["y"], stats, dr, dy, work, gate=c["gate"], dr=dr, dy=dy)
    for k, t in (("r_out", r), ("n", y), ("dr", dr), ("dy", dy)):
        assert torch.equal(t, want[k]), k


# ------------------------------------------------------------------ 4-bit weights

# (m, rows, cols, group, zeros, type). More than 256 workgroups of more than 16 rows: two parts of the columns, three steps
# in LDS, up to 17 steps and three slabs of scales. Then four parts, four or three steps, room for 4, 8, 16, 24 and 32
# rows, up to 18 steps. The groups of a row are no multiple of eight, so that the last of a slab's pieces is moved
W4 = [(17, 8225, 4256, 32, True, BF16), (24, 8225, 4288, 64, False, F16), (32, 8225, 4224, 128, True, F16),
      (29, 8225, 4256, 32, True, F16), (70, 2740, 4288, 64, True, BF16),
      (3, 100, 8352, 32, True, BF16), (4, 70, 8512, 64, False, F16), (8, 100, 8352, 32, True, F16), (6, 70, 8576, 128, True, BF16),
      (16, 100, 8352, 32, True, BF16), (11, 70, 8512, 64, True, F16), (24, 100, 8352, 32, True, F16),
      (20, 70, 8576, 128, False, BF16), (32, 100, 8352, 32, True, BF16), (27, 70, 8512, 64, True, F16),
      (40, 70, 9088, 128, True, F16)]


def w4_on_device(rows, cols, group, zeros, dtype, seed):
    return [None if t is None else t.to(DEV) for t in w4_case(rows, cols, group, zeros, dtype, seed)]


@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", W4)
def test_w4_matmul_of_many_steps(m, rows, cols, group, zeros, dtype):
    c = w4_on_device(rows, cols, group, zeros, dtype, seed=cols)
    x = normal(generator(m), (m, cols), dtype)
    v, e = ref.w4_product(x, *c, group)
    y = empty(m, rows, dtype, 8 + rows % 2)
    moe.moe_w4_matmul(w4_make(c, group), strided(x, 8), y)
    ref.check(y, v.cpu(), (e + ref.U[dtype] * (v.abs() + e) + ref.TINY[dtype]).cpu(), f"[{m}, {cols}] x [{rows}]")
    assert untouched(y)


@pytest.mark.parametrize("m,rows,cols,group,zeros,dtype", W4)
def test_w4_gated_of_many_steps(m, rows, cols, group, zeros, dtype):
    rows = rows // 2 + 1
    cg, cu = (w4_on_device(rows, cols, group, zeros, dtype, seed=s) for s in (cols, cols + 1))
    x = normal(generator(m), (m, cols), dtype)
    (g, eg), (u, eu) = ref.w4_product(x, *cg, group), ref.w4_product(x, *cu, group)
    a, da, uc = ref.gated(g, u, "silu", 0.0)
    v = a * uc
    # |act''| <= 1.2, as for the dense block: the second order of g's error
    e = (da * uc).abs() * eg + a.abs() * eu + 2 * eg * eu + 0.6 * eg * eg * uc.abs() + ref.ACC * v.abs()
    h = empty(m, rows, dtype)
    moe.moe_w4_gated(w4_make(cg, group), w4_make(cu, group), x, h, act="silu", limit=0.0)
    ref.check(h, v.cpu(), (e + ref.U[dtype] * (v.abs() + e) + ref.TINY[dtype]).cpu(), f"gated [{m}, {cols}] x [{rows}]")
    assert untouched(h)
