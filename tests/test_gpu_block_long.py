"""GPU: the operators around the layer where a workgroup takes many steps: rows after rows, rings of
buffers that come round again, the largest tiles and their joins. Against float64, on the device."""
import pytest
import torch

import block_reference as ref
from test_gpu_block import BF16, DEV, F16, ffn_run, untouched

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


# 17 to 64 rows: slabs of 256, eight in flight, up to four rounds of them, room for 24, 32, 40, 48 and 64 rows
@pytest.mark.parametrize("m,dim,inter", [(17, 4360, 520), (24, 520, 4360), (32, 8200, 264), (26, 136, 8200), (33, 4104, 264),
                                         (40, 264, 4232), (48, 4360, 136), (43, 136, 4104), (64, 136, 8200), (49, 8200, 72),
                                         (20, 16384, 16), (31, 16, 16384)])
def test_ffn_more_rows_in_slabs(m, dim, inter):
    ffn_against_float64(m, dim, inter, BF16 if m % 2 else F16, "gelu", 0.0, extra=16)
