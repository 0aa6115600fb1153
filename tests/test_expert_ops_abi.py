"""CPU: the refusals of sorting by expert, of products with bias, activation and residual, and of dropout. Every call
below has to be refused, or to have nothing to do, before the library touches a device (there is none here)."""
import ctypes
import os
import re

import numpy
import pytest
import torch

import expert_reference as ref
import mixture_experts_ffn_gemv_amd as moe

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")
P = 1 << 20   # an aligned stand-in for a device pointer: never followed
NAN = float("nan")
EINVAL, ESCRATCH, OK = moe.MOE_EINVAL, moe.MOE_ESCRATCH, moe.MOE_OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.lib()


@pytest.mark.parametrize("name", ["moe_linear", "moe_dropout"])
def test_structs_match_the_header(name):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
    fields = [(" ".join(t.split()), f) for t, f in re.findall(r"([A-Za-z_][\w ]*\*?)\s+(\w+);", body)]
    binding = getattr(moe, name)._fields_
    assert [f for _, f in fields] == [f for f, _ in binding]
    types = {"int32_t": ctypes.c_int32, "double": ctypes.c_double, "const void*": ctypes.c_void_p}
    assert [types[t] for t, _ in fields] == [t for _, t in binding]


# ------------------------------------------------------------------ sort

def sort_size(lib, m, topk, n_experts):
    size = ctypes.c_size_t()
    return lib.moe_sort_workspace(m, topk, n_experts, ctypes.byref(size)), size.value


def test_sort_is_refused(lib):
    for bad in ((-1, 6, 384), (3, 0, 384), (3, 65, 384), (3, 6, 0), (3, 6, 1025), (1 << 21, 64, 384)):
        assert sort_size(lib, *bad)[0] == EINVAL, bad
        assert lib.moe_sort(P, *bad, P, P, P, P, 1 << 30, None) == EINVAL, bad
    assert lib.moe_sort_workspace(3, 6, 384, None) == EINVAL

    def call(idx=P, m=9000, row_of=P, pick_of=P, offsets=P, work=P, nwork=1 << 30):
        return lib.moe_sort(idx, m, 6, 384, row_of, pick_of, offsets, work, nwork, None)

    for bad in (dict(idx=None), dict(idx=P + 2), dict(row_of=None), dict(row_of=P + 1), dict(pick_of=P + 2), dict(offsets=None),
                dict(offsets=P + 3), dict(work=None), dict(work=P + 16)):
        assert call(**bad) == EINVAL, bad
    rc, need = sort_size(lib, 9000, 6, 384)
    assert rc == OK and need > 0 and need % 256 == 0 and call(nwork=need - 1) == ESCRATCH


@pytest.mark.parametrize("topk,n_experts", [(1, 1), (6, 384), (64, 1024)])
def test_sort_workspaces_fit_fewer_tokens(lib, topk, n_experts):
    last = 0
    for m in sorted({*range(0, 300, 7), *range(300, 60000, 997), 1 << 18, 1 << 20}):
        rc, need = sort_size(lib, m, topk, n_experts)
        assert rc == OK and need >= last, m
        last = need


def test_moves_are_refused(lib):
    def dispatch(dtype=0, dim=64, x=P, ldx=64, row_of=P, m=3, topk=6, xs=P, ldxs=64, rows=18):
        return lib.moe_dispatch_forward(dtype, dim, x, ldx, row_of, m, topk, xs, ldxs, rows, None)

    def back(dtype=0, dim=64, x=P, ldx=64, row_of=P, m=3, topk=6, xs=P, ldxs=64, rows=18):
        return lib.moe_dispatch_backward(dtype, dim, xs, ldxs, rows, row_of, m, topk, x, ldx, None)

    def combine(dtype=0, dim=64, x=P, ldx=64, row_of=P, m=3, topk=6, xs=P, ldxs=64, rows=18, weights=P):
        return lib.moe_combine_forward(dtype, dim, xs, ldxs, rows, weights, row_of, m, topk, x, ldx, None)

    def combine_back(dtype=0, dim=64, x=P, ldx=64, row_of=P, m=3, topk=6, xs=P, ldxs=64, rows=18, weights=P, de=P, ldde=64, dw=P):
        return lib.moe_combine_backward(dtype, dim, x, ldx, xs, ldxs, rows, weights, row_of, m, topk, de, ldde, dw, None)

    for call in (dispatch, back, combine, combine_back):
        for bad in (dict(dtype=3), dict(dtype=-1), dict(dim=0), dict(dim=(1 << 20) + 1), dict(x=None), dict(x=P + 1), dict(ldx=63),
                    dict(xs=None), dict(xs=P + 1), dict(ldxs=0), dict(row_of=None), dict(row_of=P + 2), dict(m=-1), dict(topk=0),
                    dict(topk=65), dict(rows=-1), dict(rows=(1 << 26) + 1), dict(dtype=2, x=P + 2), dict(m=1 << 26)):
            assert call(**bad) == EINVAL, (call, bad)
        assert call(m=0, x=None, xs=None, row_of=None) == OK
    for call in (combine, combine_back):
        assert call(weights=None) == call(weights=P + 2) == EINVAL
    assert combine_back(de=P + 1) == combine_back(ldde=63) == combine_back(dw=P + 2) == EINVAL
    assert dispatch(rows=0, xs=None) == combine_back(de=None, dw=None) == OK   # nothing to do


# ------------------------------------------------------------------ linear

def linear(**kw):
    v = dict(cols=64, rows=37, experts=1, dtype=moe.MOE_BF16, act=moe.MOE_ACT_SILU, w=P, bias=P)
    v.update(kw)
    return moe.moe_linear(**v)


def sizes(lib, f, m):
    out = [ctypes.c_size_t() for _ in range(3)]
    rc = lib.moe_linear_workspace(f, m, *[ctypes.byref(o) for o in out])
    return (rc, *(o.value for o in out))


def forward(lib, f, x=P, ldx=64, offsets=None, m=300, r=P, ldr=37, y=P, ldy=37, saved=P, nsaved=1 << 30, work=P, nwork=1 << 30):
    return lib.moe_linear_forward(f, x, ldx, offsets, m, r, ldr, y, ldy, saved, nsaved, work, nwork, None)


def backward(lib, f, x=P, ldx=64, offsets=None, m=300, dy=P, lddy=37, saved=P, nsaved=1 << 30, dx=P, lddx=64, dw=P, dbias=P, work=P,
             nwork=1 << 30):
    return lib.moe_linear_backward(f, x, ldx, offsets, m, dy, lddy, saved, nsaved, dx, lddx, dw, dbias, work, nwork, None)


@pytest.mark.parametrize("bad", [dict(cols=0), dict(cols=60), dict(cols=65544), dict(rows=0), dict(rows=(1 << 17) + 1), dict(experts=0),
                                 dict(experts=1025), dict(dtype=moe.MOE_F32), dict(dtype=-1), dict(act=3), dict(act=-1), dict(w=None),
                                 dict(w=P + 8), dict(bias=P + 1)])
def test_linear_descriptions_are_refused(lib, bad):
    f = ctypes.byref(linear(**bad))
    assert sizes(lib, f, 3)[0] == forward(lib, f, offsets=P) == backward(lib, f, offsets=P) == EINVAL


def test_linear_arguments_are_refused(lib):
    f, plain, no_bias, two = (ctypes.byref(linear(**kw)) for kw in ({}, dict(act=moe.MOE_ACT_NONE), dict(bias=None), dict(experts=2)))
    rc, need, saved, back = sizes(lib, f, 300)
    assert rc == OK and saved >= 300 * 40 * 4 and back >= 300 * 40 * 2 and all(v % 256 == 0 for v in (need, saved, back))
    assert sizes(lib, plain, 300)[2] == 0
    assert sizes(lib, f, -1)[0] == sizes(lib, f, (1 << 24) + 1)[0] == sizes(lib, None, 1)[0] == EINVAL
    assert lib.moe_linear_workspace(f, 3, None, None, None) == EINVAL
    for bad in (dict(m=-1), dict(m=(1 << 24) + 1), dict(x=None), dict(x=P + 8), dict(ldx=56), dict(ldx=68), dict(ldx=(1 << 22) + 8),
                dict(offsets=P + 2), dict(saved=P + 16), dict(work=P + 16)):
        assert forward(lib, f, **bad) == backward(lib, f, **bad) == EINVAL, bad
    assert forward(lib, two) == backward(lib, two) == EINVAL   # a matrix per expert needs its offsets
    for bad in (dict(y=None), dict(y=P + 1), dict(ldy=36), dict(r=P + 1), dict(ldr=36)):
        assert forward(lib, f, **bad) == EINVAL, bad
    for bad in (dict(dy=None), dict(dy=P + 1), dict(lddy=36), dict(saved=None), dict(dx=P + 8), dict(lddx=60), dict(lddx=68),
                dict(dw=P + 8), dict(dbias=P + 1), dict(work=None)):
        assert backward(lib, f, **bad) == EINVAL, bad
    assert backward(lib, no_bias) == EINVAL                    # the gradient of no bias
    assert forward(lib, f, nsaved=saved - 1) == ESCRATCH
    assert backward(lib, f, nsaved=saved - 1) == backward(lib, f, nwork=back - 1) == ESCRATCH
    wide = ctypes.byref(linear(cols=8192))
    need = sizes(lib, wide, 300)[1]
    assert need > 0 and forward(lib, wide, ldx=8192, work=None) == EINVAL and forward(lib, wide, ldx=8192, nwork=need - 1) == ESCRATCH
    assert forward(lib, f, m=0, x=None, y=None, r=None, saved=None, work=None, nwork=0) == OK


@pytest.mark.parametrize("cols,rows,experts", [(8, 1, 1), (64, 37, 1), (64, 37, 5), (1544, 4101, 1), (5120, 2304, 1), (2048, 1408, 32),
                                               (65536, 131072, 1)])
def test_linear_workspaces_fit_fewer_rows(lib, cols, rows, experts):
    f, last = ctypes.byref(linear(cols=cols, rows=rows, experts=experts)), (0, 0, 0)
    for m in sorted({*range(0, 300), *range(300, 9000, 37), 1000, 1536, 8192, 1 << 20, 1 << 24}):
        rc, *now = sizes(lib, f, m)
        assert rc == OK and all(a <= b and b % 256 == 0 for a, b in zip(last, now)), m
        last = now


# ------------------------------------------------------------------ dropout

def test_dropout_is_refused(lib):
    def call(dim=64, dtype=0, p=0.1, rng=P, x=P, ldx=64, r=P, ldr=64, m=3, y=P, ldy=64):
        return lib.moe_dropout_forward(ctypes.byref(moe.moe_dropout(dim, dtype, p)), rng, x, ldx, r, ldr, m, y, ldy, None)

    for bad in (dict(dim=0), dict(dim=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1), dict(p=-0.1), dict(p=1.01), dict(p=NAN), dict(rng=None),
                dict(rng=P + 4), dict(x=None), dict(x=P + 1), dict(ldx=63), dict(r=P + 1), dict(ldr=0), dict(m=-1), dict(m=(1 << 30) + 1),
                dict(y=None), dict(y=P + 1), dict(ldy=63), dict(dtype=2, x=P + 2)):
        assert call(**bad) == EINVAL, bad
    f = ctypes.byref(moe.moe_dropout(64, 0, 0.1))
    assert lib.moe_dropout_forward(None, P, P, 64, P, 64, 3, P, 64, None) == EINVAL
    for bad in ((None, P, 64, 3, P, 64), (P, None, 64, 3, P, 64), (P, P, 63, 3, P, 64), (P, P, 64, -1, P, 64), (P, P, 64, 3, None, 64),
                (P, P, 64, 3, P, 63)):
        assert lib.moe_dropout_backward(f, *bad, None) == EINVAL, bad
    assert call(m=0, x=None, y=None, r=None, rng=None) == OK


def test_generator_reference_against_published_vectors():
    # the known answers published with the generator (Random123's kat_vectors, philox4x32, 10 rounds)
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = ref.philox([numpy.array([c]) for c in counter], key)
        assert tuple(int(w[0]) for w in got) == want


def test_binding_refuses_tensors_of_the_host():
    w, i = torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(8, 2, dtype=torch.int32)
    f = torch.zeros(8, 2)
    for call in (lambda: moe.make_linear(w), lambda: moe.make_linear(w[0]), lambda: moe.make_linear(w, act="relu"),
                 lambda: moe.make_dropout(8, torch.int32, 0.1), lambda: moe.moe_sort(i, 4, i, None, i[0], None),
                 lambda: moe.moe_sort(w, 4, i, None, i[0], None), lambda: moe.moe_dispatch_forward(w, i, w),
                 lambda: moe.moe_dispatch_forward(w[:3], i, w), lambda: moe.moe_dispatch_forward(w, i, w.float()),
                 lambda: moe.moe_dispatch_backward(w, i, w), lambda: moe.moe_combine_forward(w, f, i, w),
                 lambda: moe.moe_combine_backward(w, w, f, i, de=w)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == EINVAL
