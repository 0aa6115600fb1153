"""CPU: the refusals of the operators around the layer. Every call below has to be
refused before the library touches a device (there is none here)."""
import ctypes
import os
import re

import pytest
import torch

import mixture_experts_ffn_gemv_amd as moe

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")
P = 1 << 20   # an aligned stand-in for a device pointer: never followed
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.lib()


@pytest.mark.parametrize("name", ["moe_ffn", "moe_norm", "moe_w4"])
def test_structs_match_the_header(name):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
    fields = [(" ".join(t.split()), f) for t, f in re.findall(r"([A-Za-z_][\w ]*\*?)\s+(\w+);", body)]
    binding = getattr(moe, name)._fields_
    assert [f for _, f in fields] == [f for f, _ in binding]
    types = {"int32_t": ctypes.c_int32, "float": ctypes.c_float, "const void*": ctypes.c_void_p}
    assert [types[t] for t, _ in fields] == [t for _, t in binding]


def ffn(**kw):
    v = dict(dim=64, inter=128, dtype=moe.MOE_BF16, act=moe.MOE_ACT_SILU, limit=0.0, w_gate=P, w_up=P, w_down=P)
    v.update(kw)
    return moe.moe_ffn(**v)


BAD_FFN = [dict(dim=0), dict(dim=60), dict(dim=16392), dict(inter=4), dict(inter=130), dict(dtype=moe.MOE_F32),
           dict(dtype=-1), dict(act=2), dict(limit=NAN), dict(w_gate=None), dict(w_up=P + 8), dict(w_down=P + 2)]


def ffn_sizes(lib, f, m):
    out = [ctypes.c_size_t() for _ in range(3)]
    rc = lib.moe_ffn_workspace(f, m, *[ctypes.byref(o) for o in out])
    return (rc, *(o.value for o in out))


def ffn_forward(lib, f, m=3, x=P, ldx=64, y=P, ldy=64, saved=P, nsaved=1 << 30, work=P, nwork=1 << 30):
    return lib.moe_ffn_forward(f, x, ldx, m, y, ldy, saved, nsaved, work, nwork, None)


def ffn_backward(lib, f, m=3, x=P, ldx=64, dy=P, lddy=64, saved=P, nsaved=1 << 30, dx=P, lddx=64, dwg=P, dwu=P, dwd=P,
                 work=P, nwork=1 << 30):
    return lib.moe_ffn_backward(f, x, ldx, dy, lddy, m, saved, nsaved, dx, lddx, dwg, dwu, dwd, work, nwork, None)


@pytest.mark.parametrize("bad", BAD_FFN)
def test_ffn_descriptions_are_refused(lib, bad):
    f = ctypes.byref(ffn(**bad))
    assert ffn_sizes(lib, f, 3)[0] == moe.MOE_EINVAL
    assert ffn_forward(lib, f) == moe.MOE_EINVAL
    assert ffn_backward(lib, f) == moe.MOE_EINVAL


def test_ffn_arguments_are_refused(lib):
    f = ctypes.byref(ffn())
    rc, forward, saved, backward = ffn_sizes(lib, f, 3)
    assert rc == moe.MOE_OK and forward >= 3 * 128 * 2 and saved >= 3 * 128 * 8 and backward >= 3 * forward
    assert ffn_sizes(lib, f, 0)[0] == moe.MOE_OK
    assert ffn_sizes(lib, f, -1)[0] == ffn_sizes(lib, f, (1 << 24) + 1)[0] == ffn_sizes(lib, None, 1)[0] == moe.MOE_EINVAL
    assert lib.moe_ffn_workspace(f, 3, None, None, None) == moe.MOE_EINVAL
    for bad in (dict(m=-1), dict(m=(1 << 24) + 1), dict(x=None), dict(x=P + 8), dict(ldx=56), dict(ldx=68),
                dict(ldx=(1 << 22) + 8), dict(work=None), dict(work=P + 16), dict(saved=P + 16)):
        assert ffn_forward(lib, f, **bad) == moe.MOE_EINVAL, bad
        assert ffn_backward(lib, f, **bad) == moe.MOE_EINVAL, bad
    for bad in (dict(y=None), dict(y=P + 2), dict(ldy=0), dict(ldy=65)):
        assert ffn_forward(lib, f, **bad) == moe.MOE_EINVAL, bad
    for bad in (dict(dy=None), dict(lddy=60), dict(saved=None), dict(dx=P + 4), dict(lddx=63), dict(dwg=P + 8),
                dict(dwu=P + 8), dict(dwd=P + 8)):
        assert ffn_backward(lib, f, **bad) == moe.MOE_EINVAL, bad
    assert ffn_forward(lib, f, nwork=forward - 1) == moe.MOE_ESCRATCH
    assert ffn_forward(lib, f, nsaved=saved - 1) == moe.MOE_ESCRATCH
    assert ffn_backward(lib, f, nwork=backward - 1) == moe.MOE_ESCRATCH
    assert ffn_backward(lib, f, nsaved=saved - 1) == moe.MOE_ESCRATCH
    assert ffn_forward(lib, f, m=0, x=None, y=None, saved=None, work=None, nwork=0) == moe.MOE_OK


def norm(**kw):
    v = dict(dim=64, dtype=moe.MOE_BF16, eps=1e-6, res_scale=1.0, w_post=P, w_pre=P)
    v.update(kw)
    return moe.moe_norm(**v)


def norm_forward(lib, f, r=P, ldr=64, y=P, ldy=64, gate=None, kind=0, m=3, r_out=P, ldro=64, n=P, ldn=64, stats=P):
    return lib.moe_norm_forward(f, r, ldr, y, ldy, gate, kind, m, r_out, ldro, n, ldn, stats, None)


def norm_backward(lib, f, r=P, ldr=64, y=P, ldy=64, gate=None, kind=0, m=3, stats=P, do=P, lddo=64, dn=P, lddn=64, dr=P,
                  lddr=64, dy=P, lddy=64, dgate=None, dwp=P, dwn=P, work=P, nwork=1 << 30):
    return lib.moe_norm_backward(f, r, ldr, y, ldy, gate, kind, m, stats, do, lddo, dn, lddn, dr, lddr, dy, lddy, dgate,
                                 dwp, dwn, work, nwork, None)


@pytest.mark.parametrize("bad", [dict(dim=0), dict(dim=16385), dict(dtype=3), dict(dtype=-1), dict(eps=0.0), dict(eps=-1.0),
                                 dict(eps=NAN), dict(eps=INF), dict(res_scale=NAN), dict(res_scale=INF)])
def test_norm_descriptions_are_refused(lib, bad):
    f = ctypes.byref(norm(**bad))
    size = ctypes.c_size_t()
    assert lib.moe_norm_workspace(f, 3, ctypes.byref(size)) == moe.MOE_EINVAL
    assert norm_forward(lib, f) == moe.MOE_EINVAL
    assert norm_backward(lib, f) == moe.MOE_EINVAL


def test_norm_arguments_are_refused(lib):
    f, no_post, no_pre = (ctypes.byref(norm(**kw)) for kw in ({}, dict(w_post=None), dict(w_pre=None)))
    size = ctypes.c_size_t()
    assert lib.moe_norm_workspace(f, 3, ctypes.byref(size)) == moe.MOE_OK and size.value >= 64 * 4
    assert lib.moe_norm_workspace(f, -1, ctypes.byref(size)) == lib.moe_norm_workspace(f, 3, None) == moe.MOE_EINVAL
    for bad in (dict(m=-1), dict(r=None), dict(r=P + 1), dict(ldr=63), dict(y=None), dict(ldy=0), dict(kind=1),
                dict(kind=4, gate=P), dict(kind=-1), dict(gate=P), dict(gate=P + 1, kind=2), dict(gate=P + 1, kind=1),
                dict(stats=P + 2)):
        assert norm_forward(lib, f, **bad) == moe.MOE_EINVAL, bad
        assert norm_backward(lib, f, **bad) == moe.MOE_EINVAL, bad
    for bad in (dict(n=None), dict(ldro=63), dict(ldn=1), dict(n=P + 1)):
        assert norm_forward(lib, f, **bad) == moe.MOE_EINVAL, bad
    assert norm_forward(lib, no_pre) == moe.MOE_EINVAL                              # n without its weight
    assert norm_forward(lib, no_pre, n=None, r_out=None) == moe.MOE_EINVAL          # nothing to compute
    assert norm_forward(lib, no_post, y=None, gate=P, kind=1) == moe.MOE_EINVAL     # a gate of nothing
    for bad in (dict(do=None, dn=None), dict(stats=None), dict(dgate=P), dict(lddo=1), dict(lddn=1), dict(lddr=63),
                dict(lddy=63), dict(dwp=P + 1), dict(work=None), dict(work=P + 16)):
        assert norm_backward(lib, f, **bad) == moe.MOE_EINVAL, bad
    assert norm_backward(lib, f, nwork=16) == moe.MOE_ESCRATCH
    assert norm_backward(lib, no_pre, dn=None) == norm_backward(lib, no_pre, dwn=None) == moe.MOE_EINVAL
    assert norm_backward(lib, no_post) == moe.MOE_EINVAL
    assert norm_backward(lib, no_post, y=None, dwp=None) == moe.MOE_EINVAL          # dy of no y
    assert norm_forward(lib, f, m=0, r=None, y=None, r_out=None, n=None) == moe.MOE_OK


@pytest.mark.parametrize("dim,inter", [(8, 8), (64, 128), (1544, 4104), (5120, 2304), (8192, 2048), (16384, 16384)])
def test_workspaces_fit_fewer_rows(lib, dim, inter):
    # what is enough for m rows is enough for any fewer: a program sizes its workspace once, for its largest batch
    f, n, size = ctypes.byref(ffn(dim=dim, inter=inter)), ctypes.byref(norm(dim=dim)), ctypes.c_size_t()
    rows = sorted({*range(0, 300), *range(300, 9000, 37), 1000, 1536, 8192, 1 << 20, 1 << 24})
    last = (0, 0, 0, 0)
    for m in rows:
        rc, *sizes = ffn_sizes(lib, f, m)
        assert rc == moe.MOE_OK and lib.moe_norm_workspace(n, m, ctypes.byref(size)) == moe.MOE_OK
        sizes.append(size.value)
        assert all(a <= b and b % 256 == 0 for a, b in zip(last, sizes)), m
        last = sizes


def w4(**kw):
    v = dict(rows=48, cols=256, group=64, dtype=moe.MOE_BF16, codes=P, scales=P, zeros=None)
    v.update(kw)
    return moe.moe_w4(**v)


@pytest.mark.parametrize("bad", [dict(rows=0), dict(rows=(1 << 22) + 1), dict(cols=0), dict(cols=96), dict(cols=65600),
                                 dict(group=16), dict(group=0), dict(group=256), dict(dtype=moe.MOE_F32), dict(codes=None),
                                 dict(codes=P + 8), dict(scales=None), dict(scales=P + 1)])
def test_w4_descriptions_are_refused(lib, bad):
    w, good = ctypes.byref(w4(**bad)), ctypes.byref(w4())
    assert lib.moe_w4_matmul(w, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    assert lib.moe_w4_gated(w, good, 0, 0.0, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    assert lib.moe_w4_gated(good, w, 0, 0.0, P, 256, 3, P, 48, None) == moe.MOE_EINVAL


def test_w4_arguments_are_refused(lib):
    w = ctypes.byref(w4())
    assert lib.moe_w4_matmul(None, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    for x, ldx, m, y, ldy in ((None, 256, 3, P, 48), (P + 8, 256, 3, P, 48), (P, 248, 3, P, 48), (P, 260, 3, P, 48),
                              (P, (1 << 24) + 8, 3, P, 48), (P, 256, -1, P, 48), (P, 256, 3, None, 48), (P, 256, 3, P + 1, 48),
                              (P, 256, 3, P, 47), (P, 256, 64 * 65535 + 1, P, 48)):
        assert lib.moe_w4_matmul(w, x, ldx, m, y, ldy, None) == moe.MOE_EINVAL
        assert lib.moe_w4_gated(w, w, 0, 0.0, x, ldx, m, y, ldy, None) == moe.MOE_EINVAL
    for other in (dict(rows=32), dict(cols=128), dict(group=32), dict(dtype=moe.MOE_F16), dict(zeros=P)):
        assert lib.moe_w4_gated(w, ctypes.byref(w4(**other)), 0, 0.0, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    assert lib.moe_w4_gated(w, w, 2, 0.0, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    assert lib.moe_w4_gated(w, w, 0, NAN, P, 256, 3, P, 48, None) == moe.MOE_EINVAL
    assert lib.moe_w4_matmul(w, None, 256, 0, None, 48, None) == moe.MOE_OK


def test_binding_refuses_tensors_of_the_host():
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    for call in (lambda: moe.make_ffn(w, w, w), lambda: moe.make_norm(8, torch.bfloat16, w_pre=w[0]),
                 lambda: moe.make_norm(8, torch.int32), lambda: moe.make_ffn(w, w, w, act="relu"),
                 lambda: moe.make_w4(torch.zeros(8, 16, dtype=torch.uint8), w[:, :1])):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_EINVAL
