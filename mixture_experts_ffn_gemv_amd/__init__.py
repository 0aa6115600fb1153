"""Python binding of libmoe (include/moe.h): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
plain pointers and sizes; tensors are torch tensors on the current HIP device
(PyTorch supplies memory and streams, nothing else). Every step of the layer
runs in the HIP kernels of libmoe.so; if the library is not built this module
raises on first use instead of falling back to anything.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_EINVAL = -1
MOE_ENOMEM = -2
MOE_EHIP = -3
MOE_ENONFINITE = -4
MOE_ENOTRESIDENT = -5
MOE_ESTATE = -6
MOE_ESCRATCH = -7

MOE_SHARED_NONE = 0
MOE_SHARED_BF16 = 1
MOE_SHARED_KQUANT = 2

MOE_EXPERT_KQUANT = 0
MOE_EXPERT_MXFP4 = 1

MOE_DISPATCH_MMQ = 0
MOE_DISPATCH_MIXED = 1

MOE_PATH_DECODE = 0
MOE_PATH_GEMV = 1
MOE_PATH_MMQ = 2

MOE_STATIC_SCRATCH_BYTES = 8 << 20

MOE_BF16 = 0
MOE_F16 = 1
MOE_F32 = 2

MOE_ACT_SILU = 0
MOE_ACT_GELU = 1
MOE_ACT_NONE = 2

MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_GATE_FULL = 3

EXPORTED = (
    "moe_create", "moe_destroy", "moe_expert_layout", "moe_pack_expert", "moe_set_slots", "moe_slot_bind",
    "moe_slot_evict",
    "moe_slot_of", "moe_set_host_arena", "moe_route", "moe_forward", "moe_forward_ex", "moe_check",
    "moe_get_stats", "moe_reset_stats", "moe_strerror", "moe_quantize_q8_1", "moe_set_profiling",
    "moe_kernel_times", "moe_set_dispatch", "moe_plan_call", "moe_forward_static",
    "moe_ffn_workspace", "moe_ffn_forward", "moe_ffn_backward",
    "moe_norm_workspace", "moe_norm_forward", "moe_norm_backward",
    "moe_w4_matmul", "moe_w4_gated",
    "moe_sort_workspace", "moe_sort", "moe_dispatch_forward", "moe_dispatch_backward",
    "moe_combine_forward", "moe_combine_backward",
    "moe_linear_workspace", "moe_linear_forward", "moe_linear_backward",
    "moe_dropout_forward", "moe_dropout_backward",
)

KERNEL_CLASSES = ("router", "quant_h", "topk", "bucket", "gateup", "shared_gateup", "down", "shared_down",
                  "combine")


class moe_cfg(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("n_routed", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("gate_temp", ctypes.c_float),
        ("norm_topk_prob", ctypes.c_int32),
        ("route_scale", ctypes.c_float),
        ("swiglu_limit", ctypes.c_float),
        ("max_tokens", ctypes.c_int32),
        ("expert_fmt", ctypes.c_int32),
    ]


class moe_weights(ctypes.Structure):
    _fields_ = [
        ("router_w", ctypes.c_void_p),
        ("router_bias", ctypes.c_void_p),
        ("shared_fmt", ctypes.c_int32),
        ("shared_w1", ctypes.c_void_p),
        ("shared_w3", ctypes.c_void_p),
        ("shared_w2", ctypes.c_void_p),
    ]


class moe_stats(ctypes.Structure):
    _fields_ = [
        ("calls", ctypes.c_uint64),
        ("hits", ctypes.c_uint64),
        ("misses", ctypes.c_uint64),
        ("bytes_copied", ctypes.c_uint64),
        ("waves", ctypes.c_uint64),
        ("route_ms", ctypes.c_double),
        ("fetch_ms", ctypes.c_double),
        ("compute_ms", ctypes.c_double),
        ("near_ties", ctypes.c_uint64),
    ]


class moe_plan(ctypes.Structure):
    _fields_ = [
        ("small_routing", ctypes.c_int32),
        ("expert_path", ctypes.c_int32),
        ("shared_rows_router", ctypes.c_int32),
        ("shared_rows_topk", ctypes.c_int32),
        ("shared_rows_gateup", ctypes.c_int32),
    ]


class moe_ffn(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("limit", ctypes.c_float),
        ("w_gate", ctypes.c_void_p),
        ("w_up", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p),
    ]


class moe_norm(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("res_scale", ctypes.c_float),
        ("w_post", ctypes.c_void_p),
        ("w_pre", ctypes.c_void_p),
    ]


class moe_w4(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("zeros", ctypes.c_void_p),
    ]


class moe_linear(ctypes.Structure):
    _fields_ = [
        ("cols", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("experts", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("w", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
    ]


class moe_dropout(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("p", ctypes.c_double),
    ]


class MoeError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


_lib = None


def lib():
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        sigs = {
            "moe_create": [P(moe_cfg), P(vp)],
            "moe_destroy": [vp],
            "moe_expert_layout": [P(moe_cfg), P(sz), P(sz), P(sz), P(sz)],
            "moe_pack_expert": [P(moe_cfg), vp, vp, vp],
            "moe_set_slots": [vp, vp, i32],
            "moe_slot_bind": [vp, i32, i32],
            "moe_slot_evict": [vp, i32],
            "moe_slot_of": [vp, i32, P(i32)],
            "moe_set_host_arena": [vp, vp, sz],
            "moe_route": [vp, P(moe_weights), vp, i32, vp, vp, vp],
            "moe_forward": [vp, P(moe_weights), vp, i32, vp, vp],
            "moe_forward_ex": [vp, P(moe_weights), vp, i32, vp, vp, vp, vp],
            "moe_check": [vp, vp],
            "moe_get_stats": [vp, P(moe_stats)],
            "moe_reset_stats": [vp],
            "moe_quantize_q8_1": [vp, i32, i32, vp, vp, vp],
            "moe_set_profiling": [vp, i32],
            "moe_set_dispatch": [vp, i32],
            "moe_kernel_times": [vp, P(ctypes.c_double), P(ctypes.c_int64), i32],
            "moe_plan_call": [vp, i32, i32, P(moe_plan)],
            "moe_forward_static": [P(moe_cfg), P(moe_weights), vp, vp, vp, i32, vp, vp, vp, vp, vp],
            "moe_ffn_workspace": [P(moe_ffn), i32, P(sz), P(sz), P(sz)],
            "moe_ffn_forward": [P(moe_ffn), vp, i64, i32, vp, i64, vp, sz, vp, sz, vp],
            "moe_ffn_backward": [P(moe_ffn), vp, i64, vp, i64, i32, vp, sz, vp, i64, vp, vp, vp, vp, sz, vp],
            "moe_norm_workspace": [P(moe_norm), i32, P(sz)],
            "moe_norm_forward": [P(moe_norm), vp, i64, vp, i64, vp, i32, i32, vp, i64, vp, i64, vp, vp],
            "moe_norm_backward": [P(moe_norm), vp, i64, vp, i64, vp, i32, i32, vp, vp, i64, vp, i64, vp, i64, vp, i64,
                                  vp, vp, vp, vp, sz, vp],
            "moe_w4_matmul": [P(moe_w4), vp, i64, i32, vp, i64, vp],
            "moe_w4_gated": [P(moe_w4), P(moe_w4), i32, ctypes.c_float, vp, i64, i32, vp, i64, vp],
            "moe_sort_workspace": [i32, i32, i32, P(sz)],
            "moe_sort": [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp],
            "moe_dispatch_forward": [i32, i32, vp, i64, vp, i32, i32, vp, i64, i32, vp],
            "moe_dispatch_backward": [i32, i32, vp, i64, i32, vp, i32, i32, vp, i64, vp],
            "moe_combine_forward": [i32, i32, vp, i64, i32, vp, vp, i32, i32, vp, i64, vp],
            "moe_combine_backward": [i32, i32, vp, i64, vp, i64, i32, vp, vp, i32, i32, vp, i64, vp, vp],
            "moe_linear_workspace": [P(moe_linear), i32, P(sz), P(sz), P(sz)],
            "moe_linear_forward": [P(moe_linear), vp, i64, vp, i32, vp, i64, vp, i64, vp, sz, vp, sz, vp],
            "moe_linear_backward": [P(moe_linear), vp, i64, vp, i32, vp, i64, vp, sz, vp, i64, vp, vp, vp, sz, vp],
            "moe_dropout_forward": [P(moe_dropout), vp, vp, i64, vp, i64, i32, vp, i64, vp],
            "moe_dropout_backward": [P(moe_dropout), vp, vp, i64, i32, vp, i64, vp],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_strerror.argtypes = [ctypes.c_int]
        L.moe_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(code):
    return lib().moe_strerror(code).decode()


def _check(rc, where):
    if rc != MOE_OK:
        raise MoeError(rc, where)
    return rc


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without a Stream object around it (0.3 against 2.6 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def make_cfg(dim, inter, n_routed, topk, gate_temp=1.0, norm_topk_prob=True, route_scale=1.5,
             swiglu_limit=10.0, max_tokens=1, expert_fmt=MOE_EXPERT_KQUANT):
    return moe_cfg(dim, inter, n_routed, topk, gate_temp, int(bool(norm_topk_prob)), route_scale,
                   swiglu_limit, max_tokens, expert_fmt)


def make_weights(router_w, router_bias, shared_fmt=MOE_SHARED_NONE, shared_w1=None, shared_w3=None,
                 shared_w2=None):
    return moe_weights(_ptr(router_w), _ptr(router_bias), shared_fmt, _ptr(shared_w1), _ptr(shared_w3),
                       _ptr(shared_w2))


# ----------------------------------------------------------------------------- entry points

def moe_create(cfg):
    ctx = ctypes.c_void_p()
    _check(lib().moe_create(ctypes.byref(cfg), ctypes.byref(ctx)), "moe_create")
    return ctx


def moe_destroy(ctx):
    return _check(lib().moe_destroy(ctx), "moe_destroy")


def moe_expert_layout(cfg):
    """-> (slot_bytes, off_w1, off_w3, off_w2)"""
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().moe_expert_layout(ctypes.byref(cfg), *[ctypes.byref(o) for o in out]), "moe_expert_layout")
    return tuple(o.value for o in out)


def moe_pack_expert(cfg, src, dst, stream=None):
    return _check(lib().moe_pack_expert(ctypes.byref(cfg), _ptr(src), _ptr(dst), _stream(stream)), "moe_pack_expert")


def pack_experts(cfg, arena, stream=None):
    """Expert slices in plain GGUF row order, uint8 [n, slot_bytes] on the
    device -> a new tensor of the same shape in the slot layout."""
    out = torch.empty_like(arena)
    for e in range(arena.shape[0]):
        moe_pack_expert(cfg, arena[e], out[e], stream)
    return out


def moe_set_slots(ctx, arena, n_slots):
    return _check(lib().moe_set_slots(ctx, _ptr(arena), n_slots), "moe_set_slots")


def moe_slot_bind(ctx, expert, slot):
    return _check(lib().moe_slot_bind(ctx, expert, slot), "moe_slot_bind")


def moe_slot_evict(ctx, expert):
    return _check(lib().moe_slot_evict(ctx, expert), "moe_slot_evict")


def moe_slot_of(ctx, expert):
    s = ctypes.c_int32()
    _check(lib().moe_slot_of(ctx, expert, ctypes.byref(s)), "moe_slot_of")
    return s.value


def moe_set_host_arena(ctx, pinned, stride):
    return _check(lib().moe_set_host_arena(ctx, _ptr(pinned), stride), "moe_set_host_arena")


def moe_route(ctx, w, x, m, weights_out, idx_out, stream=None):
    return _check(lib().moe_route(ctx, ctypes.byref(w), _ptr(x), m, _ptr(weights_out), _ptr(idx_out),
                                  _stream(stream)), "moe_route")


def moe_forward(ctx, w, x, m, out, stream=None):
    return _check(lib().moe_forward(ctx, ctypes.byref(w), _ptr(x), m, _ptr(out), _stream(stream)), "moe_forward")


def moe_forward_ex(ctx, w, x, m, out, weights_out=None, idx_out=None, stream=None):
    return _check(lib().moe_forward_ex(ctx, ctypes.byref(w), _ptr(x), m, _ptr(out), _ptr(weights_out),
                                       _ptr(idx_out), _stream(stream)), "moe_forward_ex")


def moe_plan_call(ctx, m, shared_fmt):
    """-> dict of the moe_plan fields for a call of m tokens."""
    p = moe_plan()
    _check(lib().moe_plan_call(ctx, m, shared_fmt, ctypes.byref(p)), "moe_plan_call")
    return {f: getattr(p, f) for f, _ in moe_plan._fields_}


def moe_forward_static(cfg, w, arena, slot_table, x, m, out, weights_out=None, idx_out=None, status=None,
                       stream=None):
    return _check(lib().moe_forward_static(ctypes.byref(cfg), ctypes.byref(w), _ptr(arena), _ptr(slot_table),
                                           _ptr(x), m, _ptr(out), _ptr(weights_out), _ptr(idx_out), _ptr(status),
                                           _stream(stream)), "moe_forward_static")


def moe_quantize_q8_1(x, rows, cols, q_out, d_out, stream=None):
    return _check(lib().moe_quantize_q8_1(_ptr(x), rows, cols, _ptr(q_out), _ptr(d_out), _stream(stream)),
                  "moe_quantize_q8_1")


def moe_check(ctx, stream=None):
    """Synchronise and return the device status code (does not raise)."""
    return lib().moe_check(ctx, _stream(stream))


def moe_set_dispatch(ctx, mode):
    """MOE_DISPATCH_MMQ (the default) or MOE_DISPATCH_MIXED (GEMVs for groups of <= 8 rows, MMQ above)."""
    return _check(lib().moe_set_dispatch(ctx, int(mode)), "moe_set_dispatch")


def moe_set_profiling(ctx, on):
    return _check(lib().moe_set_profiling(ctx, int(bool(on))), "moe_set_profiling")


def moe_kernel_times(ctx):
    """-> {kernel class: (summed ms, launches)} since profiling was switched on or last read."""
    n = len(KERNEL_CLASSES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(lib().moe_kernel_times(ctx, ms, cnt, n), "moe_kernel_times")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_CLASSES)}


def moe_get_stats(ctx):
    s = moe_stats()
    _check(lib().moe_get_stats(ctx, ctypes.byref(s)), "moe_get_stats")
    return {f: getattr(s, f) for f, _ in moe_stats._fields_}


def moe_reset_stats(ctx):
    return _check(lib().moe_reset_stats(ctx), "moe_reset_stats")


# ----------------------------------------------------------------------------- operators around the layer
#
# Tensors are checked here for what C cannot see (device, type, shape, rows whose
# values are consecutive); everything else is checked by the entry point.

_DTYPES = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32}
_ACTS = {"silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}


_MOST = 2 ** 31 - 1   # sizes are 32 bits in C, and ctypes would cut off what is above them


def _small(where, *sizes):
    if max(sizes) > _MOST:
        raise MoeError(MOE_EINVAL, where)


def _dtype(t, where):
    if t not in _DTYPES:
        raise MoeError(MOE_EINVAL, where)
    return _DTYPES[t]


def _act(act, where):
    act = _ACTS.get(act, act)
    if act not in (MOE_ACT_SILU, MOE_ACT_GELU):
        raise MoeError(MOE_EINVAL, where)
    return act


def _rows(t, m, dim, dtype, where):
    """A device matrix [m, dim] with consecutive values in each row -> (pointer, row stride); None -> (None, 0)."""
    if t is None:
        return None, 0
    if t.shape != (m, dim) or t.dtype is not dtype or not t.is_cuda or m > _MOST:
        raise MoeError(MOE_EINVAL, where)
    ld, one = t.stride()
    if one != 1 and dim != 1:
        raise MoeError(MOE_EINVAL, where)
    return t.data_ptr(), ld if m > 1 else dim   # (one row: its stride leads nowhere)


def _whole(t, shape, dtype, where):
    """A contiguous device tensor of that shape and type -> its pointer; None -> None."""
    if t is None:
        return None
    if not t.is_cuda or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise MoeError(MOE_EINVAL, where)
    return t.data_ptr()


def _bytes(t, where):
    """A workspace -> (pointer, bytes); None -> (None, 0)."""
    if t is None:
        return None, 0
    if not t.is_cuda or not t.is_contiguous():
        raise MoeError(MOE_EINVAL, where)
    return t.data_ptr(), t.numel() * t.element_size()


def make_ffn(w_gate, w_up, w_down, act="silu", limit=0.0):
    """Describe a dense gated feed-forward block: w_gate, w_up [inter, dim], w_down [dim, inter]
    (kept alive by the result); act "silu" or "gelu"; limit <= 0: no clamps."""
    if w_gate.dim() != 2:
        raise MoeError(MOE_EINVAL, "make_ffn")
    inter, dim = w_gate.shape
    _small("make_ffn", inter, dim)
    dt = w_gate.dtype
    f = moe_ffn(dim, inter, _dtype(dt, "make_ffn"), _act(act, "make_ffn"), limit,
                _whole(w_gate, (inter, dim), dt, "make_ffn"), _whole(w_up, (inter, dim), dt, "make_ffn"),
                _whole(w_down, (dim, inter), dt, "make_ffn"))
    f.torch_dtype, f.tensors = dt, (w_gate, w_up, w_down)
    return f


def moe_ffn_workspace(f, m):
    """-> (forward, saved, backward) bytes for m rows."""
    _small("moe_ffn_workspace", m)
    out = [ctypes.c_size_t() for _ in range(3)]
    _check(lib().moe_ffn_workspace(ctypes.byref(f), m, *[ctypes.byref(o) for o in out]), "moe_ffn_workspace")
    return tuple(o.value for o in out)


def moe_ffn_forward(f, x, y, work, saved=None, stream=None):
    """y = block(x), x and y [m, dim]; saved: what moe_ffn_backward takes."""
    me, m, dt = "moe_ffn_forward", x.shape[0], f.torch_dtype
    return _check(lib().moe_ffn_forward(ctypes.byref(f), *_rows(x, m, f.dim, dt, me), m, *_rows(y, m, f.dim, dt, me),
                                        *_bytes(saved, me), *_bytes(work, me), _stream(stream)), me)


def moe_ffn_backward(f, x, dy, saved, work, dx=None, dw_gate=None, dw_up=None, dw_down=None, stream=None):
    """Gradients of the block into the tensors that are given."""
    me, m, dt = "moe_ffn_backward", x.shape[0], f.torch_dtype
    wide = (f.inter, f.dim)
    return _check(lib().moe_ffn_backward(
        ctypes.byref(f), *_rows(x, m, f.dim, dt, me), *_rows(dy, m, f.dim, dt, me), m, *_bytes(saved, me),
        *_rows(dx, m, f.dim, dt, me), _whole(dw_gate, wide, dt, me), _whole(dw_up, wide, dt, me),
        _whole(dw_down, (f.dim, f.inter), dt, me), *_bytes(work, me), _stream(stream)), me)


def make_norm(dim, dtype, w_post=None, w_pre=None, eps=1e-6, res_scale=1.0):
    """Describe the norms around a block: w_post and w_pre [dim] or None (kept alive by the result)."""
    _small("make_norm", dim)
    f = moe_norm(dim, _dtype(dtype, "make_norm"), eps, res_scale, _whole(w_post, (dim,), dtype, "make_norm"),
                 _whole(w_pre, (dim,), dtype, "make_norm"))
    f.torch_dtype, f.tensors = dtype, (w_post, w_pre)
    return f


def moe_norm_workspace(f, m):
    """-> workspace bytes of moe_norm_backward for m rows."""
    _small("moe_norm_workspace", m)
    out = ctypes.c_size_t()
    _check(lib().moe_norm_workspace(ctypes.byref(f), m, ctypes.byref(out)), "moe_norm_workspace")
    return out.value


def _gate(gate, m, dim, dtype, where):
    """-> (pointer, MOE_GATE_*) of a gate [dim] (per channel), [m, 1] (per token) or [m, dim]."""
    if gate is None:
        return None, MOE_GATE_NONE
    shape = tuple(gate.shape)
    kind = {(m, 1): MOE_GATE_TOKEN, (m, dim): MOE_GATE_FULL, (dim,): MOE_GATE_CHANNEL}.get(shape)
    if kind is None:
        raise MoeError(MOE_EINVAL, where)
    return _whole(gate, shape, dtype, where), kind


def moe_norm_forward(f, r, y, r_out, n, gate=None, stats=None, stream=None):
    """r_out = res_scale r + gate norm(y), n = norm(r_out). gate [dim] (per channel), [m, 1] (per token)
    or [m, dim]. y, r_out and n may be None as moe.h says."""
    me, m, dt, d = "moe_norm_forward", r.shape[0], f.torch_dtype, f.dim
    return _check(lib().moe_norm_forward(
        ctypes.byref(f), *_rows(r, m, d, dt, me), *_rows(y, m, d, dt, me), *_gate(gate, m, d, dt, me), m,
        *_rows(r_out, m, d, dt, me), *_rows(n, m, d, dt, me), _whole(stats, (m, 2), torch.float32, me),
        _stream(stream)), me)


def moe_norm_backward(f, r, y, stats, dr_out, dn, work, gate=None, dr=None, dy=None, dgate=None, dw_post=None,
                      dw_pre=None, stream=None):
    """Gradients of moe_norm_forward into the tensors that are given."""
    me, m, dt, d = "moe_norm_backward", r.shape[0], f.torch_dtype, f.dim
    if dgate is not None and (gate is None or dgate.shape != gate.shape):
        raise MoeError(MOE_EINVAL, me)
    return _check(lib().moe_norm_backward(
        ctypes.byref(f), *_rows(r, m, d, dt, me), *_rows(y, m, d, dt, me), *_gate(gate, m, d, dt, me), m,
        _whole(stats, (m, 2), torch.float32, me), *_rows(dr_out, m, d, dt, me), *_rows(dn, m, d, dt, me),
        *_rows(dr, m, d, dt, me), *_rows(dy, m, d, dt, me), _gate(dgate, m, d, dt, me)[0],
        _whole(dw_post, (d,), dt, me), _whole(dw_pre, (d,), dt, me), *_bytes(work, me), _stream(stream)), me)


def make_w4(codes, scales, zeros=None, group=None):
    """Describe a matrix of 4-bit weights: codes uint8 [rows, cols / 2], scales [rows, cols / group] (bf16 or
    f16), zeros uint8 [rows, cols / group] or None (kept alive by the result)."""
    me = "make_w4"
    if codes.dim() != 2 or scales.dim() != 2 or not scales.shape[1]:
        raise MoeError(MOE_EINVAL, me)
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    _small(me, rows, cols)
    group = cols // scales.shape[1] if group is None else group
    if group <= 0 or cols % group:
        raise MoeError(MOE_EINVAL, me)
    shape = (rows, cols // group)
    w = moe_w4(rows, cols, group, _dtype(scales.dtype, me), _whole(codes, (rows, cols // 2), torch.uint8, me),
               _whole(scales, shape, scales.dtype, me), _whole(zeros, shape, torch.uint8, me))
    w.torch_dtype, w.tensors = scales.dtype, (codes, scales, zeros)
    return w


def moe_w4_matmul(w, x, y, stream=None):
    """y [m, rows] = x [m, cols] W^T."""
    me, m, dt = "moe_w4_matmul", x.shape[0], w.torch_dtype
    return _check(lib().moe_w4_matmul(ctypes.byref(w), *_rows(x, m, w.cols, dt, me), m, *_rows(y, m, w.rows, dt, me),
                                      _stream(stream)), me)


def moe_w4_gated(w_gate, w_up, x, h, act="silu", limit=0.0, stream=None):
    """h [m, rows] = act(x Wg^T) * (x Wu^T), clamped as in make_ffn."""
    me, m, dt = "moe_w4_gated", x.shape[0], w_gate.torch_dtype
    return _check(lib().moe_w4_gated(ctypes.byref(w_gate), ctypes.byref(w_up), _act(act, me), limit,
                                     *_rows(x, m, w_gate.cols, dt, me), m, *_rows(h, m, w_gate.rows, dt, me),
                                     _stream(stream)), me)


_several = None   # whether there are devices that a tensor could be on but the current one


def _stream_of(stream, where, *tensors):
    """The stream of a call on these tensors (None among them: not given). Their device has to be the current one."""
    global _several
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if _several:
        here = torch.cuda.current_device()
        if any(t is not None and t.get_device() != here for t in tensors):
            raise MoeError(MOE_EINVAL, where)
    return _stream(stream)


def _any_rows(t, dtype, where):
    """A device matrix of that type with consecutive values in each row -> (pointer, row stride, rows, values of a row)."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 2 or not t.is_cuda:
        raise MoeError(MOE_EINVAL, where)
    m, dim = shape
    ld, one = t.stride()
    if (one != 1 and dim != 1) or m > _MOST or dim > _MOST:
        raise MoeError(MOE_EINVAL, where)
    return t.data_ptr(), ld if m > 1 else dim, m, dim   # (one row: its stride leads nowhere)


def _picks(t, where):
    """A contiguous int32 device matrix [m, topk] -> (pointer, m, topk)."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 2 or not t.is_cuda or not t.is_contiguous():
        raise MoeError(MOE_EINVAL, where)
    m, topk = shape
    if m > _MOST or topk > _MOST:
        raise MoeError(MOE_EINVAL, where)
    return t.data_ptr(), m, topk


def moe_sort_workspace(m, topk, n_experts):
    """-> the bytes that moe_sort works in."""
    _small("moe_sort_workspace", m, topk, n_experts)
    size = ctypes.c_size_t()
    _check(lib().moe_sort_workspace(m, topk, n_experts, ctypes.byref(size)), "moe_sort_workspace")
    return size.value


def moe_sort(idx, n_experts, row_of, pick_of, offsets, work, stream=None):
    """The order by expert of the picks idx int32 [m, topk]: row_of [m, topk], pick_of [m * topk] (or None) and
    offsets [n_experts + 1], all int32."""
    me = "moe_sort"
    picks, m, topk = _picks(idx, me)
    if n_experts > _MOST:
        raise MoeError(MOE_EINVAL, me)
    return _check(lib().moe_sort(
        picks, m, topk, n_experts, _whole(row_of, (m, topk), torch.int32, me), _whole(pick_of, (m * topk,), torch.int32, me),
        _whole(offsets, (n_experts + 1,), torch.int32, me), *_bytes(work, me),
        _stream_of(stream, me, idx, row_of, pick_of, offsets, work)), me)


def _moved(tokens, sorted_rows, row_of, where):
    """Token rows [m, dim], sorted rows [rows, dim] and row_of [m, topk] of one call -> their pointers and sizes."""
    at, m, topk = _picks(row_of, where)
    dt = tokens.dtype
    if dt not in _DTYPES:
        raise MoeError(MOE_EINVAL, where)
    t, ldt, n, dim = _any_rows(tokens, dt, where)
    s, lds, rows, width = _any_rows(sorted_rows, dt, where)
    if n != m or width != dim:
        raise MoeError(MOE_EINVAL, where)
    return _DTYPES[dt], dim, t, ldt, s, lds, rows, at, m, topk


def moe_dispatch_forward(x, row_of, xs, stream=None):
    """xs[row_of[t, j]] = x[t]: x [m, dim], row_of [m, topk], xs [rows, dim]."""
    me = "moe_dispatch_forward"
    dt, dim, x_, ldx, xs_, ldxs, rows, at, m, topk = _moved(x, xs, row_of, me)
    return _check(lib().moe_dispatch_forward(dt, dim, x_, ldx, at, m, topk, xs_, ldxs, rows,
                                             _stream_of(stream, me, x, row_of, xs)), me)


def moe_dispatch_backward(dxs, row_of, dx, stream=None):
    """dx[t] = sum over j of dxs[row_of[t, j]]."""
    me = "moe_dispatch_backward"
    dt, dim, dx_, lddx, dxs_, lddxs, rows, at, m, topk = _moved(dx, dxs, row_of, me)
    return _check(lib().moe_dispatch_backward(dt, dim, dxs_, lddxs, rows, at, m, topk, dx_, lddx,
                                              _stream_of(stream, me, dxs, row_of, dx)), me)


def moe_combine_forward(e, weights, row_of, y, stream=None):
    """y[t] = sum over j of weights[t, j] e[row_of[t, j]]: e [rows, dim], weights f32 [m, topk], y [m, dim]."""
    me = "moe_combine_forward"
    dt, dim, y_, ldy, e_, lde, rows, at, m, topk = _moved(y, e, row_of, me)
    return _check(lib().moe_combine_forward(dt, dim, e_, lde, rows, _whole(weights, (m, topk), torch.float32, me), at, m, topk, y_, ldy,
                                            _stream_of(stream, me, e, weights, row_of, y)), me)


def moe_combine_backward(dy, e, weights, row_of, de=None, dweights=None, stream=None):
    """Gradients of moe_combine_forward into the tensors that are given."""
    me = "moe_combine_backward"
    dt, dim, dy_, lddy, e_, lde, rows, at, m, topk = _moved(dy, e, row_of, me)
    return _check(lib().moe_combine_backward(
        dt, dim, dy_, lddy, e_, lde, rows, _whole(weights, (m, topk), torch.float32, me), at, m, topk, *_rows(de, rows, dim, dy.dtype, me),
        _whole(dweights, (m, topk), torch.float32, me), _stream_of(stream, me, dy, e, weights, row_of, de, dweights)), me)


_LINEAR_ACTS = {**_ACTS, "none": MOE_ACT_NONE, None: MOE_ACT_NONE}


def make_linear(w, bias=None, act="none"):
    """Describe a product with bias and activation: w [rows, cols] and bias [rows], or a matrix per expert, w [experts,
    rows, cols] and bias [experts, rows] (kept alive by the result); act "none", "silu" or "gelu"."""
    me = "make_linear"
    if w.dim() not in (2, 3):
        raise MoeError(MOE_EINVAL, me)
    rows, cols = w.shape[-2:]
    experts, dt = w.shape[0] if w.dim() == 3 else 1, w.dtype
    _small(me, rows, cols, experts)
    act = _LINEAR_ACTS.get(act, act)
    if act not in (MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_NONE):
        raise MoeError(MOE_EINVAL, me)
    f = moe_linear(cols, rows, experts, _dtype(dt, me), act, _whole(w, w.shape, dt, me), _whole(bias, w.shape[:-1], dt, me))
    f.torch_dtype, f.tensors = dt, (w, bias)
    return f


def moe_linear_workspace(f, m):
    """-> (forward, saved, backward) bytes for m rows."""
    _small("moe_linear_workspace", m)
    out = [ctypes.c_size_t() for _ in range(3)]
    _check(lib().moe_linear_workspace(ctypes.byref(f), m, *[ctypes.byref(o) for o in out]), "moe_linear_workspace")
    return tuple(o.value for o in out)


def moe_linear_forward(f, x, y, work, offsets=None, residual=None, saved=None, stream=None):
    """y = act(x W^T + bias) + residual, x [m, cols], y and residual [m, rows]; offsets int32 [experts + 1]: the rows of
    each expert; saved: what moe_linear_backward takes."""
    me, m, dt = "moe_linear_forward", x.shape[0], f.torch_dtype
    return _check(lib().moe_linear_forward(
        ctypes.byref(f), *_rows(x, m, f.cols, dt, me), _whole(offsets, (f.experts + 1,), torch.int32, me), m,
        *_rows(residual, m, f.rows, dt, me), *_rows(y, m, f.rows, dt, me), *_bytes(saved, me), *_bytes(work, me),
        _stream_of(stream, me, *f.tensors, x, y, work, offsets, residual, saved)), me)


def moe_linear_backward(f, x, dy, saved, work, offsets=None, dx=None, dw=None, dbias=None, stream=None):
    """Gradients of moe_linear_forward into the tensors that are given; dw and dbias have the shapes of w and bias."""
    me, m, dt = "moe_linear_backward", x.shape[0], f.torch_dtype
    w, bias = f.tensors
    return _check(lib().moe_linear_backward(
        ctypes.byref(f), *_rows(x, m, f.cols, dt, me), _whole(offsets, (f.experts + 1,), torch.int32, me), m,
        *_rows(dy, m, f.rows, dt, me), *_bytes(saved, me), *_rows(dx, m, f.cols, dt, me), _whole(dw, w.shape, dt, me),
        _whole(dbias, w.shape[:-1], dt, me), *_bytes(work, me),
        _stream_of(stream, me, *f.tensors, x, dy, saved, work, offsets, dx, dw, dbias)), me)


def make_dropout(dim, dtype, p):
    """Describe dropout of rows of dim values of that type with probability p."""
    _small("make_dropout", dim)
    f = moe_dropout(dim, _dtype(dtype, "make_dropout"), p)
    f.torch_dtype = dtype
    return f


def moe_dropout_forward(f, rng, x, y, residual=None, stream=None):
    """y = residual + keep x / (1 - p); rng int64 [2]: seed and use, on the device."""
    me, m, dt = "moe_dropout_forward", x.shape[0], f.torch_dtype
    return _check(lib().moe_dropout_forward(
        ctypes.byref(f), _whole(rng, (2,), torch.int64, me), *_rows(x, m, f.dim, dt, me), *_rows(residual, m, f.dim, dt, me), m,
        *_rows(y, m, f.dim, dt, me), _stream_of(stream, me, rng, x, y, residual)), me)


def moe_dropout_backward(f, rng, dy, dx, stream=None):
    """dx = keep dy / (1 - p) with the mask of the forward call."""
    me, m, dt = "moe_dropout_backward", dy.shape[0], f.torch_dtype
    return _check(lib().moe_dropout_backward(ctypes.byref(f), _whole(rng, (2,), torch.int64, me), *_rows(dy, m, f.dim, dt, me), m,
                                             *_rows(dx, m, f.dim, dt, me), _stream_of(stream, me, rng, dy, dx)), me)
