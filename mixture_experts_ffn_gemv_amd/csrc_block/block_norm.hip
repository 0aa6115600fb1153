// The norm after a block, its gate, the scaled residual and the norm before the
// next block, forward and backward (moe_norm_* in include/moe.h).
//
// A row lives in the registers of the threads that own it from its first load to
// its last store, so each array passes through memory once in each direction. A
// thread holds C chunks of V consecutive values (16-byte chunks where pointers and
// strides allow it, else V = 1); chunk j of thread t is chunk t + j * tpr of the
// row. A row is owned by tpr threads: a power of two up to 64 (several rows per
// wavefront, sums by lane exchange) or a multiple of 64 (a workgroup per row, sums
// over the wavefronts through LDS).
//
// Backward: each workgroup takes rows blockIdx, blockIdx + grid, ... and keeps its
// columns' sums for the weights and a per-channel gate in registers; at the end it
// writes them as one row of partial sums, and a second kernel adds these in
// workgroup order. No atomics, so the sums do not depend on scheduling.
#include "block_common.h"

namespace moe {
namespace {

constexpr int EPT = 16;            // values of a row that one thread holds at most
constexpr int MAX_DIM = 16384;     // EPT * 1024
constexpr int FWD_BLOCKS = 1 << 20;  // a forward workgroup takes a second row only beyond this (threads of a grid < 2^32)
constexpr int BWD_BLOCKS = 512;      // workgroups that share the rows of a backward pass

struct NormArgs {
    const void *r, *y, *gate, *w_post, *w_pre;
    void *r_out, *n;
    float* stats;
    int64_t ldr, ldy, ldro, ldn;
    int dim, m, gate_kind, tpr;
    float eps, res_scale;
    // backward
    const void *dr_out, *dn;
    void *dr, *dy, *dgate;
    int64_t lddro, lddn, lddr, lddy;
    float* partial;   // [grid][3][dim]: dw_post, dw_pre, dgate (channel); NULL: none of them wanted
};

// chunk of V values; `on` false: zeros
template <typename T, int V>
MOE_DEV void load_chunk(const void* base, int64_t at, bool on, float* v) {
    const typename T::bits* p = reinterpret_cast<const typename T::bits*>(base) + at;
    if (V == 1) {
        v[0] = on ? T::load(p[0]) : 0.f;
    } else if (V == 4) {
        const float4 q = on ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
        const uint4 q = on ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = T::load((typename T::bits)(w[i] & 0xFFFFu));
            v[2 * i + 1] = T::load((typename T::bits)(w[i] >> 16));
        }
    }
}
template <typename T, int V>
MOE_DEV void store_chunk(void* base, int64_t at, const float* v) {
    typename T::bits* p = reinterpret_cast<typename T::bits*>(base) + at;
    if constexpr (V == 1) {
        p[0] = T::store(v[0]);
    } else if constexpr (V == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]),
                                                  T::pack2(v[6], v[7]));
    }
}

// Sum over the tpr threads of a row. For tpr > 64 every thread of the workgroup
// calls it; `lds` has a float per wavefront and is used once per call site and row.
MOE_DEV float row_sum(float v, int tpr, float* lds) {
    if (tpr <= 64) {
        for (int off = tpr >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off);
        return v;
    }
    v = wave_sum(v);
    const int wv = threadIdx.x >> 6, nw = tpr >> 6;
    if ((threadIdx.x & 63) == 0) lds[wv] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += lds[i];
    return s;
}

template <typename T, int V, int C>
__global__ __launch_bounds__(1024) void norm_forward_kernel(NormArgs a) {
    __shared__ float lds[2][2][16];
    const int tpr = a.tpr, rpb = tpr <= 64 ? blockDim.x / tpr : 1;
    const int t = tpr <= 64 ? threadIdx.x % tpr : threadIdx.x, rg = tpr <= 64 ? threadIdx.x / tpr : 0;
    const bool has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * rpb + rg; row < a.m; row += (int64_t)gridDim.x * rpb, turn ^= 1) {
        int col[C];
        float rv[C][V], yv[C][V], gv[C][V], wp[C][V], wn[C][V];
        const float gt = a.gate_kind == MOE_GATE_TOKEN ? T::load(reinterpret_cast<const typename T::bits*>(a.gate)[row]) : 1.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            col[j] = (t + j * tpr) * V;
            const bool on = col[j] < a.dim;
            load_chunk<T, V>(a.r, row * a.ldr + col[j], on, rv[j]);
            load_chunk<T, V>(a.y, row * a.ldy + col[j], on && a.y != nullptr, yv[j]);
            if (a.gate_kind == MOE_GATE_FULL || a.gate_kind == MOE_GATE_CHANNEL)
                load_chunk<T, V>(a.gate, (a.gate_kind == MOE_GATE_FULL ? row * a.dim : 0) + col[j], on, gv[j]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) gv[j][i] = gt;
            if (has_post) load_chunk<T, V>(a.w_post, col[j], on, wp[j]);
            if (has_pre) load_chunk<T, V>(a.w_pre, col[j], on, wn[j]);
        }
        float rs1 = 0.f;
        if (has_post) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) s += yv[j][i] * yv[j][i];
            rs1 = 1.0f / sqrtf(row_sum(s, tpr, lds[turn][0]) / (float)a.dim + a.eps);
        }
        float s2 = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = has_post ? yv[j][i] * rs1 * wp[j][i] : yv[j][i];
                rv[j][i] = a.res_scale * rv[j][i] + gv[j][i] * p;
                s2 += rv[j][i] * rv[j][i];
            }
        if (a.r_out != nullptr) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (col[j] < a.dim) store_chunk<T, V>(a.r_out, row * a.ldro + col[j], rv[j]);
        }
        float rs2 = 0.f;
        if (has_pre) {
            rs2 = 1.0f / sqrtf(row_sum(s2, tpr, lds[turn][1]) / (float)a.dim + a.eps);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = rv[j][i] * rs2 * wn[j][i];
                if (col[j] < a.dim) store_chunk<T, V>(a.n, row * a.ldn + col[j], o);
            }
        }
        if (a.stats != nullptr && t == 0) {
            a.stats[2 * row] = rs1;
            a.stats[2 * row + 1] = rs2;
        }
    }
}

template <typename T, int V, int C>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormArgs a) {
    __shared__ float lds[2][3][16];
    extern __shared__ float sums[];   // tpr <= 64: [3][rows per workgroup][tpr * V * C]
    const int tpr = a.tpr, rpb = tpr <= 64 ? blockDim.x / tpr : 1;
    const int t = tpr <= 64 ? threadIdx.x % tpr : threadIdx.x, rg = tpr <= 64 ? threadIdx.x / tpr : 0;
    const bool has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr && a.dn != nullptr;
    const float inv_dim = 1.0f / (float)a.dim;
    int col[C];
    float wp[C][V], wn[C][V], gc[C][V];
    float s_post[C][V], s_pre[C][V], s_gate[C][V];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        col[j] = (t + j * tpr) * V;
        const bool on = col[j] < a.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) wp[j][i] = gc[j][i] = 1.f, wn[j][i] = s_post[j][i] = s_pre[j][i] = s_gate[j][i] = 0.f;
        if (has_post) load_chunk<T, V>(a.w_post, col[j], on, wp[j]);
        if (has_pre) load_chunk<T, V>(a.w_pre, col[j], on, wn[j]);
        if (a.gate_kind == MOE_GATE_CHANNEL) load_chunk<T, V>(a.gate, col[j], on, gc[j]);
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * rpb + rg; row < a.m; row += (int64_t)gridDim.x * rpb, turn ^= 1) {
        float rv[C][V], yv[C][V], gv[C][V], ev[C][V], dv[C][V];
        const float gt = a.gate_kind == MOE_GATE_TOKEN ? T::load(reinterpret_cast<const typename T::bits*>(a.gate)[row]) : 1.f;
        const float rs1 = has_post ? a.stats[2 * row] : 1.f, rs2 = has_pre ? a.stats[2 * row + 1] : 0.f;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const bool on = col[j] < a.dim;
            load_chunk<T, V>(a.r, row * a.ldr + col[j], on, rv[j]);
            load_chunk<T, V>(a.y, row * a.ldy + col[j], on && a.y != nullptr, yv[j]);
            load_chunk<T, V>(a.dn, row * a.lddn + col[j], on && has_pre, dv[j]);
            load_chunk<T, V>(a.dr_out, row * a.lddro + col[j], on && a.dr_out != nullptr, ev[j]);
            if (a.gate_kind == MOE_GATE_FULL) load_chunk<T, V>(a.gate, row * a.dim + col[j], on, gv[j]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) gv[j][i] = a.gate_kind == MOE_GATE_CHANNEL ? gc[j][i] : gt;
        }
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // rv becomes r' from here on
                rv[j][i] = a.res_scale * rv[j][i] + gv[j][i] * (yv[j][i] * rs1 * wp[j][i]);
                s += rv[j][i] * (wn[j][i] * dv[j][i]);
            }
        const float c2 = has_pre ? row_sum(s, tpr, lds[turn][0]) * inv_dim * rs2 * rs2 : 0.f;
        float sy = 0.f, sg = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s_pre[j][i] += dv[j][i] * rv[j][i] * rs2;
                ev[j][i] += rs2 * (wn[j][i] * dv[j][i] - rv[j][i] * c2);
                const float yn = yv[j][i] * rs1;          // y / rms(y)
                const float dp = gv[j][i] * ev[j][i];
                s_post[j][i] += dp * yn;
                s_gate[j][i] += ev[j][i] * (yn * wp[j][i]);
                sg += ev[j][i] * (yn * wp[j][i]);
                dv[j][i] = wp[j][i] * dp;                 // b
                sy += yv[j][i] * dv[j][i];
                rv[j][i] = a.res_scale * ev[j][i];        // dr
            }
        if (a.dr != nullptr) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (col[j] < a.dim) store_chunk<T, V>(a.dr, row * a.lddr + col[j], rv[j]);
        }
        if (a.dgate != nullptr && a.gate_kind == MOE_GATE_FULL) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = ev[j][i] * (yv[j][i] * rs1 * wp[j][i]);
                if (col[j] < a.dim) store_chunk<T, V>(a.dgate, row * a.dim + col[j], o);
            }
        }
        if (a.dgate != nullptr && a.gate_kind == MOE_GATE_TOKEN) {
            sg = row_sum(sg, tpr, lds[turn][2]);
            if (t == 0) reinterpret_cast<typename T::bits*>(a.dgate)[row] = T::store(sg);
        }
        if (a.dy != nullptr) {
            const float c1 = has_post ? row_sum(sy, tpr, lds[turn][1]) * inv_dim * rs1 * rs1 : 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = rs1 * (dv[j][i] - yv[j][i] * c1);
                if (col[j] < a.dim) store_chunk<T, V>(a.dy, row * a.lddy + col[j], o);
            }
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + (size_t)blockIdx.x * 3 * a.dim;
    if (tpr > 64) {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (col[j] + i < a.dim) {
                    out[col[j] + i] = s_post[j][i];
                    out[a.dim + col[j] + i] = s_pre[j][i];
                    out[2 * a.dim + col[j] + i] = s_gate[j][i];
                }
        return;
    }
    const int width = tpr * V * C;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sums[(0 * rpb + rg) * width + col[j] + i] = s_post[j][i];
            sums[(1 * rpb + rg) * width + col[j] + i] = s_pre[j][i];
            sums[(2 * rpb + rg) * width + col[j] + i] = s_gate[j][i];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 3 * a.dim; c += blockDim.x) {
        const int which = c / a.dim, cc = c - which * a.dim;
        float v = 0.f;
        for (int g = 0; g < rpb; ++g) v += sums[(which * rpb + g) * width + cc];
        out[c] = v;
    }
}

// out[which][c] = the sum over `blocks` partial rows, in order within each of the
// four slices of a workgroup, then over the slices
template <typename T>
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* partial, int blocks, int dim, void* o0, void* o1,
                                                        void* o2) {
    __shared__ float lds[4][64];
    const int lane = threadIdx.x & 63, sl = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    void* o = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
    if (o == nullptr) return;
    float v = 0.f;
    if (c < dim)
        for (int b = sl; b < blocks; b += 4) v += partial[((size_t)b * 3 + blockIdx.y) * dim + c];
    lds[sl][lane] = v;
    __syncthreads();
    if (sl == 0 && c < dim)
        reinterpret_cast<typename T::bits*>(o)[c] = T::store(lds[0][lane] + lds[1][lane] + lds[2][lane] + lds[3][lane]);
}

struct NormPlan {
    int v, c, tpr, threads, rpb;
};

// V from the alignment, then the fewest chunks per thread that keep a row within 512 threads
NormPlan norm_plan(int dim, int v) {
    NormPlan p;
    p.v = v;
    const int chunks = (dim + v - 1) / v, cmax = EPT / v;
    p.c = 1;
    while (p.c < cmax && chunks > 512 * p.c) p.c *= 2;
    int t = (chunks + p.c - 1) / p.c;
    if (t <= 64) {
        p.tpr = 1;
        while (p.tpr < t) p.tpr *= 2;
        p.threads = 256;
        p.rpb = 256 / p.tpr;
    } else {
        p.tpr = p.threads = (t + 63) / 64 * 64;
        p.rpb = 1;
    }
    return p;
}

int check_norm(const moe_norm* f) {
    if (f == nullptr) return MOE_EINVAL;
    if (f->dim < 1 || f->dim > MAX_DIM || f->dtype < MOE_BF16 || f->dtype > MOE_F32) return MOE_EINVAL;
    if (!(f->eps > 0.f) || !(f->eps < INFINITY) || !(fabsf(f->res_scale) < INFINITY)) return MOE_EINVAL;
    return MOE_OK;
}

size_t value_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// collects what the vector path needs: every pointer and row stride a multiple of 16 bytes
struct Alignment {
    size_t size;
    bool vec = true, ok = true;
    void rows(const void* p, int64_t ld, int dim) {
        if (p == nullptr) return;
        if (ld < dim) ok = false;
        if (!aligned_to(p, size)) ok = false;
        if (!aligned_to(p, 16) || (ld * (int64_t)size) % 16) vec = false;
    }
};

int row_blocks(const NormPlan& p, int m, int most) { return (int)std::min<int64_t>(((int64_t)m + p.rpb - 1) / p.rpb, most); }
int backward_blocks(const NormPlan& p, int m) { return row_blocks(p, m, BWD_BLOCKS); }

template <typename T, bool BWD>
hipError_t launch_norm(const NormPlan& p, const NormArgs& a, hipStream_t st) {
    void (*k)(NormArgs) = nullptr;
#define PICK(V, C) (BWD ? norm_backward_kernel<T, V, C> : norm_forward_kernel<T, V, C>)
    constexpr int VEC = sizeof(typename T::bits) == 4 ? 4 : 8;
    if (p.v == 1)
        k = p.c == 1 ? PICK(1, 1) : p.c == 2 ? PICK(1, 2) : p.c == 4 ? PICK(1, 4) : p.c == 8 ? PICK(1, 8) : PICK(1, 16);
    else
        k = p.c == 1 ? PICK(VEC, 1) : p.c == 2 ? PICK(VEC, 2) : PICK(VEC, EPT / VEC);
#undef PICK
    const int grid = row_blocks(p, a.m, BWD ? BWD_BLOCKS : FWD_BLOCKS);
    const size_t lds = BWD && p.tpr <= 64 && a.partial != nullptr ? sizeof(float) * 3 * p.rpb * p.tpr * p.v * p.c : 0;
    return launch_kernel(k, dim3(grid), dim3(p.threads), lds, st, a);
}

template <bool BWD>
hipError_t launch_norm_of(int dtype, const NormPlan& p, const NormArgs& a, hipStream_t st) {
    if (dtype == MOE_BF16) return launch_norm<Bf16, BWD>(p, a, st);
    if (dtype == MOE_F16) return launch_norm<F16, BWD>(p, a, st);
    return launch_norm<F32, BWD>(p, a, st);
}

// what both directions check of the description, the gate and the rows they share
int check_rows(const moe_norm* f, const void* r, const void* y, const void* gate, int gate_kind, int m, Alignment& al) {
    if (r == nullptr || m < 0 || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EINVAL;
    if ((gate == nullptr) != (gate_kind == MOE_GATE_NONE)) return MOE_EINVAL;
    if (y == nullptr && (f->w_post != nullptr || gate_kind != MOE_GATE_NONE)) return MOE_EINVAL;
    al.rows(f->w_post, f->dim, f->dim);
    al.rows(f->w_pre, f->dim, f->dim);
    if (gate_kind == MOE_GATE_TOKEN) al.ok = al.ok && aligned_to(gate, al.size);
    else al.rows(gate, f->dim, f->dim);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_workspace(const moe_norm* f, int32_t m, size_t* backward) {
    const int rc = check_norm(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || backward == nullptr) return MOE_EINVAL;
    // the layout of the rows decides how many workgroups share them: the most of the two
    int blocks = 0;
    for (int v : {1, f->dtype == MOE_F32 ? 4 : 8}) blocks = std::max(blocks, backward_blocks(norm_plan(f->dim, v), m));
    *backward = round_up((size_t)blocks * 3 * f->dim * sizeof(float), 256);
    return MOE_OK;
}

int moe_norm_forward(const moe_norm* f, const void* r, int64_t ldr, const void* y, int64_t ldy, const void* gate,
                     int32_t gate_kind, int32_t m, void* r_out, int64_t ldro, void* n, int64_t ldn, float* stats,
                     void* stream) {
    int rc = check_norm(f);
    if (rc != MOE_OK) return rc;
    Alignment al{value_bytes(f->dtype)};
    if (m == 0) return MOE_OK;
    if ((rc = check_rows(f, r, y, gate, gate_kind, m, al)) != MOE_OK) return rc;
    if ((n == nullptr) != (f->w_pre == nullptr) || (n == nullptr && r_out == nullptr)) return MOE_EINVAL;
    al.rows(r, ldr, f->dim);
    al.rows(y, ldy, f->dim);
    al.rows(r_out, ldro, f->dim);
    al.rows(n, ldn, f->dim);
    if (!al.ok || !aligned_to(stats, 4)) return MOE_EINVAL;
    NormArgs a{};
    a.r = r, a.y = y, a.gate = gate, a.w_post = f->w_post, a.w_pre = f->w_pre, a.r_out = r_out, a.n = n, a.stats = stats;
    a.ldr = ldr, a.ldy = ldy, a.ldro = ldro, a.ldn = ldn;
    a.dim = f->dim, a.m = m, a.gate_kind = gate_kind, a.eps = f->eps, a.res_scale = f->res_scale;
    const int vec = f->dtype == MOE_F32 ? 4 : 8;
    const NormPlan p = norm_plan(f->dim, al.vec && f->dim % vec == 0 ? vec : 1);
    a.tpr = p.tpr;
    return status_of(launch_norm_of<false>(f->dtype, p, a, (hipStream_t)stream));
}

int moe_norm_backward(const moe_norm* f, const void* r, int64_t ldr, const void* y, int64_t ldy, const void* gate,
                      int32_t gate_kind, int32_t m, const float* stats, const void* dr_out, int64_t lddro,
                      const void* dn, int64_t lddn, void* dr, int64_t lddr, void* dy, int64_t lddy, void* dgate,
                      void* dw_post, void* dw_pre, void* work, size_t work_bytes, void* stream) {
    int rc = check_norm(f);
    if (rc != MOE_OK) return rc;
    const hipStream_t st = (hipStream_t)stream;
    Alignment al{value_bytes(f->dtype)};
    if (m < 0 || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EINVAL;
    if ((dgate != nullptr && gate_kind == MOE_GATE_NONE) || (dw_post != nullptr && f->w_post == nullptr) ||
        (dw_pre != nullptr && f->w_pre == nullptr))
        return MOE_EINVAL;
    for (const void* p : {dgate, dw_post, dw_pre})
        if (!aligned_to(p, al.size)) return MOE_EINVAL;
    void* const d_channel = gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
    const bool sums = dw_post != nullptr || dw_pre != nullptr || d_channel != nullptr;
    int blocks = 0;
    if (m > 0) {
        if ((rc = check_rows(f, r, y, gate, gate_kind, m, al)) != MOE_OK) return rc;
        if (dr_out == nullptr && dn == nullptr) return MOE_EINVAL;
        if ((dn != nullptr && f->w_pre == nullptr) || (dy != nullptr && y == nullptr)) return MOE_EINVAL;
        if (stats == nullptr && (f->w_post != nullptr || dn != nullptr)) return MOE_EINVAL;
        al.rows(r, ldr, f->dim);
        al.rows(y, ldy, f->dim);
        al.rows(dr_out, lddro, f->dim);
        al.rows(dn, lddn, f->dim);
        al.rows(dr, lddr, f->dim);
        al.rows(dy, lddy, f->dim);
        if (gate_kind == MOE_GATE_FULL) al.rows(dgate, f->dim, f->dim);
        if (!al.ok || !aligned_to(stats, 4)) return MOE_EINVAL;
        const int vec = f->dtype == MOE_F32 ? 4 : 8;
        const NormPlan p = norm_plan(f->dim, al.vec && f->dim % vec == 0 ? vec : 1);
        blocks = backward_blocks(p, m);
        if (sums) {
            if (work == nullptr || !aligned_to(work, 256)) return MOE_EINVAL;
            if (work_bytes < (size_t)blocks * 3 * f->dim * sizeof(float)) return MOE_ESCRATCH;
        }
        NormArgs a{};
        a.r = r, a.y = y, a.gate = gate, a.w_post = f->w_post, a.w_pre = f->w_pre, a.stats = const_cast<float*>(stats);
        a.ldr = ldr, a.ldy = ldy, a.dim = f->dim, a.m = m, a.gate_kind = gate_kind, a.eps = f->eps;
        a.res_scale = f->res_scale, a.tpr = p.tpr;
        a.dr_out = dr_out, a.dn = dn, a.dr = dr, a.dy = dy, a.dgate = dgate;
        a.lddro = lddro, a.lddn = lddn, a.lddr = lddr, a.lddy = lddy;
        a.partial = sums ? reinterpret_cast<float*>(work) : nullptr;
        const hipError_t e = launch_norm_of<true>(f->dtype, p, a, st);
        if (e != hipSuccess) return MOE_EHIP;
    }
    if (!sums) return MOE_OK;
    const dim3 grid((f->dim + 63) / 64, 3);
    const float* part = reinterpret_cast<const float*>(work);
    hipError_t e;
    if (f->dtype == MOE_BF16)
        e = launch_kernel(norm_sums_kernel<Bf16>, grid, 256, 0, st, part, blocks, f->dim, dw_post, dw_pre, d_channel);
    else if (f->dtype == MOE_F16)
        e = launch_kernel(norm_sums_kernel<F16>, grid, 256, 0, st, part, blocks, f->dim, dw_post, dw_pre, d_channel);
    else
        e = launch_kernel(norm_sums_kernel<F32>, grid, 256, 0, st, part, blocks, f->dim, dw_post, dw_pre, d_channel);
    return status_of(e);
}

}  // extern "C"
