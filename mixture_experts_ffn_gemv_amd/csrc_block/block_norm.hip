// The norm after a block, its gate, the scaled residual and the norm before the
// next block, forward and backward (moe_norm_* in include/moe.h).
//
// A row lives in the registers of the threads that own it from its first load to
// its last store, so each array passes through memory once in each direction. A
// thread holds C chunks of V consecutive values (16 bytes, wherever the row starts);
// chunk j of thread t is chunk t + j * tpr of the row. A row is owned by tpr threads:
// a power of two up to 64 (several rows per wavefront, sums by lane exchange) or a
// multiple of 64 (a workgroup per row, sums over the wavefronts through LDS). A workgroup takes rows blockIdx, blockIdx +
// grid, ... and requests its next row, as it lies in memory, before it works on the
// current one; the weights and a per-channel gate stay in registers.
//
// Backward: each workgroup keeps two sums per column in registers,
//   S = sum e y rs1 (times the gate, unless it is per channel) and sum dn r' rs2;
// at the end it writes them as one row of partial sums, and a second kernel adds
// these in a fixed order and makes dw_post = gate S, dgate = w_post S and dw_pre of
// them. No atomics, so the sums do not depend on scheduling.
//
// Bound by memory. At 8192 x 5120 bf16: forward 69 us for 336 MB (4.9 TB/s), backward
// 106 us for 503 MB (4.7 TB/s) and 5 us for its sums, where a copy of 1 GiB reaches
// 6.2 TB/s. One token: 3.8 us, a launch and two dependent reductions. Measured at that
// size and not taken: two rows requested ahead (forward the same, backward the same,
// short calls slower: 1003 x 1111 f32 16 against 11 us), 30 wavefronts of workgroups
// per CU instead of 20 (forward 86 us), single values where rows are not 16-byte
// aligned (107 and 173 us, since the tail's loads stood in branches).
#include "block_rows.h"

namespace moe {
namespace {

constexpr int MAX_DIM = 16384;   // 1024 threads with 16 values each
// wavefronts per CU for which workgroups are launched: about as many as are resident, so that
// each workgroup keeps requesting rows ahead from the first to the last
constexpr int FWD_WAVES = 20, BWD_WAVES = 12;

struct NormArgs {
    const void *r, *y, *gate, *w_post, *w_pre;
    void *r_out, *n;
    float* stats;
    int64_t ldr, ldy, ldro, ldn;
    int dim, m, gate_kind, tpr;
    float eps, res_scale;
    bool past_l2;   // each output is larger than the L2s (32 MB): stored past them (backward 113 -> 103 us at 8192 x 5120 bf16)
    // backward
    const void *dr_out, *dn;
    void *dr, *dy, *dgate;
    int64_t lddro, lddn, lddr, lddy;
    // an array that is not there has another's address, so that loads need no condition
    bool has_y, has_dn, has_dr;
    float* partial;   // [grid][2][dim]; NULL: no sum over rows is wanted
};

// Holds a chunk as it lies in memory: unpacked anew for each row, it takes fewer registers
template <typename T>
MOE_DEV void keep(Raw<T>& r) {
    if constexpr (Raw<T>::V == 8) asm volatile("" : "+v"(r.q.x), "+v"(r.q.y), "+v"(r.q.z), "+v"(r.q.w));
}

// Sum over the tpr threads of a row. WIDE: every thread of the workgroup calls it;
// `lds` has a float per wavefront and is used once per call site and row.
template <bool WIDE>
MOE_DEV float row_sum(float v, int tpr, float* lds) {
    if (!WIDE) {
        for (int off = tpr >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off);
        return v;
    }
    v = wave_sum(v);
    const int wv = threadIdx.x >> 6, nw = tpr >> 6;
    if ((threadIdx.x & 63) == 0) lds[wv] = v;
    barrier_lds();   // the next row's loads stay in flight
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += lds[i];
    return s;
}

// WIDE: a row per workgroup, so that its number is the same in every lane.
// G: which gate, SCALAR (none, or one per row), MOE_GATE_CHANNEL or MOE_GATE_FULL
constexpr int SCALAR = MOE_GATE_NONE;
template <typename T, int C, int G, Tail TAIL, bool WIDE, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_forward_kernel(NormArgs a) {
    constexpr int V = Raw<T>::V;
    __shared__ float lds[2][2][16];
    const int tpr = WIDE ? (int)blockDim.x : a.tpr, rpb = WIDE ? 1 : blockDim.x / tpr;
    const int t = WIDE ? threadIdx.x : threadIdx.x % tpr, rg = WIDE ? 0 : threadIdx.x / tpr;
    const bool has_y = a.has_y, has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr;
    const bool token = G == SCALAR && a.gate_kind == MOE_GATE_TOKEN;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int col[C], skip[C];
    struct Row {   // a requested row
        Raw<T> r[C], y[C], g[C];
        typename T::bits gate;
    } q;
    Raw<T> wp[C], wn[C], gc[C];
    auto request = [&](int64_t row) {
        row = min(row, (int64_t)a.m - 1);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            q.r[j].template load<TAIL>(a.r, row * a.ldr, col[j], a.dim);
            q.y[j].template load<TAIL>(a.y, row * a.ldy, col[j], a.dim);
            if (G == MOE_GATE_FULL) q.g[j].template load<TAIL>(a.gate, row * a.dim, col[j], a.dim);
        }
        if (token) q.gate = reinterpret_cast<const typename T::bits*>(a.gate)[row];
    };
    int64_t row = (int64_t)blockIdx.x * rpb + rg;
#pragma unroll
    for (int j = 0; j < C; ++j) place_chunk<TAIL>(t + j * tpr, V, a.dim, col[j], skip[j]);
    request(row);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        wp[j].template load<TAIL>(has_post ? a.w_post : a.r, 0, col[j], a.dim);
        wn[j].template load<TAIL>(has_pre ? a.w_pre : a.r, 0, col[j], a.dim);
        if (G == MOE_GATE_CHANNEL) gc[j].template load<TAIL>(a.gate, 0, col[j], a.dim);
    }
    for (int turn = 0; row < a.m; row += step, turn ^= 1) {
        float rv[C][V], yv[C][V];
        Raw<T> g_[C];   // this row's gate, as it lies in memory
        const float gt = token ? T::load(q.gate) : 1.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            q.r[j].template get<TAIL>(rv[j], skip[j]);
            q.y[j].template get<TAIL>(yv[j], skip[j], has_y);
            if (G != SCALAR) g_[j] = G == MOE_GATE_FULL ? q.g[j] : gc[j];
        }
        request(row + step);
        float rs1 = 0.f;
        if (has_post) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) s += yv[j][i] * yv[j][i];
            rs1 = 1.0f / sqrtf(row_sum<WIDE>(s, tpr, lds[turn][0]) / (float)a.dim + a.eps);
        }
        float s2 = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float w[V], g[V];
            keep(wp[j]);
            wp[j].template get<WHOLE>(w, skip[j]);
            if (G != SCALAR) keep(g_[j]), g_[j].template get<WHOLE>(g, skip[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = has_post ? yv[j][i] * rs1 * w[i] : yv[j][i];
                rv[j][i] = a.res_scale * rv[j][i] + (G != SCALAR ? g[i] : gt) * p;
                s2 += rv[j][i] * rv[j][i];
            }
            if (a.r_out != nullptr) store_chunk<T, TAIL>(a.r_out, row * a.ldro, col[j], a.dim, skip[j], a.past_l2, rv[j]);
        }
        float rs2 = 0.f;
        if (has_pre) {
            rs2 = 1.0f / sqrtf(row_sum<WIDE>(s2, tpr, lds[turn][1]) / (float)a.dim + a.eps);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float w[V];
                keep(wn[j]);
                wn[j].template get<WHOLE>(w, skip[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] *= rv[j][i] * rs2;
                store_chunk<T, TAIL>(a.n, row * a.ldn, col[j], a.dim, skip[j], a.past_l2, w);
            }
        }
        if (a.stats != nullptr && t == 0) {
            a.stats[2 * row] = rs1;
            a.stats[2 * row + 1] = rs2;
        }
    }
}

template <typename T, int C, int G, Tail TAIL, bool WIDE, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_backward_kernel(NormArgs a) {
    constexpr int V = Raw<T>::V;
    __shared__ float lds[2][3][16];
    extern __shared__ float sums[];   // not WIDE: [2][rows per workgroup][tpr * V]
    const int tpr = WIDE ? (int)blockDim.x : a.tpr, rpb = WIDE ? 1 : blockDim.x / tpr;
    const int t = WIDE ? threadIdx.x : threadIdx.x % tpr, rg = WIDE ? 0 : threadIdx.x / tpr;
    const bool has_y = a.has_y, has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr && a.has_dn;
    const bool token = G == SCALAR && a.gate_kind == MOE_GATE_TOKEN;
    const float inv_dim = 1.0f / (float)a.dim;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int col[C], skip[C];
    struct Row {   // a requested row
        Raw<T> r[C], y[C], dn[C], dr[C], g[C];
        typename T::bits gate;
        float rs1, rs2;
    } q;
    Raw<T> wp[C], wn[C], gc[C];
    auto request = [&](int64_t row) {
        row = min(row, (int64_t)a.m - 1);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            q.r[j].template load<TAIL>(a.r, row * a.ldr, col[j], a.dim);
            q.y[j].template load<TAIL>(a.y, row * a.ldy, col[j], a.dim);
            q.dn[j].template load<TAIL>(a.dn, row * a.lddn, col[j], a.dim);
            q.dr[j].template load<TAIL>(a.dr_out, row * a.lddro, col[j], a.dim);
            if (G == MOE_GATE_FULL) q.g[j].template load<TAIL>(a.gate, row * a.dim, col[j], a.dim);
        }
        if (token) q.gate = reinterpret_cast<const typename T::bits*>(a.gate)[row];
        q.rs1 = a.stats[2 * row];
        q.rs2 = a.stats[2 * row + 1];
    };
    int64_t row = (int64_t)blockIdx.x * rpb + rg;
    float s_post[C][V], s_pre[C][V];
#pragma unroll
    for (int j = 0; j < C; ++j) place_chunk<TAIL>(t + j * tpr, V, a.dim, col[j], skip[j]);
    request(row);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        wp[j].template load<TAIL>(has_post ? a.w_post : a.r, 0, col[j], a.dim);
        wn[j].template load<TAIL>(has_pre ? a.w_pre : a.r, 0, col[j], a.dim);
        if (G == MOE_GATE_CHANNEL) gc[j].template load<TAIL>(a.gate, 0, col[j], a.dim);
#pragma unroll
        for (int i = 0; i < V; ++i) s_post[j][i] = s_pre[j][i] = 0.f;
    }
    for (int turn = 0; row < a.m; row += step, turn ^= 1) {
        // t: r'; yn: y rs1; d: dn, then b = w_post dp; e: dr_out, then e. With no norm after r', or no
        // gradient of it, w_pre and r' read as zeros: what they hold must not reach e, finite or not
        float tv[C][V], yn[C][V], dv[C][V], ev[C][V];
        Raw<T> g_[C];   // this row's gate, as it lies in memory
        const float rs1 = has_post ? q.rs1 : 1.f, rs2 = has_pre ? q.rs2 : 0.f, gt = token ? T::load(q.gate) : 1.f;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float w[V], n[V], g[V];
            q.r[j].template get<TAIL>(tv[j], skip[j]);
            q.y[j].template get<TAIL>(yn[j], skip[j], has_y);
            q.dn[j].template get<TAIL>(dv[j], skip[j], has_pre);
            q.dr[j].template get<TAIL>(ev[j], skip[j], a.has_dr);
            keep(wp[j]), keep(wn[j]);
            wp[j].template get<WHOLE>(w, skip[j]);
            wn[j].template get<WHOLE>(n, skip[j], has_pre);
            if (G != SCALAR) g_[j] = G == MOE_GATE_FULL ? q.g[j] : gc[j], keep(g_[j]), g_[j].template get<WHOLE>(g, skip[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                yn[j][i] *= rs1;
                tv[j][i] = a.res_scale * tv[j][i] + (G != SCALAR ? g[i] : gt) * (has_post ? yn[j][i] * w[i] : yn[j][i]);
                tv[j][i] = has_pre ? tv[j][i] : 0.f;
                s += tv[j][i] * (n[i] * dv[j][i]);
            }
        }
        request(row + step);
        const float c2 = has_pre ? row_sum<WIDE>(s, tpr, lds[turn][0]) * inv_dim * rs2 * rs2 : 0.f;
        float sy = 0.f, sg = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float w[V], n[V], g[V], o[V];
            keep(wp[j]), keep(wn[j]);
            wp[j].template get<WHOLE>(w, skip[j]);
            wn[j].template get<WHOLE>(n, skip[j], has_pre);
            if (G != SCALAR) keep(g_[j]), g_[j].template get<WHOLE>(g, skip[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s_pre[j][i] += dv[j][i] * tv[j][i] * rs2;
                ev[j][i] += rs2 * (n[i] * dv[j][i] - tv[j][i] * c2);
                const float wi = has_post ? w[i] : 1.f, gi = G != SCALAR ? g[i] : gt, ey = ev[j][i] * yn[j][i];
                s_post[j][i] += G == MOE_GATE_CHANNEL ? ey : gi * ey;
                sg += ey * wi;
                dv[j][i] = wi * gi * ev[j][i];
                sy += yn[j][i] * dv[j][i];
                o[i] = a.res_scale * ev[j][i];
            }
            if (a.dr != nullptr) store_chunk<T, TAIL>(a.dr, row * a.lddr, col[j], a.dim, skip[j], a.past_l2, o);
            if (G == MOE_GATE_FULL && a.dgate != nullptr) {
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = ev[j][i] * (has_post ? yn[j][i] * w[i] : yn[j][i]);
                store_chunk<T, TAIL>(a.dgate, row * a.dim, col[j], a.dim, skip[j], a.past_l2, o);
            }
        }
        if (token && a.dgate != nullptr) {
            sg = row_sum<WIDE>(sg, tpr, lds[turn][2]);
            if (t == 0) reinterpret_cast<typename T::bits*>(a.dgate)[row] = T::store(sg);
        }
        if (a.dy != nullptr) {
            const float c1 = has_post ? row_sum<WIDE>(sy, tpr, lds[turn][1]) * inv_dim : 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
#pragma unroll
                for (int i = 0; i < V; ++i) dv[j][i] = rs1 * (dv[j][i] - yn[j][i] * c1);
                store_chunk<T, TAIL>(a.dy, row * a.lddy, col[j], a.dim, skip[j], a.past_l2, dv[j]);
            }
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + (size_t)blockIdx.x * 2 * a.dim;
    if (WIDE) {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= skip[j] && (TAIL != SHORT || i < a.dim)) {
                    out[col[j] + i] = s_post[j][i];
                    out[a.dim + col[j] + i] = s_pre[j][i];
                }
        return;
    }
    const int width = tpr * V * C;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= skip[j]) {
                sums[rg * width + col[j] + i] = s_post[j][i];
                sums[(rpb + rg) * width + col[j] + i] = s_pre[j][i];
            }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.dim; c += blockDim.x) {
        const int which = c / a.dim, cc = c - which * a.dim;
        float v = 0.f;
        for (int g = 0; g < rpb; ++g) v += sums[(which * rpb + g) * width + cc];
        out[c] = v;
    }
}

// The sums over the partial rows: 32 columns per workgroup, its 32 half wavefronts
// take every 32nd row each (eight loads in flight), and the first adds theirs in
// order. blockIdx.y 0: S -> dw_post = gate S, dgate = w_post S; 1: dw_pre.
template <typename T>
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* partial, int blocks, int dim, const void* gate,
                                                         const void* w_post, void* dw_post, void* dgate, void* dw_pre) {
    __shared__ float lds[32][32];
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    if (blockIdx.y == 0 ? dw_post == nullptr && dgate == nullptr : dw_pre == nullptr) return;
    float v = 0.f;
    if (c < dim) {
        const float* p = partial + (size_t)blockIdx.y * dim + c;
        const size_t row = 2 * (size_t)dim;
        int b = sl;
        for (; b + 32 * 7 < blocks; b += 32 * 8) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = p[(b + 32 * i) * row];
#pragma unroll
            for (int i = 0; i < 8; ++i) v += q[i];
        }
        for (; b < blocks; b += 32) v += p[b * row];
    }
    lds[sl][lane] = v;
    __syncthreads();
    if (sl != 0 || c >= dim) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += lds[i][lane];
    typedef typename T::bits bits;
    auto at = [&](const void* p) { return p != nullptr ? T::load(reinterpret_cast<const bits*>(p)[c]) : 1.f; };
    if (blockIdx.y == 1) {
        reinterpret_cast<bits*>(dw_pre)[c] = T::store(v);
        return;
    }
    if (dw_post != nullptr) reinterpret_cast<bits*>(dw_post)[c] = T::store(v * at(gate));
    if (dgate != nullptr) reinterpret_cast<bits*>(dgate)[c] = T::store(v * at(w_post));
}

struct NormPlan {
    int c, maxt;              // chunks per thread, the instance's largest workgroup
    int tpr, threads, rpb;
};

// A row of up to 64 chunks is held by part of a wavefront (C = 1). Longer ones: the
// fewest chunks per thread, within the instances that launch_norm has.
NormPlan norm_plan(int dim, int dtype) {
    NormPlan p;
    const int v = dtype == MOE_F32 ? 4 : 8, chunks = (dim + v - 1) / v;
    if (chunks <= 64) {
        p.c = p.tpr = 1;
        while (p.tpr < chunks) p.tpr *= 2;
        p.maxt = p.threads = 256;
        p.rpb = 256 / p.tpr;
        return p;
    }
    if (v == 8) p.c = chunks <= 640 ? 1 : 2, p.maxt = chunks <= 640 ? 640 : chunks <= 1024 ? 512 : 1024;
    else p.c = chunks <= 640 ? 1 : chunks <= 2048 ? 2 : 4, p.maxt = chunks <= 640 ? 640 : 1024;
    p.tpr = p.threads = ((chunks + p.c - 1) / p.c + 63) / 64 * 64;
    p.rpb = 1;
    return p;
}

int check_norm(const moe_norm* f) {
    if (f == nullptr) return MOE_EINVAL;
    if (f->dim < 1 || f->dim > MAX_DIM || f->dtype < MOE_BF16 || f->dtype > MOE_F32) return MOE_EINVAL;
    if (!(f->eps > 0.f) || !(f->eps < INFINITY) || !(fabsf(f->res_scale) < INFINITY)) return MOE_EINVAL;
    return MOE_OK;
}


bool past_l2(const moe_norm* f, int m) { return (size_t)m * f->dim * value_bytes(f->dtype) > (32u << 20); }

// a matrix whose pointer is aligned to its values and whose rows do not overlap (NULL passes)
bool rows_ok(const void* p, int64_t ld, int dim, size_t size) { return p == nullptr || (ld >= dim && aligned_to(p, size)); }

int row_blocks(const NormPlan& p, int m, int waves_per_cu) {
    const int most = 256 * std::max(1, waves_per_cu / (p.threads / 64));
    return (int)std::min<int64_t>(((int64_t)m + p.rpb - 1) / p.rpb, most);
}
int backward_blocks(const NormPlan& p, int m) { return row_blocks(p, m, BWD_WAVES); }

size_t backward_bytes(const moe_norm* f, int m) {
    return round_up((size_t)backward_blocks(norm_plan(f->dim, f->dtype), m) * 2 * f->dim * sizeof(float), 256);
}

template <typename T, bool BWD, int G, Tail TAIL>
void (*pick_norm(const NormPlan& p))(NormArgs) {
#define PICK(C, W, M) (BWD ? norm_backward_kernel<T, C, G, TAIL, W, M> : norm_forward_kernel<T, C, G, TAIL, W, M>)
    constexpr int V = Raw<T>::V;
    if (TAIL == SHORT || p.maxt == 256) return PICK(1, false, 256);
    if constexpr (TAIL != SHORT) {
        if (p.c == 1) return PICK(1, true, 640);
        if (V == 8) return p.maxt == 512 ? PICK(2, true, 512) : PICK(2, true, 1024);
        if constexpr (V == 4) return p.c == 2 ? PICK(2, true, 1024) : PICK(4, true, 1024);
    }
#undef PICK
    return nullptr;
}

template <typename T, bool BWD, int G>
hipError_t launch_norm(const NormPlan& p, const NormArgs& a, hipStream_t st) {
    constexpr int V = Raw<T>::V;
    void (*const k)(NormArgs) = a.dim % V == 0 ? pick_norm<T, BWD, G, WHOLE>(p)
                                : a.dim > V    ? pick_norm<T, BWD, G, SHIFTED>(p)
                                               : pick_norm<T, BWD, G, SHORT>(p);
    const int grid = row_blocks(p, a.m, BWD ? BWD_WAVES : FWD_WAVES);
    const size_t lds = BWD && p.maxt == 256 && a.partial != nullptr ? sizeof(float) * 2 * p.threads * V : 0;
    return launch_kernel(k, dim3(grid), dim3(p.threads), lds, st, a);
}

template <typename T, bool BWD>
hipError_t launch_norm(const NormPlan& p, const NormArgs& a, hipStream_t st) {
    if (a.gate_kind == MOE_GATE_CHANNEL) return launch_norm<T, BWD, MOE_GATE_CHANNEL>(p, a, st);
    if (a.gate_kind == MOE_GATE_FULL) return launch_norm<T, BWD, MOE_GATE_FULL>(p, a, st);
    return launch_norm<T, BWD, SCALAR>(p, a, st);
}

template <bool BWD>
hipError_t launch_norm_of(int dtype, const NormPlan& p, const NormArgs& a, hipStream_t st) {
    if (dtype == MOE_BF16) return launch_norm<Bf16, BWD>(p, a, st);
    if (dtype == MOE_F16) return launch_norm<F16, BWD>(p, a, st);
    return launch_norm<F32, BWD>(p, a, st);
}

// what both directions check of the description, the gate and the rows they share
int check_rows(const moe_norm* f, const void* r, int64_t ldr, const void* y, int64_t ldy, const void* gate, int gate_kind) {
    const size_t size = value_bytes(f->dtype);
    if (r == nullptr || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EINVAL;
    if ((gate == nullptr) != (gate_kind == MOE_GATE_NONE)) return MOE_EINVAL;
    if (y == nullptr && (f->w_post != nullptr || gate_kind != MOE_GATE_NONE)) return MOE_EINVAL;
    for (const void* p : {gate, f->w_post, f->w_pre})
        if (!aligned_to(p, size)) return MOE_EINVAL;
    return rows_ok(r, ldr, f->dim, size) && rows_ok(y, ldy, f->dim, size) ? MOE_OK : MOE_EINVAL;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_workspace(const moe_norm* f, int32_t m, size_t* backward) {
    const int rc = check_norm(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || backward == nullptr) return MOE_EINVAL;
    *backward = backward_bytes(f, m);
    return MOE_OK;
}

int moe_norm_forward(const moe_norm* f, const void* r, int64_t ldr, const void* y, int64_t ldy, const void* gate,
                     int32_t gate_kind, int32_t m, void* r_out, int64_t ldro, void* n, int64_t ldn, float* stats,
                     void* stream) {
    int rc = check_norm(f);
    if (rc != MOE_OK) return rc;
    if (m < 0) return MOE_EINVAL;
    if (m == 0) return MOE_OK;
    if ((rc = check_rows(f, r, ldr, y, ldy, gate, gate_kind)) != MOE_OK) return rc;
    if ((n == nullptr) != (f->w_pre == nullptr) || (n == nullptr && r_out == nullptr)) return MOE_EINVAL;
    const size_t size = value_bytes(f->dtype);
    if (!rows_ok(r_out, ldro, f->dim, size) || !rows_ok(n, ldn, f->dim, size) || !aligned_to(stats, 4)) return MOE_EINVAL;
    NormArgs a{};
    a.r = r, a.y = y, a.gate = gate, a.w_post = f->w_post, a.w_pre = f->w_pre, a.r_out = r_out, a.n = n, a.stats = stats;
    a.has_y = y != nullptr, a.past_l2 = past_l2(f, m);
    if (!a.has_y) a.y = r, ldy = ldr;
    a.ldr = ldr, a.ldy = ldy, a.ldro = ldro, a.ldn = ldn;
    a.dim = f->dim, a.m = m, a.gate_kind = gate_kind, a.eps = f->eps, a.res_scale = f->res_scale;
    const NormPlan p = norm_plan(f->dim, f->dtype);
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
    const size_t size = value_bytes(f->dtype);
    if (m < 0 || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EINVAL;
    if ((dgate != nullptr && gate_kind == MOE_GATE_NONE) || (dw_post != nullptr && f->w_post == nullptr) ||
        (dw_pre != nullptr && f->w_pre == nullptr))
        return MOE_EINVAL;
    for (const void* p : {dgate, dw_post, dw_pre})
        if (!aligned_to(p, size)) return MOE_EINVAL;
    void* const d_channel = gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr;
    const bool sums = dw_post != nullptr || dw_pre != nullptr || d_channel != nullptr;
    const NormPlan p = norm_plan(f->dim, f->dtype);
    if (m > 0) {
        if ((rc = check_rows(f, r, ldr, y, ldy, gate, gate_kind)) != MOE_OK) return rc;
        if (dr_out == nullptr && dn == nullptr) return MOE_EINVAL;
        if ((dn != nullptr && f->w_pre == nullptr) || (dy != nullptr && y == nullptr)) return MOE_EINVAL;
        if (stats == nullptr) return MOE_EINVAL;
        if (!rows_ok(dr_out, lddro, f->dim, size) || !rows_ok(dn, lddn, f->dim, size) || !rows_ok(dr, lddr, f->dim, size) ||
            !rows_ok(dy, lddy, f->dim, size) || !aligned_to(stats, 4))
            return MOE_EINVAL;
        if (sums) {
            if (work == nullptr || !aligned_to(work, 256)) return MOE_EINVAL;
            if (work_bytes < backward_bytes(f, m)) return MOE_ESCRATCH;
        }
        NormArgs a{};
        a.r = r, a.y = y, a.gate = gate, a.w_post = f->w_post, a.w_pre = f->w_pre, a.stats = const_cast<float*>(stats);
        a.past_l2 = past_l2(f, m);
        a.has_y = y != nullptr, a.has_dn = dn != nullptr, a.has_dr = dr_out != nullptr;
        if (!a.has_y) a.y = r, ldy = ldr;
        if (!a.has_dn) dn = r, lddn = ldr;
        if (!a.has_dr) dr_out = r, lddro = ldr;
        a.ldr = ldr, a.ldy = ldy, a.dim = f->dim, a.m = m, a.gate_kind = gate_kind, a.eps = f->eps;
        a.res_scale = f->res_scale, a.tpr = p.tpr;
        a.dr_out = dr_out, a.dn = dn, a.dr = dr, a.dy = dy, a.dgate = dgate;
        a.lddro = lddro, a.lddn = lddn, a.lddr = lddr, a.lddy = lddy;
        a.partial = sums ? reinterpret_cast<float*>(work) : nullptr;
        const hipError_t e = launch_norm_of<true>(f->dtype, p, a, st);
        if (e != hipSuccess) return MOE_EHIP;
    }
    if (!sums) return MOE_OK;
    const dim3 grid((f->dim + 31) / 32, 2);
    const float* part = reinterpret_cast<const float*>(work);
    // (no rows: zeros, whatever the factors hold)
    const void* const channel = gate_kind == MOE_GATE_CHANNEL && m > 0 ? gate : nullptr;
    const void* const w_post = m > 0 ? f->w_post : nullptr;
    auto* const k = f->dtype == MOE_BF16 ? norm_sums_kernel<Bf16> : f->dtype == MOE_F16 ? norm_sums_kernel<F16> : norm_sums_kernel<F32>;
    return status_of(launch_kernel(k, grid, dim3(1024), 0, st, part, backward_blocks(p, m), f->dim, channel, w_post, dw_post,
                                   d_channel, dw_pre));
}

}  // extern "C"
