// Tokens sorted by the experts they picked and back, with the routing weights applied, and the
// gradients (moe_sort, moe_dispatch_*, moe_combine_* in include/moe.h).
//
// moe_sort is a stable counting sort. A pick's row is the number of picks of lower experts, plus
// the picks of its expert in the steps of 1024 before its own, in the wavefronts before its own,
// and in the lanes before its own: the last from ballots over the bits of the expert's number, the one
// before from a byte per (expert, wavefront) in LDS. Only counts are added atomically, in LDS, so the
// result does not depend on scheduling.
//
// The rows are moved in chunks of 16 bytes; each row is read once and written once. Weighted sums are made
// in f32 in the order of a token's picks. dw = dy . e and de = w dy share dy, and so come of one pass.
//
// Memory bounds the moves: 8192 tokens of 5120 bf16 with six picks each are brought to their rows in 103 us (587 MB, 5.7
// TB/s), summed in 102 to 118 (587 MB), and the sums' gradients made in 220 to 242 (1.09 GB, 4.5 to 5.0 TB/s); their 49152
// picks are sorted in 8.2 (10.4 between a step's other kernels). For one token each of the three is a launch of 3 us.
#include "block_rows.h"

namespace moe {
namespace {

constexpr int MAX_EXPERTS = 1024, MAX_TOPK = 64, MAX_DIM = 1 << 20;
constexpr int MAX_PICKS = 1 << 26;

// ------------------------------------------------------------------ sort

constexpr int STEP = 1024;      // picks per step of a workgroup, a lane each
// As many steps or fewer are sorted by one launch, in which every workgroup counts all the picks. One launch and two, calls one
// after another: picks of 384 experts, 8190 5.6 and 8.3 us, 24576 6.1 and 8.5, 40962 7.5 and 8.6, 49152 8.2 and 8.6, 57342 8.9
// and 9.1, 65538 9.5 and 8.8; of 1024, 49152 8.4 and 11.1; of eight, whose counts more lanes add to at a time, 32768 9.1 and
// 8.4, 49152 13.1 and 8.5. So the bound is where many experts gain little more, and with a few experts it comes late.
constexpr int WHOLE_STEPS = 48;
constexpr int MAX_BLOCKS = 256;

struct SortArgs {
    const int32_t* idx;
    int32_t *row_of, *pick_of, *offsets;
    int32_t* counts;   // [grid][experts]: picks of each segment
    int n, experts, segment;
};

// picks per workgroup of the two-launch form
int segment_of(int n) { return std::max(1, (n + MAX_BLOCKS * STEP - 1) / (MAX_BLOCKS * STEP)) * STEP; }

__global__ __launch_bounds__(STEP) void sort_count_kernel(SortArgs a) {
    __shared__ int count[MAX_EXPERTS];
    const int tid = threadIdx.x, first = blockIdx.x * a.segment, last = min(a.n, first + a.segment);
    if (tid < a.experts) count[tid] = 0;
    __syncthreads();
    for (int i = first + tid; i < last; i += STEP) {
        const int e = a.idx[i];
        if ((unsigned)e < (unsigned)a.experts) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (tid < a.experts) a.counts[(size_t)blockIdx.x * a.experts + tid] = count[tid];
}

// WHOLE: the one launch. Every workgroup counts all the picks itself.
template <bool WHOLE>
__global__ __launch_bounds__(STEP) void sort_place_kernel(SortArgs a) {
    __shared__ int before[MAX_EXPERTS], rest[MAX_EXPERTS];   // picks of each expert before this segment, and from it on
    __shared__ int sums[STEP / 64];
    __shared__ __align__(16) uint8_t waves[MAX_EXPERTS][STEP / 64];   // picks in each wavefront of the step
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, E = a.experts;
    const int first = blockIdx.x * a.segment, last = min(a.n, first + a.segment);
    if (tid < E) {
        before[tid] = 0, rest[tid] = 0;
        *reinterpret_cast<uint4*>(waves[tid]) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (WHOLE) {
        constexpr int U = 8;   // picks that a lane requests at a time
        for (int i0 = tid; i0 < a.n; i0 += U * STEP) {
            int e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) e[u] = i0 + u * STEP < a.n ? a.idx[i0 + u * STEP] : -1;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((unsigned)e[u] < (unsigned)E) atomicAdd(i0 + u * STEP < first ? &before[e[u]] : &rest[e[u]], 1);
        }
    } else {
        const int wide = (E + 63) / 64 * 64, groups = STEP / wide, e = tid % wide, grp = tid / wide;
        if (e < E && grp < groups) {
            int b = 0, r = 0;
#pragma unroll 8
            for (int s = grp; s < (int)gridDim.x; s += groups) {
                const int c = a.counts[(size_t)s * E + e];
                if (s < (int)blockIdx.x) b += c;
                else r += c;
            }
            atomicAdd(&before[e], b);
            atomicAdd(&rest[e], r);
        }
    }
    __syncthreads();
    // the experts' first rows: an exclusive sum over them
    const int mine = tid < E ? before[tid] + rest[tid] : 0, upto = wave_inclusive_scan(mine);
    if (lane == 63) sums[wv] = upto;
    __syncthreads();
    int total = 0, at = upto - mine;
    for (int i = 0; i < STEP / 64; ++i) {
        if (i < wv) at += sums[i];
        total += sums[i];
    }
    if (tid < E) before[tid] += at;   // now: the row of this segment's first pick of the expert
    if (blockIdx.x == 0) {
        if (tid < E) a.offsets[tid] = at;
        if (tid == 0) a.offsets[E] = total;
    }
    const int bits = 32 - __builtin_clz(E);   // (E itself stands for no expert)
    for (int base = first; base < last; base += STEP) {
        const int i = base + tid;
        int e = i < last ? a.idx[i] : E;
        if ((unsigned)e > (unsigned)E) e = E;
        uint64_t same = ~0ull;   // the wavefront's lanes with the same expert
        for (int b = 0; b < bits; ++b) {
            const bool on = e >> b & 1;
            const uint64_t v = __ballot(on);
            same &= on ? v : ~v;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (e < E && rank == 0) waves[e][wv] = (uint8_t)__popcll(same);
        __syncthreads();   // (also: `before` is written)
        int row = -1;
        if (e < E) {
            const uint4 w = *reinterpret_cast<const uint4*>(waves[e]);
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
            row = before[e] + rank;
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // the wavefronts before this one
                const int k = min(max(wv - 4 * j, 0), 4);
                row = sdot4(k == 4 ? q[j] : q[j] & ((1u << (8 * k)) - 1), 0x01010101u, row);
            }
        }
        if (i < last) {
            a.row_of[i] = row;
            if (a.pick_of != nullptr && row >= 0) a.pick_of[row] = i;
            if (a.pick_of != nullptr && i >= total) a.pick_of[i] = -1;
        }
        if (base + STEP >= last) break;
        __syncthreads();
        if (tid < E) {
            const uint4 w = *reinterpret_cast<const uint4*>(waves[tid]);
            int c = before[tid];
            for (uint32_t q : {w.x, w.y, w.z, w.w}) c = sdot4(q, 0x01010101u, c);
            before[tid] = c;
            *reinterpret_cast<uint4*>(waves[tid]) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ rows to experts and back

struct MoveArgs {
    const void *x, *e;   // rows of tokens, and sorted rows
    void *out, *de;
    const float* weights;
    float* dweights;
    const int32_t* row_of;
    int64_t ldx, lde, ldo, ldde;
    int dim, m, topk, rows;
    bool past_l2;
    Walk walk;
};

// the sorted row of a token's j-th pick; -1: none
MOE_DEV int row_at(const MoveArgs& a, int64_t t, int j) {
    const int row = a.row_of[t * a.topk + j];
    return (unsigned)row < (unsigned)a.rows ? row : -1;
}

// a chunk as it is
template <typename T, Tail TAIL>
MOE_DEV void copy_chunk(const Raw<T>& from, void* base, int64_t row, int col, int dim, int skip, bool past_l2) {
    typename T::bits* p = reinterpret_cast<typename T::bits*>(base) + row + col;
    if (skip >= Raw<T>::V) return;
    if (TAIL == SHORT || (TAIL == SHIFTED && skip != 0)) {
#pragma unroll
        for (int i = 0; i < Raw<T>::V; ++i)
            if (i >= skip && col + i < dim) p[i] = from.b[i];
        return;
    }
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    const words w = {from.q.x, from.q.y, from.q.z, from.q.w};
    if (past_l2) __builtin_nontemporal_store(w, reinterpret_cast<words*>(p));
    else *reinterpret_cast<words*>(p) = w;
}

template <typename T, Tail TAIL>
__global__ __launch_bounds__(256) void dispatch_kernel(MoveArgs a) {
    for (Place p = first_place(a.walk); p.row < a.m; p = p.next(a.walk)) {
        int col, skip;
        place_chunk<TAIL>(p.chunk, Raw<T>::V, a.dim, col, skip);
        Raw<T> x;
        x.template load<TAIL>(a.x, p.row * a.ldx, col, a.dim);
        for (int j = 0; j < a.topk; ++j) {
            const int row = row_at(a, p.row, j);
            if (row >= 0) copy_chunk<T, TAIL>(x, a.out, row * a.ldo, col, a.dim, skip, a.past_l2);
        }
    }
}

// out[t] = sum over j of w[t, j] e[row_of[t, j]] (WEIGHTED; else w = 1), `J` rows at a time: none is added before the last is
// requested. (Each row's number is waited for, and with it the row before: within a wavefront they come one after another.)
template <typename T, Tail TAIL, bool WEIGHTED, bool ONCE, int J>
__global__ __launch_bounds__(256) void combine_kernel(MoveArgs a) {
    constexpr int V = Raw<T>::V;
    for (Place p = first_place(a.walk); p.row < a.m; p = p.next(a.walk)) {
        int col, skip;
        place_chunk<TAIL>(p.chunk, V, a.dim, col, skip);
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.f;
        for (int j0 = 0; j0 < a.topk; j0 += J) {
            Raw<T> e[J];
            float w[J];
            bool there[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // (a pick without a row reads the first one and adds none of it)
                const int row = j0 + j < a.topk ? row_at(a, p.row, j0 + j) : -1;
                there[j] = row >= 0;
                w[j] = WEIGHTED && there[j] ? a.weights[p.row * a.topk + j0 + j] : 1.f;
                e[j].template load_of<TAIL, ONCE>(a.e, max(row, 0) * a.lde, col, a.dim);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v[V];
                e[j].template get<WHOLE>(v, 0, there[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] = WEIGHTED ? sum[i] + (there[j] ? w[j] * v[i] : 0.f) : sum[i] + v[i];
            }
        }
        store_chunk<T, TAIL>(a.out, p.row * a.ldo, col, a.dim, skip, a.past_l2, sum);
    }
}

// de[row] = w dy[t] and dw[t, j] = dy[t] . e[row]: `tpr` threads per token (a power of two up to 64, or the whole
// workgroup: WIDE), J picks at a time
template <typename T, Tail TAIL, bool WIDE, int J>
__global__ __launch_bounds__(256) void combine_backward_kernel(MoveArgs a, int tpr) {
    constexpr int V = Raw<T>::V;
    __shared__ float lds[4][J];
    const int t = WIDE ? threadIdx.x : threadIdx.x % tpr, per = WIDE ? 1 : 256 / tpr;
    const int64_t token = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * per + (WIDE ? 0 : threadIdx.x / tpr);
    const int64_t at = min(token, (int64_t)a.m - 1);
    const int chunks = (a.dim + V - 1) / V, step = WIDE ? 256 : tpr;
    for (int j0 = 0; j0 < a.topk; j0 += J) {
        int row[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            row[j] = j0 + j < a.topk && token < a.m ? row_at(a, at, j0 + j) : -1;
            w[j] = row[j] >= 0 ? a.weights[at * a.topk + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int c = t; c < chunks; c += step) {
            int col, skip;
            place_chunk<TAIL>(c, V, a.dim, col, skip);
            Raw<T> x, e[J];
            x.template load<TAIL>(a.x, at * a.ldx, col, a.dim);
#pragma unroll
            for (int j = 0; j < J; ++j) e[j].template load<TAIL>(a.e, max(row[j], 0) * a.lde, col, a.dim);
            float dy[V];
            x.template get<TAIL>(dy, skip);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v[V], d[V];
                e[j].template get<TAIL>(v, skip, row[j] >= 0);
#pragma unroll
                for (int i = 0; i < V; ++i) dot[j] += dy[i] * v[i], d[i] = w[j] * dy[i];
                if (row[j] >= 0 && a.de != nullptr) store_chunk<T, TAIL>(a.de, row[j] * a.ldde, col, a.dim, skip, a.past_l2, d);
            }
        }
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (WIDE) dot[j] = wave_sum(dot[j]);
            else
                for (int off = tpr >> 1; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        }
        if (WIDE) {
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int j = 0; j < J; ++j) lds[threadIdx.x >> 6][j] = dot[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < J; ++j) dot[j] = (lds[0][j] + lds[1][j]) + (lds[2][j] + lds[3][j]);
            __syncthreads();
        }
        if (t == 0 && token < a.m) {
#pragma unroll
            for (int j = 0; j < J; ++j)   // (a pick without a row: 0, whatever dy holds)
                if (j0 + j < a.topk) a.dweights[token * a.topk + j0 + j] = row[j] >= 0 ? dot[j] : 0.f;
        }
    }
}

int check_picks(int32_t m, int32_t topk) {
    return m < 0 || topk < 1 || topk > MAX_TOPK || (int64_t)m * topk > MAX_PICKS ? MOE_EINVAL : MOE_OK;
}
int check_move(int32_t dtype, int32_t dim, int32_t m, int32_t topk, int32_t rows, const int32_t* row_of) {
    if (dtype < MOE_BF16 || dtype > MOE_F32 || dim < 1 || dim > MAX_DIM || rows < 0 || rows > MAX_PICKS) return MOE_EINVAL;
    const int rc = check_picks(m, topk);
    if (rc != MOE_OK || m == 0) return rc;
    return row_of != nullptr && aligned_to(row_of, 4) ? MOE_OK : MOE_EINVAL;
}

bool overlap(const void* p, size_t bytes, const void* q, size_t other) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p != nullptr && q != nullptr && a < b + other && b < a + bytes;
}

// Whether results are written past the L2s, which hold 32 MB: six rows each of 8192 x 5120 bf16 there and back 202 us so
// and 233 through them, of 1999 44.3 and 45.0, and no difference for fewer.
bool past_l2(int64_t rows, int dim, size_t size) { return (size_t)rows * dim * size > (32u << 20); }

template <typename K>
hipError_t launch_walk(K* k, MoveArgs a, int v, bool past, hipStream_t st) {
    const int per_row = (a.dim + v - 1) / v;
    const int64_t blocks = walk_blocks((int64_t)per_row * a.m, past);
    a.walk = walk(per_row, blocks * 256);
    return launch_kernel(k, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

template <typename T>   // (a copy does not look at the values: 16-bit types are one)
hipError_t launch_dispatch(const MoveArgs& a, hipStream_t st) {
    constexpr int V = Raw<T>::V;
    const Tail tail = tail_of(a.dim, V);
    return launch_walk(tail == SHORT ? dispatch_kernel<T, SHORT> : tail == WHOLE ? dispatch_kernel<T, WHOLE> : dispatch_kernel<T, SHIFTED>,
                       a, V, a.past_l2, st);
}

template <typename T, bool WEIGHTED, bool ONCE, int J>
hipError_t launch_combine_j(const MoveArgs& a, hipStream_t st) {
    constexpr int V = Raw<T>::V;
    const Tail tail = tail_of(a.dim, V);
    return launch_walk(tail == SHORT ? combine_kernel<T, SHORT, WEIGHTED, false, J>
                       : tail == WHOLE ? combine_kernel<T, WHOLE, WEIGHTED, ONCE, J> : combine_kernel<T, SHIFTED, WEIGHTED, ONCE, J>, a, V, ONCE, st);
}
// As many of a token's rows are taken at a time as it has, up to eight, and a request for a row that it does not have costs
// as much as one for another: sums of two rows of 8192 x 5120 bf16 42 us so and 63 with eight at a time, of six 101 and
// 106; the gradients of six rows of 1999 44.6 and 45.9.
template <typename T, bool WEIGHTED, bool ONCE>
hipError_t launch_combine_t(const MoveArgs& a, hipStream_t st) {
    if (a.topk == 1) return launch_combine_j<T, WEIGHTED, ONCE, 1>(a, st);
    if (a.topk == 2) return launch_combine_j<T, WEIGHTED, ONCE, 2>(a, st);
    if (a.topk <= 4) return launch_combine_j<T, WEIGHTED, ONCE, 4>(a, st);
    if (a.topk <= 6) return launch_combine_j<T, WEIGHTED, ONCE, 6>(a, st);
    return launch_combine_j<T, WEIGHTED, ONCE, 8>(a, st);
}
template <typename T>
hipError_t launch_combine_of(const MoveArgs& a, hipStream_t st) {
    const bool once = past_caches((std::min((size_t)a.m * a.topk, (size_t)a.rows) + a.m) * a.dim * sizeof(typename T::bits));
    if (a.weights != nullptr) return once ? launch_combine_t<T, true, true>(a, st) : launch_combine_t<T, true, false>(a, st);
    return once ? launch_combine_t<T, false, true>(a, st) : launch_combine_t<T, false, false>(a, st);
}

template <typename T, int J>
hipError_t launch_backward_j(const MoveArgs& a, hipStream_t st) {
    constexpr int V = Raw<T>::V;
    const Tail tail = tail_of(a.dim, V);
    const int chunks = (a.dim + V - 1) / V;
    int tpr = 1;
    while (tpr < 64 && tpr < chunks) tpr *= 2;
    const bool wide = chunks > 128;   // (8192 x 5120 bf16, six picks: 219 us, a wavefront per token 223)
    const int per = wide ? 1 : 256 / tpr;
    auto pick = [&](auto* narrow, auto* whole) { return wide ? whole : narrow; };
    auto* const k = tail == SHORT ? combine_backward_kernel<T, SHORT, false, J>
                    : tail == WHOLE ? pick(combine_backward_kernel<T, WHOLE, false, J>, combine_backward_kernel<T, WHOLE, true, J>)
                                    : pick(combine_backward_kernel<T, SHIFTED, false, J>, combine_backward_kernel<T, SHIFTED, true, J>);
    const int blocks = (a.m + per - 1) / per, across = std::min(blocks, 1 << 20);   // (a grid holds fewer than 2^32 threads along x)
    return launch_kernel(k, dim3(across, (blocks + across - 1) / across), dim3(256), 0, st, a, tpr);
}
template <typename T>
hipError_t launch_backward_t(const MoveArgs& a, hipStream_t st) {
    if (a.topk == 1) return launch_backward_j<T, 1>(a, st);
    if (a.topk == 2) return launch_backward_j<T, 2>(a, st);
    if (a.topk <= 4) return launch_backward_j<T, 4>(a, st);
    if (a.topk <= 6) return launch_backward_j<T, 6>(a, st);
    return launch_backward_j<T, 8>(a, st);
}

// out[t] = the (weighted) sum of a token's sorted rows
int sum_rows(int32_t dtype, int32_t dim, const void* e, int64_t lde, int32_t rows, const float* weights, const int32_t* row_of,
             int32_t m, int32_t topk, void* out, int64_t ldo, void* stream) {
    const int rc = check_move(dtype, dim, m, topk, rows, row_of);
    if (rc != MOE_OK || m == 0) return rc;
    const size_t size = value_bytes(dtype);
    if (!value_rows_ok(out, ldo, dim, size) || (rows > 0 && !value_rows_ok(e, lde, dim, size)) || !aligned_to(weights, 4)) return MOE_EINVAL;
    MoveArgs a{};
    // (no sorted rows: what is read in their place is not used)
    a.e = rows > 0 ? e : out, a.lde = rows > 0 ? lde : 0, a.out = out, a.ldo = ldo, a.weights = weights, a.row_of = row_of;
    a.dim = dim, a.m = m, a.topk = topk, a.rows = rows, a.past_l2 = past_l2(m, dim, size);
    const hipStream_t st = (hipStream_t)stream;
    return status_of(dtype == MOE_BF16 ? launch_combine_of<Bf16>(a, st) : dtype == MOE_F16 ? launch_combine_of<F16>(a, st) : launch_combine_of<F32>(a, st));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_sort_workspace(int32_t m, int32_t topk, int32_t n_experts, size_t* bytes) {
    const int rc = check_picks(m, topk);
    if (rc != MOE_OK) return rc;
    if (n_experts < 1 || n_experts > MAX_EXPERTS || bytes == nullptr) return MOE_EINVAL;
    const int n = m * topk;
    *bytes = n <= WHOLE_STEPS * STEP ? 0 : round_up((size_t)std::min((n + STEP - 1) / STEP, MAX_BLOCKS) * n_experts * 4, 256);
    return MOE_OK;
}

int moe_sort(const int32_t* idx, int32_t m, int32_t topk, int32_t n_experts, int32_t* row_of, int32_t* pick_of, int32_t* offsets,
             void* work, size_t work_bytes, void* stream) {
    size_t need = 0;
    const int rc = moe_sort_workspace(m, topk, n_experts, &need);
    if (rc != MOE_OK) return rc;
    if (offsets == nullptr) return MOE_EINVAL;
    for (const void* p : {(const void*)idx, (const void*)row_of, (const void*)pick_of, (const void*)offsets})
        if (!aligned_to(p, 4)) return MOE_EINVAL;
    if (m > 0 && (idx == nullptr || row_of == nullptr)) return MOE_EINVAL;
    if (need > 0 && (work == nullptr || !aligned_to(work, 256))) return MOE_EINVAL;
    if (work_bytes < need) return MOE_ESCRATCH;
    // (a workgroup reads picks of which others write the rows)
    const size_t picks = (size_t)m * topk * 4;
    if (overlap(idx, picks, row_of, picks) || overlap(idx, picks, pick_of, picks) || overlap(idx, picks, offsets, ((size_t)n_experts + 1) * 4))
        return MOE_EINVAL;
    SortArgs a{};
    a.idx = idx, a.row_of = row_of, a.pick_of = pick_of, a.offsets = offsets, a.counts = reinterpret_cast<int32_t*>(work);
    a.n = m * topk, a.experts = n_experts;
    const hipStream_t st = (hipStream_t)stream;
    if (need == 0) {
        a.segment = STEP;
        return status_of(launch_kernel(sort_place_kernel<true>, dim3(std::max(1, (a.n + STEP - 1) / STEP)), dim3(STEP), 0, st, a));
    }
    a.segment = segment_of(a.n);
    const dim3 grid((a.n + a.segment - 1) / a.segment);
    const hipError_t e = launch_kernel(sort_count_kernel, grid, dim3(STEP), 0, st, a);
    return status_of(e != hipSuccess ? e : launch_kernel(sort_place_kernel<false>, grid, dim3(STEP), 0, st, a));
}

int moe_dispatch_forward(int32_t dtype, int32_t dim, const void* x, int64_t ldx, const int32_t* row_of, int32_t m, int32_t topk,
                         void* xs, int64_t ldxs, int32_t rows, void* stream) {
    const int rc = check_move(dtype, dim, m, topk, rows, row_of);
    if (rc != MOE_OK || m == 0 || rows == 0) return rc;
    const size_t size = value_bytes(dtype);
    if (!value_rows_ok(x, ldx, dim, size) || !value_rows_ok(xs, ldxs, dim, size)) return MOE_EINVAL;
    MoveArgs a{};
    a.x = x, a.ldx = ldx, a.out = xs, a.ldo = ldxs, a.row_of = row_of;
    a.dim = dim, a.m = m, a.topk = topk, a.rows = rows, a.past_l2 = past_l2(rows, dim, size);
    return status_of(dtype == MOE_F32 ? launch_dispatch<F32>(a, (hipStream_t)stream) : launch_dispatch<Bf16>(a, (hipStream_t)stream));
}

int moe_dispatch_backward(int32_t dtype, int32_t dim, const void* dxs, int64_t lddxs, int32_t rows, const int32_t* row_of, int32_t m,
                          int32_t topk, void* dx, int64_t lddx, void* stream) {
    return sum_rows(dtype, dim, dxs, lddxs, rows, nullptr, row_of, m, topk, dx, lddx, stream);
}

int moe_combine_forward(int32_t dtype, int32_t dim, const void* e, int64_t lde, int32_t rows, const float* weights,
                        const int32_t* row_of, int32_t m, int32_t topk, void* y, int64_t ldy, void* stream) {
    if (weights == nullptr && m > 0) return MOE_EINVAL;
    return sum_rows(dtype, dim, e, lde, rows, weights, row_of, m, topk, y, ldy, stream);
}

int moe_combine_backward(int32_t dtype, int32_t dim, const void* dy, int64_t lddy, const void* e, int64_t lde, int32_t rows,
                         const float* weights, const int32_t* row_of, int32_t m, int32_t topk, void* de, int64_t ldde,
                         float* dweights, void* stream) {
    const int rc = check_move(dtype, dim, m, topk, rows, row_of);
    if (rc != MOE_OK || m == 0 || (de == nullptr && dweights == nullptr)) return rc;
    const size_t size = value_bytes(dtype);
    if (weights == nullptr || !aligned_to(weights, 4) || !aligned_to(dweights, 4) || !value_rows_ok(dy, lddy, dim, size)) return MOE_EINVAL;
    if (rows > 0 && (!value_rows_ok(e, lde, dim, size) || (de != nullptr && !value_rows_ok(de, ldde, dim, size)))) return MOE_EINVAL;
    MoveArgs a{};
    a.x = dy, a.ldx = lddy, a.e = rows > 0 ? e : dy, a.lde = rows > 0 ? lde : 0, a.de = de, a.ldde = ldde;
    a.weights = weights, a.dweights = dweights, a.row_of = row_of;
    a.dim = dim, a.m = m, a.topk = topk, a.rows = rows, a.past_l2 = past_l2(rows, dim, size);
    const hipStream_t st = (hipStream_t)stream;
    return status_of(dtype == MOE_BF16 ? launch_backward_t<Bf16>(a, st) : dtype == MOE_F16 ? launch_backward_t<F16>(a, st) : launch_backward_t<F32>(a, st));
}

}  // extern "C"
