// Matrix products with bias, activation and residual in their epilogue, of one matrix or of one per
// expert over rows sorted by expert, forward and backward (moe_linear_* in include/moe.h).
//
//   FWD  z = x W^T + b -> y = act(z) + residual  (and z in f32 for the backward pass)
//   dz   = dy act'(z), with the column sums that are db: a pass over the rows
//   DX   dx = dz W
//   DW   dW = dz^T x
//
// How a product is made of tiles is in block_tiles.h. With a matrix per expert a tile belongs to one expert: the
// host knows only how many tiles there may be, and each workgroup finds its own from the offsets, which a
// wavefront adds up 64 at a time. A workgroup without a tile ends at once.
//
// dz is rounded to 16 bits, as an operand of the matrix cores, and nothing else before the results: with many rows the
// gradients have sqrt(2) of the error that their own rounding gives them. With few rows a handful of large dz may make up
// most of a gradient, and their errors do not average out: of 1 to 16 rows of 64 to 256 outputs dx and dW were up to twice as
// far off as their own rounding. There dz is in two parts, its rounding and that of what the first leaves: 2^-16 of dz is
// lost in bf16, 2^-22 in f16. (Of eight rows or fewer of one matrix dz stays in f32: their backward pass is a kernel of its
// own.) z is kept in f32.
//
// What bounds it: with few rows the weights' bytes (one row of 2304 x 5120 bf16: 8.0 us a call, 23.6 MB; six experts of
// 5120 x 2304, one row each: 29 us, 4.9 TB/s; 64 experts of 2048 x 1408 f16, 47 rows each: 86 to 92 us, 390 MB); with many
// the matrix cores (8192 rows of 5120 x 2304 bf16: forward 190 us and the join of its last tiles 11, together 0.96 PFLOP/s;
// dz 29 us; dx and dW 384 us, 1.0 PFLOP/s; 16184 rows of 32 experts of 2048 x 1408: forward 138 to 151 us, dx 145, dW 157,
// 93 GFLOP each; kernels in a profiled run, whose sum is 4% above the calls'). A tile's K step of 256 x 256 takes 1.45 us
// forward, 1.65 in dx and 1.75 in dW; the rest are the ends of tiles, where z, y and the residual pass through all CUs at
// once, and rounds that are not full.
#include <cmath>

#include "block_rows.h"
#include "block_tiles.h"

namespace moe {
namespace {

enum Kind { FWD, DX, DW };
constexpr bool p_by_rows(Kind k) { return k != FWD; }   // p (not k) is P's consecutive index
constexpr bool q_by_rows(Kind k) { return k == DW; }

struct LinArgs {
    const uint16_t *x, *w, *bias, *residual, *dy, *dz;
    float* z;              // [m, padded(N)]
    uint16_t *y, *dx, *dw, *dbias, *dz_out;
    uint16_t* dz_rest;     // the second part of dz, of matrices with few rows; NULL: dz is exact, or no matrix has few rows
    const int32_t* offsets;   // [experts + 1]; NULL: one matrix for all rows
    int64_t ldx, ldr, ldy, lddy, lddz, lddx;
    int m, N, K, experts, act;
    float* partial;        // column sums, [chunk + expert][N]
};
// A matrix of so many rows or fewer has dz in two parts, and where the matrices have no more on average, all of them. In dx
// the parts are the halves of a tile of 128 rows, so that the weights are read once; in dW the halves of a K step. Backward
// with two parts and with one: 64 rows of 5120 x 2304 32.8 and 32.2 us; of 32 experts of 2048 x 1408, 64 rows 105.9 and 105.5,
// 1024 rows 121 and 115, 2048 rows 149 and 124. Where they have more on average the experts with few rows are the last tiles
// of the same launch, by code of their own (16184 rows, none of them few: 327 and 326), since a test in each K step, or a
// loop around a tile's, cost registers (486 and 642).
constexpr int TWO_PARTS = 64;
MOE_DEV __host__ bool all_two(int m, int experts) { return m <= (int64_t)TWO_PARTS * experts; }
enum Only { ALL, MANY, FEW };   // of which experts: any, with more rows, with so many or fewer
// Where the second part of `row` lies, which is one of a matrix's rows from row0 on. (One matrix has room for few rows.)
MOE_DEV uint16_t* rest_of(const LinArgs& a, int row, int row0) {
    return a.dz_rest + (a.experts > 1 || a.m <= TWO_PARTS ? row : row - row0) * a.lddz;
}
// rows of z and dz are padded to whole chunks of eight values
MOE_DEV __host__ int padded(int N) { return (N + 7) / 8 * 8; }

// act(v) with the hardware's reciprocal, which is off by 2^-23 (a division is ten instructions)
template <int ACT>
MOE_DEV float act_of(float v) {
    if (ACT == MOE_ACT_NONE) return v;
    float z = v;
    if (ACT == MOE_ACT_GELU) {
        const float c = fminf(fmaxf(v, -100.f), 100.f);   // (there tanh is 1 to the last bit, and c^3 finite)
        z = 2.f * 0.7978845608028654f * (c + 0.044715f * c * c * c);
    }
    return v * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// act'(v), NaN where v is
MOE_DEV float act_slope(float v, int act) {
    if (act == MOE_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
        return s * (1.f + v * (1.f - s));
    }
    const float c = clamp_up(v, 100.f), k = 2.f * 0.7978845608028654f;   // (fminf and fmaxf would make a number of a NaN)
    const float z = k * (c + 0.044715f * c * c * c);
    // (1 + tanh) / 2 and (1 - tanh) / 2, neither as a difference
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z)), q = __builtin_amdgcn_rcpf(1.f + __expf(z));
    return s + c * s * q * k * (1.f + 0.134145f * c * c);
}

// 64 offsets at a time, one per lane; what lies outside 0..m or goes back does not count
MOE_DEV int offset_at(const LinArgs& a, int i) { return min(max(a.offsets[min(i, a.experts)], 0), a.m); }

// the same of one i for the whole wavefront
MOE_DEV int offset_of(const LinArgs& a, int i) { return __builtin_amdgcn_readfirstlane(offset_at(a, i)); }

// an expert's rows, 0 if it is not meant
template <Only ONLY>
MOE_DEV int rows_of(int begin, int end) {
    const int n = max(end - begin, 0);
    return ONLY == ALL || (n > TWO_PARTS) == (ONLY == MANY) ? n : 0;
}

// A tile among those of `rows`-row tiles of the experts' rows: which expert, where it begins, its
// rows; np tiles side by side. Every lane of the wavefront calls it.
struct Slice {
    int expert, row0, rows;    // the expert's rows
    int tile;                  // which of the expert's tiles (q and p)
};
template <Only ONLY>
MOE_DEV int tiles_total(const LinArgs& a, int rows) {
    const int lane = threadIdx.x & 63;
    int n = 0;
#pragma unroll 4
    for (int e = lane; e < a.experts; e += 64) n += (rows_of<ONLY>(offset_at(a, e), offset_at(a, e + 1)) + rows - 1) / rows;
    n = wave_inclusive_scan(n);
    return __builtin_amdgcn_readlane(n, 63);
}
// false: there are not so many
template <Only ONLY>
MOE_DEV bool find_slice(const LinArgs& a, int rows, int np, int tile, Slice& s) {
    const int lane = threadIdx.x & 63;
    // 256 experts at a time, but one load after another: the second of an expert's two is behind a branch, before which the
    // compiler waits for the first (eight trips to the L2 for up to 256 experts, sixteen for 384)
    constexpr int U = 4;
    s = {0, 0, 0, 0};
    int before = 0;   // tiles of the experts before these
    for (int e0 = 0; e0 < a.experts; e0 += 64 * U) {
        int lo[U], cnt[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + 64 * u + lane;
            lo[u] = offset_at(a, e);
            cnt[u] = e < a.experts ? rows_of<ONLY>(lo[u], offset_at(a, e + 1)) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = (cnt[u] + rows - 1) / rows * np, upto = before + wave_inclusive_scan(n);
            const uint64_t past = __ballot(upto > tile);
            if (past != 0) {
                const int l = __builtin_ctzll(past);
                s.expert = e0 + 64 * u + l;
                s.row0 = __builtin_amdgcn_readlane(lo[u], l);
                s.rows = __builtin_amdgcn_readlane(cnt[u], l);
                s.tile = tile - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
                return true;
            }
            before = __builtin_amdgcn_readlane(upto, 63);
        }
    }
    return false;
}

// eight consecutive 16-bit values of a row, of which `left` > 0 are there; no alignment but a value's
MOE_DEV uint4 load8(const uint16_t* p, int left) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (left >= 8) {
        __builtin_memcpy(&q, p, 16);
    } else {   // four, two and one of them
        if (left & 4) __builtin_memcpy(&q, p, 8);
        uint32_t two = 0;
        if (left & 2) __builtin_memcpy(&two, p + (left & 4), 4);
        const uint32_t one = left & 1 ? p[left - 1] : 0u, at = left & 6;
        if (left & 4) q.z = two;
        else q.x = two;
        if (at == 0) q.x = one;
        if (at == 2) q.y = one;
        if (at == 4) q.z = one;
        if (at == 6) q.w = one;
    }
    return q;
}
MOE_DEV void store8(uint16_t* p, int left, uint4 q) {
    if (left >= 8) {
        __builtin_memcpy(p, &q, 16);
    } else {
        if (left & 4) __builtin_memcpy(p, &q, 8);
        const uint32_t two = left & 4 ? q.z : q.x, at = left & 6;
        if (left & 2) __builtin_memcpy(p + (left & 4), &two, 4);
        if (left & 1) p[left - 1] = (uint16_t)(at == 0 ? q.x : at == 2 ? q.y : at == 4 ? q.z : q.w);
    }
}
template <typename T>
MOE_DEV void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = T::lo(w[i]), v[2 * i + 1] = T::hi(w[i]);
}
template <typename T>
MOE_DEV uint4 pack8(const float (&v)[8]) {
    return make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7]));
}

// Where a tile lies and what it multiplies
struct Tile {
    Operand P, Q;       // Q's second matrix: the second part of dz, with TWO
    int q0, p0;
    int expert, row0;   // q (DW: k) counts from this row
};
// order: of DW with offsets, the experts with the most rows first. TWO: dz is in two parts; BQ: rows of q, of either
template <Kind KIND, bool GROUPED, int BQ, int BP, bool TWO, Only ONLY>
MOE_DEV Tile locate(const LinArgs& a, int tile, int nq, int np, const uint16_t* order) {
    Tile t;
    t.expert = 0, t.row0 = 0;
    int rows = a.m;
    if (GROUPED) {
        if (KIND == DW) {
            const int each = nq * np;
            t.expert = tile / each;
            tile -= t.expert * each;
            t.expert = __builtin_amdgcn_readfirstlane(order[t.expert]);
            t.row0 = offset_of(a, t.expert);
            rows = max(offset_of(a, t.expert + 1) - t.row0, 0);
        } else {
            Slice s;
            find_slice<ONLY>(a, BQ, np, tile, s);
            t.expert = s.expert, t.row0 = s.row0, rows = s.rows, tile = s.tile;
            nq = (rows + BQ - 1) / BQ;
        }
    }
    const uint16_t* const w = a.w + (size_t)t.expert * a.N * a.K;
    const uint16_t* const x = a.x + t.row0 * a.ldx;
    const uint16_t* const dz = a.dz + t.row0 * a.lddz;
    const uint16_t* const rest = TWO ? rest_of(a, t.row0, t.row0) : dz;
    // (dz's rows are padded to whole chunks with zeros)
    if (KIND == FWD) t.P = {w, w, a.K, a.N, a.K}, t.Q = {x, x, a.ldx, rows, a.K};
    if (KIND == DX) t.P = {w, w, a.K, a.K, a.N}, t.Q = {dz, rest, a.lddz, rows, padded(a.N)};
    if (KIND == DW) t.P = {x, x, a.ldx, a.K, rows}, t.Q = {dz, rest, a.lddz, padded(a.N), rows};
    // eight q tiles deep, so that the tiles an XCD works on at a time share their operands in its L2
    const int deep = 8 * np, gr = tile / deep, gq = min(8, nq - gr * 8), in = tile - gr * deep;
    t.q0 = (gr * 8 + in % gq) * BQ;
    t.p0 = in / gq * BP;
    return t;
}

// what other lanes of the wavefront wrote to LDS before is read after, and the other way round
MOE_DEV void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// A wavefront's own piece of LDS, through which its sums pass on their way out: a few rows of TP values at a time
template <int TP>
struct Slab {
    static constexpr int LPR = TP / 8, ROWS = 64 / LPR >= 16 ? 16 : 8, STRIDE = TP + 4;   // lanes per row
    static constexpr int BYTES = ROWS * STRIDE * 4;
};
// eight values (KIND FWD: sums, with the bias and the residual as they lie) on their way to memory
template <typename T, int ACT>
MOE_DEV void put_forward(const LinArgs& a, int64_t row, int p, int left, float (&o)[8], const uint4& bias, const uint4& residual) {
    float b[8], res[8];
    unpack8<T>(bias, b);
    unpack8<T>(residual, res);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += b[i];
    if (ACT != MOE_ACT_NONE && a.z != nullptr) {
        float* z = a.z + row * padded(a.N) + p;
        *reinterpret_cast<f32x4*>(z) = (f32x4){o[0], o[1], o[2], o[3]};
        *reinterpret_cast<f32x4*>(z + 4) = (f32x4){o[4], o[5], o[6], o[7]};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = act_of<ACT>(o[i]) + res[i];
    store8(a.y + row * a.ldy + p, left, pack8<T>(o));
}
// What a wavefront does with its sums of 16 NJ q (from qw) and TP p (from pw): v[i][j] of a lane is p = 16 i +
// 4 g + 0..3 of q = 16 j + l16. They pass through the wavefront's own piece of LDS, a few rows at a time, so
// that a lane has eight values of one row, and its neighbours the ones beside them: memory is read and written in
// whole lines (four values a lane wrote quarters of them).
template <typename T, Kind KIND, int ACT, int TP, int NI, int NJ>
MOE_DEV void finish(const LinArgs& a, const Tile& t, int qw, int pw, const f32x4 (&v)[NI][NJ], float* slab) {
    typedef Slab<TP> S;
    const int lane = lane_here(), l16 = lane & 15, g = lane >> 4;
    const int r = lane / S::LPR, c = lane % S::LPR * 8;
    const int rows = KIND == DW ? a.N : t.Q.rows, p = t.p0 + pw + c, left = (KIND == FWD ? a.N : a.K) - p;
    if (qw >= rows) return;
    const bool mine = lane < S::ROWS * S::LPR && left > 0;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 bias = KIND == FWD && a.bias != nullptr && mine ? load8(a.bias + (size_t)t.expert * a.N + p, left) : none;
    auto residual = [&](int q) { return a.residual != nullptr && mine && q < rows ? load8(a.residual + (t.row0 + q) * a.ldr + p, left) : none; };
    uint4 next = KIND == FWD ? residual(qw + r) : none;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < 16 / S::ROWS; ++h) {
            if (S::ROWS == 16 || (l16 >> 3) == h) {
#pragma unroll
                for (int i = 0; i < NI; ++i) *reinterpret_cast<f32x4*>(&slab[(l16 & (S::ROWS - 1)) * S::STRIDE + 16 * i + 4 * g]) = v[i][j];
            }
            wave_fence();
            const int at = mine ? r * S::STRIDE + c : 0;
            const f32x4 lo = *reinterpret_cast<const f32x4*>(&slab[at]), hi = *reinterpret_cast<const f32x4*>(&slab[at + 4]);
            wave_fence();
            const int q = qw + 16 * j + S::ROWS * h + r;
            const int64_t row = t.row0 + q;
            float o[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if constexpr (KIND == FWD) {
                const uint4 here = next;
                next = residual(q + S::ROWS);
                if (mine && q < rows) put_forward<T, ACT>(a, row, p, left, o, bias, here);
            } else if (mine && q < rows) {   // (K is a multiple of 8)
                uint16_t* const to = KIND == DX ? a.dx + row * a.lddx : a.dw + ((size_t)t.expert * a.N + q) * a.K;
                *reinterpret_cast<uint4*>(to + p) = pack8<T>(o);
            }
        }
}

// order[i]: the experts with more than TWO_PARTS rows and then the others, so that either are one run; up to 64 of them (a lane
// each) with the most rows first, equal ones in their order, and more as they come. counts: room for E of them. -> how many
// have more than TWO_PARTS. Every workgroup does this before its first load. dW with the most rows first (of more than 64, each
// compared with each) and as they come: 32 experts of 2048 x 1408, 16184 rows 140 and 172 us; 64 of 1024 x 1024, 8000 rows
// 49 and 53; 128 of 512 x 512, 4000 rows 24.6 and 21.2; 384 of 256 x 256, 2500 rows 29.7 and 20.5; 1024 of 72 x 40, 2500 rows
// 123 and 13.
MOE_DEV int sort_experts(const LinArgs& a, int threads, int* counts, uint16_t* order) {
    for (int e = threadIdx.x; e < a.experts; e += threads) counts[e] = max(offset_at(a, e + 1) - offset_at(a, e), 0);
    __syncthreads();
    const int lane = threadIdx.x & 63;
    int many = 0;
    if (a.experts <= 64) {
        const int mine = lane < a.experts ? counts[lane] : -1;
        int before = 0;
        for (int i = 0; i < a.experts; ++i) {
            const int n = __builtin_amdgcn_readlane(mine, i);
            before += n > mine || (n == mine && i < lane) ? 1 : 0;
        }
        if (threadIdx.x < a.experts) order[before] = (uint16_t)lane;
        many = __popcll(__ballot(mine > TWO_PARTS));
    } else {
        auto has_many = [&](int e) { return e < a.experts && counts[min(e, a.experts - 1)] > TWO_PARTS; };
        for (int e0 = 0; e0 < a.experts; e0 += 64) many += __popcll(__ballot(has_many(e0 + lane)));
        int more = 0;   // experts before these with more than TWO_PARTS
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane;
            const bool on = has_many(e);
            const uint64_t all = __ballot(on);
            const int of = __popcll(all & ((1ull << lane) - 1));
            if (e < a.experts && threadIdx.x < 64) order[on ? more + of : many + (e0 - more) + (lane - of)] = (uint16_t)e;
            more += __popcll(all);
        }
    }
    __syncthreads();
    return many;
}

// The work of one product: the first `whole` tiles, each in one piece, and the `rest` in `splits` pieces along k.
// With offsets nothing is split, and of a product of the tokens' rows `whole` is only a bound.
struct Plan {
    int nq, np;          // tiles along q and p
    int whole, rest, splits;
    float* partial;      // [split][rest][j][i][thread] of the split tiles' sums, four f32 each
};

// TWO: of matrices with dz in two parts
template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP, bool TWO = false>
struct LinTile : TileProduct<T, p_by_rows(KIND), q_by_rows(KIND), false, BQ, BP, WQ, WP, TWO && KIND == DX, TWO && KIND == DW> {
    typedef TileProduct<T, p_by_rows(KIND), q_by_rows(KIND), false, BQ, BP, WQ, WP, TWO && KIND == DX, TWO && KIND == DW> Base;
    static constexpr bool FOLDED = TWO && KIND == DX;
    // rows of q in results: of a wavefront's 64 rows of dx the first 32 are of the first part, the others of the second
    static constexpr int BQ_OUT = FOLDED ? BQ / 2 : BQ, TQ_OUT = FOLDED ? Base::TQ / 2 : Base::TQ, NJ_OUT = FOLDED ? Base::NJ / 2 : Base::NJ;
    static_assert(!FOLDED || Base::TQ % 64 == 0, "");
    static MOE_DEV auto& results(f32x4 (&acc)[Base::NI][Base::NJ], f32x4 (&out)[Base::NI][NJ_OUT]) {
        if constexpr (FOLDED) {
#pragma unroll
            for (int i = 0; i < Base::NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ_OUT; ++j) out[i][j] = acc[i][j / 2 * 4 + j % 2] + acc[i][j / 2 * 4 + j % 2 + 2];
            return out;
        } else {
            return acc;
        }
    }
};

struct Piece {
    Tile t;
    int tile, split, kt0, nk;   // split < 0: a whole tile
};
// Pieces that an XCD has of a product: an eighth of the whole tiles, side by side, and of the others
struct Share {
    int w0, whole, s0, pieces;
};
MOE_DEV Share share_of(const Plan& plan, int whole, int xcd) {
    const int64_t pieces = (int64_t)plan.rest * plan.splits;
    Share s;
    s.w0 = (int)((int64_t)whole * xcd >> 3), s.whole = (int)((int64_t)whole * (xcd + 1) >> 3) - s.w0;
    s.s0 = (int)(pieces * xcd >> 3), s.pieces = (int)(pieces * (xcd + 1) >> 3) - s.s0;
    return s;
}
MOE_DEV void piece_at(const Plan& plan, const Share& s, int place, Piece& x) {
    x.split = -1;
    if (place < s.whole) {
        x.tile = s.w0 + place;
    } else {
        const int item = s.s0 + place - s.whole;
        x.split = item / plan.rest;
        x.tile = plan.whole + item - x.split * plan.rest;
    }
}
template <Kind KIND, bool GROUPED, int BQ, int BP, bool TWO, int SPAN, Only ONLY>
MOE_DEV void open_piece(const LinArgs& a, const Plan& plan, const uint16_t* order, Piece& x) {
    x.t = locate<KIND, GROUPED, BQ, BP, TWO, ONLY>(a, x.tile, plan.nq, plan.np, order);
    const int steps = (x.t.P.k + SPAN - 1) / SPAN;
    x.kt0 = GROUPED || x.split < 0 ? 0 : (int)((int64_t)x.split * steps / plan.splits);
    x.nk = (GROUPED || x.split < 0 ? steps : (int)((int64_t)(x.split + 1) * steps / plan.splits)) - x.kt0;
}
template <int TH, int NI, int NJ>
MOE_DEV void store_sums(const Plan& plan, const Piece& x, const f32x4 (&acc)[NI][NJ]) {
    f32x4* o = reinterpret_cast<f32x4*>(plan.partial) + (size_t)(x.split * plan.rest + x.tile - plan.whole) * NI * NJ * TH + threadIdx.x;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) o[(j * NI + i) * TH] = acc[i][j];
}

// Both kernels: a workgroup takes one piece after another. The loads of the next piece's first two steps are under
// way while it finishes the one before. The pointers into LDS are a lambda's own restricted ones there, so that the
// compiler does not wait for these loads before it reads the slab. In dx and dW it waits nowhere in a tile's end; forward it
// does, once or twice in each of the sixteen passes from the third on: the branches of load8 and store8 for a row's tail keep
// it from counting what is under way, in whole tiles too. GROUPED: with offsets.
template <typename T, bool GROUPED, int ACT, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void linear_forward_kernel(LinArgs a, Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    typedef LinTile<T, FWD, BQ, BP, WQ, WP> Product;
    constexpr int NI = Product::NI, NJ = Product::NJ;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wq = wv / WP, wp = wv % WP;
    float* const slab = reinterpret_cast<float*>(smem + Product::LDS + wv * Slab<Product::TP>::BYTES);
    const Share mine = share_of(plan, GROUPED ? tiles_total<ALL>(a, BQ) * plan.np : plan.whole, blockIdx.x & 7);
    int place = blockIdx.x >> 3;
    if (place >= mine.whole + mine.pieces) return;
    Piece now;
    piece_at(plan, mine, place, now);
    open_piece<FWD, GROUPED, BQ, BP, false, Product::KSPAN, ALL>(a, plan, nullptr, now);
    Product::begin({now.t.P, now.t.Q, 1, now.t.q0, now.t.p0, now.kt0, now.nk}, smem);
    for (;;) {
        f32x4 acc[NI][NJ];
        Product::template sums<true>({now.t.P, now.t.Q, 1, now.t.q0, now.t.p0, now.kt0, now.nk}, smem, acc);
        Piece next;
        place += gridDim.x >> 3;
        const bool more = place < mine.whole + mine.pieces;
        if (more) {
            piece_at(plan, mine, place, next);
            open_piece<FWD, GROUPED, BQ, BP, false, Product::KSPAN, ALL>(a, plan, nullptr, next);
        }
        barrier_lds();   // every wavefront has read the last step
        [&](uint8_t* __restrict buffers, float* __restrict own) {
            if (more) Product::begin({next.t.P, next.t.Q, 1, next.t.q0, next.t.p0, next.kt0, next.nk}, buffers);
            if (!GROUPED && now.split >= 0) store_sums<Product::TH>(plan, now, acc);
            else finish<T, FWD, ACT, Product::TP, NI, NJ>(a, now.t, now.t.q0 + wq * Product::TQ, wp * Product::TP, acc, own);
        }(smem, slab);
        if (!more) return;
        now = next;
    }
}

// What a workgroup has of one product's pieces in the backward pass. The XCD's pieces, `count` of this product
// after `base` of another, go to its workgroups forth and back; run: with offsets, dW's tiles side by side on an XCD.
template <typename T, Kind KIND, bool GROUPED, int B, int WQ, int WP, bool TWO, Only ONLY>
MOE_DEV void run_pieces(const LinArgs& a, const Plan& plan, const Share& mine, int base, int count, int run, int& turn,
                        const uint16_t* order, uint8_t* smem, float* slab) {
    typedef LinTile<T, KIND, B, B, WQ, WP, TWO> Product;
    constexpr int NI = Product::NI, NJ = Product::NJ, NJ_OUT = Product::NJ_OUT;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wq = wv / WP, wp = wv % WP;
    auto take = [&](Piece& x) -> bool {
        const int step = gridDim.x >> 3, at = blockIdx.x >> 3, xcd = blockIdx.x & 7;
        for (;;) {
            const int place = turn * step + (turn & 1 ? step - 1 - at : at) - base;
            if (place >= count) return false;
            ++turn;
            if (GROUPED && KIND == DW) {
                x.tile = (place / run * 8 + xcd) * run + place % run, x.split = -1;
                if (x.tile >= plan.whole) continue;
            } else {
                piece_at(plan, mine, place, x);
            }
            open_piece<KIND, GROUPED, Product::BQ_OUT, B, TWO, Product::KSPAN, ONLY>(a, plan, order, x);
            return true;
        }
    };
    Piece now;
    if (!take(now)) return;
    barrier_lds();   // (what was in the buffers is read)
    Product::begin({now.t.P, now.t.Q, 1, now.t.q0, now.t.p0, now.kt0, now.nk}, smem);
    for (;;) {
        f32x4 acc[NI][NJ];
        Product::template sums<true>({now.t.P, now.t.Q, 1, now.t.q0, now.t.p0, now.kt0, now.nk}, smem, acc);
        f32x4 out[NI][NJ_OUT];
        auto& v = Product::results(acc, out);
        Piece next;
        const bool more = take(next);
        barrier_lds();   // every wavefront has read the last step
        [&](uint8_t* __restrict buffers, float* __restrict own) {
            if (more) Product::begin({next.t.P, next.t.Q, 1, next.t.q0, next.t.p0, next.kt0, next.nk}, buffers);
            if (!GROUPED && now.split >= 0) store_sums<Product::TH>(plan, now, v);
            else finish<T, KIND, MOE_ACT_NONE, Product::TP, NI, NJ_OUT>(a, now.t, now.t.q0 + wq * Product::TQ_OUT, wp * Product::TP, v, own);
        }(smem, slab);
        if (!more) return;
        now = next;
    }
}

// dx and dW of one matrix in one launch, so that the longer pieces of the one (W_FIRST: dW's) are filled up with the other's:
// neither fills the CUs evenly by itself.
template <typename T, bool W_FIRST, int B, int WQ, int WP, bool TWO>
__global__ __launch_bounds__(64 * WQ * WP) void linear_backward_kernel(LinArgs a, Plan px, Plan pw) {
    extern __shared__ __align__(16) uint8_t smem[];
    typedef LinTile<T, DX, B, B, WQ, WP, TWO> ProductX;
    typedef LinTile<T, DW, B, B, WQ, WP, TWO> ProductW;
    constexpr size_t LDS = ProductX::LDS > ProductW::LDS ? ProductX::LDS : ProductW::LDS;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), xcd = blockIdx.x & 7;
    float* const slab = reinterpret_cast<float*>(smem + LDS + wv * Slab<ProductX::TP>::BYTES);
    const Share sx = share_of(px, px.whole, xcd), sw = share_of(pw, pw.whole, xcd);
    const int nx = sx.whole + sx.pieces, nw = sw.whole + sw.pieces;
    int turn = 0;
    if (W_FIRST) run_pieces<T, DW, false, B, WQ, WP, TWO, ALL>(a, pw, sw, 0, nw, 1, turn, nullptr, smem, slab);
    run_pieces<T, DX, false, B, WQ, WP, TWO, ALL>(a, px, sx, W_FIRST ? nw : 0, nx, 1, turn, nullptr, smem, slab);
    if (!W_FIRST) run_pieces<T, DW, false, B, WQ, WP, TWO, ALL>(a, pw, sw, nx, nw, 1, turn, nullptr, smem, slab);
}

// dx or dW of a matrix per expert, with dz in one part (PARTS 1), in two (2), or in two of those with few rows (BOTH). dW's
// tiles have as many steps as their expert has rows: each XCD has an eighth of each expert's, those with the most rows
// first (experts of 8 to 2000 rows, 506 on average: no workgroup has more than a quarter above the mean, where an eighth of the
// experts for each XCD left one with twice the mean).
constexpr int BOTH = 3;
template <typename T, Kind KIND, int B, int WQ, int WP, int PARTS>
__global__ __launch_bounds__(64 * WQ * WP) void linear_experts_backward_kernel(LinArgs a, Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    typedef LinTile<T, KIND, B, B, WQ, WP, PARTS == 2> Product;
    typedef LinTile<T, KIND, B, B, WQ, WP, true> Few;
    constexpr int SLAB = Slab<Product::TP>::BYTES;
    constexpr Only FIRST = PARTS == BOTH ? MANY : ALL;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), xcd = blockIdx.x & 7;
    float* const slab = reinterpret_cast<float*>(smem + Product::LDS + wv * SLAB);
    uint16_t* const order = reinterpret_cast<uint16_t*>(smem + Product::LDS + WQ * WP * SLAB);
    int turn = 0;
    if (KIND == DW) {
        const int many = sort_experts(a, Product::TH, reinterpret_cast<int*>(smem), order), each = plan.nq * plan.np;
        const int run = max((each + 7) >> 3, 1);
        auto count = [&](int tiles) { return (tiles + 8 * run - 1) / (8 * run) * run; };
        if (PARTS == BOTH) plan.whole = many * each;
        const int n = count(plan.whole);
        run_pieces<T, KIND, true, B, WQ, WP, PARTS == 2, FIRST>(a, plan, Share{}, 0, n, run, turn, order, smem, slab);
        if (PARTS == BOTH) {
            plan.whole = (a.experts - many) * each;
            run_pieces<T, KIND, true, B, WQ, WP, true, FEW>(a, plan, Share{}, n, count(plan.whole), run, turn, order + many, smem, slab);
        }
    } else {
        const Share mine = share_of(plan, tiles_total<FIRST>(a, Product::BQ_OUT) * plan.np, xcd);
        run_pieces<T, KIND, true, B, WQ, WP, PARTS == 2, FIRST>(a, plan, mine, 0, mine.whole, 1, turn, nullptr, smem, slab);
        if (PARTS == BOTH) {
            const Share few = share_of(plan, tiles_total<FEW>(a, Few::BQ_OUT) * plan.np, xcd);
            run_pieces<T, KIND, true, B, WQ, WP, true, FEW>(a, plan, few, mine.whole, few.whole, 1, turn, nullptr, smem, slab);
        }
    }
}

// The split tiles' sums, added in order of k, and what is done with them: a workgroup per
// tile and j (16 q of each wavefront)
template <typename T, Kind KIND, int ACT, int BQ, int BP, int WQ, int WP, bool TWO>
__global__ __launch_bounds__(64 * WQ * WP) void linear_join_kernel(LinArgs a, Plan plan) {
    typedef LinTile<T, KIND, BQ, BP, WQ, WP, TWO> Product;
    constexpr int TH = Product::TH, NI = Product::NI, NJ = Product::NJ_OUT;
    __shared__ __align__(16) float slab[WQ * WP][Slab<Product::TP>::BYTES / 4];
    const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), wq = wv / WP, wp = wv % WP;
    const int r = blockIdx.x / NJ, j = blockIdx.x % NJ;
    const f32x4* from = reinterpret_cast<const f32x4*>(plan.partial) + ((size_t)r * NJ + j) * NI * TH + tid;
    f32x4 v[NI][1];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i][0] = from[i * TH];
#pragma unroll 2
    for (int s = 1; s < plan.splits; ++s) {
        const f32x4* f = from + (size_t)s * plan.rest * NI * NJ * TH;
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i][0] += f[i * TH];
    }
    const Tile t = locate<KIND, false, Product::BQ_OUT, BP, TWO, ALL>(a, plan.whole + r, plan.nq, plan.np, nullptr);
    finish<T, KIND, ACT, Product::TP, NI, 1>(a, t, t.q0 + wq * Product::TQ_OUT + 16 * j, wp * Product::TP, v, slab[wv]);
}

// ------------------------------------------------------------------ dz and its column sums

// A workgroup owns a chunk of rows and 512 columns, eight per lane, a row per wavefront at a time. The rows may be
// several experts': where one ends the sums of its columns go to the row (chunk + expert) of `partial`, a number of
// its own for every expert in every chunk.
constexpr int DZ_COLS = 512;
// rows of a chunk: 16, or as many more as leave at least 512 chunks, up to 64 (1013 x 4101: 28.7 us with 64, 11.8
// with 16)
MOE_DEV __host__ int dz_rows(int m) { return m >= 512 * 64 ? 64 : m >= 512 * 32 ? 32 : 16; }
// at most as many chunks have m rows or fewer
int dz_chunks(int m) { return std::max({(m + 63) / 64, std::min((m + 15) / 16, 1024), std::min((m + 31) / 32, 1024)}); }

// The experts of rising rows: 64 experts' rows at a time wait in the lanes
struct ExpertWalk {
    int base, begin, end;   // the lane's: where expert base + lane begins and ends
};
MOE_DEV ExpertWalk walk_experts(const LinArgs& a, int row) {
    const int lane = threadIdx.x & 63;
    int n = 0;   // experts that end at `row` or before
    for (int e0 = 0; e0 < a.experts; e0 += 64) n += __popcll(__ballot(e0 + lane < a.experts && offset_at(a, e0 + lane + 1) <= row));
    return {n, offset_at(a, n + lane), offset_at(a, n + lane + 1)};
}
// the expert of `row` and where it begins and ends (experts that are not there end with the last)
MOE_DEV int expert_of(const LinArgs& a, ExpertWalk& w, int row, int& begin, int& end) {
    uint64_t past;
    while ((past = __ballot(w.end > row)) == 0 && w.base + 64 < a.experts) {
        w.base += 64;
        w.begin = offset_at(a, w.base + (threadIdx.x & 63));
        w.end = offset_at(a, w.base + (threadIdx.x & 63) + 1);
    }
    const int l = past != 0 ? __builtin_ctzll(past) : 0;
    begin = __builtin_amdgcn_readlane(w.begin, l);
    end = __builtin_amdgcn_readlane(w.end, l);
    return min(w.base + l, a.experts - 1);
}

// STORE: dz is wanted (else it is dy itself, and only the sums are)
template <typename T, bool STORE>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinArgs a) {
    __shared__ float lds[4][DZ_COLS];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    constexpr int U = 4;   // rows that a wavefront requests at a time
    const int chunk = dz_rows(a.m), first = blockIdx.x * chunk, n0 = blockIdx.y * DZ_COLS + lane * 8, left = a.N - n0;
    const int last = min(first + chunk, a.offsets != nullptr ? offset_of(a, a.experts) : a.m);
    const bool parts = a.offsets != nullptr && a.partial != nullptr;   // each expert's sums are wanted
    const bool two = STORE && a.dz_rest != nullptr;
    ExpertWalk walk{0, 0, 0};
    uint64_t few = ~0ull;   // the chunk's rows that have a second part
    const bool some = two && !all_two(a.m, a.experts);
    if ((parts || some) && first < last) walk = walk_experts(a, first);
    if (some) {
        few = 0;
        ExpertWalk w = walk;
        for (int row = first; row < last;) {
            int begin, end;
            expert_of(a, w, row, begin, end);
            const bool all = end - begin <= TWO_PARTS;
            end = max(min(last, end), row + 1);
            // (whatever the offsets hold, what is written lies among 64 rows)
            if (all && row >= begin && end - begin <= TWO_PARTS) few |= (~0ull >> (64 - (end - row))) << (row - first);
            row = end;
        }
    }
    const int row0 = some ? offset_of(a, 0) : 0;
    int row = first;
    while (row < last) {
        int e = 0, begin = 0, end = last;
        if (parts) {
            e = expert_of(a, walk, row, begin, end);
            end = max(min(last, end), row + 1);   // (offsets that go back must not hold the loop up)
        }
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
        for (int r0 = row + wv; r0 < end && left > 0; r0 += 4 * U) {
            uint4 dy[U];
            f32x4 z[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = min(r0 + 4 * u, end - 1);
                dy[u] = load8(a.dy + r * a.lddy + n0, left);
                if (a.act != MOE_ACT_NONE) {
                    const float* from = a.z + (size_t)r * padded(a.N) + n0;
                    z[u][0] = *reinterpret_cast<const f32x4*>(from), z[u][1] = *reinterpret_cast<const f32x4*>(from + 4);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + 4 * u;
                float d[8];
                unpack8<T>(dy[u], d);
                if (a.act != MOE_ACT_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = i < left ? d[i] * act_slope(z[u][i >> 2][i & 3], a.act) : 0.f;
                }
                if (r < end) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += d[i];
                    if (STORE) {
                        const uint4 q = pack8<T>(d);
                        *reinterpret_cast<uint4*>(a.dz_out + r * a.lddz + n0) = q;
                        if (two && (few >> (r - first) & 1)) {
                            float hi[8];
                            unpack8<T>(q, hi);   // (what is infinite or NaN leaves nothing)
#pragma unroll
                            for (int i = 0; i < 8; ++i) hi[i] = fabsf(hi[i]) <= 3.4e38f ? d[i] - hi[i] : 0.f;
                            *reinterpret_cast<uint4*>(rest_of(a, r, row0) + n0) = pack8<T>(hi);
                        }
                    }
                }
            }
        }
        if (a.partial != nullptr) {
            *reinterpret_cast<f32x4*>(&lds[wv][lane * 8]) = (f32x4){sum[0], sum[1], sum[2], sum[3]};
            *reinterpret_cast<f32x4*>(&lds[wv][lane * 8 + 4]) = (f32x4){sum[4], sum[5], sum[6], sum[7]};
            __syncthreads();
            for (int c = tid; c < DZ_COLS; c += 256) {
                const int n = blockIdx.y * DZ_COLS + c;
                if (n < a.N) a.partial[(size_t)(blockIdx.x + e) * a.N + n] = (lds[0][c] + lds[1][c]) + (lds[2][c] + lds[3][c]);
            }
            __syncthreads();
        }
        row = end;
    }
}

// dbias: the sums of an expert's chunks in a fixed order, 64 columns by 16 threads each
template <typename T>
__global__ __launch_bounds__(1024) void linear_bias_kernel(LinArgs a) {
    __shared__ float lds[16][64];
    const int c = threadIdx.x & 63, g = threadIdx.x >> 6, e = blockIdx.y, n = blockIdx.x * 64 + c;
    const int r0 = a.offsets != nullptr ? offset_of(a, e) : 0, r1 = a.offsets != nullptr ? offset_of(a, e + 1) : a.m;
    float s = 0.f;
    const int chunk = dz_rows(a.m);
    if (n < a.N && r1 > r0)
#pragma unroll 8
        for (int b = r0 / chunk + g; b <= (r1 - 1) / chunk; b += 16) s += a.partial[(size_t)(b + e) * a.N + n];
    lds[g][c] = s;
    __syncthreads();
    if (g == 0 && n < a.N) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += lds[i][c];
        a.dbias[(size_t)e * a.N + n] = T::store(s);
    }
}

// ------------------------------------------------------------------ few rows

// Up to 16 rows of each matrix: FWD with the weights read straight into registers, since nothing would be
// read twice. A workgroup multiplies 16 weight rows at a time, each wavefront a part of k, and their sums are joined through
// LDS in wavefront order. x comes into LDS whole.
constexpr int FEW_WAVES = 8, FEW_ROWS = 16;
constexpr int FEW_LDS = 64 << 10;
// values of k of a row in LDS, whole runs of 1024 bytes
MOE_DEV __host__ int few_row(int K) { return (K + 511) / 512 * 512; }

template <typename T, int ACT>
__global__ __launch_bounds__(64 * FEW_WAVES) void linear_few_kernel(LinArgs a, int room) {
    constexpr int AHEAD = 5;
    extern __shared__ __align__(16) uint8_t smem[];   // x; then sums [wavefront][256]
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, row_bytes = few_row(a.K) * 2, runs = row_bytes / 1024;
    Slice s{0, 0, a.m, 0};
    if (a.offsets != nullptr) {
        if (!find_slice<ALL>(a, room, 1, blockIdx.y, s)) return;
    } else {
        s.tile = blockIdx.y;
    }
    const int rows = min(s.rows - s.tile * room, room), row0 = s.row0 + s.tile * room;
    const uint16_t* const w0 = a.w + (size_t)s.expert * a.N * a.K;
    const uint16_t* const w = w0 + (size_t)min(n0 + l16, a.N - 1) * a.K;
    const auto X = buffer_rsrc(a.x + row0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K) * 2);
    const int xt = min(l16, rows - 1);   // (a token that does not exist reads another's; its sums are not used)
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    // the first wavefront finishes: eight values of row lane / 2 a lane. What it adds is requested before the weights
    const int er = lane >> 1, ep = n0 + (lane & 1) * 8, left = a.N - ep;
    const bool ends = wv == 0 && er < rows && left > 0;
    uint4 bias = make_uint4(0, 0, 0, 0), residual = bias;
    if (ends && a.bias != nullptr) bias = load8(a.bias + (size_t)s.expert * a.N + ep, left);
    if (ends && a.residual != nullptr) residual = load8(a.residual + (row0 + er) * a.ldr + ep, left);
    const int chunks = (a.K + 31) / 32, c0 = wv * chunks / FEW_WAVES, c1 = (wv + 1) * chunks / FEW_WAVES;
    for (int r = wv; r < rows * runs; r += FEW_WAVES) {
        // 16-byte chunk c of a row lies at c ^ (row & 15)
        const int row = r / runs, k = (r - row * runs) * 512 + (lane ^ (row & 15)) * 8;
        buffer_load_lds16(X, smem + r * 1024, k < a.K ? (uint32_t)(row * a.ldx + k) * 2 : PAST);
    }
    __atomic_signal_fence(__ATOMIC_SEQ_CST);   // (x is requested before any weight: the wait below counts back from the last)
    uint4 wq[AHEAD];
    auto request = [&](int i, int c) { wq[i] = *reinterpret_cast<const uint4*>(w + min(32 * min(c, chunks - 1) + 8 * g, a.K - 8)); };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) request(i, c0 + i);
    wait_vm_loads<AHEAD>();   // this wavefront's part of x has landed
    barrier_lds();
    auto multiply = [&](int i, int c) {
        // a weight that stands in for one past K is not one (x is zero there)
        const uint32_t on = 32 * c + 8 * g < a.K ? ~0u : 0u;
        const u32x4 wm = {wq[i].x & on, wq[i].y & on, wq[i].z & on, wq[i].w & on};
        const int cx = c * 4 + g;
        acc = T::mfma(__builtin_bit_cast(s16x8, wm), *reinterpret_cast<const s16x8*>(smem + xt * row_bytes + ((cx ^ (xt & 15)) << 4)), acc);
    };
    int c = c0;
    for (; c + AHEAD < c1; c += AHEAD)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            multiply(i, c + i);
            request(i, c + AHEAD + i);
        }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (c + i < c1) multiply(i, c + i);   // (a chunk of another's part is left out)
    __syncthreads();   // x is read; the sums take its place
    float* red = reinterpret_cast<float*>(smem);
    *reinterpret_cast<f32x4*>(&red[wv * 256 + lane * 4]) = acc;
    __syncthreads();
    if (!ends) return;
    // weight row 4 g + r of token l16 lies at 64 g + 4 l16 + r of a wavefront's sums
    float o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < FEW_WAVES; ++i) v += *reinterpret_cast<const f32x4*>(&red[i * 256 + (2 * (lane & 1) + h) * 64 + er * 4]);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[4 * h + r] = v[r];
    }
    put_forward<T, ACT>(a, row0 + er, ep, left, o, bias, residual);
}

// Up to eight rows of one matrix, backward, in one pass over the weights: with so few rows the products are bound by reading W and
// writing dW, dz can stay in f32 (a lane multiplies it itself), and nothing but dx's sums needs a second launch. A
// workgroup has 512 columns of k, eight a lane, and `rows` weight rows, every fourth a wavefront; dz of 64 of them at a
// time waits in LDS. Silu, all three gradients, weights from memory (K x N), and with dz, its sums and tiles instead: one row
// of 5120 x 2304 18.3 us and 31.0 (47 MB), eight 23.0 and 31.3; of 4096 x 16384 70 and 121, eight 75 and 121 (268 MB); of 952 x
// 364 10.6 and 13.3; eight of 8192 x 512 16.1 and 16.6. Sixteen rows of x and dx would not fit the registers.
constexpr int FEW_BACK = 8, FEW_BACK_COLS = 512, FEW_BACK_ROWS = 64;

template <typename T, int M>
__global__ __launch_bounds__(256) void linear_few_backward_kernel(LinArgs a, int rows) {
    __shared__ __align__(16) float dzs[FEW_BACK_ROWS][M];
    __shared__ __align__(16) float red[4][FEW_BACK_COLS];
    constexpr int U = 4;   // weight rows that a wavefront requests at a time
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int k = blockIdx.x * FEW_BACK_COLS + lane * 8, first = blockIdx.y * rows, last = min(first + rows, a.N);
    const bool live = k < a.K;
    const int at = live ? k : 0;   // (a lane past K reads the first columns and writes none)
    float x[M][8], dx[M][8];
#pragma unroll
    for (int t = 0; t < M; ++t) {
        uint4 q = make_uint4(0, 0, 0, 0);   // (a row that does not exist: its dz is zero too)
        if (t < a.m && a.dw != nullptr) q = *reinterpret_cast<const uint4*>(a.x + t * a.ldx + at);
        unpack8<T>(q, x[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dx[t][i] = 0.f;
    }
    for (int n0 = first; n0 < last; n0 += FEW_BACK_ROWS) {
        const int here = min(last - n0, FEW_BACK_ROWS);
        for (int i = tid; i < FEW_BACK_ROWS * M; i += 256) {
            const int t = i / FEW_BACK_ROWS, r = i % FEW_BACK_ROWS, n = n0 + r;
            float d = 0.f;
            if (t < a.m && r < here) {
                d = T::load(a.dy[t * a.lddy + n]);
                if (a.act != MOE_ACT_NONE) d *= act_slope(a.z[(size_t)t * padded(a.N) + n], a.act);
            }
            dzs[r][t] = d;
        }
        __syncthreads();
        if (a.dbias != nullptr && blockIdx.x == 0 && tid < here) {
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < M; ++t) s += dzs[tid][t];
            a.dbias[n0 + tid] = T::store(s);
        }
        if (a.dx != nullptr || a.dw != nullptr)
            for (int r0 = wv; r0 < here; r0 += 4 * U) {
                uint4 w[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    w[u] = make_uint4(0, 0, 0, 0);
                    if (a.dx != nullptr) w[u] = *reinterpret_cast<const uint4*>(a.w + (size_t)(n0 + min(r0 + 4 * u, here - 1)) * a.K + at);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + 4 * u;
                    if (r >= here) break;
                    float v[8], o[8], dz[M];
                    unpack8<T>(w[u], v);
#pragma unroll
                    for (int t = 0; t < M; ++t) dz[t] = dzs[r][t];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll
                    for (int t = 0; t < M; ++t)
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] += dz[t] * x[t][i], dx[t][i] += dz[t] * v[i];
                    if (a.dw != nullptr && live) *reinterpret_cast<uint4*>(a.dw + (size_t)(n0 + r) * a.K + k) = pack8<T>(o);
                }
            }
        __syncthreads();   // dz is read
    }
    if (a.dx == nullptr) return;
    // the wavefronts' sums in their order, a row at a time
#pragma unroll
    for (int t = 0; t < M; ++t) {
        if (t < a.m) {
            *reinterpret_cast<f32x4*>(&red[wv][lane * 8]) = (f32x4){dx[t][0], dx[t][1], dx[t][2], dx[t][3]};
            *reinterpret_cast<f32x4*>(&red[wv][lane * 8 + 4]) = (f32x4){dx[t][4], dx[t][5], dx[t][6], dx[t][7]};
            __syncthreads();
            for (int c = tid; c < FEW_BACK_COLS; c += 256) {
                const int col = blockIdx.x * FEW_BACK_COLS + c;
                const float s = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
                if (col < a.K) {
                    if (gridDim.y == 1) a.dx[t * a.lddx + col] = T::store(s);
                    else a.partial[((size_t)blockIdx.y * a.m + t) * a.K + col] = s;
                }
            }
            __syncthreads();
        }
    }
}

// dx: the sums of `pieces` parts of the weight rows in a fixed order, 256 columns of a row by 16 wavefronts
template <typename T>
__global__ __launch_bounds__(1024) void linear_few_join_kernel(LinArgs a, int pieces) {
    __shared__ __align__(16) f32x4 lds[16][64];
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6, k = blockIdx.x * 256 + lane * 4, t = blockIdx.y;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (k < a.K)
#pragma unroll 8
        for (int i = g; i < pieces; i += 16) s += *reinterpret_cast<const f32x4*>(a.partial + ((size_t)i * a.m + t) * a.K + k);
    lds[g][lane] = s;
    __syncthreads();
    if (g == 0 && k < a.K) {
        s = lds[0][lane];
#pragma unroll
        for (int i = 1; i < 16; ++i) s += lds[i][lane];
        *reinterpret_cast<uint2*>(a.dx + t * a.lddx + k) = make_uint2(T::pack2(s[0], s[1]), T::pack2(s[2], s[3]));
    }
}

// ------------------------------------------------------------------ plans

int cdiv(int a, int b) { return (a + b - 1) / b; }

constexpr int N_CU = 256, MAX_SPLITS = 16;

// The tiles that there are: BQ x BP, of how many the CUs hold at a time (LDS), and what a K step of so many at once
// takes, in us (forward; dx and dW, whose operands are transposed on their way from LDS), and the beginning and the
// end of one. Few rows only where they are the tokens'. Forward with each of the four: 8192 rows of 5120 x 2304 192, 216,
// 248 and 356 us; 64 experts of 2048 x 1408 with 47 rows each 132, 102, 92 and 96; 1013 rows of 1544 x 4101 52, 38.5, 37.9 and
// 48; 23 rows of 8192 x 2048 27.8, 18.5, 14.7 and 13.1. dx and dW with the first two: 382 and 445; 32 experts of 2048 x
// 1408, 16184 rows, 326 and 322; 1013 rows 62.8 and 61.8 (with dz and dbias).
struct Shape {
    int bq, bp, slots;
    double step, back, ends;
};
constexpr Shape SHAPES[] = {{256, 256, N_CU, 1.5, 1.7, 8}, {128, 128, 2 * N_CU, 1.0, 1.1, 6}, {64, 128, 2 * N_CU, 0.65, 0, 5}, {32, 128, 3 * N_CU, 0.65, 0, 5}};
constexpr int N_SHAPES = 4, BACK_SHAPES = 2;

struct Extent {
    int nq, np, tiles, steps;
    double likely;   // tiles that there will be
};
// tiles along q and p, all of them (with offsets: at most), K steps of one
Extent extent(Kind kind, int m, int N, int K, int experts, bool grouped, const Shape& s) {
    Extent e;
    e.steps = cdiv(kind == FWD ? K : kind == DX ? N : grouped ? cdiv(m, experts) : m, BK);
    e.nq = cdiv(kind == DW ? N : m, s.bq), e.np = cdiv(kind == FWD ? N : K, s.bp);
    e.tiles = kind == DW ? experts * e.nq * e.np : grouped ? (m / s.bq + std::min(experts, m)) * e.np : e.nq * e.np;
    e.likely = grouped && kind != DW ? std::min((double)e.tiles, (m / (double)s.bq + 0.5 * std::min(experts, m)) * e.np) : e.tiles;
    return e;
}
// Bytes that hold the split tiles' sums of any plan for m rows or fewer: the pieces are at most the
// slots, and at most the tiles times the splits
size_t partial_bytes(Kind kind, int m, int N, int K, int experts) {
    if (experts > 1) return 0;
    size_t most = 0;
    for (int i = 0; i < (kind == FWD ? N_SHAPES : BACK_SHAPES); ++i) {
        const Shape& s = SHAPES[i];
        const Extent e = extent(kind, m, N, K, 1, false, s);
        const int splits = std::min(MAX_SPLITS, e.steps / 2);
        if (splits >= 2) most = std::max(most, (size_t)std::min<int64_t>(s.slots, (int64_t)e.tiles * splits) * s.bq * s.bp * sizeof(float));
    }
    return round_up(most, 256);
}
// what the sums of n pieces cost: they pass through memory twice, at 5 TB/s, and their join is a launch
double join_cost(const Shape& s, int pieces) { return 6 + 2.0 * s.bq * s.bp * 4 / 5e6 * pieces; }

// How a forward pass is cut up: which tiles, and by how much those past the last full round of the CUs are split along
// k. With offsets nothing is split.
Plan plan_forward(int m, int N, int K, int experts, bool grouped, int* shape) {
    Plan best{};
    double best_cost = 1e300;
    for (int i = 0; i < N_SHAPES; ++i) {
        const Shape& s = SHAPES[i];
        const Extent e = extent(FWD, m, N, K, experts, grouped, s);
        Plan p{e.nq, e.np, e.tiles, 0, 1, nullptr};
        const double tile = e.steps * s.step + s.ends;
        double cost = std::max(1.0, std::ceil(e.likely / s.slots)) * tile;
        const int rest = e.tiles % s.slots;
        if (!grouped && rest > 0) {
            const double full = e.tiles / s.slots * tile;
            for (int n = 2; n <= MAX_SPLITS && n * 2 <= e.steps && rest * n <= s.slots; ++n) {
                const double c = full + cdiv(e.steps, n) * s.step + s.ends + join_cost(s, rest * n);
                if (c < cost) cost = c, p.whole = e.tiles - rest, p.rest = rest, p.splits = n;
            }
        }
        if (cost < best_cost) best_cost = cost, best = p, *shape = i;
    }
    return best;
}

// How dx and dW (where wanted) are: one kind of tiles for both, and in how many pieces along k those of either. With
// both (of one matrix), what they take together, and two fifths of the shorter piece for its end; with one, whole rounds.
// two: of matrices with dz in two parts, whose dx has tiles of one kind.
constexpr int TWO_SHAPE = 1;
struct BackPlan {
    Plan x, w;
    int shape;
    bool w_first;
};
BackPlan plan_backward(int m, int N, int K, int experts, bool grouped, bool two, bool want_x, bool want_w) {
    BackPlan best{};
    double best_cost = 1e300;
    for (int i = 0; i < BACK_SHAPES; ++i) {
        if (two && (want_x || !grouped) && i != TWO_SHAPE) continue;
        const Shape& s = SHAPES[i];
        const Shape half{s.bq / 2, s.bp, s.slots, s.step, s.back, s.ends};
        Extent e[2];
        Plan p[2]{};
        for (int k = 0; k < 2; ++k) {
            e[k] = extent(k == 0 ? DX : DW, m, N, K, experts, grouped, two && k == 0 ? half : s);
            if (k == 0 ? want_x : want_w) p[k] = {e[k].nq, e[k].np, e[k].tiles, 0, 1, nullptr};
            else e[k].tiles = 0, e[k].likely = 0;
        }
        auto splits_of = [&](int k, int n) { return n == 1 || (!grouped && e[k].tiles > 0 && n * 2 <= e[k].steps && (int64_t)e[k].tiles * n <= s.slots); };
        for (int nx = 1; nx <= MAX_SPLITS; ++nx) {
            if (!splits_of(0, nx)) continue;
            for (int nw = 1; nw <= MAX_SPLITS; ++nw) {
                if (!splits_of(1, nw)) continue;
                const int n[2] = {nx, nw};
                double piece[2], total = 0, joins = 0;
                for (int k = 0; k < 2; ++k) {
                    piece[k] = cdiv(e[k].steps, n[k]) * s.back + s.ends;
                    total += e[k].likely * n[k] * piece[k] / s.slots;
                    if (n[k] > 1) joins += join_cost(s, e[k].tiles * n[k]);
                }
                double cost;
                if (want_x && want_w) {
                    cost = std::max({total + 0.4 * std::min(piece[0], piece[1]), piece[0], piece[1]});
                } else {
                    const int k = want_x ? 0 : 1;
                    cost = std::max(1.0, std::ceil(e[k].likely * n[k] / s.slots)) * piece[k];
                }
                cost += joins;
                if (cost >= best_cost) continue;
                best_cost = cost;
                best.shape = i, best.w_first = piece[1] >= piece[0];
                best.x = p[0], best.w = p[1];
                for (int k = 0; k < 2; ++k)
                    if (n[k] > 1) {
                        Plan& q = k == 0 ? best.x : best.w;
                        q.rest = q.whole, q.whole = 0, q.splits = n[k];
                    }
            }
        }
    }
    return best;
}

template <typename T, Kind KIND, int ACT, int I, int WQ, int WP, bool TWO = false>
hipError_t launch_join(const LinArgs& a, const Plan& plan, hipStream_t st) {
    constexpr Shape S = SHAPES[I];
    typedef LinTile<T, KIND, S.bq, S.bp, WQ, WP, TWO> P;
    if (plan.rest == 0) return hipSuccess;
    return launch_kernel(linear_join_kernel<T, KIND, ACT, S.bq, S.bp, WQ, WP, TWO>, dim3(plan.rest * P::NJ_OUT), dim3(P::TH), 0, st, a, plan);
}
int grid_of(int64_t pieces, int slots) { return (int)std::min<int64_t>(slots, (pieces + 7) / 8 * 8); }
int64_t pieces_of(const Plan& p) { return p.whole + (int64_t)p.rest * p.splits; }

template <typename T, int ACT, int I, int WQ, int WP>
hipError_t launch_forward_tiles(const LinArgs& a, const Plan& plan, hipStream_t st) {
    constexpr Shape S = SHAPES[I];
    typedef LinTile<T, FWD, S.bq, S.bp, WQ, WP> P;
    auto* const k = a.offsets != nullptr ? linear_forward_kernel<T, true, ACT, S.bq, S.bp, WQ, WP> : linear_forward_kernel<T, false, ACT, S.bq, S.bp, WQ, WP>;
    const hipError_t e = launch_kernel(k, dim3(grid_of(pieces_of(plan), S.slots)), dim3(P::TH), P::LDS + WQ * WP * Slab<P::TP>::BYTES, st, a, plan);
    return e != hipSuccess ? e : launch_join<T, FWD, ACT, I, WQ, WP>(a, plan, st);
}
template <typename T, int ACT>
hipError_t launch_forward(const LinArgs& a, float* partial, hipStream_t st) {
    int shape = 0;
    Plan p = plan_forward(a.m, a.N, a.K, a.experts, a.offsets != nullptr, &shape);
    p.partial = partial;
    switch (shape) {
        case 0: return launch_forward_tiles<T, ACT, 0, 2, 4>(a, p, st);
        case 1: return launch_forward_tiles<T, ACT, 1, 2, 2>(a, p, st);
        case 2: return launch_forward_tiles<T, ACT, 2, 1, 4>(a, p, st);
        default: return launch_forward_tiles<T, ACT, 3, 1, 4>(a, p, st);
    }
}

template <typename T, int I, int WQ, int WP, bool TWO>
hipError_t launch_backward_tiles(const LinArgs& a, const BackPlan& b, hipStream_t st) {
    constexpr Shape S = SHAPES[I];
    typedef LinTile<T, DX, S.bq, S.bp, WQ, WP, TWO> X;
    typedef LinTile<T, DW, S.bq, S.bp, WQ, WP, TWO> W;
    const size_t lds = std::max(X::LDS, W::LDS) + WQ * WP * Slab<X::TP>::BYTES;
    auto* const k = b.w_first ? linear_backward_kernel<T, true, S.bq, WQ, WP, TWO> : linear_backward_kernel<T, false, S.bq, WQ, WP, TWO>;
    hipError_t e = launch_kernel(k, dim3(grid_of(pieces_of(b.x) + pieces_of(b.w), S.slots)), dim3(X::TH), lds, st, a, b.x, b.w);
    if (e == hipSuccess) e = launch_join<T, DX, MOE_ACT_NONE, I, WQ, WP, TWO>(a, b.x, st);
    return e != hipSuccess || TWO ? e : launch_join<T, DW, MOE_ACT_NONE, I, WQ, WP>(a, b.w, st);   // (TWO: a step or two along k)
}
template <typename T, Kind KIND, int I, int WQ, int WP, int PARTS>
hipError_t launch_experts_tiles(const LinArgs& a, const Plan& plan, hipStream_t st) {
    constexpr Shape S = SHAPES[I];
    typedef LinTile<T, KIND, S.bq, S.bp, WQ, WP> P;
    const size_t lds = P::LDS + WQ * WP * Slab<P::TP>::BYTES + (KIND == DW ? (size_t)a.experts * 2 : 0);
    return launch_kernel(linear_experts_backward_kernel<T, KIND, S.bq, WQ, WP, PARTS>, dim3(grid_of(pieces_of(plan), S.slots)), dim3(P::TH), lds, st, a, plan);
}
template <typename T, Kind KIND, int PARTS>
hipError_t launch_experts_of(const LinArgs& a, hipStream_t st) {
    const BackPlan b = plan_backward(a.m, a.N, a.K, a.experts, true, PARTS == 2, KIND == DX, KIND == DW);
    const Plan& plan = KIND == DX ? b.x : b.w;
    if constexpr (!(KIND == DX && PARTS == 2))
        if (b.shape == 0) return launch_experts_tiles<T, KIND, 0, 2, 4, PARTS>(a, plan, st);
    return launch_experts_tiles<T, KIND, 1, 2, 2, PARTS>(a, plan, st);
}
template <typename T, Kind KIND>
hipError_t launch_experts(const LinArgs& a, hipStream_t st) {
    if (a.dz_rest == nullptr) return launch_experts_of<T, KIND, 1>(a, st);
    return all_two(a.m, a.experts) ? launch_experts_of<T, KIND, 2>(a, st) : launch_experts_of<T, KIND, BOTH>(a, st);
}
template <typename T>
hipError_t launch_backward(const LinArgs& a, float* partial_x, float* partial_w, hipStream_t st) {
    const bool want_x = a.dx != nullptr && a.m > 0, want_w = a.dw != nullptr, two = a.dz_rest != nullptr;
    if (a.offsets != nullptr) {
        // each by itself: tiles of dx that run side by side share an expert's weights in their XCD's L2, and pieces of dW
        // between them part them (16184 rows of 32 experts, 2048 x 1408: 142 and 155 us, together 309)
        const hipError_t e = want_x ? launch_experts<T, DX>(a, st) : hipSuccess;
        return e == hipSuccess && want_w ? launch_experts<T, DW>(a, st) : e;
    }
    BackPlan b = plan_backward(a.m, a.N, a.K, 1, false, two, want_x, want_w);
    b.x.partial = partial_x, b.w.partial = partial_w;
    if (two) return launch_backward_tiles<T, TWO_SHAPE, 2, 2, true>(a, b, st);
    return b.shape == 0 ? launch_backward_tiles<T, 0, 2, 4, false>(a, b, st) : launch_backward_tiles<T, 1, 2, 2, false>(a, b, st);
}

constexpr int MAX_M = 1 << 24, MAX_N = 1 << 17, MAX_K = 1 << 16, MAX_EXPERTS = 1024;

int check_linear(const moe_linear* f) {
    if (f == nullptr || f->cols < 8 || f->cols > MAX_K || f->cols % 8) return MOE_EINVAL;
    if (f->rows < 1 || f->rows > MAX_N || f->experts < 1 || f->experts > MAX_EXPERTS) return MOE_EINVAL;
    if (f->dtype != MOE_BF16 && f->dtype != MOE_F16) return MOE_EINVAL;
    if (f->act != MOE_ACT_NONE && f->act != MOE_ACT_SILU && f->act != MOE_ACT_GELU) return MOE_EINVAL;
    return f->w != nullptr && aligned_to(f->w, 16) && aligned_to(f->bias, 2) ? MOE_OK : MOE_EINVAL;
}

// 16-byte rows of an operand of the matrix cores; the longest stride keeps a tile's offsets within 32 bits
bool rows_ok(const void* p, int64_t ld, int dim) {
    return p != nullptr && aligned_to(p, 16) && ld >= dim && ld % 8 == 0 && ld <= (1 << 22);
}

size_t forward_bytes(const moe_linear* f, int m) { return partial_bytes(FWD, m, f->rows, f->cols, f->experts); }
size_t saved_bytes_of(const moe_linear* f, int m) {
    return f->act == MOE_ACT_NONE ? 0 : round_up((size_t)m * padded(f->rows) * 4, 256);
}
// of either part of dz; the second is that of 64 rows or fewer, which with a matrix per expert may be any
size_t dz_bytes(const moe_linear* f, int m) { return round_up((size_t)m * padded(f->rows) * 2, 256); }
size_t rest_bytes(const moe_linear* f, int m) {
    return f->act == MOE_ACT_NONE ? 0 : dz_bytes(f, f->experts > 1 ? m : std::min(m, TWO_PARTS));
}
size_t sums_bytes(const moe_linear* f, int m) {
    return f->bias == nullptr ? 0 : round_up((size_t)(dz_chunks(m) + f->experts) * f->rows * 4, 256);
}
size_t dx_bytes(const moe_linear* f, int m) { return partial_bytes(DX, m, f->rows, f->cols, f->experts); }
size_t dw_bytes(const moe_linear* f, int m) { return partial_bytes(DW, m, f->rows, f->cols, f->experts); }
// weight rows of a workgroup: as many as make about two workgroups a CU, but 512 parts of the rows at most, and 16 rows at least
int few_back_rows(int N, int K) {
    const int parts = std::min(cdiv(2 * N_CU, cdiv(K, FEW_BACK_COLS)), 512);
    return std::max(16, cdiv(cdiv(N, parts), 4) * 4);
}

// dx's sums of few rows
size_t few_back_bytes(const moe_linear* f, int m) {
    return f->experts > 1 ? 0 : round_up((size_t)cdiv(f->rows, few_back_rows(f->rows, f->cols)) * std::min(m, FEW_BACK) * f->cols * 4, 256);
}
size_t backward_bytes(const moe_linear* f, int m) {
    return std::max(dz_bytes(f, m) + rest_bytes(f, m) + std::max(sums_bytes(f, m), dx_bytes(f, m) + dw_bytes(f, m)), few_back_bytes(f, m));
}

LinArgs describe(const moe_linear* f, int m, const int32_t* offsets) {
    LinArgs a{};
    a.w = reinterpret_cast<const uint16_t*>(f->w);
    a.bias = reinterpret_cast<const uint16_t*>(f->bias);
    a.offsets = offsets;
    a.m = m, a.N = f->rows, a.K = f->cols, a.experts = f->experts, a.act = f->act;
    return a;
}

// Whether m rows take the kernel for few rows; `room`: rows of x that a workgroup of it has LDS for, all of them or with
// offsets twice the average (more of one expert read its weights again, from the L2). x has to fit whole, and with offsets
// it is for so few experts that tiles of 32 rows leave CUs idle; with short k, of which each wavefront has but a load or two,
// for fewer (the bounds, a quarter of K's values up to 200 or 256 tiles, are fitted to these figures). That kernel and those
// tiles, weights from memory, K x N:
//   4096 x 4096          1 row 9.9 and 15.7 us, 8 rows 10.4 and 15.5, 16 rows (not whole) 15.2 and 15.5
//   8192 x 1024          1 row 11.2 and 14.5 us, 16 rows (not whole) 19.1 and 14.4
//   2048 x 65536         1 row 55.6 and 64.4 us, 16 rows 63.9 and 64.9
//   384 of 2304 x 5120   2 rows 18.1 and 33.1 us, 4 rows 27.8 and 34.8, 6 rows 39.7 and 37.2, 12 rows 71.5 and 52.3
//   384 of 2304 x 1280   6 rows 13.9 and 33.0 us, 16 rows 28.2 and 34.7, 96 rows 136 and 99, 1536 rows 597 and 373
//   384 of 256 x 2048    2 rows 7.5 and 7.4 us, 6 rows 12.1 and 7.6
//   64 of 1024 x 2048    6 rows 8.4 and 15.9 us, 24 rows 23.6 and 19.8
//   122 of 432 x 1813    6 rows 6.9 and 10.4 us, 16 rows 15.0 and 11.2
//   8 of 4096 x 4096     6 rows 42.0 and 58.2 us, 16 rows 55.3 and 63.4
bool few_rows(const LinArgs& a, int& room) {
    const int each = cdiv(a.m, a.experts);   // rows of an expert, on average
    if (each > FEW_ROWS) return false;
    room = std::min(a.m, a.offsets != nullptr ? std::min(2 * each, FEW_ROWS) : FEW_ROWS);
    if (room * few_row(a.K) * 2 > FEW_LDS) return false;
    if (a.offsets == nullptr) return true;
    const double picked = a.experts * (1 - std::pow(1 - 1.0 / a.experts, a.m));   // experts with a row, where every row picks one of all
    return picked * cdiv(a.N, 128) < std::min(a.K / 4, a.K < 4096 ? 200 : N_CU);
}

template <typename T, int ACT>
hipError_t forward_act(const LinArgs& a, float* partial, hipStream_t st) {
    int room = 0;
    if (!few_rows(a, room)) return launch_forward<T, ACT>(a, partial, st);
    const int items = a.offsets != nullptr ? a.m / room + std::min(a.experts, a.m) : 1;
    const size_t lds = std::max<size_t>((size_t)room * few_row(a.K) * 2, sizeof(float) * FEW_WAVES * 256);
    return launch_kernel(linear_few_kernel<T, ACT>, dim3(cdiv(a.N, 16), items), dim3(64 * FEW_WAVES), lds, st, a, room);
}
template <typename T>
hipError_t forward(const LinArgs& a, float* partial, hipStream_t st) {
    return a.act == MOE_ACT_NONE   ? forward_act<T, MOE_ACT_NONE>(a, partial, st)
           : a.act == MOE_ACT_SILU ? forward_act<T, MOE_ACT_SILU>(a, partial, st)
                                   : forward_act<T, MOE_ACT_GELU>(a, partial, st);
}

template <typename T, int M>
hipError_t few_backward_of(const LinArgs& a, hipStream_t st) {
    const int rows = few_back_rows(a.N, a.K), parts = cdiv(a.N, rows);
    const bool columns = a.dx != nullptr || a.dw != nullptr;
    const hipError_t e = launch_kernel(linear_few_backward_kernel<T, M>, dim3(columns ? cdiv(a.K, FEW_BACK_COLS) : 1, parts), dim3(256), 0, st, a, rows);
    if (e != hipSuccess || a.dx == nullptr || parts == 1) return e;
    return launch_kernel(linear_few_join_kernel<T>, dim3(cdiv(a.K, 256), a.m), dim3(1024), 0, st, a, parts);
}
template <typename T>
hipError_t few_backward(LinArgs a, float* partial, hipStream_t st) {
    if (a.dx == nullptr && a.dw == nullptr && a.dbias == nullptr) return hipSuccess;
    a.partial = partial;
    return a.m == 1 ? few_backward_of<T, 1>(a, st) : a.m == 2 ? few_backward_of<T, 2>(a, st) : a.m <= 4 ? few_backward_of<T, 4>(a, st) : few_backward_of<T, 8>(a, st);
}

template <typename T>
hipError_t backward(LinArgs a, uint8_t* work, size_t work_dz, size_t work_dx, bool direct, hipStream_t st) {
    if (a.m > 0 && a.m <= FEW_BACK && a.offsets == nullptr) return few_backward<T>(a, reinterpret_cast<float*>(work), st);
    hipError_t e = hipSuccess;
    float* const partial = reinterpret_cast<float*>(work + work_dz);
    if (a.m > 0 && (!direct || a.dbias != nullptr)) {
        LinArgs d = a;
        if (a.dbias != nullptr) d.partial = partial;
        e = launch_kernel(direct ? linear_dz_kernel<T, false> : linear_dz_kernel<T, true>, dim3(cdiv(a.m, dz_rows(a.m)), cdiv(a.N, DZ_COLS)),
                          dim3(256), 0, st, d);
    }
    if (e == hipSuccess && a.dbias != nullptr) {
        LinArgs d = a;
        d.partial = partial;
        e = launch_kernel(linear_bias_kernel<T>, dim3(cdiv(a.N, 64), a.experts), dim3(1024), 0, st, d);
    }
    if (e == hipSuccess && ((a.dx != nullptr && a.m > 0) || a.dw != nullptr))
        e = launch_backward<T>(a, partial, reinterpret_cast<float*>(work + work_dz + work_dx), st);
    return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear_workspace(const moe_linear* f, int32_t m, size_t* forward, size_t* saved, size_t* backward) {
    const int rc = check_linear(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M || forward == nullptr || saved == nullptr || backward == nullptr) return MOE_EINVAL;
    *forward = forward_bytes(f, m);
    *saved = saved_bytes_of(f, m);
    *backward = backward_bytes(f, m);
    return MOE_OK;
}

int moe_linear_forward(const moe_linear* f, const void* x, int64_t ldx, const int32_t* offsets, int32_t m, const void* residual,
                       int64_t ldr, void* y, int64_t ldy, void* saved, size_t saved_bytes, void* work, size_t work_bytes,
                       void* stream) {
    const int rc = check_linear(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M || !aligned_to(offsets, 4) || (offsets == nullptr && f->experts > 1)) return MOE_EINVAL;
    if (m == 0) return MOE_OK;
    if (!rows_ok(x, ldx, f->cols) || !value_rows_ok(y, ldy, f->rows, 2)) return MOE_EINVAL;
    if (residual != nullptr && !value_rows_ok(residual, ldr, f->rows, 2)) return MOE_EINVAL;
    const size_t need = forward_bytes(f, m);
    if ((need > 0 && work == nullptr) || !aligned_to(work, 256) || !aligned_to(saved, 256)) return MOE_EINVAL;
    if (work_bytes < need || (saved != nullptr && saved_bytes < saved_bytes_of(f, m))) return MOE_ESCRATCH;
    LinArgs a = describe(f, m, offsets);
    a.x = reinterpret_cast<const uint16_t*>(x), a.ldx = ldx;
    a.residual = reinterpret_cast<const uint16_t*>(residual), a.ldr = ldr;
    a.y = reinterpret_cast<uint16_t*>(y), a.ldy = ldy;
    a.z = f->act == MOE_ACT_NONE ? nullptr : reinterpret_cast<float*>(saved);
    float* const partial = reinterpret_cast<float*>(work);
    const hipStream_t st = (hipStream_t)stream;
    return status_of(f->dtype == MOE_BF16 ? forward<Bf16>(a, partial, st) : forward<F16>(a, partial, st));
}

int moe_linear_backward(const moe_linear* f, const void* x, int64_t ldx, const int32_t* offsets, int32_t m, const void* dy,
                        int64_t lddy, const void* saved, size_t saved_bytes, void* dx, int64_t lddx, void* dw, void* dbias,
                        void* work, size_t work_bytes, void* stream) {
    const int rc = check_linear(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M || !aligned_to(offsets, 4) || (offsets == nullptr && f->experts > 1)) return MOE_EINVAL;
    if (!aligned_to(dw, 16) || !aligned_to(dbias, 2) || (dbias != nullptr && f->bias == nullptr)) return MOE_EINVAL;
    LinArgs a = describe(f, m, offsets);
    bool direct = false;
    if (m > 0) {
        if (!rows_ok(x, ldx, f->cols) || !value_rows_ok(dy, lddy, f->rows, 2) || (dx != nullptr && !rows_ok(dx, lddx, f->cols)))
            return MOE_EINVAL;
        if (work == nullptr || !aligned_to(work, 256) || !aligned_to(saved, 256) || (f->act != MOE_ACT_NONE && saved == nullptr))
            return MOE_EINVAL;
        if (work_bytes < backward_bytes(f, m) || saved_bytes < saved_bytes_of(f, m)) return MOE_ESCRATCH;
        a.x = reinterpret_cast<const uint16_t*>(x), a.ldx = ldx;
        a.dy = reinterpret_cast<const uint16_t*>(dy), a.lddy = lddy;
        a.dx = reinterpret_cast<uint16_t*>(dx), a.lddx = lddx;
        a.z = reinterpret_cast<float*>(const_cast<void*>(saved));
        // with no activation dy is the operand itself, where its rows are whole chunks
        direct = f->act == MOE_ACT_NONE && f->rows % 8 == 0 && rows_ok(dy, lddy, f->rows);
        a.dz_out = reinterpret_cast<uint16_t*>(work);
        a.dz = direct ? a.dy : a.dz_out, a.lddz = direct ? lddy : padded(f->rows);
        if (f->act != MOE_ACT_NONE && (offsets != nullptr || m <= TWO_PARTS))
            a.dz_rest = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(work) + dz_bytes(f, m));
    }
    a.dw = reinterpret_cast<uint16_t*>(dw);
    a.dbias = reinterpret_cast<uint16_t*>(dbias);
    uint8_t* const w = reinterpret_cast<uint8_t*>(work);
    const hipStream_t st = (hipStream_t)stream;
    const size_t work_dz = m > 0 ? dz_bytes(f, m) + rest_bytes(f, m) : 0, work_dx = m > 0 ? dx_bytes(f, m) : 0;
    return status_of(f->dtype == MOE_BF16 ? backward<Bf16>(a, w, work_dz, work_dx, direct, st) : backward<F16>(a, w, work_dz, work_dx, direct, st));
}

}  // extern "C"
