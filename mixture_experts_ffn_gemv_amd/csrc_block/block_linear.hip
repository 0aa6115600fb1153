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
// wavefront adds up 64 at a time. Workgroups past the last tile end at once.
//
// dz is rounded to 16 bits, as an operand of the matrix cores, and nothing else before the results: the
// gradients have sqrt(2) of the error that their own rounding gives them. z is kept in f32.
#include "block_rows.h"
#include "block_tiles.h"

namespace moe {
namespace {

enum Kind { FWD, DX, DW };
constexpr bool p_by_rows(Kind k) { return k != FWD; }   // p (not k) is P's consecutive index
constexpr bool q_by_rows(Kind k) { return k == DW; }

struct LinArgs {
    const uint16_t *x, *w, *bias, *residual, *dy, *dz;
    float* z;              // [m, z_ld(N)]
    uint16_t *y, *dx, *dw, *dbias, *dz_out;
    const int32_t* offsets;   // [experts + 1]; NULL: one matrix for all rows
    int64_t ldx, ldr, ldy, lddy, lddz, lddx;
    int m, N, K, experts, act;
    float* partial;        // column sums, [chunk + expert][N]
};
MOE_DEV __host__ int z_ld(int N) { return (N + 3) / 4 * 4; }
MOE_DEV __host__ int dz_ld(int N) { return (N + 7) / 8 * 8; }

MOE_DEV float act_any(float v, int act) { return act == MOE_ACT_NONE ? v : act_value(v, act); }

// 64 offsets at a time, one per lane; what lies outside 0..m or goes back does not count
MOE_DEV int offset_at(const LinArgs& a, int i) { return min(max(a.offsets[min(i, a.experts)], 0), a.m); }

// A tile among those of `rows`-row tiles of the experts' rows: which expert, where it begins, its
// rows; np tiles side by side. Every lane of the wavefront calls it.
struct Slice {
    int expert, row0, rows;    // the expert's rows
    int tile;                  // which of the expert's tiles (q and p)
};
MOE_DEV int tiles_total(const LinArgs& a, int rows) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e = lane; e < a.experts; e += 64) n += (max(offset_at(a, e + 1) - offset_at(a, e), 0) + rows - 1) / rows;
    n = wave_inclusive_scan(n);
    return __builtin_amdgcn_readlane(n, 63);
}
MOE_DEV Slice find_slice(const LinArgs& a, int rows, int np, int tile) {
    const int lane = threadIdx.x & 63;
    Slice s{0, 0, 0, 0};
    int before = 0;   // tiles of the experts before these 64
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int lo = offset_at(a, e0 + lane), cnt = e0 + lane < a.experts ? max(offset_at(a, e0 + lane + 1) - lo, 0) : 0;
        const int n = (cnt + rows - 1) / rows * np, upto = before + wave_inclusive_scan(n);
        const uint64_t past = __ballot(upto > tile);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            s.expert = e0 + l;
            s.row0 = __builtin_amdgcn_readlane(lo, l);
            s.rows = __builtin_amdgcn_readlane(cnt, l);
            s.tile = tile - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
            break;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return s;
}

// four consecutive values at p + 0..3 of a row, of which `left` are there; no alignment but the values'
template <typename T>
MOE_DEV void load4(const uint16_t* p, int left, float (&v)[4]) {
    uint2 q = make_uint2(0, 0);
    if (left >= 4) __builtin_memcpy(&q, p, 8);
    else {
        uint16_t b[4] = {0, 0, 0, 0};
        for (int i = 0; i < 3; ++i)
            if (i < left) b[i] = p[i];
        q = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
    }
    v[0] = T::lo(q.x), v[1] = T::hi(q.x), v[2] = T::lo(q.y), v[3] = T::hi(q.y);
}
template <typename T>
MOE_DEV void store4(uint16_t* p, int left, const float (&v)[4]) {
    const uint2 q = make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
    if (left >= 4) __builtin_memcpy(p, &q, 8);
    else {
        const uint16_t b[4] = {(uint16_t)q.x, (uint16_t)(q.x >> 16), (uint16_t)q.y, (uint16_t)(q.y >> 16)};
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = b[i];
    }
}

// Where a tile lies and what it multiplies
struct Tile {
    Operand P, Q;
    int q0, p0;
    int expert, row0;   // q (DW: k) counts from this row
};
template <Kind KIND, int BQ, int BP>
MOE_DEV Tile locate(const LinArgs& a, int tile, int nq, int np) {
    Tile t;
    t.expert = 0, t.row0 = 0;
    int rows = a.m;
    if (a.offsets != nullptr) {
        if (KIND == DW) {
            const int each = nq * np;
            t.expert = tile / each;
            tile -= t.expert * each;
            t.row0 = offset_at(a, t.expert);
            rows = max(offset_at(a, t.expert + 1) - t.row0, 0);
        } else {
            const Slice s = find_slice(a, BQ, np, tile);
            t.expert = s.expert, t.row0 = s.row0, rows = s.rows, tile = s.tile;
            nq = (rows + BQ - 1) / BQ;
        }
    }
    const uint16_t* const w = a.w + (size_t)t.expert * a.N * a.K;
    const uint16_t* const x = a.x + t.row0 * a.ldx;
    const uint16_t* const dz = a.dz + t.row0 * a.lddz;
    // (dz's rows are padded to whole chunks with zeros)
    if (KIND == FWD) t.P = {w, w, a.K, a.N, a.K}, t.Q = {x, x, a.ldx, rows, a.K};
    if (KIND == DX) t.P = {w, w, a.K, a.K, a.N}, t.Q = {dz, dz, a.lddz, rows, dz_ld(a.N)};
    if (KIND == DW) t.P = {x, x, a.ldx, a.K, rows}, t.Q = {dz, dz, a.lddz, dz_ld(a.N), rows};
    // eight q tiles deep, so that the tiles an XCD works on at a time share their operands in its L2
    const int deep = 8 * np, gr = tile / deep, gq = min(8, nq - gr * 8), in = tile - gr * deep;
    t.q0 = (gr * 8 + in % gq) * BQ;
    t.p0 = in / gq * BP;
    return t;
}

// What a wavefront does with the sums of 16 q (q = qw + l16) and its TP p: a lane holds p =
// 16 i + 4 g + 0..3 in v[i], counted from pw
template <typename T, Kind KIND, int NI>
MOE_DEV void finish(const LinArgs& a, const Tile& t, int qw, int pw, const f32x4 (&v)[NI]) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4, q = qw + l16;
    const int extent = KIND == FWD ? a.N : a.K;
    if (q >= (KIND == DW ? a.N : t.Q.rows)) return;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int p = t.p0 + pw + 16 * i + 4 * g, left = extent - p;
        if (left <= 0) continue;
        float o[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
        if constexpr (KIND == FWD) {
            const int64_t row = t.row0 + q;
            if (a.bias != nullptr) {
                float b[4];
                load4<T>(a.bias + (size_t)t.expert * a.N + p, left, b);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] += b[r];
            }
            if (a.z != nullptr) *reinterpret_cast<f32x4*>(a.z + row * z_ld(a.N) + p) = (f32x4){o[0], o[1], o[2], o[3]};
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = act_any(o[r], a.act);
            if (a.residual != nullptr) {
                float b[4];
                load4<T>(a.residual + row * a.ldr + p, left, b);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] += b[r];
            }
            store4<T>(a.y + row * a.ldy + p, left, o);
        } else if constexpr (KIND == DX) {
            store4<T>(a.dx + (t.row0 + q) * a.lddx + p, 4, o);   // (K is a multiple of 8)
        } else {
            store4<T>(a.dw + ((size_t)t.expert * a.N + q) * a.K + p, 4, o);
        }
    }
}

// The work of one launch: the first `whole` tiles by a workgroup each, the `rest` (what does
// not fill the CUs once more) by `splits` workgroups each, every one with its part of k. With an
// expert's rows per tile `whole` is only a bound.
struct Plan {
    int nq, np;          // tiles along q and p
    int whole, rest, splits;
    float* partial;      // [split][rest][j][i][thread] of the split tiles' sums, four f32 each
};

template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
using LinTile = TileProduct<T, p_by_rows(KIND), q_by_rows(KIND), false, BQ, BP, WQ, WP>;

template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void linear_kernel(LinArgs a, Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    typedef LinTile<T, KIND, BQ, BP, WQ, WP> Product;
    constexpr int TH = Product::TH, NI = Product::NI, NJ = Product::NJ;
    const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), wq = wv / WP, wp = wv % WP;

    // consecutive tiles (of a split part: those of one part of k) on one XCD
    const int whole_blocks = (plan.whole + 7) / 8 * 8;
    int tile, split = -1;
    if ((int)blockIdx.x < whole_blocks) {
        const int whole = a.offsets != nullptr && KIND != DW ? tiles_total(a, BQ) * plan.np : plan.whole;
        tile = xcd_logical_block(blockIdx.x, whole);
        if (tile >= whole) return;
    } else {
        const int items = plan.rest * plan.splits, item = xcd_logical_block(blockIdx.x - whole_blocks, items);
        if (item >= items) return;
        split = item / plan.rest;
        tile = plan.whole + item - split * plan.rest;
    }
    const Tile t = locate<KIND, BQ, BP>(a, tile, plan.nq, plan.np);
    const int steps = (t.P.k + BK - 1) / BK;
    const int kt0 = split < 0 ? 0 : (int)((int64_t)split * steps / plan.splits);
    const int nk = (split < 0 ? steps : (int)((int64_t)(split + 1) * steps / plan.splits)) - kt0;
    f32x4 acc[NI][NJ];
    Product::run(t.P, t.Q, 1, t.q0, t.p0, kt0, nk, smem, acc);

    if (split >= 0) {
        f32x4* o = reinterpret_cast<f32x4*>(plan.partial) + (size_t)(split * plan.rest + tile - plan.whole) * NI * NJ * TH + tid;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i) o[(j * NI + i) * TH] = acc[i][j];
        return;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        f32x4 v[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = acc[i][j];
        finish<T, KIND, NI>(a, t, t.q0 + wq * Product::TQ + 16 * j, wp * Product::TP, v);
    }
}

// The split tiles' sums, added in order of k, and what is done with them: a workgroup per
// tile and j (16 q of each wavefront)
template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void linear_join_kernel(LinArgs a, Plan plan) {
    typedef LinTile<T, KIND, BQ, BP, WQ, WP> Product;
    constexpr int TH = Product::TH, NI = Product::NI, NJ = Product::NJ;
    const int tid = threadIdx.x, wv = tid >> 6, wq = wv / WP, wp = wv % WP;
    const int r = blockIdx.x / NJ, j = blockIdx.x % NJ;
    const f32x4* from = reinterpret_cast<const f32x4*>(plan.partial) + ((size_t)r * NJ + j) * NI * TH + tid;
    f32x4 v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = from[i * TH];
#pragma unroll 2
    for (int s = 1; s < plan.splits; ++s) {
        const f32x4* f = from + (size_t)s * plan.rest * NI * NJ * TH;
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] += f[i * TH];
    }
    const Tile t = locate<KIND, BQ, BP>(a, plan.whole + r, plan.nq, plan.np);
    finish<T, KIND, NI>(a, t, t.q0 + wq * Product::TQ + 16 * j, wp * Product::TP, v);
}

// ------------------------------------------------------------------ dz and its column sums

// A workgroup owns DZ_ROWS rows and 512 columns, eight per lane, a row per wavefront at a time. The rows may be
// several experts': where one ends the sums of its columns go to the row (chunk + expert) of `partial`, a number of
// its own for every expert in every chunk.
constexpr int DZ_ROWS = 64, DZ_COLS = 512;

// the number of experts whose rows end at `row` or before: the expert of that row
MOE_DEV int expert_of(const LinArgs& a, int row) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) n += __popcll(__ballot(e0 + lane < a.experts && offset_at(a, e0 + lane + 1) <= row));
    return n;
}

// STORE: dz is wanted (else it is dy itself, and only the sums are)
template <typename T, bool STORE>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinArgs a) {
    __shared__ float lds[4][DZ_COLS];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int first = blockIdx.x * DZ_ROWS, n0 = blockIdx.y * DZ_COLS + lane * 8, left = a.N - n0;
    const int last = min(first + DZ_ROWS, a.offsets != nullptr ? offset_at(a, a.experts) : a.m);
    int row = first;
    while (row < last) {
        const int e = a.offsets != nullptr ? expert_of(a, row) : 0;
        // (offsets that go back must not hold the loop up)
        const int end = a.offsets != nullptr ? max(min(last, offset_at(a, e + 1)), row + 1) : last;
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
        for (int r = row + wv; r < end && left > 0; r += 4) {
            float d[8], lo[4], hi[4];
            const uint16_t* dy = a.dy + r * a.lddy + n0;
            load4<T>(dy, left, lo);
            if (left > 4) load4<T>(dy + 4, left - 4, hi);
            else hi[0] = hi[1] = hi[2] = hi[3] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = lo[i], d[4 + i] = hi[i];
            if (a.act != MOE_ACT_NONE) {
                const float* z = a.z + (size_t)r * z_ld(a.N) + n0;
                const f32x4 z0 = *reinterpret_cast<const f32x4*>(z), z1 = left > 4 ? *reinterpret_cast<const f32x4*>(z + 4) : z0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float f, df;
                    act_both(i < 4 ? z0[i] : z1[i - 4], a.act, f, df);
                    d[i] = i < left ? d[i] * df : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += d[i];
            if (STORE)
                *reinterpret_cast<uint4*>(a.dz_out + r * a.lddz + n0) =
                    make_uint4(T::pack2(d[0], d[1]), T::pack2(d[2], d[3]), T::pack2(d[4], d[5]), T::pack2(d[6], d[7]));
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
    const int r0 = a.offsets != nullptr ? offset_at(a, e) : 0, r1 = a.offsets != nullptr ? offset_at(a, e + 1) : a.m;
    float s = 0.f;
    if (n < a.N && r1 > r0)
        for (int b = r0 / DZ_ROWS + g; b <= (r1 - 1) / DZ_ROWS; b += 16) s += a.partial[(size_t)(b + e) * a.N + n];
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
// read twice. A workgroup owns 16 weight rows, each of its eight wavefronts a part of k, and their sums are
// joined through LDS in wavefront order. x comes into LDS whole, or as much of k at a time as fits.
constexpr int FEW_WAVES = 8, FEW_ROWS = 16;
constexpr int FEW_LDS = 64 << 10;
// values of k that a pass takes, a multiple of 512: whole runs of 1024 bytes
MOE_DEV __host__ int few_pass(int rows, int K) {
    const int whole = (K + 511) / 512 * 512, fit = FEW_LDS / (rows * 1024) * 512;
    return whole < fit ? whole : fit;
}

template <typename T>
__global__ __launch_bounds__(64 * FEW_WAVES) void linear_few_kernel(LinArgs a, int room) {
    constexpr int AHEAD = 5;
    extern __shared__ __align__(16) uint8_t smem[];   // x; then sums [wavefront][256]
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, pass_k = few_pass(room, a.K), row_bytes = pass_k * 2, runs = row_bytes / 1024;
    Slice s{0, 0, a.m, 0};
    if (a.offsets != nullptr) {
        if ((int)blockIdx.y >= tiles_total(a, room)) return;
        s = find_slice(a, room, 1, blockIdx.y);
    } else {
        s.tile = blockIdx.y;
    }
    const int rows = min(s.rows - s.tile * room, room), row0 = s.row0 + s.tile * room;
    const uint16_t* const w0 = a.w + (size_t)s.expert * a.N * a.K;
    const uint16_t* const w = w0 + (size_t)min(n0 + l16, a.N - 1) * a.K;
    const auto X = buffer_rsrc(a.x + row0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K) * 2);
    const int xt = min(l16, rows - 1);   // (a token that does not exist reads another's; its sums are not used)
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.K; k0 += pass_k) {
        const int chunks = (min(pass_k, a.K - k0) + 31) / 32;
        const int c0 = wv * chunks / FEW_WAVES, c1 = (wv + 1) * chunks / FEW_WAVES;
        for (int r = wv; r < rows * runs; r += FEW_WAVES) {
            // 16-byte chunk c of a row lies at c ^ (row & 15)
            const int row = r / runs, k = k0 + (r - row * runs) * 512 + (lane ^ (row & 15)) * 8;
            buffer_load_lds16(X, smem + r * 1024, k < a.K ? (uint32_t)(row * a.ldx + k) * 2 : PAST);
        }
        uint4 wq[AHEAD];
        auto request = [&](int i, int c) { wq[i] = *reinterpret_cast<const uint4*>(w + min(k0 + 32 * min(c, chunks - 1) + 8 * g, a.K - 8)); };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) request(i, c0 + i);
        wait_vm_loads<AHEAD>();   // this wavefront's part of x has landed
        barrier_lds();
        auto multiply = [&](int i, int c) {
            // a weight that stands in for one past K is not one (x is zero there)
            const uint32_t on = k0 + 32 * c + 8 * g < a.K ? ~0u : 0u;
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
        __syncthreads();   // x is read; the next part, or the sums, take its place
    }
    float* red = reinterpret_cast<float*>(smem);
    *reinterpret_cast<f32x4*>(&red[wv * 256 + lane * 4]) = acc;
    __syncthreads();
    if (tid >= 64) return;
    f32x4 v[1] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < FEW_WAVES; ++i) v[0] += *reinterpret_cast<const f32x4*>(&red[i * 256 + lane * 4]);
    Tile t;
    t.expert = s.expert, t.row0 = row0, t.p0 = n0, t.Q.rows = rows;
    finish<T, FWD, 1>(a, t, 0, 0, v);
}

// ------------------------------------------------------------------ plans

int cdiv(int a, int b) { return (a + b - 1) / b; }

constexpr int N_CU = 256, MAX_SPLITS = 16;
struct Product {
    Plan plan;
    int tile;         // 256 or 128
};
struct Extent {
    int nq, np, tiles, steps, slots;
};
// tiles of B x B along q and p, all of them (with a matrix per expert: at most), K steps of one, and how many the
// CUs hold at a time
Extent extent(Kind kind, int m, int N, int K, int experts, int B) {
    Extent e;
    e.steps = cdiv(kind == FWD ? K : kind == DX ? N : m, BK);
    e.nq = cdiv(kind == DW ? N : m, B), e.np = cdiv(kind == FWD ? N : K, B);
    e.tiles = kind == DW ? experts * e.nq * e.np : experts == 1 ? e.nq * e.np : (m / B + std::min(experts, m)) * e.np;
    e.slots = B == 256 ? N_CU : 2 * N_CU;
    return e;
}
// Bytes that hold the split tiles' sums of any plan for m rows or fewer
size_t partial_bytes(Kind kind, int m, int N, int K, int experts) {
    if (experts > 1) return 0;
    size_t most = 0;
    for (int B : {256, 128}) {
        const Extent e = extent(kind, m, N, K, 1, B);
        const int splits = std::min(MAX_SPLITS, e.steps / 2);
        if (splits >= 2) most = std::max(most, (size_t)std::min<int64_t>(e.slots, (int64_t)e.tiles * splits) * B * B * sizeof(float));
    }
    return most;
}

// How a product is cut up: 256 x 256 or 128 x 128 tiles, and by how much the tiles past the last full
// round of the CUs are split along k. Costs in units of one K step of a 256 x 256 tile on a CU
// (about 1.65 us): a 128 x 128 tile's step takes 0.33 of it (a quarter of the products, at three quarters
// of the rate); the split tiles' sums pass through memory twice (0.06 a 256 x 256 tile and split, and 4 for
// the second launch). With a matrix per expert nothing is split.
Product plan_product(Kind kind, int m, int N, int K, int experts) {
    Product best{};
    double best_cost = 1e300;
    for (int B : {256, 128}) {
        const Extent e = extent(kind, m, N, K, experts, B);
        Product p{};
        p.tile = B;
        p.plan.nq = e.nq, p.plan.np = e.np;
        const double step = B == 256 ? 1 : 0.66, share = B == 256 ? 0.06 : 0.015;   // (two workgroups share a CU)
        p.plan.whole = e.tiles, p.plan.splits = 1;
        double cost;
        if (experts > 1) {
            const int steps = kind == DW ? cdiv(cdiv(m, experts), BK) : e.steps;
            cost = cdiv(e.tiles, e.slots) * (double)steps * step;
        } else {
            const int rounds = e.tiles / e.slots, rest = e.tiles % e.slots;
            cost = rounds * (double)e.steps * step;
            if (rest > 0) {
                double tail = e.steps * step;
                for (int s = 2; s <= MAX_SPLITS && s * 2 <= e.steps && rest * s <= e.slots; ++s) {
                    const double t = cdiv(e.steps, s) * step + 4 + share * rest * s;
                    if (t < tail) tail = t, p.plan.whole = e.tiles - rest, p.plan.rest = rest, p.plan.splits = s;
                }
                cost += tail;
            }
        }
        if (cost < best_cost) best_cost = cost, best = p;
    }
    return best;
}

template <typename T, Kind KIND, int B, int WQ, int WP>
hipError_t launch_tiles(const LinArgs& a, const Plan& plan, hipStream_t st) {
    const int grid = (plan.whole + 7) / 8 * 8 + (plan.rest * plan.splits + 7) / 8 * 8;
    if (grid == 0) return hipSuccess;
    typedef LinTile<T, KIND, B, B, WQ, WP> P;
    const hipError_t e = launch_kernel(linear_kernel<T, KIND, B, B, WQ, WP>, dim3(grid), dim3(P::TH), P::LDS, st, a, plan);
    if (e != hipSuccess || plan.rest == 0) return e;
    return launch_kernel(linear_join_kernel<T, KIND, B, B, WQ, WP>, dim3(plan.rest * P::NJ), dim3(P::TH), 0, st, a, plan);
}

template <typename T, Kind KIND>
hipError_t launch_product(const LinArgs& a, float* partial, hipStream_t st) {
    Product p = plan_product(KIND, a.m, a.N, a.K, a.offsets != nullptr ? std::max(a.experts, 2) : 1);
    if (a.offsets != nullptr && a.experts == 1 && KIND == DW) p = plan_product(KIND, a.m, a.N, a.K, 1);
    p.plan.partial = partial;
    return p.tile == 256 ? launch_tiles<T, KIND, 256, 2, 4>(a, p.plan, st) : launch_tiles<T, KIND, 128, 2, 2>(a, p.plan, st);
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

size_t forward_bytes(const moe_linear* f, int m) { return round_up(partial_bytes(FWD, m, f->rows, f->cols, f->experts), 256); }
size_t saved_bytes_of(const moe_linear* f, int m) {
    return f->act == MOE_ACT_NONE ? 0 : round_up((size_t)m * z_ld(f->rows) * 4, 256);
}
size_t dz_bytes(const moe_linear* f, int m) { return round_up((size_t)m * dz_ld(f->rows) * 2, 256); }
size_t sums_bytes(const moe_linear* f, int m) {
    return f->bias == nullptr ? 0 : round_up((size_t)(cdiv(m, DZ_ROWS) + f->experts) * f->rows * 4, 256);
}
size_t product_bytes(const moe_linear* f, int m) {
    return round_up(std::max(partial_bytes(DX, m, f->rows, f->cols, f->experts), partial_bytes(DW, m, f->rows, f->cols, f->experts)), 256);
}
size_t backward_bytes(const moe_linear* f, int m) { return dz_bytes(f, m) + std::max(sums_bytes(f, m), product_bytes(f, m)); }

LinArgs describe(const moe_linear* f, int m, const int32_t* offsets) {
    LinArgs a{};
    a.w = reinterpret_cast<const uint16_t*>(f->w);
    a.bias = reinterpret_cast<const uint16_t*>(f->bias);
    a.offsets = offsets;
    a.m = m, a.N = f->rows, a.K = f->cols, a.experts = f->experts, a.act = f->act;
    return a;
}

template <typename T>
hipError_t forward(const LinArgs& a, float* partial, hipStream_t st) {
    const int each = cdiv(a.m, a.experts);   // rows of an expert, on average
    if (each > FEW_ROWS) return launch_product<T, FWD>(a, partial, st);
    const int room = std::min(a.m, FEW_ROWS), items = a.offsets != nullptr ? a.m / room + std::min(a.experts, a.m) : cdiv(a.m, room);
    const size_t lds = std::max<size_t>((size_t)room * few_pass(room, a.K) * 2, sizeof(float) * FEW_WAVES * 256);
    return launch_kernel(linear_few_kernel<T>, dim3(cdiv(a.N, 16), items), dim3(64 * FEW_WAVES), lds, st, a, room);
}

template <typename T>
hipError_t backward(LinArgs a, uint8_t* work, size_t work_dz, bool direct, hipStream_t st) {
    hipError_t e = hipSuccess;
    float* const partial = reinterpret_cast<float*>(work + work_dz);
    if (a.m > 0 && (!direct || a.dbias != nullptr)) {
        LinArgs d = a;
        if (a.dbias != nullptr) d.partial = partial;
        e = launch_kernel(direct ? linear_dz_kernel<T, false> : linear_dz_kernel<T, true>, dim3(cdiv(a.m, DZ_ROWS), cdiv(a.N, DZ_COLS)),
                          dim3(256), 0, st, d);
    }
    if (e == hipSuccess && a.dbias != nullptr) {
        LinArgs d = a;
        d.partial = partial;
        e = launch_kernel(linear_bias_kernel<T>, dim3(cdiv(a.N, 64), a.experts), dim3(1024), 0, st, d);
    }
    if (e == hipSuccess && a.dx != nullptr && a.m > 0) e = launch_product<T, DX>(a, partial, st);
    if (e == hipSuccess && a.dw != nullptr) e = launch_product<T, DW>(a, partial, st);
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
        a.dz = direct ? a.dy : a.dz_out, a.lddz = direct ? lddy : dz_ld(f->rows);
    }
    a.dw = reinterpret_cast<uint16_t*>(dw);
    a.dbias = reinterpret_cast<uint16_t*>(dbias);
    uint8_t* const w = reinterpret_cast<uint8_t*>(work);
    const hipStream_t st = (hipStream_t)stream;
    const size_t work_dz = m > 0 ? dz_bytes(f, m) : 0;
    return status_of(f->dtype == MOE_BF16 ? backward<Bf16>(a, w, work_dz, direct, st) : backward<F16>(a, w, work_dz, direct, st));
}

}  // extern "C"
