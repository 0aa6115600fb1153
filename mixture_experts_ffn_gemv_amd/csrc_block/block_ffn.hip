// The dense gated feed-forward block, forward and backward (moe_ffn_* in
// include/moe.h), as matrix-core products with fused epilogues.
//
//   GATEUP  g = x Wg^T, u = x Wu^T -> h = act(g) u  (and g, u in f32 for the backward pass)
//   DOWN    y = h Wd^T
//   DH      dh = dy Wd -> dg, du, h, from the saved g and u
//   DX      dx = dg Wg + du Wu, one sum over both
//   DW      dWg = dg^T x, dWu = du^T x, dWd = dy^T h, the three in one launch
//
// Every product is out[q, p] = sum_k P(k, p) Q(k, q) with p the consecutive index of
// the output. P is the matrix instruction's first operand, so that a lane's four
// results are four consecutive values of one output row. An operand either has k as
// its consecutive index (tiles of rows x 64 k; one 16-byte LDS read per lane gives
// eight k) or p / q (tiles of 64 k x rows; two transposing 8-byte LDS reads), so no
// operand is ever transposed in memory.
//
// Tiles come into LDS by buffer loads straight to LDS, 16 bytes per lane, a K step of 64
// ahead. What lies past an operand's rows or past K lands as zeros: rows by the buffer's
// length, a K tail by an offset past it. Chunks of 16 bytes are stored permuted so that
// the LDS reads of a matrix operand fall on distinct banks.
//
// h, dg and du are rounded to 16 bits, as operands of the matrix cores (h of a few rows in two parts: see
// h_in_parts); in f16 they become infinite past 65504. Rounding one operand of a product once more makes the error of y and of the gradients
// sqrt(2) of what rounding the result alone gives (bf16 2.3e-3 of the norm, f16 2.9e-4); two products
// of 16-bit parts of each would cost a second matrix product. g and u stay in f32.
//
// Bound, for many rows, by the matrix cores: at 8192 rows of 5120 x 2304 (bf16, a training
// step 1.72 ms) GATEUP takes 333 us (1.16 PFLOP/s), DOWN 187 (1.03), DH 266 (0.73), DX 346
// (1.12), DW 533 (1.09), where a library product of 8192^3 reaches 1.51 (either operand's
// k consecutive), 1.32 or 1.16 (as in DX and DW). A round of whole tiles runs at 1.3; the rest
// is the last round, which is not full, and the ends of tiles: GATEUP stores 151 MB of g and u in f32, DH reads
// them and writes 113 MB of dg, du and h, after the products of its tile. Counters: no LDS
// conflicts, matrix cores busy 0.59 (GATEUP) and 0.48 (DW) of the cycles.
// Few rows are bound by the weights' bytes: one token of 5120 x 2304 20.7 us, 70.8 MB, 3.4 TB/s.
#include "block_common.h"

namespace moe {
namespace {

constexpr int BK = 64;
constexpr uint32_t PAST = 0xFFFFFFF0u;   // an offset past every buffer: zeros

enum Kind { GATEUP, DOWN, DH, DX, DW };
constexpr bool p_by_rows(Kind k) { return k == DH || k == DX || k == DW; }   // p (not k) is P's consecutive index
constexpr bool q_by_rows(Kind k) { return k == DW; }

struct FfnArgs {
    const uint16_t *x, *dy, *wg, *wu, *wd;
    uint16_t *h, *dg, *du;   // [m, I]
    float* saved;            // g and u: blocks of 16 rows x 16 columns, see saved_at
    uint16_t *y, *dx, *dwg, *dwu, *dwd;
    int64_t ldx, lddy, ldy, lddx;
    int m, D, I, act;
    float limit;
    bool parts;              // h lies in two parts: see h_in_parts
};

// one operand of a product: up to two matrices, used side by side (GATEUP) or one
// after the other along k (DX)
struct Operand {
    const uint16_t *a, *b;
    int64_t ld;
    int rows;   // extent of p or q
};

// saved: block (q / 16, i / 16) holds g then u, 256 f32 each, in the order of the lanes that
// hold them: four consecutive i of one q per lane
MOE_DEV size_t saved_at(int q16, int i16, int I) { return ((size_t)q16 * ((I + 15) / 16) + i16) * 512; }

// Tiles in LDS. rows x 64 k (128 bytes a row): chunk c of 16 bytes of row r lies at c ^ swz_k(r),
// so that the 16 rows of an operand read fall on distinct banks.
MOE_DEV int swz_k(int row) { return row & 7; }
// 64 k x rows, rows = 128 or 256: runs of 1024 bytes, PIECE apart, each holding rows k that are
// never read together; a transposing read takes four rows k of two lane groups at a time, and
// these lie in eight runs, whose distance puts them on distinct banks. Every read of a
// lane is then one address and a constant.
constexpr int PIECE = 1024 + 32;
constexpr int tile_bytes(int rows, bool by_rows) { return by_rows ? rows / 8 * PIECE : rows * BK * 2; }
// row k of run c: its part from the wavefront's share of c and the place in the run, and from the unit
MOE_DEV int run_row_wave(int rows, int waves, int wv, int slot) {
    const int in = rows == 256 ? 4 * slot : 4 * (slot & 1) + 16 * (slot >> 1);
    return (wv & 3) + (waves == 8 ? 8 * (wv >> 2) : 0) + in;
}
constexpr int run_row_unit(int rows, int waves, int u) {
    const int far = rows == 256 ? 16 : 32;
    return waves == 8 ? far * u : 8 * (u & 1) + far * (u >> 1);
}

MOE_DEV s16x4 read_tr(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// Asks the compiler for this order of half a step's instructions: READS LDS reads, and
// the first LOADS of the loads into LDS, spread between MFMAS matrix products
template <int READS, int MFMAS, int LOADS, int R = 0>
MOE_DEV void interleave() {
    if constexpr (R < READS) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // an LDS read
        if constexpr (R < LOADS) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);   // a load
        constexpr int n = (R + 1) * MFMAS / READS - R * MFMAS / READS;
        if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x8, n, 0);
        interleave<READS, MFMAS, LOADS, R + 1>();
    }
}

// Where a tile lies and what it multiplies
struct Tile {
    Operand P, Q;
    uint16_t* out;   // [q, p] with row stride ldo (DOWN, DX, DW)
    int64_t ldo;
    int K, segs, q0, p0;   // segs matrices one after another, K of k each
};
// Tile `tile` of a product with nq x np tiles of BQ x BP (DW: along I and along D): eight q tiles
// deep, so that the tiles an XCD works on at a time share their operands in its L2
template <Kind KIND, int BQ, int BP>
MOE_DEV Tile locate(const FfnArgs& a, int tile, int nq, int np) {
    Tile t;
    t.K = a.D, t.segs = 1, t.out = nullptr, t.ldo = 0;
    if (KIND == GATEUP) t.P = {a.wg, a.wu, a.D, a.I}, t.Q = {a.x, a.x, a.ldx, a.m};
    if (KIND == DOWN) t.P = {a.wd, a.wd, a.I, a.D}, t.Q = {a.h, a.h, a.I, a.m}, t.K = a.I, t.out = a.y, t.ldo = a.ldy;
    if (KIND == DH) t.P = {a.wd, a.wd, a.I, a.I}, t.Q = {a.dy, a.dy, a.lddy, a.m};
    if (KIND == DX) t.P = {a.wg, a.wu, a.D, a.D}, t.Q = {a.dg, a.du, a.I, a.m}, t.K = a.I, t.segs = 2, t.out = a.dx, t.ldo = a.lddx;
    if (KIND == DW) {
        // products whose output is not wanted have no tiles
        t.K = a.m;
        const int each = nq * np, n0 = a.dwg != nullptr ? each : 0, n1 = a.dwu != nullptr ? each : 0;
        if (tile < n0 + n1) {
            const bool up = tile >= n0;
            if (up) tile -= n0;
            t.P = {a.x, a.x, a.ldx, a.D}, t.Q = {up ? a.du : a.dg, nullptr, a.I, a.I};
            t.out = up ? a.dwu : a.dwg, t.ldo = a.D;
        } else {
            tile -= n0 + n1;
            t.P = {a.h, a.h, a.I, a.I}, t.Q = {a.dy, a.dy, a.lddy, a.D};
            t.out = a.dwd, t.ldo = a.I;
            nq = (a.D + BQ - 1) / BQ, np = (a.I + BP - 1) / BP;
        }
    }
    const int deep = 8 * np, gr = tile / deep, gq = min(8, nq - gr * 8), in = tile - gr * deep;
    t.q0 = (gr * 8 + in % gq) * BQ;
    t.p0 = in / gq * (KIND == GATEUP ? BP / 2 : BP);   // GATEUP: 32 rows of Wg, the same 32 of Wu, and so on
    return t;
}

// What a wavefront does with the sums of 16 q (q = qw + l16) and its TP p: a lane holds p =
// 16 i + 4 g + 0..3 in v[i], counted from pw
template <typename T, Kind KIND, int NI>
MOE_DEV void finish(const FfnArgs& a, const Tile& t, int qw, int pw, const f32x4 (&v)[NI]) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4, q = qw + l16;
    if constexpr (KIND == GATEUP) {
        if (qw >= a.m) return;
#pragma unroll
        for (int b = 0; b < NI / 4; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 gv = v[4 * b + i], uv = v[4 * b + 2 + i];
                const int at = t.p0 + (pw + 64 * b) / 2 + 16 * i, p = at + 4 * g;
                if (at >= a.I) continue;
                if (a.saved != nullptr) {
                    float* s = a.saved + saved_at(qw / 16, at / 16, a.I) + lane * 4;
                    *reinterpret_cast<f32x4*>(s) = gv;
                    *reinterpret_cast<f32x4*>(s + 256) = uv;
                }
                float h[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) h[r] = act_value(clamp_gate(gv[r], a.limit), a.act) * clamp_up(uv[r], a.limit);
                if (q < a.m && p < a.I)
                    *reinterpret_cast<uint2*>(a.h + (size_t)q * a.I + p) = make_uint2(T::pack2(h[0], h[1]), T::pack2(h[2], h[3]));
            }
    } else if constexpr (KIND == DH) {
        if (qw >= a.m) return;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = t.p0 + pw + 16 * i, p = at + 4 * g;
            if (at >= a.I) continue;
            const float* s = a.saved + saved_at(qw / 16, at / 16, a.I) + lane * 4;
            const f32x4 gv = *reinterpret_cast<const f32x4*>(s), uv = *reinterpret_cast<const f32x4*>(s + 256);
            float dg[4], du[4], h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float uc = clamp_up(uv[r], a.limit), dh = v[i][r];
                float f, df;
                act_both(clamp_gate(gv[r], a.limit), a.act, f, df);
                const bool clamped = a.limit > 0.f;
                dg[r] = clamped && gv[r] > a.limit ? 0.f : dh * uc * df;
                du[r] = clamped && fabsf(uv[r]) > a.limit ? 0.f : dh * f;
                h[r] = f * uc;
            }
            if (q < a.m && p < a.I) {
                const size_t o = (size_t)q * a.I + p;
                *reinterpret_cast<uint2*>(a.dg + o) = make_uint2(T::pack2(dg[0], dg[1]), T::pack2(dg[2], dg[3]));
                *reinterpret_cast<uint2*>(a.du + o) = make_uint2(T::pack2(du[0], du[1]), T::pack2(du[2], du[3]));
                *reinterpret_cast<uint2*>(a.h + o) = make_uint2(T::pack2(h[0], h[1]), T::pack2(h[2], h[3]));
            }
        }
    } else {
        if (q >= t.Q.rows) return;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int p = t.p0 + pw + 16 * i + 4 * g;
            if (p < t.P.rows)
                *reinterpret_cast<uint2*>(t.out + (size_t)q * t.ldo + p) = make_uint2(T::pack2(v[i][0], v[i][1]), T::pack2(v[i][2], v[i][3]));
        }
    }
}

// The work of one launch: the first `whole` tiles by a workgroup each, the `rest` (what does
// not fill the CUs once more) by `splits` workgroups each, every one with its part of k
struct Plan {
    int nq, np;          // tiles along q and p
    int whole, rest, splits;
    float* partial;      // [split][rest][j][i][thread] of the split tiles' sums, four f32 each
};

// BQ x BP tile of the output, WQ x WP wavefronts
template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void ffn_gemm_kernel(FfnArgs a, Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int TH = 64 * WQ * WP, TQ = BQ / WQ, TP = BP / WP, NI = TP / 16, NJ = TQ / 16;
    constexpr int UP = BP * 8 / TH, UQ = BQ * 8 / TH, NW = TH / 64;   // 16-byte units per thread
    constexpr bool PR = p_by_rows(KIND), QR = q_by_rows(KIND);
    constexpr int P_BYTES = tile_bytes(BP, PR), STEP = P_BYTES + tile_bytes(BQ, QR);
    static_assert(NW == 8 || NW == 4, "");
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, wq = wv / WP, wp = wv % WP;

    // consecutive tiles (of a split part: those of one part of k) on one XCD
    const int whole_blocks = (plan.whole + 7) / 8 * 8;
    int tile, split = -1;
    if ((int)blockIdx.x < whole_blocks) {
        tile = xcd_logical_block(blockIdx.x, plan.whole);
        if (tile >= plan.whole) return;
    } else {
        const int items = plan.rest * plan.splits, item = xcd_logical_block(blockIdx.x - whole_blocks, items);
        if (item >= items) return;
        split = item / plan.rest;
        tile = plan.whole + item - split * plan.rest;
    }
    const Tile t = locate<KIND, BQ, BP>(a, tile, plan.nq, plan.np);
    const Operand &P = t.P, &Q = t.Q;
    const int K = t.K, segs = t.segs, q0 = t.q0, p0 = t.p0;
    constexpr int PSPAN = KIND == GATEUP ? BP / 2 : BP;

    // This thread's first unit of each tile: its byte offset from the tile's corner; unit u is
    // unit_rows(u) rows further. A K-contiguous tile's units of a thread share their chunk of k.
    const int slot_p = PR ? lane / (BP / 8) : 0, slot_q = QR ? lane / (BQ / 8) : 0;
    const int row_k = wv * 8 + (lane >> 3), chunk = (lane & 7) ^ swz_k(row_k);
    const int first = KIND == GATEUP ? (row_k & 31) : row_k;
    const uint32_t off_p = PR ? (uint32_t)(run_row_wave(BP, NW, wv, slot_p) * P.ld + lane % (BP / 8) * 8) * 2
                              : (uint32_t)(first * P.ld + chunk * 8) * 2;
    const uint32_t off_q = QR ? (uint32_t)(run_row_wave(BQ, NW, wv, slot_q) * Q.ld + lane % (BQ / 8) * 8) * 2
                              : (uint32_t)(row_k * Q.ld + chunk * 8) * 2;

    const int seg_steps = (K + BK - 1) / BK, steps = seg_steps * segs;
    const int kt0 = split < 0 ? 0 : (int)((int64_t)split * steps / plan.splits);
    const int nk = (split < 0 ? steps : (int)((int64_t)(split + 1) * steps / plan.splits)) - kt0;
    auto stage = [&](int kt, uint8_t* buf) {
        const bool past = kt >= nk;
        kt += kt0;
        const int seg = segs == 2 && kt >= seg_steps ? 1 : 0;
        const int k0 = (kt - seg * seg_steps) * BK, kleft = min(BK, K - k0);
        const uint32_t beyond = chunk * 8 >= kleft ? PAST : 0u;   // a K tail's missing chunks
        auto side = [&](uint32_t off, const Operand& o, bool by_rows, int R, int at, int span, bool paired, int U, uint8_t* dst) {
            const uint16_t* base = seg ? o.b : o.a;
            const int left = min(o.rows - at, span);
            if (by_rows) {
                const auto buffer = buffer_rsrc(base + (size_t)k0 * o.ld + at, past ? 0u : (uint32_t)((kleft - 1) * o.ld + left) * 2);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    buffer_load_lds16(buffer, dst + (u * NW + wv) * PIECE, off + (uint32_t)(run_row_unit(R, NW, u) * o.ld * 2));
            } else {
                const uint32_t bytes = past ? 0u : (uint32_t)((left - 1) * o.ld + kleft) * 2;
                const size_t corner = (size_t)at * o.ld + k0;
                // GATEUP: rows 32..63 of every 64 are the second matrix's: with eight wavefronts those
                // of wavefronts 4..7, with four those of every second unit
                const bool second = paired && NW == 8 && (wv & 4);
                const auto buffer = buffer_rsrc((second ? o.b : base) + corner, bytes);
                const auto other = paired && NW == 4 ? buffer_rsrc(o.b + corner, bytes) : buffer;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int rows = paired ? (u * NW * 8 >> 6) * 32 : u * NW * 8;
                    const uint32_t v = (off + (uint32_t)(rows * o.ld * 2)) | beyond;
                    uint8_t* to = dst + (u * NW + wv) * 1024;
                    if (paired && NW == 4 && (u & 1)) buffer_load_lds16(other, to, v);
                    else buffer_load_lds16(buffer, to, v);
                }
            }
        };
        side(off_p, P, PR, BP, p0, PSPAN, KIND == GATEUP, UP, buf);
        side(off_q, Q, QR, BQ, q0, BQ, false, UQ, buf + P_BYTES);
    };

    // LDS byte offset of this lane's operand reads for half kk of a step; operand i lies 16 rows
    // further, which is a constant in either layout
    auto read_base = [&](bool by_rows, int R, int base, int kk) {
        if (by_rows) {
            const int run = (l16 >> 2) + 4 * (g & 1) + (R == 256 ? 8 * (g >> 1) : 0);
            return (run + kk * (R / 16)) * PIECE + (R == 256 ? 0 : (g >> 1) * 512) + base * 2 + (l16 & 3) * 8;
        }
        return (base + l16) * (BK * 2) + (((g + 4 * kk) ^ swz_k(l16)) << 4);
    };
    const int rdp0 = read_base(PR, BP, wp * TP, 0), rdp1 = read_base(PR, BP, wp * TP, 1);
    const int rdq0 = read_base(QR, BQ, wq * TQ, 0), rdq1 = read_base(QR, BQ, wq * TQ, 1);
    auto fragment = [&](const uint8_t* p, bool by_rows, int R, int i) -> s16x8 {
        if (by_rows) {
            const s16x4 lo = read_tr(p + i * 32), hi = read_tr(p + i * 32 + R * 2);   // k + 0..3, k + 4..7
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return *reinterpret_cast<const s16x8*>(p + i * 16 * BK * 2);
    };

    f32x4 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    // Half a K step (32 k) at a time: while one half is multiplied, the operands of the
    // next are read from LDS into registers. A step's buffer is free once its second half
    // is in registers, in the middle of its products: the barrier there lets the loads of
    // the step after next go into it, a whole step before they are needed.
    s16x8 fp[2][NI], fq[2][NJ];
    auto read_half = [&](const uint8_t* buf, int kk, int to) {
        const uint8_t *bp = buf + (kk ? rdp1 : rdp0), *bq = buf + P_BYTES + (kk ? rdq1 : rdq0);
#pragma unroll
        for (int i = 0; i < NI; ++i) fp[to][i] = fragment(bp, PR, BP, i);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fq[to][j] = fragment(bq, QR, BQ, j);
    };
    auto multiply = [&](int from) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[i][j] = T::mfma(fp[from][i], fq[from][j], acc[i][j]);
    };
    constexpr int READS = NI * (PR ? 2 : 1) + NJ * (QR ? 2 : 1), MFMAS = NI * NJ;
    // Two steps, one of each buffer. The buffers are the lambda's own restricted pointers so
    // that the compiler sees that the loads into one do not touch what is read from the other:
    // it would wait for every load before the next LDS read.
    auto two_steps = [&](uint8_t* __restrict b0, uint8_t* __restrict b1, int kt) {
        read_half(b0, 1, 1);
        multiply(0);
        interleave<READS, MFMAS, 0>();
        wait_vm_loads<0>();   // step kt + 1 has landed
        barrier_lds();        // for every wavefront, and every one has read the last of step kt
        stage(kt + 2, b0);
        read_half(b1, 0, 0);
        multiply(1);
        interleave<READS, MFMAS, UP + UQ>();
        read_half(b1, 1, 1);
        multiply(0);
        interleave<READS, MFMAS, 0>();
        wait_vm_loads<0>();
        barrier_lds();
        stage(kt + 3, b1);    // (past the last step: zeros)
        read_half(b0, 0, 0);
        multiply(1);
        interleave<READS, MFMAS, UP + UQ>();
    };
    if (nk > 0) {
        stage(0, smem);
        stage(1, smem + STEP);
        wait_vm_loads<UP + UQ>();
        barrier_lds();
        read_half(smem, 0, 0);
        int kt = 0;
        for (; kt + 2 < nk; kt += 2) two_steps(smem, smem + STEP, kt);
        read_half(smem, 1, 1);
        multiply(0);
        multiply(1);
        wait_vm_loads<0>();   // (no load into LDS outlives the workgroup)
        if (kt + 1 < nk) {
            barrier_lds();
            read_half(smem + STEP, 0, 0);
            read_half(smem + STEP, 1, 1);
            multiply(0);
            multiply(1);
        }
    }

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
        finish<T, KIND, NI>(a, t, q0 + wq * TQ + 16 * j, wp * TP, v);
    }
}

// The split tiles' sums, added in order of k, and what is done with them: a workgroup per
// tile and j (16 q of each wavefront)
template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void ffn_join_kernel(FfnArgs a, Plan plan) {
    constexpr int TH = 64 * WQ * WP, TQ = BQ / WQ, TP = BP / WP, NI = TP / 16, NJ = TQ / 16;
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
    finish<T, KIND, NI>(a, t, t.q0 + wq * TQ + 16 * j, wp * TP, v);
}

constexpr int SKINNY_WAVES = 8, SKINNY_LOADERS = 2, SKINNY_RING = 4;   // RING: slabs of x
// The sums of a workgroup's eight wavefronts, acc[t] of tokens 16 t + l16 and weight rows 4 g +
// 0..3, joined through LDS (which takes the place of x), and what is done with them
template <typename T, Kind KIND, int NT, int THREADS>
MOE_DEV void skinny_finish(const FfnArgs& a, float* red, int n0, const f32x4 (&acc)[NT]) {
    constexpr int RB = KIND == GATEUP ? 8 : 16;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, N = KIND == GATEUP ? a.I : a.D;
    __syncthreads();
    if (wv < SKINNY_WAVES) {
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(&red[(wv * NT + t) * 256 + lane * 4]) = acc[t];
    }
    __syncthreads();
    auto total = [&](int tok, int r) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < SKINNY_WAVES; ++i) v += red[(i * NT + (tok >> 4)) * 256 + ((r >> 2) * 16 + (tok & 15)) * 4 + (r & 3)];
        return v;
    };
    for (int e = tid; e < a.m * RB; e += THREADS) {
        const int tok = e / RB, c = e % RB, n = n0 + c;
        if (n >= N) continue;
        if (KIND == GATEUP) {
            const float gv = total(tok, c), uv = total(tok, c + 8);
            if (a.saved != nullptr) {
                float* s = a.saved + saved_at(tok >> 4, n >> 4, a.I) + (((n & 15) >> 2) * 16 + (tok & 15)) * 4 + (n & 3);
                s[0] = gv;
                s[256] = uv;
            }
            const float h = act_value(clamp_gate(gv, a.limit), a.act) * clamp_up(uv, a.limit);
            const auto rounded = T::store(h);
            a.h[(size_t)tok * a.I + n] = rounded;
            if (a.parts) {
                const float rest = h - T::load(rounded);
                a.h[(size_t)(a.m + tok) * a.I + n] = T::store(fabsf(rest) < INFINITY ? rest : 0.f);
            }
        } else {
            a.y[(size_t)tok * a.ldy + n] = T::store(total(tok, c));
        }
    }
}

// Up to 16 rows whose x fits into LDS whole: GATEUP or DOWN with the weights read straight into
// registers, since nothing would be read twice. A workgroup owns 16 weight rows (GATEUP: eight
// of Wg and the same eight of Wu), each of its eight wavefronts a part of k, and their sums are
// joined through LDS in wavefront order. There is one wait for x, and the wavefronts then
// go their own ways through k, AHEAD chunks of 32 of their weights in flight. One token of 5120 x
// 2304: 12.5 us (47 MB, 3.8 TB/s) and 6.7 us, 7.0 with h in two parts.
constexpr size_t FEW_LDS = 64 << 10;
MOE_DEV __host__ int few_row(int K) { return (K + 511) / 512 * 1024; }   // bytes of a token's row there

// Where h fits into LDS twice it is held in two 16-bit parts, its rounded value and what that leaves out
// (rows m and on), and DOWN multiplies both by a weight that it has read once: y is then rounded once. One
// token of 5120 x 2304: y's error 1.7e-3 of the norm, 2.4e-3 with h rounded, in 20.7 us against 20.2 (both
// products); 2 rows of 1544 x 4104 14.8 against 14.2. Past that the parts cost more: 8 rows of 5120 x
// 2304, in slabs, 31.9 against 29.0, 12 of 2048 x 2048 12.6 against 11.0, and many rows a second product.
bool h_in_parts(int m, int I) { return m <= 16 && 2 * m * (size_t)few_row(I) <= FEW_LDS; }
// the sums of the two parts: the second is small, and means nothing where it is not finite (an infinite
// weight times a zero, or with another sign)
MOE_DEV f32x4 join_parts(f32x4 v, f32x4 rest) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += fabsf(rest[r]) < INFINITY ? rest[r] : 0.f;
    return v;
}

// PARTS: of h, DOWN only
template <typename T, Kind KIND, bool PARTS>
__global__ __launch_bounds__(64 * SKINNY_WAVES) void ffn_few_kernel(FfnArgs a) {
    constexpr int RB = KIND == GATEUP ? 8 : 16, AHEAD = 5;
    extern __shared__ __align__(16) uint8_t smem[];   // x; then sums [wavefront][256]
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int K = KIND == GATEUP ? a.D : a.I, N = KIND == GATEUP ? a.I : a.D, n0 = blockIdx.x * RB;
    const int64_t ldx = KIND == GATEUP ? a.ldx : a.I;
    const int row_bytes = few_row(K), runs = row_bytes / 1024;
    const int rows = PARTS ? 2 * a.m : a.m;
    const auto X = buffer_rsrc(KIND == GATEUP ? a.x : a.h, (uint32_t)((rows - 1) * ldx + K) * 2);
    for (int r = wv; r < rows * runs; r += SKINNY_WAVES) {
        // 16-byte chunk c of a row lies at c ^ (row & 15)
        const int row = r / runs, k = (r - row * runs) * 512 + (lane ^ (row & 15)) * 8;
        buffer_load_lds16(X, smem + r * 1024, k < K ? (uint32_t)(row * ldx + k) * 2 : PAST);
    }
    const int chunks = (K + 31) / 32, c0 = wv * chunks / SKINNY_WAVES, c1 = (wv + 1) * chunks / SKINNY_WAVES;
    const int row = min(n0 + (l16 & (RB - 1)), N - 1);
    const uint16_t* w = (KIND == DOWN ? a.wd : l16 < 8 ? a.wg : a.wu) + (size_t)row * K;
    uint4 wq[AHEAD];
    auto request = [&](int i, int c) { wq[i] = *reinterpret_cast<const uint4*>(w + min(32 * min(c, chunks - 1) + 8 * g, K - 8)); };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) request(i, c0 + i);
    wait_vm_loads<AHEAD>();   // this wavefront's part of x has landed
    barrier_lds();
    const int xt = min(l16, a.m - 1);   // (a token that does not exist reads another's; its sums are not used)
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}}, rest = {0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int i, int c) {
        // a weight that stands in for one past K is not one (x is zero there)
        const uint32_t on = 32 * c + 8 * g < K ? ~0u : 0u;
        const u32x4 wm = {wq[i].x & on, wq[i].y & on, wq[i].z & on, wq[i].w & on};
        const int cx = c * 4 + g;
        auto product = [&](int row, f32x4 v) {
            return T::mfma(__builtin_bit_cast(s16x8, wm), *reinterpret_cast<const s16x8*>(smem + row * row_bytes + ((cx ^ (row & 15)) << 4)), v);
        };
        acc[0] = product(xt, acc[0]);
        if (PARTS) rest = product(a.m + xt, rest);
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
        if (c + i < c1) multiply(i, c + i);   // (a chunk of another's part is left out: its x times a zero weight is NaN if infinite)
    if (PARTS) acc[0] = join_parts(acc[0], rest);
    skinny_finish<T, KIND, 1, 64 * SKINNY_WAVES>(a, reinterpret_cast<float*>(smem), n0, acc);
}

// Few rows (m <= ROWS) whose x does not: the same weight rows, but the eight wavefronts split
// every slab of KS k between them. x comes into LDS a slab at a time, whole lines of
// it (a load that gathers 16 rows takes about 90 cycles of a CU's load path, one of whole
// lines 16, so that x straight from the L2s cost as much as the weights). Two wavefronts of
// their own load it: loads complete in the order of a wavefront's requests, so that one which
// waited for x would wait for every weight that it had requested before. 47 rows of 8192 x 2048:
// 25.2 us (67 MB, 2.7 TB/s) and 17.4 us; 32 rows 34.0 us together. A slab of
// x is three times its weights there, and is what bounds it.
constexpr int skinny_slab(int rows) { return rows <= 16 ? 512 : 256; }
template <typename T, Kind KIND, int ROWS>
__global__ __launch_bounds__(64 * (SKINNY_WAVES + SKINNY_LOADERS)) void ffn_skinny_kernel(FfnArgs a) {
    constexpr int RB = KIND == GATEUP ? 8 : 16, NT = (ROWS + 15) / 16;   // RB: output columns
    constexpr int KS = skinny_slab(ROWS), PER = KS / 32 / SKINNY_WAVES, ROW = KS * 2, RUN = 1024 / ROW;   // RUN: rows per load into LDS
    constexpr int AHEAD = KS == 512 ? 5 : 8;   // slabs of weights in flight
    extern __shared__ __align__(16) uint8_t smem[];   // RING slabs of x [token][KS]; then sums [wavefront][NT][256]
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int K = KIND == GATEUP ? a.D : a.I, N = KIND == GATEUP ? a.I : a.D, n0 = blockIdx.x * RB;
    const int slabs = (K + KS - 1) / KS;
    const int64_t ldx = KIND == GATEUP ? a.ldx : a.I;
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (wv >= SKINNY_WAVES) {
        constexpr int LOADS = ROWS / RUN / SKINNY_LOADERS;   // of one loader and slab
        const auto X = buffer_rsrc(KIND == GATEUP ? a.x : a.h, (uint32_t)((a.m - 1) * ldx + K) * 2);
        const int in_run = lane / (64 / RUN), slot = lane % (64 / RUN);
        auto stage = [&](int b) {   // (past the last slab, past m or K: zeros)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int r = ((wv - SKINNY_WAVES) * LOADS + i) * RUN, tok = r + in_run;
                // 16-byte chunk c of a token's row lies at c ^ (token & 15)
                const int k = b * KS + (slot ^ (tok & 15)) * 8;
                buffer_load_lds16(X, smem + (b % SKINNY_RING * ROWS + r) * ROW, tok < a.m && k < K ? (uint32_t)(tok * ldx + k) * 2 : PAST);
            }
        };
#pragma unroll
        for (int b = 0; b < SKINNY_RING - 1; ++b) stage(b);
        for (int b = 0; b < slabs; ++b) {
            wait_vm_loads<(SKINNY_RING - 2) * LOADS>();   // slab b has landed
            barrier_lds();                                // every wavefront is done with slab b - 1
            stage(b + SKINNY_RING - 1);
        }
        wait_vm_loads<0>();
    } else {
        const int row = min(n0 + (l16 & (RB - 1)), N - 1);
        const uint16_t* w = (KIND == DOWN ? a.wd : l16 < 8 ? a.wg : a.wu) + (size_t)row * K;
        auto k_of = [&](int b, int i) { return b * KS + (wv * PER + i) * 32 + 8 * g; };
        uint4 wq[AHEAD][PER];
        auto request = [&](int at, int b) {
#pragma unroll
            for (int i = 0; i < PER; ++i) wq[at][i] = *reinterpret_cast<const uint4*>(w + min(k_of(b, i), K - 8));
        };
        int xrow[NT];   // this lane's token rows
#pragma unroll
        for (int t = 0; t < NT; ++t) xrow[t] = min(16 * t + l16, ROWS - 1);
        auto slab = [&](int at, int b) {
            barrier_lds();   // slab b of x has landed
            const uint8_t* x = smem + b % SKINNY_RING * ROWS * ROW;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                // (a weight past K is another of its row: x is zero there, but a NaN must not come in)
                const uint32_t on = k_of(b, i) < K ? ~0u : 0u;
                const u32x4 wm = {wq[at][i].x & on, wq[at][i].y & on, wq[at][i].z & on, wq[at][i].w & on};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int c = (wv * PER + i) * 4 + g;
                    const s16x8 xv = *reinterpret_cast<const s16x8*>(x + xrow[t] * ROW + ((c ^ (xrow[t] & 15)) << 4));
                    acc[t] = T::mfma(__builtin_bit_cast(s16x8, wm), xv, acc[t]);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) request(i, min(i, slabs - 1));
        int b = 0;
        for (; b + 2 * AHEAD <= slabs; b += AHEAD)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                slab(i, b + i);
                request(i, b + AHEAD + i);
            }
        for (; b < slabs; b += AHEAD)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (b + i < slabs) {
                    slab(i, b + i);
                    if (b + AHEAD + i < slabs) request(i, b + AHEAD + i);
                }
    }
    skinny_finish<T, KIND, NT, 64 * (SKINNY_WAVES + SKINNY_LOADERS)>(a, reinterpret_cast<float*>(smem), n0, acc);
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

// Tiles of B x B, B = 256 (eight wavefronts, one workgroup per CU) or 128 (four, two per CU)
constexpr int N_CU = 256, MAX_SPLITS = 16;
struct Product {
    Plan plan;
    int tile;         // 256 or 128
};
// tiles along q and p, all of them, K steps of one, and how many the CUs hold at a time. DW: of
// `products` outputs
struct Extent {
    int nq, np, tiles, steps, slots;
};
Extent extent(Kind kind, int m, int D, int I, int products, int B) {
    Extent e;
    e.steps = kind == DX ? 2 * cdiv(I, BK) : cdiv(kind == DOWN ? I : kind == DW ? m : D, BK);
    if (kind == DW) e.nq = cdiv(I, B), e.np = cdiv(D, B);
    else e.nq = cdiv(m, B), e.np = cdiv(kind == GATEUP ? 2 * I : kind == DH ? I : D, B);
    e.tiles = e.nq * e.np * (kind == DW ? products : 1);
    e.slots = B == 256 ? N_CU : 2 * N_CU;
    return e;
}
// Bytes that hold the split tiles' sums of any plan for m rows or fewer: the parts are at most the
// slots, and at most the tiles times the splits. (The sums of one plan jump with m: 6.8 MB for
// 1536 rows of 5120 x 2304, 58 MB for 1000, so that a workspace of just that size would be too
// small for a smaller batch. This is 64 MiB at most.)
size_t partial_bytes(Kind kind, int m, int D, int I, int products) {
    size_t most = 0;
    for (int B : {256, 128}) {
        const Extent e = extent(kind, m, D, I, products, B);
        const int splits = std::min(MAX_SPLITS, e.steps / 2);
        if (splits >= 2) most = std::max(most, (size_t)std::min<int64_t>(e.slots, (int64_t)e.tiles * splits) * B * B * sizeof(float));
    }
    return most;
}

// How a product is cut up: 256 x 256 or 128 x 128 tiles, and by how much the tiles past the last full
// round of the CUs are split along k. Costs in units of one K step of a 256 x 256 tile on a CU
// (about 1.65 us): a 128 x 128 tile's step takes 0.33 of it (a quarter of the products, at three quarters
// of the rate); the split tiles' sums pass through memory twice (0.06 a 256 x 256 tile and split, and 4 for
// the second launch). What the end of a tile loads and stores is not counted; of a product with few
// steps it is half the time (GATEUP of 1013 rows of 1544 x 4104, 25 steps in one round: 50 us, its steps
// alone by these costs 27). 8192 rows of 5120 x 2304 in the large tiles and in the small: GATEUP 334 and
// 377 us, DOWN 187 and 196, DH 266 and 271, DX 346 and 422, DW 533 and 624.
Product plan_product(Kind kind, int m, int D, int I, int products) {
    Product best{};
    double best_cost = 1e30;
    for (int B : {256, 128}) {
        const Extent e = extent(kind, m, D, I, products, B);
        Product p{};
        p.tile = B;
        p.plan.nq = e.nq, p.plan.np = e.np;
        const double step = B == 256 ? 1 : 0.66, share = B == 256 ? 0.06 : 0.015;   // (two workgroups share a CU)
        const int rounds = e.tiles / e.slots, rest = e.tiles % e.slots;
        double cost = rounds * (double)e.steps * step;
        p.plan.whole = e.tiles, p.plan.splits = 1;
        if (rest > 0) {
            double tail = e.steps * step;
            for (int s = 2; s <= MAX_SPLITS && s * 2 <= e.steps && rest * s <= e.slots; ++s) {
                const double t = cdiv(e.steps, s) * step + 4 + share * rest * s;
                if (t < tail) tail = t, p.plan.whole = e.tiles - rest, p.plan.rest = rest, p.plan.splits = s;
            }
            cost += tail;
        }
        if (cost < best_cost) best_cost = cost, best = p;
    }
    return best;
}

template <typename T, Kind KIND, int B, int WQ, int WP>
hipError_t launch_tiles(const FfnArgs& a, const Plan& plan, hipStream_t st) {
    const int grid = (plan.whole + 7) / 8 * 8 + (plan.rest * plan.splits + 7) / 8 * 8;
    if (grid == 0) return hipSuccess;
    constexpr int NJ = B / WQ / 16;
    const hipError_t e = launch_kernel(ffn_gemm_kernel<T, KIND, B, B, WQ, WP>, dim3(grid), dim3(64 * WQ * WP),
                                       2 * (tile_bytes(B, p_by_rows(KIND)) + tile_bytes(B, q_by_rows(KIND))), st, a, plan);
    if (e != hipSuccess || plan.rest == 0) return e;
    return launch_kernel(ffn_join_kernel<T, KIND, B, B, WQ, WP>, dim3(plan.rest * NJ), dim3(64 * WQ * WP), 0, st, a, plan);
}

template <typename T, Kind KIND>
hipError_t launch_product(const FfnArgs& a, float* partial, hipStream_t st) {
    Product p = plan_product(KIND, a.m, a.D, a.I, (a.dwg != nullptr) + (a.dwu != nullptr) + (a.dwd != nullptr));
    p.plan.partial = partial;
    return p.tile == 256 ? launch_tiles<T, KIND, 256, 2, 4>(a, p.plan, st) : launch_tiles<T, KIND, 128, 2, 2>(a, p.plan, st);
}

constexpr int MAX_M = 1 << 24;
constexpr int TILES_ABOVE = 32;   // as many rows or fewer of a forward pass never go in tiles

int check_ffn(const moe_ffn* f) {
    if (f == nullptr) return MOE_EINVAL;
    for (int v : {f->dim, f->inter})
        if (v < 8 || v > 16384 || v % 8) return MOE_EINVAL;
    if ((f->dtype != MOE_BF16 && f->dtype != MOE_F16) || (f->act != MOE_ACT_SILU && f->act != MOE_ACT_GELU)) return MOE_EINVAL;
    if (f->limit != f->limit) return MOE_EINVAL;
    for (const void* w : {f->w_gate, f->w_up, f->w_down})
        if (w == nullptr || !aligned_to(w, 16)) return MOE_EINVAL;
    return MOE_OK;
}

// 16-byte rows; the longest stride keeps a tile's offsets within 32 bits
bool rows_ok(const void* p, int64_t ld, int dim) {
    return p != nullptr && aligned_to(p, 16) && ld >= dim && ld % 8 == 0 && ld <= (1 << 22);
}

size_t rows_bytes(const moe_ffn* f, int m) { return round_up((size_t)m * f->inter * 2, 256); }
// room for the split tiles' sums of the products of one direction, whichever outputs are wanted
size_t forward_partial(const moe_ffn* f, int m) {
    if (m <= TILES_ABOVE) return 0;
    return std::max(partial_bytes(GATEUP, m, f->dim, f->inter, 0), partial_bytes(DOWN, m, f->dim, f->inter, 0));
}
size_t backward_partial(const moe_ffn* f, int m) {
    return std::max({partial_bytes(DH, m, f->dim, f->inter, 0), partial_bytes(DX, m, f->dim, f->inter, 0),
                     partial_bytes(DW, m, f->dim, f->inter, 3)});
}
// (h: 16 rows in two parts are as many as 32)
size_t h_bytes(const moe_ffn* f, int m) { return m <= 16 ? 2 * rows_bytes(f, m) : rows_bytes(f, std::max(m, 32)); }
size_t forward_bytes(const moe_ffn* f, int m) { return h_bytes(f, m) + forward_partial(f, m); }
size_t backward_bytes(const moe_ffn* f, int m) { return 3 * rows_bytes(f, m) + backward_partial(f, m); }
size_t saved_bytes_of(const moe_ffn* f, int m) { return (size_t)cdiv(m, 16) * cdiv(f->inter, 16) * 2048; }

FfnArgs describe(const moe_ffn* f, int m) {
    FfnArgs a{};
    a.wg = reinterpret_cast<const uint16_t*>(f->w_gate);
    a.wu = reinterpret_cast<const uint16_t*>(f->w_up);
    a.wd = reinterpret_cast<const uint16_t*>(f->w_down);
    a.m = m, a.D = f->dim, a.I = f->inter, a.act = f->act, a.limit = f->limit;
    return a;
}

template <typename T, Kind KIND, int ROWS>
hipError_t launch_skinny(const FfnArgs& a, hipStream_t st) {
    const size_t lds = std::max<size_t>(SKINNY_RING * ROWS * skinny_slab(ROWS) * 2, sizeof(float) * SKINNY_WAVES * cdiv(ROWS, 16) * 256);
    return launch_kernel(ffn_skinny_kernel<T, KIND, ROWS>, dim3(KIND == GATEUP ? cdiv(a.I, 8) : cdiv(a.D, 16)),
                         dim3(64 * (SKINNY_WAVES + SKINNY_LOADERS)), lds, st, a);
}

// LDS room for 16, 24, 32, 40, 48 or 64 rows of x
constexpr int skinny_room(int m) { return m <= 16 ? 16 : m <= 48 ? (m + 7) / 8 * 8 : 64; }

// 33 to 64 rows: whether weight rows are faster than tiles, by what either costs in us. By weight rows
// each 256 workgroups take 4 and what a CU loads, K times the room for x and 16 weight rows, at 55
// bytes a ns, whether a CU has two of them at a time or one after the other. Tiles take 14, or 3 and one for
// each K step where that is less, and the weights at 5.5 TB/s. Over 155 forward calls (33 to 64 rows, 31 widths of
// 264 x 4232 to 16384 x 4096) the two choices of a call cost 0.4% more than the best two on average, 6.5% at most; going by
// the number of workgroups alone cost 7.5% and 64%. GATEUP, weight rows against tiles, 40 and 64 rows: 2048 x
// 2048 (D x I) 9.1 against 17.0 us, 10.3 against 17.2; 5120 x 2304 28.6 against 24.2, 34.8 against 25.1; 8192 x 2048
// 23.8 against 27.8, 28.6 against 26.9; 10240 x 2560 55.4 against 34.0, 67.9 against 34.2; 14336 x 1024 36.7
// against 25.0, 45.3 against 25.5. DOWN: 4096 x 4096 13.9 against 17.7, 16.6 against 18.1; 8192 x 1024 9.5 against
// 18.7, 14.1 against 18.8; 8192 x 256 7.5 against 5.3, 10.6 against 5.5; 16384 x 2048 29.9 against 25.3, 37.4
// against 25.7.
bool by_weight_rows(int m, int K, int blocks) {
    const double rows = cdiv(blocks, N_CU) * (4 + K * (skinny_room(m) + 16.0) * 2 / 55e3);
    const double tiles = std::min(14.0, 3 + K / 64.0) + blocks * 16.0 * K * 2 / 5.5e6;
    return rows < tiles;
}

// GATEUP or DOWN of the forward pass. Few rows go by weight rows, more in tiles: 32 rows of 5120 x
// 2304 (D x I, both products) take 36.5 against 39.6 us, of 8192 x 2048 33.8 against 46.0, of 1024 x
// 1024 11.6 against 22.2 (of 8192 x 8192 114.8 against 108.3).
template <typename T, Kind KIND>
hipError_t launch_forward(const FfnArgs& a, float* partial, hipStream_t st) {
    const int K = KIND == GATEUP ? a.D : a.I, blocks = KIND == GATEUP ? cdiv(a.I, 8) : cdiv(a.D, 16);
    if (a.m > 64 || (a.m > TILES_ABOVE && !by_weight_rows(a.m, K, blocks))) return launch_product<T, KIND>(a, partial, st);
    // up to 16 rows that fit into LDS whole: one row of 5120 x 2304 21.8 against 27.7 us in slabs, of
    // 8192 x 2048 23.7 against 27.0, 16 rows of 1024 x 1024 7.9 against 11.4
    const bool parts = KIND == DOWN && a.parts;
    const size_t whole = (parts ? 2 : 1) * a.m * (size_t)few_row(K);
    if (a.m <= 16 && whole <= FEW_LDS)
        return launch_kernel(parts ? ffn_few_kernel<T, KIND, KIND == DOWN> : ffn_few_kernel<T, KIND, false>, dim3(blocks),
                             dim3(64 * SKINNY_WAVES), std::max<size_t>(whole, sizeof(float) * SKINNY_WAVES * 256), st, a);
    // (room for 24 and 40 rows: 20 rows of 5120 x 2304 33.8 against 35.1 us in room for 32, 36 rows of 8192
    // x 2048 36.6 against 40.3 in room for 48, which two workgroups of a CU do not have)
    switch (skinny_room(a.m)) {
        case 16: return launch_skinny<T, KIND, 16>(a, st);
        case 24: return launch_skinny<T, KIND, 24>(a, st);
        case 32: return launch_skinny<T, KIND, 32>(a, st);
        case 40: return launch_skinny<T, KIND, 40>(a, st);
        case 48: return launch_skinny<T, KIND, 48>(a, st);
        default: return launch_skinny<T, KIND, 64>(a, st);
    }
}

template <typename T>
hipError_t forward(const FfnArgs& a, float* partial, hipStream_t st) {
    const hipError_t e = launch_forward<T, GATEUP>(a, partial, st);
    return e != hipSuccess ? e : launch_forward<T, DOWN>(a, partial, st);
}

template <typename T>
hipError_t backward(const FfnArgs& a, float* partial, hipStream_t st) {
    hipError_t e = a.m > 0 ? launch_product<T, DH>(a, partial, st) : hipSuccess;
    if (e == hipSuccess && a.m > 0 && a.dx != nullptr) e = launch_product<T, DX>(a, partial, st);
    if (e == hipSuccess) e = launch_product<T, DW>(a, partial, st);
    return e;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_ffn_workspace(const moe_ffn* f, int32_t m, size_t* forward, size_t* saved, size_t* backward) {
    const int rc = check_ffn(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M || forward == nullptr || saved == nullptr || backward == nullptr) return MOE_EINVAL;
    *forward = forward_bytes(f, m);
    *saved = saved_bytes_of(f, m);
    *backward = backward_bytes(f, m);
    return MOE_OK;
}

int moe_ffn_forward(const moe_ffn* f, const void* x, int64_t ldx, int32_t m, void* y, int64_t ldy, void* saved,
                    size_t saved_bytes, void* work, size_t work_bytes, void* stream) {
    const int rc = check_ffn(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M) return MOE_EINVAL;
    if (m == 0) return MOE_OK;
    if (!rows_ok(x, ldx, f->dim) || !rows_ok(y, ldy, f->dim)) return MOE_EINVAL;
    if (work == nullptr || !aligned_to(work, 256) || !aligned_to(saved, 256)) return MOE_EINVAL;
    if (work_bytes < forward_bytes(f, m) || (saved != nullptr && saved_bytes < saved_bytes_of(f, m))) return MOE_ESCRATCH;
    FfnArgs a = describe(f, m);
    a.x = reinterpret_cast<const uint16_t*>(x), a.ldx = ldx;
    a.y = reinterpret_cast<uint16_t*>(y), a.ldy = ldy;
    a.h = reinterpret_cast<uint16_t*>(work);
    a.saved = reinterpret_cast<float*>(saved);
    a.parts = h_in_parts(m, f->inter);
    float* const partial = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(work) + h_bytes(f, m));
    const hipStream_t st = (hipStream_t)stream;
    return status_of(f->dtype == MOE_BF16 ? forward<Bf16>(a, partial, st) : forward<F16>(a, partial, st));
}

int moe_ffn_backward(const moe_ffn* f, const void* x, int64_t ldx, const void* dy, int64_t lddy, int32_t m,
                     const void* saved, size_t saved_bytes, void* dx, int64_t lddx, void* dw_gate, void* dw_up,
                     void* dw_down, void* work, size_t work_bytes, void* stream) {
    const int rc = check_ffn(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_M) return MOE_EINVAL;
    for (const void* p : {dw_gate, dw_up, dw_down})
        if (!aligned_to(p, 16)) return MOE_EINVAL;
    FfnArgs a = describe(f, m);
    if (m > 0) {
        if (!rows_ok(x, ldx, f->dim) || !rows_ok(dy, lddy, f->dim) || (dx != nullptr && !rows_ok(dx, lddx, f->dim)))
            return MOE_EINVAL;
        if (saved == nullptr || !aligned_to(saved, 256) || work == nullptr || !aligned_to(work, 256)) return MOE_EINVAL;
        if (work_bytes < backward_bytes(f, m) || saved_bytes < saved_bytes_of(f, m)) return MOE_ESCRATCH;
        a.x = reinterpret_cast<const uint16_t*>(x), a.ldx = ldx;
        a.dy = reinterpret_cast<const uint16_t*>(dy), a.lddy = lddy;
        a.dx = reinterpret_cast<uint16_t*>(dx), a.lddx = lddx;
        a.saved = reinterpret_cast<float*>(const_cast<void*>(saved));
        uint8_t* w = reinterpret_cast<uint8_t*>(work);
        a.dg = reinterpret_cast<uint16_t*>(w);
        a.du = reinterpret_cast<uint16_t*>(w + rows_bytes(f, m));
        a.h = reinterpret_cast<uint16_t*>(w + 2 * rows_bytes(f, m));
    }
    a.dwg = reinterpret_cast<uint16_t*>(dw_gate);
    a.dwu = reinterpret_cast<uint16_t*>(dw_up);
    a.dwd = reinterpret_cast<uint16_t*>(dw_down);
    float* const partial = m > 0 ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(work) + 3 * rows_bytes(f, m)) : nullptr;
    const hipStream_t st = (hipStream_t)stream;
    return status_of(f->dtype == MOE_BF16 ? backward<Bf16>(a, partial, st) : backward<F16>(a, partial, st));
}

}  // extern "C"
