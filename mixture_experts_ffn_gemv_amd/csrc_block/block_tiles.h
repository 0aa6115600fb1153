// Tiles of matrix products for the matrix cores, through LDS: what the dense products of
// the operators around the layer share.
//
// Every product is out[q, p] = sum_k P(k, p) Q(k, q) with p the consecutive index of
// the output. P is the matrix instruction's first operand, so that a lane's four
// results are four consecutive values of one output row. An operand either has k as
// its consecutive index (tiles of rows x 64 k; one 16-byte LDS read per lane gives
// eight k) or p / q (tiles of 64 k x rows; two transposing 8-byte LDS reads), so no
// operand is ever transposed in memory.
//
// Tiles come into LDS by buffer loads straight to LDS, 16 bytes per lane, a K step of 64
// ahead. What lies past an operand's rows or past its k lands as zeros: rows by the buffer's
// length, a K tail by an offset past it. Chunks of 16 bytes are stored permuted so that
// the LDS reads of a matrix operand fall on distinct banks.
#pragma once

#include "block_common.h"

namespace moe {
namespace {

constexpr int BK = 64;
constexpr uint32_t PAST = 0xFFFFFFF0u;   // an offset past every buffer: zeros

// one operand of a product: up to two matrices, used side by side (PAIRED) or one
// after the other along k
struct Operand {
    const uint16_t *a, *b;
    int64_t ld;
    int rows;   // extent of p or q
    int k;      // of one matrix
};

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

// The lane, opaque to the compiler: what follows from it is worked out where it is used, and not kept in registers
// over another tile's products
MOE_DEV int lane_here() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// A BQ x BP tile of the output by WQ x WP wavefronts: acc[i][j] of a lane holds p = 16 i + 4 (lane / 16) +
// 0..3 and q = 16 j + lane % 16 of its wavefront's part. PR, QR: p or q (not k) is the operand's
// consecutive index. PAIRED: of every 64 p, the first 32 are P's first matrix, the others the second;
// Q_PAIRED: the same of q. K_PAIRED (both operands by rows): a K step is 32 k of the operands' first matrices and the same 32
// of their second.
template <typename T, bool PR, bool QR, bool PAIRED, int BQ, int BP, int WQ, int WP, bool Q_PAIRED = false, bool K_PAIRED = false>
struct TileProduct {
    static constexpr int TH = 64 * WQ * WP, TQ = BQ / WQ, TP = BP / WP, NI = TP / 16, NJ = TQ / 16;
    static constexpr int UP = BP * 8 / TH, UQ = BQ * 8 / TH, NW = TH / 64;   // 16-byte units per thread
    static constexpr int P_BYTES = tile_bytes(BP, PR), STEP = P_BYTES + tile_bytes(BQ, QR);
    static constexpr int PSPAN = PAIRED ? BP / 2 : BP, QSPAN = Q_PAIRED ? BQ / 2 : BQ, KSPAN = K_PAIRED ? BK / 2 : BK;
    static constexpr size_t LDS = 2 * STEP;
    static_assert(NW == 8 || NW == 4, "");
    static_assert(!(PAIRED && PR) && !(Q_PAIRED && QR), "");
    static_assert(!K_PAIRED || (PR && QR && BP == BQ && BQ == 32 * NW), "");   // (a unit's k are below 32 or none is)
    static_assert((!PR || BP == 128 || BP == 256) && (!QR || BQ == 128 || BQ == 256), "");

    // A product's tile and its K steps kt0 .. kt0 + nk - 1; segs matrices one after another along k
    struct Work {
        const Operand &P, &Q;
        int segs, q0, p0, kt0, nk;
    };

    // This thread's first unit of each tile: its byte offset from the tile's corner; unit u is
    // unit_rows(u) rows further. A K-contiguous tile's units of a thread share their chunk of k.
    struct Units {
        uint32_t off_p, off_q;
        int chunk;
    };
    static MOE_DEV Units units(const Work& w) {
        const int lane = lane_here(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int slot_p = PR ? lane / (BP / 8) : 0, slot_q = QR ? lane / (BQ / 8) : 0;
        const int row_k = wv * 8 + (lane >> 3), chunk = (lane & 7) ^ swz_k(row_k);
        const int first = PAIRED ? (row_k & 31) : row_k;
        Units s;
        s.chunk = chunk;
        s.off_p = PR ? (uint32_t)(run_row_wave(BP, NW, wv, slot_p) * w.P.ld + lane % (BP / 8) * 8) * 2
                     : (uint32_t)(first * w.P.ld + chunk * 8) * 2;
        s.off_q = QR ? (uint32_t)(run_row_wave(BQ, NW, wv, slot_q) * w.Q.ld + lane % (BQ / 8) * 8) * 2
                     : (uint32_t)((Q_PAIRED ? row_k & 31 : row_k) * w.Q.ld + chunk * 8) * 2;
        return s;
    }

    // requests step kt's tiles (past the last: zeros)
    static MOE_DEV void stage(const Work& w, const Units& s, int kt, uint8_t* buf) {
        const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int seg_steps = (w.P.k + KSPAN - 1) / KSPAN;
        const bool past = kt >= w.nk;
        kt += w.kt0;
        const int seg = w.segs == 2 && kt >= seg_steps ? 1 : 0;
        const int k0 = (kt - seg * seg_steps) * KSPAN;
        auto side = [&](uint32_t off, const Operand& o, bool by_rows, int R, int at, int span, bool paired, int U, uint8_t* dst) {
            const uint16_t* base = seg ? o.b : o.a;
            const int left = min(o.rows - at, span), kleft = min(KSPAN, o.k - k0);
            const uint32_t beyond = s.chunk * 8 >= kleft ? PAST : 0u;   // a K tail's missing chunks
            if (by_rows) {
                const auto buffer = buffer_rsrc(base + (size_t)k0 * o.ld + at, past ? 0u : (uint32_t)((kleft - 1) * o.ld + left) * 2);
                // (with both operands by rows the units' offsets would not fit into the registers beside the sums)
                if (PR && QR) asm volatile("" : "+v"(off));
                if constexpr (K_PAIRED) {
                    const auto other = buffer_rsrc(o.b + (size_t)k0 * o.ld + at, past ? 0u : (uint32_t)((kleft - 1) * o.ld + left) * 2);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int row = run_row_unit(R, NW, u);
                        buffer_load_lds16(row < KSPAN ? buffer : other, dst + (u * NW + wv) * PIECE, off + (uint32_t)(row % KSPAN * o.ld * 2));
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        buffer_load_lds16(buffer, dst + (u * NW + wv) * PIECE, off + (uint32_t)(run_row_unit(R, NW, u) * o.ld * 2));
                }
            } else {
                const uint32_t bytes = past ? 0u : (uint32_t)((left - 1) * o.ld + kleft) * 2;
                const size_t corner = (size_t)at * o.ld + k0;
                // PAIRED: rows 32..63 of every 64 are the second matrix's: with eight wavefronts those
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
        side(s.off_p, w.P, PR, BP, w.p0, PSPAN, PAIRED, UP, buf);
        side(s.off_q, w.Q, QR, BQ, w.q0, QSPAN, Q_PAIRED, UQ, buf + P_BYTES);
    }

    // requests the first two steps, into buffers that nobody reads any more
    static MOE_DEV void begin(const Work& w, uint8_t* smem) {
        if (w.nk <= 0) return;
        const Units s = units(w);
        stage(w, s, 0, smem);
        stage(w, s, 1, smem + STEP);
    }

    // the sums, after begin; AFTER: other memory operations may have followed begin's. At the end this
    // wavefront has read all that it will of the buffers.
    template <bool AFTER>
    static MOE_DEV void sums(const Work& w, uint8_t* smem, f32x4 (&acc)[NI][NJ]) {
        const int lane = lane_here(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int l16 = lane & 15, g = lane >> 4, wq = wv / WP, wp = wv % WP;
        const int nk = w.nk;
        const Units s = units(w);
        // LDS byte offset of this lane's operand reads for half kk of a step; operand i lies 16 rows
        // further, which is a constant in either layout, as the second half is in one by rows
        auto read_base = [&](bool by_rows, int R, int base, int kk) {
            if (by_rows) {
                const int run = (l16 >> 2) + 4 * (g & 1) + (R == 256 ? 8 * (g >> 1) : 0);
                return (run + kk * (R / 16)) * PIECE + (R == 256 ? 0 : (g >> 1) * 512) + base * 2 + (l16 & 3) * 8;
            }
            return (base + l16) * (BK * 2) + (((g + 4 * kk) ^ swz_k(l16)) << 4);
        };
        const int rdp0 = read_base(PR, BP, wp * TP, 0), rdp1 = PR ? rdp0 + BP / 16 * PIECE : read_base(PR, BP, wp * TP, 1);
        const int rdq0 = read_base(QR, BQ, wq * TQ, 0), rdq1 = QR ? rdq0 + BQ / 16 * PIECE : read_base(QR, BQ, wq * TQ, 1);
        auto fragment = [&](const uint8_t* p, bool by_rows, int R, int i) -> s16x8 {
            if (by_rows) {
                const s16x4 lo = read_tr(p + i * 32), hi = read_tr(p + i * 32 + R * 2);   // k + 0..3, k + 4..7
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
            return *reinterpret_cast<const s16x8*>(p + i * 16 * BK * 2);
        };

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
            stage(w, s, kt + 2, b0);
            read_half(b1, 0, 0);
            multiply(1);
            interleave<READS, MFMAS, UP + UQ>();
            read_half(b1, 1, 1);
            multiply(0);
            interleave<READS, MFMAS, 0>();
            wait_vm_loads<0>();
            barrier_lds();
            stage(w, s, kt + 3, b1);    // (past the last step: zeros)
            read_half(b0, 0, 0);
            multiply(1);
            interleave<READS, MFMAS, UP + UQ>();
        };
        if (nk > 0) {
            wait_vm_loads<AFTER ? 0 : UP + UQ>();
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
    }

    static MOE_DEV void run(const Work& w, uint8_t* smem, f32x4 (&acc)[NI][NJ]) {
        begin(w, smem);
        sums<false>(w, smem, acc);
    }
};

}  // namespace
}  // namespace moe
