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
// Tiles come into LDS by buffer loads straight to LDS, 16 bytes per lane, one K step of
// 64 ahead. What lies past an operand's rows or past K lands as zeros: rows by the
// buffer's length, a K tail by an offset past it. Chunks of 16 bytes are stored
// permuted so that the LDS reads of a matrix operand fall on distinct banks.
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

MOE_DEV int swz_k(int row) { return (row & 7) ^ ((row >> 3) & 1); }            // chunk permutation of a rows x 64 k tile
MOE_DEV int swz_r(int k) { return ((k & 3) | (((k >> 3) & 1) << 2)) << 1; }    // of a 64 k x rows tile

MOE_DEV s16x4 read_tr(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// BQ x BP tile of the output, WQ x WP wavefronts
template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(64 * WQ * WP) void ffn_gemm_kernel(FfnArgs a, int nq, int np, int tiles) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int TH = 64 * WQ * WP, TQ = BQ / WQ, TP = BP / WP, NI = TP / 16, NJ = TQ / 16;
    constexpr int P_BYTES = BP * BK * 2, STEP = (BP + BQ) * BK * 2;
    constexpr int UP = BP * 8 / TH, UQ = BQ * 8 / TH;   // 16-byte units per thread
    constexpr bool PR = p_by_rows(KIND), QR = q_by_rows(KIND);
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, wq = wv / WP, wp = wv % WP;

    // which tile: consecutive tiles on one XCD, eight q tiles deep, so that the tiles an XCD
    // works on at a time share their operands in its L2
    int tile = xcd_logical_block(blockIdx.x, tiles);
    int which = 0;   // DW: the product
    if (tile >= tiles) return;
    Operand P, Q;
    int K = a.D, segs = 1, tq_n = nq, tp_n = np;
    if (KIND == GATEUP) P = {a.wg, a.wu, a.D, a.I}, Q = {a.x, a.x, a.ldx, a.m};
    if (KIND == DOWN) P = {a.wd, a.wd, a.I, a.D}, Q = {a.h, a.h, a.I, a.m}, K = a.I;
    if (KIND == DH) P = {a.wd, a.wd, a.I, a.I}, Q = {a.dy, a.dy, a.lddy, a.m};
    if (KIND == DX) P = {a.wg, a.wu, a.D, a.D}, Q = {a.dg, a.du, a.I, a.m}, K = a.I, segs = 2;
    uint16_t* out = nullptr;
    int64_t ldo = 0;
    if (KIND == DOWN) out = a.y, ldo = a.ldy;
    if (KIND == DX) out = a.dx, ldo = a.lddx;
    if (KIND == DW) {
        // products whose output is not wanted have no tiles
        K = a.m;
        const int each = nq * np;   // nq: tiles along I, np: tiles along D
        const int n0 = a.dwg != nullptr ? each : 0, n1 = a.dwu != nullptr ? each : 0;
        if (tile < n0) which = 0;
        else if (tile < n0 + n1) which = 1, tile -= n0;
        else which = 2, tile -= n0 + n1;
        if (which < 2) {
            P = {a.x, a.x, a.ldx, a.D};
            Q = {which == 0 ? a.dg : a.du, nullptr, a.I, a.I};
            out = which == 0 ? a.dwg : a.dwu, ldo = a.D;
        } else {
            P = {a.h, a.h, a.I, a.I};
            Q = {a.dy, a.dy, a.lddy, a.D};
            out = a.dwd, ldo = a.I;
            tq_n = (a.D + BQ - 1) / BQ, tp_n = (a.I + BP - 1) / BP;
        }
    }
    const int deep = 8 * tp_n, gr = tile / deep, gq = min(8, tq_n - gr * 8), in = tile - gr * deep;
    const int q0 = (gr * 8 + in % gq) * BQ, ptile = in / gq;
    constexpr int PSPAN = KIND == GATEUP ? BP / 2 : BP;   // GATEUP: 32 rows of Wg, the same 32 of Wu, and so on
    const int p0 = ptile * PSPAN;

    // this thread's units of the tiles: byte offsets from the tile's corner, and chunk
    // numbers along k (for the K tail)
    uint32_t offp[UP], offq[UQ];
    int ck_p = 0, ck_q = 0;   // K-contiguous tiles: the unit's chunk (the same in every unit of a thread)
    auto offsets = [&](auto& off, const Operand& o, bool by_rows, int R, int& ck, bool paired, int U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = u * TH + tid;
            if (by_rows) {
                const int k = p / (R / 8), c = (p % (R / 8)) ^ swz_r(k);
                off[u] = (uint32_t)(k * o.ld + c * 8) * 2;
            } else {
                const int row = p >> 3, c = (p & 7) ^ swz_k(row);
                const int r = paired ? (row >> 6) * 32 + (row & 31) : row;
                ck = c;
                off[u] = (uint32_t)(r * o.ld + c * 8) * 2;
            }
        }
    };
    offsets(offp, P, PR, BP, ck_p, KIND == GATEUP, UP);
    offsets(offq, Q, QR, BQ, ck_q, false, UQ);

    const int seg_steps = (K + BK - 1) / BK, nk = seg_steps * segs;
    auto stage = [&](int kt, uint8_t* buf) {
        const int seg = segs == 2 && kt >= seg_steps ? 1 : 0;
        const int k0 = (kt - seg * seg_steps) * BK, kleft = min(BK, K - k0);
        const bool tail = kleft < BK;
        auto side = [&](auto& off, const Operand& o, bool by_rows, int at, int span, int ck, bool paired, int U, uint8_t* dst) {
            const uint16_t* base = seg ? o.b : o.a;
            const int left = min(o.rows - at, span);
            if (by_rows) {
                const auto R = buffer_rsrc(base + (size_t)k0 * o.ld + at, (uint32_t)((kleft - 1) * o.ld + left) * 2);
#pragma unroll
                for (int u = 0; u < U; ++u) buffer_load_lds16(R, dst + (u * TH + wv * 64) * 16, off[u]);
            } else {
                const uint32_t bytes = (uint32_t)((left - 1) * o.ld + kleft) * 2;
                const size_t corner = (size_t)at * o.ld + k0;
                const auto R = buffer_rsrc(base + corner, bytes);
                const auto S = paired ? buffer_rsrc(o.b + corner, bytes) : R;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // a K tail's missing chunks are within the buffer for all rows but the last
                    const uint32_t v = tail && ck * 8 >= kleft ? PAST : off[u];
                    const bool second = paired && ((((u * TH + wv * 64) >> 3) >> 5) & 1);
                    if (second) buffer_load_lds16(S, dst + (u * TH + wv * 64) * 16, v);
                    else buffer_load_lds16(R, dst + (u * TH + wv * 64) * 16, v);
                }
            }
        };
        side(offp, P, PR, p0, PSPAN, ck_p, KIND == GATEUP, UP, buf);
        side(offq, Q, QR, q0, BQ, ck_q, false, UQ, buf + P_BYTES);
    };

    // LDS byte offsets of this lane's operand reads, for k 0..31 of a step
    int rdp[NI], rdq[NJ];
    auto reads = [&](auto& rd, bool by_rows, int R, int base, int n) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int r0 = base + 16 * i;
            if (by_rows) {
                const int k = 8 * g + (l16 >> 2);
                rd[i] = k * R * 2 + (((r0 / 8 + ((l16 >> 1) & 1)) ^ swz_r(k)) << 4) + (l16 & 1) * 8;
            } else {
                rd[i] = (r0 + l16) * (BK * 2) + ((g ^ swz_k(l16)) << 4);
            }
        }
    };
    reads(rdp, PR, BP, wp * TP, NI);
    reads(rdq, QR, BQ, wq * TQ, NJ);
    auto fragment = [&](const uint8_t* tile_lds, int rd, bool by_rows, int R, int kk) -> s16x8 {
        if (by_rows) {
            const uint8_t* p = tile_lds + rd + kk * 32 * R * 2;
            const s16x4 lo = read_tr(p), hi = read_tr(p + 4 * R * 2);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return *reinterpret_cast<const s16x8*>(tile_lds + (rd ^ (kk << 6)));   // chunk g + 4 kk, permuted
    };

    f32x4 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    if (nk > 0) stage(0, smem);
    for (int kt = 0; kt < nk; ++kt) {
        wait_vm_loads<0>();
        barrier_lds();   // step kt is in LDS for every wavefront; the other buffer is free
        const uint8_t* buf = smem + (kt & 1) * STEP;
        if (kt + 1 < nk) stage(kt + 1, smem + ((kt + 1) & 1) * STEP);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            s16x8 fp[NI], fq[NJ];
#pragma unroll
            for (int i = 0; i < NI; ++i) fp[i] = fragment(buf, rdp[i], PR, BP, kk);
#pragma unroll
            for (int j = 0; j < NJ; ++j) fq[j] = fragment(buf + P_BYTES, rdq[j], QR, BQ, kk);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < NI; ++i) acc[i][j] = T::mfma(fp[i], fq[j], acc[i][j]);
        }
    }

    // a lane holds p = 16 i + 4 g + 0..3 of q = 16 j + l16 (of its wavefront's part)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int q = q0 + wq * TQ + 16 * j + l16, q16 = (q0 + wq * TQ) / 16 + j;
        if constexpr (KIND == GATEUP) {
            if (16 * q16 >= a.m) continue;
#pragma unroll
            for (int b = 0; b < NI / 4; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f32x4 gv = acc[4 * b + i][j], uv = acc[4 * b + 2 + i][j];
                    const int at = p0 + (wp * TP + 64 * b) / 2 + 16 * i, p = at + 4 * g;
                    if (at >= a.I) continue;
                    if (a.saved != nullptr) {
                        float* s = a.saved + saved_at(q16, at / 16, a.I) + lane * 4;
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
            if (16 * q16 >= a.m) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int at = p0 + wp * TP + 16 * i, p = at + 4 * g;
                if (at >= a.I) continue;
                const float* s = a.saved + saved_at(q16, at / 16, a.I) + lane * 4;
                const f32x4 gv = *reinterpret_cast<const f32x4*>(s), uv = *reinterpret_cast<const f32x4*>(s + 256);
                float dg[4], du[4], h[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float uc = clamp_up(uv[r], a.limit);
                    float v, dv;
                    act_both(clamp_gate(gv[r], a.limit), a.act, v, dv);
                    const float dh = acc[i][j][r];
                    const bool clamped = a.limit > 0.f;
                    dg[r] = clamped && gv[r] > a.limit ? 0.f : dh * uc * dv;
                    du[r] = clamped && fabsf(uv[r]) > a.limit ? 0.f : dh * v;
                    h[r] = v * uc;
                }
                if (q < a.m && p < a.I) {
                    const size_t o = (size_t)q * a.I + p;
                    *reinterpret_cast<uint2*>(a.dg + o) = make_uint2(T::pack2(dg[0], dg[1]), T::pack2(dg[2], dg[3]));
                    *reinterpret_cast<uint2*>(a.du + o) = make_uint2(T::pack2(du[0], du[1]), T::pack2(du[2], du[3]));
                    *reinterpret_cast<uint2*>(a.h + o) = make_uint2(T::pack2(h[0], h[1]), T::pack2(h[2], h[3]));
                }
            }
        } else {
            if (q >= Q.rows) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int p = p0 + wp * TP + 16 * i + 4 * g;
                const f32x4 v = acc[i][j];
                if (p < P.rows)
                    *reinterpret_cast<uint2*>(out + (size_t)q * ldo + p) = make_uint2(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]));
            }
        }
    }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <typename T, Kind KIND, int BQ, int BP, int WQ, int WP>
hipError_t launch_tiles(const FfnArgs& a, hipStream_t st) {
    int nq = cdiv(a.m, BQ), np = cdiv(KIND == GATEUP ? 2 * a.I : KIND == DH ? a.I : a.D, BP), tiles = nq * np;
    if (KIND == DW) {
        nq = cdiv(a.I, BQ), np = cdiv(a.D, BP);
        tiles = nq * np * ((a.dwg != nullptr) + (a.dwu != nullptr));
        if (a.dwd != nullptr) tiles += cdiv(a.D, BQ) * cdiv(a.I, BP);
    }
    if (tiles == 0) return hipSuccess;
    return launch_kernel(ffn_gemm_kernel<T, KIND, BQ, BP, WQ, WP>, dim3((tiles + 7) / 8 * 8), dim3(64 * WQ * WP),
                         2 * (BQ + BP) * BK * 2, st, a, nq, np, tiles);
}

template <typename T, Kind KIND>
hipError_t launch_product(const FfnArgs& a, hipStream_t st) {
    const int out_q = KIND == DW ? a.I : a.m, out_p = KIND == GATEUP ? 2 * a.I : KIND == DH ? a.I : a.D;
    if (cdiv(out_q, 256) * cdiv(out_p, 256) * (KIND == DW ? 3 : 1) >= 128) return launch_tiles<T, KIND, 256, 256, 2, 4>(a, st);
    return launch_tiles<T, KIND, 128, 128, 2, 2>(a, st);
}

constexpr int MAX_M = 1 << 24;

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
size_t forward_bytes(const moe_ffn* f, int m) { return rows_bytes(f, m); }
size_t backward_bytes(const moe_ffn* f, int m) { return 3 * rows_bytes(f, m); }
size_t saved_bytes_of(const moe_ffn* f, int m) { return (size_t)cdiv(m, 16) * cdiv(f->inter, 16) * 2048; }

FfnArgs describe(const moe_ffn* f, int m) {
    FfnArgs a{};
    a.wg = reinterpret_cast<const uint16_t*>(f->w_gate);
    a.wu = reinterpret_cast<const uint16_t*>(f->w_up);
    a.wd = reinterpret_cast<const uint16_t*>(f->w_down);
    a.m = m, a.D = f->dim, a.I = f->inter, a.act = f->act, a.limit = f->limit;
    return a;
}

template <typename T>
hipError_t forward(const FfnArgs& a, hipStream_t st) {
    const hipError_t e = launch_product<T, GATEUP>(a, st);
    return e != hipSuccess ? e : launch_product<T, DOWN>(a, st);
}

template <typename T>
hipError_t backward(const FfnArgs& a, hipStream_t st) {
    hipError_t e = a.m > 0 ? launch_product<T, DH>(a, st) : hipSuccess;
    if (e == hipSuccess && a.m > 0 && a.dx != nullptr) e = launch_product<T, DX>(a, st);
    if (e == hipSuccess) e = launch_product<T, DW>(a, st);
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
    const hipStream_t st = (hipStream_t)stream;
    return status_of(f->dtype == MOE_BF16 ? forward<Bf16>(a, st) : forward<F16>(a, st));
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
    const hipStream_t st = (hipStream_t)stream;
    return status_of(f->dtype == MOE_BF16 ? backward<Bf16>(a, st) : backward<F16>(a, st));
}

}  // extern "C"
