// Products with 4-bit weights that have a 16-bit scale, and perhaps a zero point,
// per group of 32, 64 or 128 columns (moe_w4_* in include/moe.h), for few rows of x.
//
//   y[t, n] = sum_k s[n, k/G] (q[n, k] - z[n, k/G]) x[t, k]
//           = sum_groups s ( sum_k (c + q) x - (c + z) sum_k x )
//
// The codes go to the matrix cores as the 16-bit floats c + q, which are exact and
// cost no subtraction: the code's four bits are set into the mantissa of c (128 for
// bf16, 64 for f16). The sum of x over a group comes from one more matrix product
// with ones, in the layout in which it is needed. Scale and zero point are applied
// in f32 to each group's sum, so that w is never rounded.
//
// A workgroup owns 16 rows of W (of both matrices, when gated) and up to 64 rows of
// x; its wavefronts split the columns, and their sums are joined through LDS in
// wavefront order. A wavefront takes 128 columns at a time: lane (r = lane % 16,
// g = lane / 16) loads the 16 bytes of row r, columns 32 g .. 32 g + 31, and four
// lane-group swaps turn these so that its word j holds columns 32 j + 8 g .. + 7:
// each matrix instruction then covers 32 consecutive columns, one group or part of
// one. x is the instruction's first operand, W the second, so that a lane's results
// all belong to row r, whose scales it holds. Row t of x sits at operand row
// 4 (t % 4) + t / 4: up to four tokens then leave one result per lane, up to eight
// two.
#include "block_common.h"

namespace moe {
namespace {

constexpr int STAGE = 128;       // columns a wavefront takes at a time
constexpr int BATCH = 4;         // stages requested together, one batch ahead
constexpr int MAX_WAVES = 8;
constexpr int MAX_ROWS_X = 64;   // rows of x per workgroup

struct W4Mat {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
};
struct W4Args {
    W4Mat w[2];
    const uint16_t* x;
    uint16_t* y;
    int64_t ldx, ldy;
    int N, K, m, act;
    float limit;
};

// word of eight codes -> the eight values c + q as 16-bit floats, in column order
MOE_DEV s16x8 codes_to_values(uint32_t w, Bf16) {
    // halves (nibbles 0..3 | nibbles 1..4) and (4..7 | 5..8) of the word
    const uint32_t v = w >> 4;
    const uint32_t p = __builtin_amdgcn_perm(v, w, 0x05040100u), q = __builtin_amdgcn_perm(v, w, 0x07060302u);
    u32x4 o;
    o[0] = (p & 0x000F000Fu) | 0x43004300u;
    o[1] = ((p >> 8) & 0x000F000Fu) | 0x43004300u;
    o[2] = (q & 0x000F000Fu) | 0x43004300u;
    o[3] = ((q >> 8) & 0x000F000Fu) | 0x43004300u;
    return __builtin_bit_cast(s16x8, o);
}
MOE_DEV s16x8 codes_to_values(uint32_t w, F16) {
    // as above, each code in bits 4..7: 64 + q
    const uint32_t v = w << 4;
    const uint32_t p = __builtin_amdgcn_perm(w, v, 0x05040100u), q = __builtin_amdgcn_perm(w, v, 0x07060302u);
    u32x4 o;
    o[0] = (p & 0x00F000F0u) | 0x54005400u;
    o[1] = ((p >> 8) & 0x00F000F0u) | 0x54005400u;
    o[2] = (q & 0x00F000F0u) | 0x54005400u;
    o[3] = ((q >> 8) & 0x00F000F0u) | 0x54005400u;
    return __builtin_bit_cast(s16x8, o);
}
template <typename T>
constexpr float code_offset();
template <>
constexpr float code_offset<Bf16>() { return 128.f; }
template <>
constexpr float code_offset<F16>() { return 64.f; }

// word j of lane group g <-> word g of lane group j
MOE_DEV void turn_words(uint32_t* w) {
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false));
    const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
    const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
    w[0] = c[0], w[1] = c[1], w[2] = d[0], w[3] = d[1];
}

// One wavefront's 128 columns of one matrix: 16 code bytes, and the scales and zero
// points of row r's groups there.
template <int G>
struct W4Stage {
    static constexpr int NG = STAGE / G;
    uint32_t c[4];
    uint16_t s[NG];
    uint8_t z[NG];
};

// NT: tiles of 16 rows of x. IR: results per lane and tile (tokens g + 4 i, i < IR). NM: matrices (2: gated)
template <typename T, int G, int NT, int IR, int NM>
__global__ __launch_bounds__(64 * MAX_WAVES) void w4_kernel(W4Args a) {
    extern __shared__ float red[];   // [wavefront][matrix][token][16 rows]
    constexpr int NG = STAGE / G, TOK = 16 * NT;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, rows = min(16, a.N - n0);
    const int t0 = blockIdx.y * MAX_ROWS_X, mt = min(MAX_ROWS_X, a.m - t0);
    const int row = n0 + min(r, rows - 1);
    const int kg = a.K / G;
    const int stages = (a.K + STAGE - 1) / STAGE;
    const int s0 = (int)((int64_t)wv * stages / nw), s1 = (int)((int64_t)(wv + 1) * stages / nw);
    const uint32_t row_bytes = (uint32_t)a.K / 2;
    __amdgpu_buffer_rsrc_t codes[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q) codes[q] = buffer_rsrc(a.w[q].codes + (size_t)n0 * row_bytes, rows * row_bytes);
    const auto X = buffer_rsrc(a.x + (size_t)t0 * a.ldx, (uint32_t)((mt - 1) * a.ldx + a.K) * 2);
    constexpr uint32_t PAST = 0xFFFFFFF0u;   // an offset past every buffer: zeros
    uint32_t xoff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int tok = 16 * t + (r >> 2) + 4 * (r & 3);
        xoff[t] = tok < mt ? (uint32_t)(tok * a.ldx * 2) : PAST;
    }

    auto load = [&](W4Stage<G>(&st)[BATCH][NM], int s) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const bool in = s + b < s1;
            const uint32_t k = (s + b) * STAGE;
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                const uint32_t off = in && k + 32 * g < (uint32_t)a.K && r < rows ? r * row_bytes + k / 2 + 16 * g : PAST;
                const uint4 v = buffer_load16(codes[q], off);
                st[b][q].c[0] = v.x, st[b][q].c[1] = v.y, st[b][q].c[2] = v.z, st[b][q].c[3] = v.w;
                const size_t at = (size_t)row * kg + (s + b) * NG;
                if (in && (int)k + STAGE <= a.K) {
                    __builtin_memcpy(st[b][q].s, a.w[q].scales + at, sizeof(st[b][q].s));
                    if (a.w[q].zeros != nullptr) __builtin_memcpy(st[b][q].z, a.w[q].zeros + at, sizeof(st[b][q].z));
                } else if (in) {
                    for (int i = 0; i < NG; ++i) {
                        const bool have = (s + b) * NG + i < kg;
                        st[b][q].s[i] = have ? a.w[q].scales[at + i] : 0;
                        if (a.w[q].zeros != nullptr) st[b][q].z[i] = have ? a.w[q].zeros[at + i] : 0;
                    }
                }
            }
        }
    };

    float sum[NM][NT][IR];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < IR; ++i) sum[q][t][i] = 0.f;
    const s16x8 ones = __builtin_bit_cast(s16x8, (u32x4){T::ONES, T::ONES, T::ONES, T::ONES});

    auto work = [&](W4Stage<G>(&st)[BATCH][NM], int s) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (s + b >= s1) break;
            const uint32_t k = (s + b) * STAGE + 8 * g;
#pragma unroll
            for (int q = 0; q < NM; ++q) turn_words(st[b][q].c);
            f32x4 acc[NM][NT], sx[NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s16x8 xv[NT], wv8[NM];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t off = xoff[t] != PAST && k + 32 * j < (uint32_t)a.K ? xoff[t] + 2 * (k + 32 * j) : PAST;
                    const uint4 v = buffer_load16(X, off);
                    xv[t] = __builtin_bit_cast(s16x8, v);
                }
#pragma unroll
                for (int q = 0; q < NM; ++q) wv8[q] = codes_to_values(st[b][q].c[j], T());
                const bool first = (32 * j) % G == 0, last = (32 * (j + 1)) % G == 0;
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    sx[t] = T::mfma(xv[t], ones, first ? zero : sx[t]);
#pragma unroll
                    for (int q = 0; q < NM; ++q) acc[q][t] = T::mfma(xv[t], wv8[q], first ? zero : acc[q][t]);
                }
                if (last) {
                    const int i0 = 32 * j / G;
#pragma unroll
                    for (int q = 0; q < NM; ++q) {
                        const float sc = T::load(st[b][q].s[i0]);
                        const float zp = code_offset<T>() + (a.w[q].zeros != nullptr ? (float)st[b][q].z[i0] : 8.f);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < IR; ++i)
                                sum[q][t][i] = fmaf(sc, fmaf(-zp, sx[t][i], acc[q][t][i]), sum[q][t][i]);
                    }
                }
            }
        }
    };

    W4Stage<G> cur[BATCH][NM], nxt[BATCH][NM];
    load(cur, s0);
    for (int s = s0; s < s1; s += BATCH) {
        if (s + BATCH < s1) load(nxt, s + BATCH);
        work(cur, s);
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int q = 0; q < NM; ++q) cur[b][q] = nxt[b][q];
    }

#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < IR; ++i)
                red[((wv * NM + q) * TOK + 16 * t + g + 4 * i) * 16 + r] = sum[q][t][i];
    __syncthreads();
    for (int e = threadIdx.x; e < mt * 16; e += blockDim.x) {
        const int tok = e >> 4, rr = e & 15;
        if (rr >= rows) continue;
        float v[NM];
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            v[q] = 0.f;
            for (int w = 0; w < nw; ++w) v[q] += red[((w * NM + q) * TOK + tok) * 16 + rr];
        }
        float o = v[0];
        if (NM == 2) o = act_value(clamp_gate(v[0], a.limit), a.act) * clamp_up(v[NM - 1], a.limit);
        a.y[(size_t)(t0 + tok) * a.ldy + n0 + rr] = T::store(o);
    }
}

int check_w4(const moe_w4* w) {
    if (w == nullptr || w->codes == nullptr || w->scales == nullptr) return MOE_EINVAL;
    if (w->rows < 1 || w->rows > (1 << 22) || w->cols < 32 || w->cols > 65536) return MOE_EINVAL;
    if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_EINVAL;
    if (w->cols % w->group || (w->dtype != MOE_BF16 && w->dtype != MOE_F16)) return MOE_EINVAL;
    if (!aligned_to(w->codes, 16) || !aligned_to(w->scales, 2)) return MOE_EINVAL;
    return MOE_OK;
}

template <typename T, int G, int NM>
hipError_t launch_w4(const W4Args& a, hipStream_t st) {
    const int stages = (a.K + STAGE - 1) / STAGE, nw = std::min(MAX_WAVES, stages);
    const int mt = std::min(a.m, MAX_ROWS_X);
    const dim3 grid((a.N + 15) / 16, (a.m + MAX_ROWS_X - 1) / MAX_ROWS_X);
    const int nt = mt <= 16 ? 1 : mt <= 32 ? 2 : 4;
    const size_t lds = sizeof(float) * nw * NM * nt * 256;
    void (*k)(W4Args) = mt <= 4    ? w4_kernel<T, G, 1, 1, NM>
                        : mt <= 8  ? w4_kernel<T, G, 1, 2, NM>
                        : mt <= 16 ? w4_kernel<T, G, 1, 4, NM>
                        : mt <= 32 ? w4_kernel<T, G, 2, 4, NM>
                                   : w4_kernel<T, G, 4, 4, NM>;
    return launch_kernel(k, grid, dim3(64 * nw), lds, st, a);
}

template <int NM>
int run_w4(const moe_w4* const* w, int act, float limit, const void* x, int64_t ldx, int32_t m, void* y, int64_t ldy,
           void* stream) {
    for (int q = 0; q < NM; ++q)
        if (const int rc = check_w4(w[q])) return rc;
    if (NM == 2) {
        if (w[0]->rows != w[1]->rows || w[0]->cols != w[1]->cols || w[0]->group != w[1]->group || w[0]->dtype != w[1]->dtype)
            return MOE_EINVAL;
        if ((act != MOE_ACT_SILU && act != MOE_ACT_GELU) || limit != limit) return MOE_EINVAL;
    }
    if (m < 0 || m > MAX_ROWS_X * 65535) return MOE_EINVAL;
    if (m == 0) return MOE_OK;
    if (x == nullptr || y == nullptr || !aligned_to(x, 16) || !aligned_to(y, 2)) return MOE_EINVAL;
    if (ldx < w[0]->cols || ldx % 8 || ldx > (1 << 24) || ldy < w[0]->rows) return MOE_EINVAL;
    W4Args a{};
    for (int q = 0; q < NM; ++q)
        a.w[q] = {reinterpret_cast<const uint8_t*>(w[q]->codes), reinterpret_cast<const uint16_t*>(w[q]->scales),
                  reinterpret_cast<const uint8_t*>(w[q]->zeros)};
    a.x = reinterpret_cast<const uint16_t*>(x);
    a.y = reinterpret_cast<uint16_t*>(y);
    a.ldx = ldx, a.ldy = ldy, a.N = w[0]->rows, a.K = w[0]->cols, a.m = m, a.act = act, a.limit = limit;
    const hipStream_t st = (hipStream_t)stream;
    const int g = w[0]->group;
    if (w[0]->dtype == MOE_BF16)
        return status_of(g == 32 ? launch_w4<Bf16, 32, NM>(a, st) : g == 64 ? launch_w4<Bf16, 64, NM>(a, st) : launch_w4<Bf16, 128, NM>(a, st));
    return status_of(g == 32 ? launch_w4<F16, 32, NM>(a, st) : g == 64 ? launch_w4<F16, 64, NM>(a, st) : launch_w4<F16, 128, NM>(a, st));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_w4_matmul(const moe_w4* w, const void* x, int64_t ldx, int32_t m, void* y, int64_t ldy, void* stream) {
    return run_w4<1>(&w, MOE_ACT_SILU, 0.f, x, ldx, m, y, ldy, stream);
}

int moe_w4_gated(const moe_w4* w_gate, const moe_w4* w_up, int32_t act, float limit, const void* x, int64_t ldx,
                 int32_t m, void* h, int64_t ldh, void* stream) {
    const moe_w4* w[2] = {w_gate, w_up};
    return run_w4<2>(w, act, limit, x, ldx, m, h, ldh, stream);
}

}  // extern "C"
