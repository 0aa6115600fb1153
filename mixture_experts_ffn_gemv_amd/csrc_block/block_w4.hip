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
// in f32 to each group's sum, so that w is never rounded. What c adds is taken off again in f32:
// the sums of a group round at the size of (c + 15) sum |x| rather than 15 sum |x|, three bits (bf16) or
// two (f16) of the 24. Outputs differ by 1e-4 of their norm from sums of the exact w (bf16, 5120 x
// 2304), where their own rounding is 1.6e-3; taking c off the codes first would cost an instruction for
// every one or two of them.
//
// Bound, for few rows, by the codes' bytes. 65536 x 2048, one row of x: 24.0 us, 3.1 TB/s of
// codes, scales and zero points; 8192 x 8192 11.9 us, 3.1 TB/s (a stream of reads from HBM reaches about
// 6: every code passes through LDS, with a barrier for each 8 KB); 5120 x
// 5120 7.6 us, of which a launch, the first loads and the sums' join are about 4. From 16 rows
// on x, which every workgroup brings into its LDS, costs more than the codes.
//
// A workgroup owns WR RT tiles of 16 rows of W (gated: eight rows of Wg and the same eight of
// Wu in a tile) and up to 32 rows of x. Eight wavefronts work: WR of them, with RT tiles
// each, on each of WK parts of the columns; their sums are joined through LDS in order of
// the parts. A wavefront takes stages of 128 columns: lane (r = lane % 16, g = lane / 16) loads the 16 bytes of row r,
// columns 32 g .. 32 g + 31, and four lane-group swaps turn these so that its word j holds
// columns 32 j + 8 g .. + 7: each matrix instruction then covers 32 consecutive columns,
// one group or part of one. x is the instruction's first operand, W the second, so that a
// lane's results all belong to row r, whose scales it needs. Row t of x sits at operand row
// 4 (t % 4) + t / 4: up to four tokens then leave one result per lane, up to eight two.
//
// Two more wavefronts bring x and the codes into LDS, stage by stage of every part, RING - 2
// steps ahead. A load's four neighbouring lanes read 64 bytes of one row there: where each
// reads another row, as the matrix instructions want it, a load takes four times as long on
// a CU's load path, and x straight from the L2s cost four times what the codes did. They are
// wavefronts of their own because loads complete in the order of a wavefront's requests.
// Scales and zero points come eight stages at a time, in pieces of eight groups, and wait in
// LDS: loaded stage by stage they were half the time of a wide matrix.
#include "block_common.h"

namespace moe {
namespace {

constexpr int STAGE = 128;       // columns a wavefront takes at a time
constexpr int MAX_ROWS_X = 32;   // rows of x per workgroup
constexpr int WORKERS = 8, LOADERS = 2;

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

// (a & mask) | c in one instruction: the mask has to be in a vector register
MOE_DEV uint32_t and_or(uint32_t a, uint32_t mask, uint32_t c) {
    asm("" : "+v"(mask));
    return (a & mask) | c;
}
// word of eight codes -> the eight values c + q as 16-bit floats, in column order
MOE_DEV s16x8 codes_to_values(uint32_t w, Bf16) {
    // halves (nibbles 0..3 | nibbles 1..4) and (4..7 | 5..8) of the word
    const uint32_t v = w >> 4;
    const uint32_t p = __builtin_amdgcn_perm(v, w, 0x05040100u), q = __builtin_amdgcn_perm(v, w, 0x07060302u);
    const u32x4 o = {and_or(p, 0x000F000Fu, 0x43004300u), and_or(p >> 8, 0x000F000Fu, 0x43004300u),
                     and_or(q, 0x000F000Fu, 0x43004300u), and_or(q >> 8, 0x000F000Fu, 0x43004300u)};
    return __builtin_bit_cast(s16x8, o);
}
MOE_DEV s16x8 codes_to_values(uint32_t w, F16) {
    // as above, each code in bits 4..7: 64 + q
    const uint32_t v = w << 4;
    const uint32_t p = __builtin_amdgcn_perm(w, v, 0x05040100u), q = __builtin_amdgcn_perm(w, v, 0x07060302u);
    const u32x4 o = {and_or(p, 0x00F000F0u, 0x54005400u), and_or(p >> 8, 0x00F000F0u, 0x54005400u),
                     and_or(q, 0x00F000F0u, 0x54005400u), and_or(q >> 8, 0x00F000F0u, 0x54005400u)};
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

// Chunks of 16 bytes in LDS lie at c ^ swz(row), rows of 256 bytes, or c ^ swz(row / 4), rows of 64. A
// read of 16 bytes per lane takes sixteen lanes at a time: 0..3 and 12..15 of one group of sixteen
// and 4..11 of the next, which want chunk c of their rows and chunk c + 1 of theirs. So
// two bits of the row number go 0, 3, 1, 2 -> 0, 1, 2, 3, which keeps the two apart.
MOE_DEV int swz(int row) { return (row & 12) | (((row ^ (row >> 1)) & 1) << 1) | ((row >> 1) & 1); }

// One wavefront's scales and zero points of a tile for SLAB stages: row r's at r * NG * SLAB
constexpr int SLAB = 8;
template <int NG>
struct SlabTile {
    uint16_t s[16 * NG * SLAB];
    uint8_t z[16 * NG * SLAB];
};

// results of a lane for tile t of x that are any token's
constexpr int results_of(int rows, int t) { return rows - 16 * t <= 4 ? 1 : rows - 16 * t <= 8 ? 2 : 4; }

// ROWS: rows of x there is room for. WK, WR: parts of the columns, workers on each. RT: tiles of a
// worker. RING: steps in LDS
template <typename T, int G, int ROWS, int WK, int WR, int RT, int RING, bool GATED>
__global__ __launch_bounds__(64 * (WORKERS + LOADERS)) void w4_kernel(W4Args a) {
    static_assert(WK * WR == WORKERS, "");
    constexpr int NG = STAGE / G, NT = (ROWS + 15) / 16, TOK = 16 * NT, COLS = GATED ? 8 : 16;   // COLS: results per token and tile
    constexpr int IR = results_of(ROWS, 0);   // results per lane and tile of x: tokens g + 4 i, i < IR
    constexpr int X_ROW = STAGE * 2, X_STEP = WK * ROWS * X_ROW, STEP = X_STEP + WORKERS * RT * 1024;
    // RING steps of x [part][row][128] and codes [worker][tile][16 rows][64 bytes]; slabs [worker][tile];
    // then the sums [part][tile][token][16 rows]
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n0 = blockIdx.x * COLS * WR * RT;
    const int t0 = blockIdx.y * MAX_ROWS_X, mt = min(MAX_ROWS_X, a.m - t0);
    const int stages = (a.K + STAGE - 1) / STAGE, steps = (stages + WK - 1) / WK;
    auto part = [&](int wk) { return (int)((int64_t)wk * stages / WK); };   // a part's first stage: steps or steps - 1 each
    float sum[RT][NT][IR];
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < IR; ++i) sum[q][t][i] = 0.f;
    const int r = lane & 15, g = lane >> 4, wk = wv % WK, wr = wv / WK;

    const uint32_t row_bytes = (uint32_t)a.K / 2;
    // the place in the workgroup of a worker's tile, counted over the workers (part wv % WK, rows wv / WK)
    auto tile_of = [&](int w) { return w / (RT * WK) * RT + w % RT; };
    // row r of tile t: its matrix, and its number there (past the matrix: the last row)
    auto matrix = [&](int r) { return GATED && r >= 8 ? 1 : 0; };
    auto row_of = [&](int t, int r) { return min(n0 + COLS * t + (GATED ? r & 7 : r), a.N - 1); };

    if (wv >= WORKERS) {
        constexpr int LOADS = WK * ROWS / 4 / LOADERS, CODES = WORKERS * RT / LOADERS;   // of one loader and step: four rows of 256 bytes, a tile's codes
        static_assert((RING - 2) * (LOADS + CODES) < 64 && LOADS > 0, "");
        const int id = wv - WORKERS, crow = lane >> 2;
        const auto X = buffer_rsrc(a.x + (size_t)t0 * a.ldx, (uint32_t)((mt - 1) * a.ldx + a.K) * 2);
        const uint32_t piece = ((lane & 3) ^ swz(crow >> 2)) * 16;
        const uint8_t* codes[CODES];
#pragma unroll
        for (int i = 0; i < CODES; ++i)
            codes[i] = a.w[matrix(crow)].codes + (size_t)row_of(tile_of(id * CODES + i), crow) * row_bytes;
        auto stage = [&](int b) {
            uint8_t* const to = smem + b % RING * STEP;
#pragma unroll
            for (int i = 0; i < CODES; ++i) {
                // (codes past K, or past the part, are others of the row: x is zero there)
                const int w = id * CODES + i, s = min(part(w / RT % WK) + b, stages - 1);
                load_lds16(codes[i] + min(s * (STAGE / 2) + piece, row_bytes - 16), to + X_STEP + w * 1024);
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {   // (past the part, past m or K: zeros)
                const int run = id * LOADS + i, p = run / (ROWS / 4), tok = run % (ROWS / 4) * 4 + (lane >> 4);
                const int s = part(p) + b, k = s * STAGE + ((lane & 15) ^ swz(tok)) * 8;
                const bool in = tok < mt && k < a.K && s < part(p + 1);
                buffer_load_lds16(X, to + run * 1024, in ? (uint32_t)(tok * a.ldx + k) * 2 : 0xFFFFFFF0u);
            }
        };
#pragma unroll
        for (int b = 0; b < RING - 1; ++b) stage(b);
        for (int b = 0; b < steps; ++b) {
            wait_vm_loads<(RING - 2) * (LOADS + CODES)>();   // step b has landed
            barrier_lds();                                   // every worker is done with step b - 1
            stage(b + RING - 1);
        }
        wait_vm_loads<0>();
    } else {
        const int kg = a.K / G, s0 = part(wk), s1 = part(wk + 1);
        const bool zeros = a.w[0].zeros != nullptr;   // (of both matrices or of neither)
        SlabTile<NG>* const slab = reinterpret_cast<SlabTile<NG>*>(smem + RING * STEP) + wv * RT;

        // Stages s .. s + SLAB - 1: piece lane % NG of row lane / NG, eight groups each. A piece that
        // would pass the row's end is read from its last eight groups and moved down.
        auto load_slab = [&](int s) {
            const int row = lane / NG, piece = lane % NG, first = s * NG + 8 * piece;
            if (lane >= 16 * NG) return;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const W4Mat& w = a.w[matrix(row)];
                const size_t at = (size_t)row_of(wr * RT + t, row) * kg;
                unsigned __int128 sc = 0;
                uint64_t zp = 0;
                if (first < kg) {
                    if (kg >= 8) {
                        const int from = min(first, kg - 8), down = first - from;
                        __builtin_memcpy(&sc, w.scales + at + from, 16);
                        sc >>= 16 * down;
                        if (zeros) __builtin_memcpy(&zp, w.zeros + at + from, 8);
                        else zp = 0x0808080808080808u;
                        zp >>= 8 * down;
                    } else {
                        for (int i = first; i < kg; ++i) {
                            sc |= (unsigned __int128)w.scales[at + i] << (16 * (i - first));
                            zp |= (uint64_t)(zeros ? w.zeros[at + i] : 8) << (8 * (i - first));
                        }
                    }
                }
                *reinterpret_cast<unsigned __int128*>(slab[t].s + (row * NG + piece) * 8) = sc;
                *reinterpret_cast<uint64_t*>(slab[t].z + (row * NG + piece) * 8) = zp;
            }
        };
        int xrow[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xrow[t] = min(16 * t + (r >> 2) + 4 * (r & 3), ROWS - 1);
        const s16x8 ones = __builtin_bit_cast(s16x8, (u32x4){T::ONES, T::ONES, T::ONES, T::ONES});

        const int code_at = X_STEP + wv * RT * 1024 + r * 64 + ((g ^ swz(r >> 2)) << 4);
        auto work = [&](int step, int in) {   // in: the stage's place in the slab
            // everything is requested from LDS before the codes are taken apart
            const uint8_t* const at = smem + step % RING * STEP;
            const uint8_t* const x = at + wk * ROWS * X_ROW;
            uint4 q[RT];
            s16x8 xv[4][NT];
            uint16_t sc[RT][NG];
            uint8_t zp[RT][NG];
#pragma unroll
            for (int w = 0; w < RT; ++w) q[w] = *reinterpret_cast<const uint4*>(at + code_at + w * 1024);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    xv[j][t] = *reinterpret_cast<const s16x8*>(x + xrow[t] * X_ROW + (((4 * j + g) ^ swz(xrow[t])) << 4));
#pragma unroll
            for (int w = 0; w < RT; ++w) {
                __builtin_memcpy(sc[w], __builtin_assume_aligned(slab[w].s + (r * SLAB + in) * NG, 2 * NG), 2 * NG);
                __builtin_memcpy(zp[w], __builtin_assume_aligned(slab[w].z + (r * SLAB + in) * NG, NG), NG);
            }
            f32x4 acc[RT][NT], sx[NT];
            uint32_t c[RT][4];
#pragma unroll
            for (int w = 0; w < RT; ++w) {
                c[w][0] = q[w].x, c[w][1] = q[w].y, c[w][2] = q[w].z, c[w][3] = q[w].w;
                turn_words(c[w]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool first = (32 * j) % G == 0, last = (32 * (j + 1)) % G == 0;
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < NT; ++t) sx[t] = T::mfma(xv[j][t], ones, first ? zero : sx[t]);
#pragma unroll
                for (int w = 0; w < RT; ++w) {
                    const s16x8 v = codes_to_values(c[w][j], T());
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[w][t] = T::mfma(xv[j][t], v, first ? zero : acc[w][t]);
                }
                if (last) {
#pragma unroll
                    for (int w = 0; w < RT; ++w) {
                        const float s1 = T::load(sc[w][32 * j / G]), z1 = code_offset<T>() + (float)zp[w][32 * j / G];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < results_of(ROWS, t); ++i) sum[w][t][i] = fmaf(s1, fmaf(-z1, sx[t][i], acc[w][t][i]), sum[w][t][i]);
                    }
                }
            }
        };
        if (s0 < s1) load_slab(s0);
        int in = 0;
#pragma unroll 1
        for (int step = 0; step < steps; ++step) {
            barrier_lds();   // the step's codes and x have landed
            if (s0 + step >= s1) continue;
            work(step, in);
            if (++in == SLAB && s0 + step + 1 < s1) load_slab(s0 + step + 1), in = 0;
        }
    }

    __syncthreads();   // the sums take the place of x
    float* const red = reinterpret_cast<float*>(smem);
    if (wv < WORKERS) {
#pragma unroll
        for (int q = 0; q < RT; ++q)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < results_of(ROWS, t); ++i)
                    red[(((wk * WR + wr) * RT + q) * TOK + 16 * t + g + 4 * i) * 16 + r] = sum[q][t][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < mt * COLS * WR * RT; e += blockDim.x) {
        const int c = e % COLS, tile = e / COLS % (WR * RT), tok = e / (COLS * WR * RT), n = n0 + COLS * tile + c;
        if (n >= a.N) continue;
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float* p = red + ((w * WR * RT + tile) * TOK + tok) * 16 + c;
            v[0] += p[0];
            if (GATED) v[1] += p[8];
        }
        const float o = GATED ? act_value(clamp_gate(v[0], a.limit), a.act) * clamp_up(v[1], a.limit) : v[0];
        a.y[(size_t)(t0 + tok) * a.ldy + n] = T::store(o);
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

template <typename T, int G, int ROWS, int WK, int WR, int RT, int RING, bool GATED>
hipError_t launch_tiles(const W4Args& a, hipStream_t st) {
    const int cols = (GATED ? 8 : 16) * WR * RT;
    const dim3 grid((a.N + cols - 1) / cols, (a.m + MAX_ROWS_X - 1) / MAX_ROWS_X);
    const size_t lds = std::max<size_t>(RING * (WK * ROWS * STAGE * 2 + WORKERS * RT * 1024) + WORKERS * RT * sizeof(SlabTile<STAGE / G>),
                                        sizeof(float) * WORKERS * RT * ((ROWS + 15) / 16) * 256);
    return launch_kernel(w4_kernel<T, G, ROWS, WK, WR, RT, RING, GATED>, grid, dim3(64 * (WORKERS + LOADERS)), lds, st, a);
}

// LDS room for 4, 8, 16, 24 or 32 rows of x, since a step's x is loaded whether its rows exist or not (8 rows
// of 5120 x 5120, group 64: 8.1 us, in room for 16 rows 9.6; 16 rows 9.5, in room for 32 14.8; 1 row
// 7.6, in room for 8 8.0; 20 rows 12.7, in room for 32 15.1, of 65536 x 2048 26.0 against 27.4, of 32768 x
// 8192 43.6 against 45.2). With more than 16 rows one workgroup fits a
// CU. Two wavefronts on rows make the most workgroups, and the shortest where those are one round of
// the CUs at most (32 rows of 5120 x 5120 15.4 us against 24.5, of 8192 x 8192 21.7 against 37); beyond,
// four with two tiles each read x a quarter as often (16384 x 5120 26.9 against 29.6, 65536 x 2048
// 29.6 against 69, 64 rows of 8192 x 2048 12.7 against 18.1).
template <typename T, int G, bool GATED>
hipError_t launch_w4(const W4Args& a, hipStream_t st) {
    if (a.m <= 4) return launch_tiles<T, G, 4, 4, 2, 1, 4, GATED>(a, st);
    if (a.m <= 8) return launch_tiles<T, G, 8, 4, 2, 1, 4, GATED>(a, st);
    if (a.m <= 16) return launch_tiles<T, G, 16, 4, 2, 1, 4, GATED>(a, st);
    constexpr int COLS = 2 * (GATED ? 8 : 16);
    const int64_t blocks = (int64_t)((a.N + COLS - 1) / COLS) * ((a.m + MAX_ROWS_X - 1) / MAX_ROWS_X);
    if (a.m <= 24)
        return blocks <= 256 ? launch_tiles<T, G, 24, 4, 2, 1, 4, GATED>(a, st) : launch_tiles<T, G, 24, 2, 4, 2, 3, GATED>(a, st);
    if (blocks <= 256) return launch_tiles<T, G, 32, 4, 2, 1, 3, GATED>(a, st);
    return launch_tiles<T, G, 32, 2, 4, 2, 3, GATED>(a, st);
}

template <int NM>
int run_w4(const moe_w4* const* w, int act, float limit, const void* x, int64_t ldx, int32_t m, void* y, int64_t ldy,
           void* stream) {
    for (int q = 0; q < NM; ++q)
        if (const int rc = check_w4(w[q])) return rc;
    if (NM == 2) {
        if (w[0]->rows != w[1]->rows || w[0]->cols != w[1]->cols || w[0]->group != w[1]->group || w[0]->dtype != w[1]->dtype)
            return MOE_EINVAL;
        if ((w[0]->zeros == nullptr) != (w[1]->zeros == nullptr)) return MOE_EINVAL;
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
        return status_of(g == 32 ? launch_w4<Bf16, 32, NM == 2>(a, st) : g == 64 ? launch_w4<Bf16, 64, NM == 2>(a, st) : launch_w4<Bf16, 128, NM == 2>(a, st));
    return status_of(g == 32 ? launch_w4<F16, 32, NM == 2>(a, st) : g == 64 ? launch_w4<F16, 64, NM == 2>(a, st) : launch_w4<F16, 128, NM == 2>(a, st));
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
