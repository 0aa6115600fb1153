// Dropout before the residual's addition, and its gradient, from a counter-based generator
// (moe_dropout_* in include/moe.h): the mask is made anew wherever it is needed.
//
// The generator is Philox-4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as
// 1, 2, 3; 2011). Its counter names a place, (column / 8, row, the use's two words), and its key is
// the seed, so that a value's bits depend on nothing else: not on strides, on the launch, or on which
// rows a call holds before it. The 128 bits serve eight values of 16: one generator call for each 16 bytes
// of 16-bit values. 32 bits per value would cost twice the multiplications, which are most of the
// instructions here; with 16 a probability is a multiple of 2^-16, and the scale that of the multiple.
//
// Memory bounds it: 8192 x 5120 bf16 43 us with a residual (252 MB, 5.9 TB/s) and 34 without (168 MB, 5.0 TB/s); 1003 x
// 1111 f32 is a launch, 4 to 5 us.
#include "block_rows.h"

namespace moe {
namespace {

constexpr int MAX_DIM = 1 << 20, MAX_ROWS = 1 << 30;

struct DropArgs {
    const void *x, *residual;
    void* y;
    const uint64_t* rng;   // seed, use
    int64_t ldx, ldr, ldy;
    int dim, m;
    uint32_t threshold;    // kept: 16 bits that are at least this
    float scale;
    bool past_l2;
    Walk walk;
};

// 128 bits of the counter (c, row, use)
MOE_DEV uint4 philox(uint32_t c, uint32_t row, uint64_t use, uint64_t seed) {
    uint32_t x0 = c, x1 = row, x2 = (uint32_t)use, x3 = (uint32_t)(use >> 32), k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)b;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// A thread takes eight columns of a row at a time, `N` chunks of 16 bytes
template <typename T, Tail TAIL, bool RESIDUAL, bool ONCE>
__global__ __launch_bounds__(256) void dropout_kernel(DropArgs a) {
    constexpr int V = Raw<T>::V, N = 8 / V;
    const uint64_t seed = a.rng[0], use = a.rng[1];
    for (Place p = first_place(a.walk); p.row < a.m; p = p.next(a.walk)) {
        Raw<T> x[N], r[N];
        int col[N], skip[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            place_chunk<TAIL>(p.chunk * N + n, V, a.dim, col[n], skip[n]);
            x[n].template load_of<TAIL, ONCE>(a.x, p.row * a.ldx, col[n], a.dim);
            if (RESIDUAL) r[n].template load_of<TAIL, ONCE>(a.residual, p.row * a.ldr, col[n], a.dim);
        }
        const uint4 bits = philox((uint32_t)p.chunk, (uint32_t)p.row, use, seed);
        const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
        bool keep[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) keep[2 * i] = (w[i] & 0xFFFF) >= a.threshold, keep[2 * i + 1] = (w[i] >> 16) >= a.threshold;
        uint32_t mask = 0;
        if (TAIL != WHOLE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) mask |= (keep[i] ? 1u : 0u) << i;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float v[V], res[V];
            x[n].template get<WHOLE>(v, 0);
            if (RESIDUAL) r[n].template get<WHOLE>(res, 0);
            // (a chunk that begins before its columns: theirs are its last)
            const uint32_t mine = (mask >> (n * V)) << skip[n];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool k = TAIL == WHOLE ? keep[n * V + i] : (mine >> i & 1) != 0;
                const float d = k ? v[i] * a.scale : 0.f;   // (what is dropped may be infinite or NaN)
                v[i] = RESIDUAL ? res[i] + d : d;
            }
            store_chunk<T, TAIL>(a.y, p.row * a.ldy, col[n], a.dim, skip[n], a.past_l2, v);
        }
    }
}

int check_dropout(const moe_dropout* f) {
    if (f == nullptr || f->dim < 1 || f->dim > MAX_DIM) return MOE_EINVAL;
    if (f->dtype < MOE_BF16 || f->dtype > MOE_F32) return MOE_EINVAL;
    return f->p >= 0.0 && f->p <= 1.0 ? MOE_OK : MOE_EINVAL;
}

template <typename T, bool RESIDUAL, bool ONCE>
hipError_t launch_dropout_of(DropArgs a, hipStream_t st) {
    const int per_row = (a.dim + 7) / 8;
    const int64_t blocks = walk_blocks((int64_t)per_row * a.m, ONCE);
    a.walk = walk(per_row, blocks * 256);
    const Tail tail = tail_of(a.dim, Raw<T>::V);
    auto* const k = tail == SHORT ? dropout_kernel<T, SHORT, RESIDUAL, false>
                    : tail == WHOLE ? dropout_kernel<T, WHOLE, RESIDUAL, ONCE> : dropout_kernel<T, SHIFTED, RESIDUAL, ONCE>;
    return launch_kernel(k, dim3((unsigned)blocks), dim3(256), 0, st, a);
}
template <typename T, bool RESIDUAL>
hipError_t launch_dropout(const DropArgs& a, hipStream_t st) {
    return past_caches((size_t)a.m * a.dim * sizeof(typename T::bits) * (RESIDUAL ? 3 : 2)) ? launch_dropout_of<T, RESIDUAL, true>(a, st)
                                                                                          : launch_dropout_of<T, RESIDUAL, false>(a, st);
}

int dropout(const moe_dropout* f, const uint64_t* rng, const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t m,
            void* y, int64_t ldy, void* stream) {
    const int rc = check_dropout(f);
    if (rc != MOE_OK) return rc;
    if (m < 0 || m > MAX_ROWS) return MOE_EINVAL;
    if (m == 0) return MOE_OK;
    const size_t size = value_bytes(f->dtype);
    if (rng == nullptr || !aligned_to(rng, 8) || !value_rows_ok(x, ldx, f->dim, size) || !value_rows_ok(y, ldy, f->dim, size))
        return MOE_EINVAL;
    if (residual != nullptr && !value_rows_ok(residual, ldr, f->dim, size)) return MOE_EINVAL;
    DropArgs a{};
    a.x = x, a.residual = residual, a.y = y, a.rng = rng;
    a.ldx = ldx, a.ldr = ldr, a.ldy = ldy, a.dim = f->dim, a.m = m;
    a.threshold = (uint32_t)nearbyint(f->p * 65536.0);
    a.scale = a.threshold < 65536 ? (float)(65536.0 / (65536.0 - a.threshold)) : 0.f;
    a.past_l2 = (size_t)m * f->dim * size > (32u << 20);
    const hipStream_t st = (hipStream_t)stream;
    switch (f->dtype) {
        case MOE_BF16: return status_of(residual ? launch_dropout<Bf16, true>(a, st) : launch_dropout<Bf16, false>(a, st));
        case MOE_F16: return status_of(residual ? launch_dropout<F16, true>(a, st) : launch_dropout<F16, false>(a, st));
        default: return status_of(residual ? launch_dropout<F32, true>(a, st) : launch_dropout<F32, false>(a, st));
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_dropout_forward(const moe_dropout* f, const uint64_t* rng, const void* x, int64_t ldx, const void* residual,
                        int64_t ldr, int32_t m, void* y, int64_t ldy, void* stream) {
    return dropout(f, rng, x, ldx, residual, ldr, m, y, ldy, stream);
}

int moe_dropout_backward(const moe_dropout* f, const uint64_t* rng, const void* dy, int64_t lddy, int32_t m, void* dx,
                         int64_t lddx, void* stream) {
    return dropout(f, rng, dy, lddy, nullptr, 0, m, dx, lddx, stream);
}

}  // extern "C"
