// Rows of values in chunks of 16 bytes, wherever a row starts: what the operators around the
// layer that read and write whole rows share.
#pragma once

#include "block_common.h"

namespace moe {
namespace {

// How a row of dim values falls into chunks of V. WHOLE: V divides dim. SHIFTED: the
// last chunk is the row's last V values, the first `skip` of which belong to the
// chunk before it: they read as zeros here, so that they add nothing, and are not
// stored. SHORT: dim < V, one chunk of single values. A thread without a chunk loads
// the row's first and reads it as zeros (skip = V): every load is unconditional, so
// that the compiler's waits for one row leave the next rows' loads in flight.
enum Tail { WHOLE, SHIFTED, SHORT };

// A chunk as it lies in memory: 16 bytes, which need not be aligned to more than a value
template <typename T>
struct Raw {
    static constexpr int V = 16 / sizeof(typename T::bits);
    union {
        uint4 q;
        typename T::bits b[V];
    };
    template <Tail TAIL>
    MOE_DEV void load(const void* base, int64_t row, int col, int dim) {
        const typename T::bits* p = reinterpret_cast<const typename T::bits*>(base) + row;
        if (TAIL == SHORT) {
            q = make_uint4(0, 0, 0, 0);
            for (int i = 0; i < dim; ++i) b[i] = p[i];
        } else {
            __builtin_memcpy(&q, p + col, 16);
        }
    }
    // ONCE: of an array that will not be read again while the caches still hold it: it leaves their lines to others
    template <Tail TAIL, bool ONCE>
    MOE_DEV void load_of(const void* base, int64_t row, int col, int dim) {
        if (TAIL == SHORT || !ONCE) {
            load<TAIL>(base, row, col, dim);
        } else {
            typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
            const words w = __builtin_nontemporal_load(reinterpret_cast<const words*>(reinterpret_cast<const typename T::bits*>(base) + row + col));
            q = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // (used: the array is there at all)
    template <Tail TAIL>
    MOE_DEV void get(float* v, int skip, bool used = true) const {
        const uint32_t on = skip < V && used ? ~0u : 0u;
        const uint32_t w[4] = {q.x & on, q.y & on, q.z & on, q.w & on};
        if constexpr (V == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = T::lo(w[i]), v[2 * i + 1] = T::hi(w[i]);
        }
        if (TAIL == SHIFTED) {
#pragma unroll
            for (int i = 0; i < V - 1; ++i) v[i] = i < skip ? 0.f : v[i];
        }
    }
};
template <typename T, Tail TAIL>
MOE_DEV void store_chunk(void* base, int64_t row, int col, int dim, int skip, bool past_l2, const float* v) {
    constexpr int V = Raw<T>::V;
    typename T::bits* p = reinterpret_cast<typename T::bits*>(base) + row + col;
    if (skip >= V) return;
    if (TAIL == SHORT || (TAIL == SHIFTED && skip != 0)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= skip && col + i < dim) p[i] = T::store(v[i]);
        return;
    }
    uint4 q;
    if constexpr (V == 4)
        q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        q = make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7]));
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    const words w = {q.x, q.y, q.z, q.w};
    if (past_l2) __builtin_nontemporal_store(w, reinterpret_cast<words*>(p));
    else *reinterpret_cast<words*>(p) = w;
}
// where chunk c of a row starts, and how many of its values belong to the chunk before it
template <Tail TAIL>
MOE_DEV void place_chunk(int c, int v, int dim, int& col, int& skip) {
    col = c * v;
    skip = 0;
    if (col >= dim) skip = v, col = 0;
    else if (TAIL == SHIFTED && col + v > dim) skip = col + v - dim, col = dim - v;
}

// Positions (row, chunk of it) that a thread of a grid takes one after another: its own number among
// all chunks, and as many further at a time as there are threads
struct Walk {
    int per_row, rows_on, chunks_on;   // chunks per row; a step of the whole grid in rows and chunks
};
struct Place {
    int64_t row;
    int chunk;
    MOE_DEV Place next(const Walk& w) const {
        Place p{row + w.rows_on, chunk + w.chunks_on};
        if (p.chunk >= w.per_row) p.chunk -= w.per_row, ++p.row;
        return p;
    }
};
MOE_DEV Place first_place(const Walk& w) {
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    return {(int64_t)(i / (uint32_t)w.per_row), (int)(i % (uint32_t)w.per_row)};
}
// Whether arrays of that many bytes in all are read past the caches: the last one holds 256 MiB, and what a program
// made just before is still there. Sums of six rows of 8192 x 5120 bf16 (587 MB) 102 us past them and 117 through
// them, of 1999 x 5120 (143 MB) 27 and 21.6; dropout with a residual, both ways (419 MB), 67 and 83.
inline bool past_caches(size_t bytes) { return bytes > ((size_t)192 << 20); }

// Workgroups of 256 for `places` positions: as many as are resident, or with PAST (the arrays are larger than the caches) a
// thread each, as far as a grid goes. Sums of six rows of 8192 x 5120 bf16 with and without: 5.5 and 5.2 TB/s; of 1999 x
// 5120, from the caches: 24.2 and 22.0 us.
inline int64_t walk_blocks(int64_t places, bool past) { return std::min<int64_t>((places + 255) / 256, past ? 1 << 20 : 256 * 8); }
inline Walk walk(int per_row, int64_t threads) { return {per_row, (int)(threads / per_row), (int)(threads % per_row)}; }

inline size_t value_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
inline Tail tail_of(int dim, int v) { return dim < v ? SHORT : dim % v ? SHIFTED : WHOLE; }
// a matrix of rows aligned to its values
inline bool value_rows_ok(const void* p, int64_t ld, int dim, size_t size) { return p != nullptr && aligned_to(p, size) && ld >= dim; }

}  // namespace
}  // namespace moe
