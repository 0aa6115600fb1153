// Device and host helpers of the operators around the layer (the gated
// feed-forward block, the norms, the products with 4-bit weights): the 16- and
// 32-bit value types, matrix-core wrappers, argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "moe.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Value types. `bits` is how a value lies in memory; `pack2` rounds two f32 values
// to nearest even (NaN stays NaN) into one word, the first in the low half.
struct Bf16 {
    typedef uint16_t bits;
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    static MOE_DEV float load(bits b) { return __uint_as_float((uint32_t)b << 16); }
    static MOE_DEV bits store(float f) { return __builtin_bit_cast(bits, (__bf16)f); }
    static MOE_DEV float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static MOE_DEV float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static MOE_DEV uint32_t pack2(float a, float b) {
        v2 v;
        v[0] = (__bf16)a;
        v[1] = (__bf16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    static MOE_DEV f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static constexpr uint32_t ONES = 0x3F803F80u;
};
struct F16 {
    typedef uint16_t bits;
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    static MOE_DEV float load(bits b) { return (float)__builtin_bit_cast(_Float16, b); }
    static MOE_DEV bits store(float f) { return __builtin_bit_cast(bits, (_Float16)f); }
    static MOE_DEV float lo(uint32_t w) { return (float)__builtin_bit_cast(v2, w)[0]; }
    static MOE_DEV float hi(uint32_t w) { return (float)__builtin_bit_cast(v2, w)[1]; }
    static MOE_DEV uint32_t pack2(float a, float b) {
        v2 v;
        v[0] = (_Float16)a;
        v[1] = (_Float16)b;
        return __builtin_bit_cast(uint32_t, v);
    }
    static MOE_DEV f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static constexpr uint32_t ONES = 0x3C003C00u;
};
struct F32 {
    typedef float bits;
    static MOE_DEV float load(bits b) { return b; }
    static MOE_DEV bits store(float f) { return f; }
};

// the clamps of the gated product, which keep a NaN (limit <= 0: none)
MOE_DEV float clamp_gate(float g, float limit) { return limit > 0.f && g > limit ? limit : g; }
MOE_DEV float clamp_up(float u, float limit) {
    if (limit > 0.f) u = u > limit ? limit : (u < -limit ? -limit : u);
    return u;
}

// act(v) and its derivative, NaN where v is. SILU: v s(v), s the logistic function. GELU:
// the tanh form. Beyond |v| = 100 tanh is 1 to the last bit, and the argument is held
// there so that v^3 does not overflow.
MOE_DEV float act_value(float v, int act) {
    if (act == MOE_ACT_SILU) return v / (1.0f + __expf(-v));
    const float c = fminf(fmaxf(v, -100.f), 100.f);
    const float z = 0.7978845608028654f * (c + 0.044715f * c * c * c);
    return v / (1.0f + __expf(-2.f * z));   // v/2 (1 + tanh z) without a difference
}
MOE_DEV void act_both(float v, int act, float& a, float& da) {
    if (act == MOE_ACT_SILU) {
        const float s = 1.0f / (1.0f + __expf(-v));
        a = v * s;
        da = s * (1.f + v * (1.f - s));
        return;
    }
    const float c = clamp_up(v, 100.f);   // (fminf and fmaxf would make a number of a NaN)
    const float z = 0.7978845608028654f * (c + 0.044715f * c * c * c);
    // (1 + tanh z) / 2 and (1 - tanh z) / 2, neither as a difference
    const float s = 1.f / (1.f + __expf(-2.f * z)), q = 1.f / (1.f + __expf(2.f * z));
    a = v * s;
    da = s + 2.f * c * s * q * 0.7978845608028654f * (1.f + 0.134145f * c * c);
}

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace moe
