// Operands of the adapters' second product (v B_a^T), shared by the kernels
// that add it to the projection.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

// Eight ranks k .. k + 7 of row `row` of v as hi + low in bf16: v is the sum of
// its partial sums in order, hi its rounding and low the rounding of what is
// left, so hi + low is within 2^-17 of v (2^-134 where that is more). A finite v
// stays finite: hi ends at the largest bf16, where from 3.3961e38 on it would round
// to infinity. Where v is infinite low is zero, so that it stays infinite (infinity
// less itself is not a number).
__device__ __forceinline__ void lora_v_operand(const LoraParams& lo, int64_t row, int k, u32x4& hi, u32x4& low) {
    typedef float float8_t __attribute__((ext_vector_type(8)));
    const float8_t v = sum_planes<kLoraMaxPlanes - 1>(reinterpret_cast<const float8_t*>(lo.v + row * lo.R + k), lo.planes,
                                                      lo.M * lo.R / 8);
    constexpr float kMaxBf16 = 0x1.FEp127f;
    auto in_range = [](float x) { return __builtin_isfinite(x) ? __builtin_amdgcn_fmed3f(x, -kMaxBf16, kMaxBf16) : x; };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v0 = v[2 * e], v1 = v[2 * e + 1];
        hi[e] = pack_bf16x2_rne(in_range(v0), in_range(v1));
        const float h0 = bf16_to_f32(hi[e] & 0xFFFFu), h1 = bf16_to_f32(hi[e] >> 16);
        low[e] = pack_bf16x2_rne(__builtin_isinf(h0) ? 0.0f : v0 - h0, __builtin_isinf(h1) ? 0.0f : v1 - h1);
    }
}

// B_a's eight values of ranks k .. k + 7: what lies beyond the rank is not part
// of the adapter and is left out, whatever it holds.
__device__ __forceinline__ u32x4 lora_mask_rank(u32x4 b, int k, int rank) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] &= (k + 2 * e < rank ? 0xFFFFu : 0u) | (k + 2 * e + 1 < rank ? 0xFFFF0000u : 0u);
    return b;
}

// B_a for the product with low: infinities and NaN are left out, as the product
// with hi has them already (low may be zero or have the other sign, and would turn
// an infinity into NaN). Per 16-bit half: one added to an exponent of all ones
// gives the sign bit, whose arithmetic shift is the mask.
typedef short short2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ short2_t lora_infinite_bits(uint32_t b) {
    return __builtin_bit_cast(short2_t, b & 0x7F807F80u) + (short2_t)(short)0x80;
}
__device__ __forceinline__ u32x4 lora_finite(u32x4 b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] &= ~__builtin_bit_cast(uint32_t, lora_infinite_bits(b[e]) >> (short2_t)(short)15);
    return b;
}
__device__ __forceinline__ bool lora_any_infinite(u32x4 b) {
    uint32_t any = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= __builtin_bit_cast(uint32_t, lora_infinite_bits(b[e]));
    return (any & 0x80008000u) != 0;
}

}  // namespace nvfp4
