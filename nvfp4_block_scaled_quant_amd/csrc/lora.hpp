// Operands of the adapters' second product (v B_a^T), shared by the kernels
// that add it to the projection.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

// Eight ranks k .. k + 7 of row `row` of v as hi + lo in bf16 (zeros when not
// `on`): v is the sum of its partial sums in order, hi its rounding and lo the
// rounding of what is left, so hi + lo is within 2^-17 of v.
// UNROLL partial sums are loaded at a time.
template <int UNROLL>
__device__ __forceinline__ void lora_v_operand(const LoraParams& lo, bool on, int64_t row, int k, u32x4& hi,
                                               u32x4& low) {
    float4_t v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (on) {
        const float4_t* src = reinterpret_cast<const float4_t*>(lo.v + row * lo.R + k);
        const int64_t plane = lo.M * lo.R / 4;
        v[0] = sum_planes<UNROLL>(src, lo.planes, plane);
        v[1] = sum_planes<UNROLL>(src + 1, lo.planes, plane);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v0 = v[e >> 1][2 * (e & 1)], v1 = v[e >> 1][2 * (e & 1) + 1];
        hi[e] = pack_bf16x2_rne(v0, v1);
        low[e] = pack_bf16x2_rne(v0 - bf16_to_f32(hi[e] & 0xFFFFu), v1 - bf16_to_f32(hi[e] >> 16));
    }
}

// Eight ranks k .. k + 7 of column `col` of B_a (zeros when not `on`); what lies
// beyond the rank is not part of the adapter and is left out, whatever it holds.
__device__ __forceinline__ u32x4 lora_b_operand(const LoraParams& lo, bool on, int a, int64_t col, int k, int rank) {
    u32x4 b = {0u, 0u, 0u, 0u};
    if (on && k < rank) {
        b = *reinterpret_cast<const u32x4*>(lo.b + ((int64_t)a * lo.N + col) * lo.R + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k + 2 * e >= rank) b[e] = 0u;
            else if (k + 2 * e + 1 >= rank) b[e] &= 0xFFFFu;
        }
    }
    return b;
}

}  // namespace nvfp4
