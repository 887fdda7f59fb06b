// Operands of the adapters' second product (v B_a^T), shared by the kernels
// that add it to the projection.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

// Eight values of v, as partial sums, to hi + low in bf16: v is the partial
// sums' sum in order (those beyond p.planes are zero), hi its rounding and low
// the rounding of what is left, so hi + low is within 2^-17 of v.
__device__ __forceinline__ void lora_split(const float4_t (&part)[kLoraMaxPlanes][2], u32x4& hi, u32x4& low) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            v[t] = part[0][e >> 1][2 * (e & 1) + t];
#pragma unroll
            for (int j = 1; j < kLoraMaxPlanes; ++j) v[t] += part[j][e >> 1][2 * (e & 1) + t];
        }
        hi[e] = pack_bf16x2_rne(v[0], v[1]);
        low[e] = pack_bf16x2_rne(v[0] - bf16_to_f32(hi[e] & 0xFFFFu), v[1] - bf16_to_f32(hi[e] >> 16));
    }
}

// Eight ranks k .. k + 7 of row `row` of v.
__device__ __forceinline__ void lora_v_operand(const LoraParams& lo, int64_t row, int k, u32x4& hi, u32x4& low) {
    const float4_t* src = reinterpret_cast<const float4_t*>(lo.v + row * lo.R + k);
    const int64_t plane = lo.M * lo.R / 4;
    float4_t part[kLoraMaxPlanes][2];
#pragma unroll
    for (int j = 0; j < kLoraMaxPlanes; ++j) {
        part[j][0] = part[j][1] = (float4_t){0.f, 0.f, 0.f, 0.f};
        if (j < lo.planes) {
            part[j][0] = src[j * plane];
            part[j][1] = src[j * plane + 1];
        }
    }
    lora_split(part, hi, low);
}

// B_a's eight values of ranks k .. k + 7: what lies beyond the rank is not part
// of the adapter and is left out, whatever it holds.
__device__ __forceinline__ u32x4 lora_mask_rank(u32x4 b, int k, int rank) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (k + 2 * e >= rank) b[e] = 0u;
        else if (k + 2 * e + 1 >= rank) b[e] &= 0xFFFFu;
    }
    return b;
}

// Eight ranks k .. k + 7 of column `col` of B_a (zeros when not `on`).
__device__ __forceinline__ u32x4 lora_b_operand(const LoraParams& lo, bool on, int a, int64_t col, int k, int rank) {
    u32x4 b = {0u, 0u, 0u, 0u};
    if (on && k < rank) {
        b = lora_mask_rank(*reinterpret_cast<const u32x4*>(lo.b + ((int64_t)a * lo.N + col) * lo.R + k), k, rank);
    }
    return b;
}

}  // namespace nvfp4
