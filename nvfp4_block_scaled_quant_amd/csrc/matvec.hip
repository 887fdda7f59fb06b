// A few rows times 4-bit weights with group scales (gfx950):
//
//   out[m][n] = alpha[e] * sum_k x[m][k] e2m1(code[k][n]) e4m3(scale[k / 16][n])
//
// with x in bf16 or float16, not quantized, against packed NVFP4 weights: one
// matrix for all rows, or one for each expert with the rows grouped by expert
// (offsets, as the token sort gives them). gated: the columns are [gate | up] and
// out = silu(gate) * up of the float32 sums, each with its alpha.
//
// Bound by the weights, read once (9/16 of a byte an element). A work-group owns 16
// columns (gated: and the matching 16 of the up half) of one tile of at most 16
// rows; its waves share K in groups of four 128-element steps, the unit that the
// scales are packed in, and add their sums through LDS in wave order. A lane loads
// 16 contiguous bytes of a step for its column: 32 K values, dword s of which is
// its operand of a 16x16x32 MFMA; x is read with the same K permutation, straight
// from memory, as its few rows stay in the caches.
//
// Weights enter the products exactly: e2m1 * e4m3 has 6 significant bits, which
// bf16 and float16 (whose range takes every product) both hold.
#include <type_traits>

#include "elements.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int TM = 16;             // rows of a tile
constexpr int kMaxWaves = 8;

template <typename T> struct Operand;
template <> struct Operand<__bf16> {
    typedef bf16x8_t type;
    // 8 nibbles times the scale: float32 products (exact), rounded without loss
    static __device__ __forceinline__ type dequant(uint32_t word, uint32_t code) {
        const float s = e4m3_decode(code);
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 0);
        const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 1);
        const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 2);
        const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 3);
        const u32x4 r = {pack_bf16x2_rne(a[0] * s, a[1] * s), pack_bf16x2_rne(b[0] * s, b[1] * s),
                         pack_bf16x2_rne(c[0] * s, c[1] * s), pack_bf16x2_rne(d[0] * s, d[1] * s)};
        return __builtin_bit_cast(type, r);
    }
    static __device__ __forceinline__ float4_t mfma(type a, type b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Operand<_Float16> {
    typedef half8_t type;
    static __device__ __forceinline__ type dequant(uint32_t word, uint32_t code) {
        return dequant8(word, scale_pair(code));
    }
    static __device__ __forceinline__ float4_t mfma(type a, type b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// silu(g) * u by e^-|g|, which neither sign of g lets overflow (zero from |g| =
// 87.4 on: silu is then g or below 2^-119)
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float e = exp_split(fmaxf(-__builtin_fabsf(g), -200.0f));
    return g * ((g >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e)) * u;
}

// Tile `want` of the rows grouped by expert: 16-row tiles, expert after expert.
// Each wave finds it by itself, 64 experts at a time. False: there is none.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int E, int64_t M, int64_t want, int lane,
                                          int& expert, int64_t& row0, int& rows) {
    int64_t before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, cnt = 0;
        if (e < E) {
            lo = max(offsets[e], 0);
            cnt = max((int64_t)0, min((int64_t)offsets[e + 1], M) - lo);
        }
        const int nt = (int)((cnt + TM - 1) / TM);
        int sum = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const int64_t first = before + sum - nt;
        const uint64_t hit = __ballot(want >= first && want < first + nt);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t at = (want - first) * TM;
            expert = e0 + src;
            row0 = __shfl((int)(lo + at), src);
            rows = __shfl((int)min((int64_t)TM, cnt - at), src);
            return true;
        }
        before += __shfl(sum, 63);
    }
    return false;
}

template <typename T, bool GATED>
__global__ __launch_bounds__(64 * kMaxWaves) void matvec_kernel(MatvecParams p) {
    using Op = Operand<T>;
    constexpr int NB = GATED ? 2 : 1;
    __shared__ float4_t red[kMaxWaves][NB][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x / 64;
    const int64_t blocks = (GATED ? p.N / 2 : p.N) / 16;         // column blocks of the output
    const int64_t tile = blockIdx.x / blocks, nb = blockIdx.x - tile * blocks;
    int expert = 0, rows;
    int64_t row0;
    if (p.offsets) {
        if (!find_tile(p.offsets, p.E, p.M, tile, lane, expert, row0, rows)) return;
        expert = __builtin_amdgcn_readfirstlane(expert);
        row0 = __builtin_amdgcn_readfirstlane((int)row0);
        rows = __builtin_amdgcn_readfirstlane(rows);
    } else {
        row0 = tile * TM;
        rows = (int)min((int64_t)TM, p.M - row0);
    }
    const int c = lane & 15, q = lane >> 4;
    const int64_t ldq = pitch_q(p.K), ldsf = pitch_wsf(p.K);
    const int nsteps = (int)(ldq / 64), nquads = (nsteps + 3) / 4;
    const uint8_t *bq[NB], *bsf[NB];
#pragma unroll
    for (int f = 0; f < NB; ++f) {
        const int64_t block = expert * (p.N / 16) + nb + f * blocks;
        bq[f] = p.bq + block * 16 * ldq + (q >> 1) * kWqHalf + c * 32 + (q & 1) * 16;
        bsf[f] = p.bsf + block * 16 * ldsf + c * 32 + q * 8;
    }
    // rows beyond the tile's read its last one; their sums are not stored
    const T* x = static_cast<const T*>(p.x) + (row0 + min(c, rows - 1)) * p.K + 32 * q;

    float4_t acc[NB];
#pragma unroll
    for (int f = 0; f < NB; ++f) acc[f] = (float4_t){0.f, 0.f, 0.f, 0.f};
    for (int qd = wave; qd < nquads; qd += waves) {
        u32x4 w[4][NB];
        u32x2 sf[NB];
#pragma unroll
        for (int f = 0; f < NB; ++f)
            sf[f] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(bsf[f] + (int64_t)qd * kWsfQuad));
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int f = 0; f < NB; ++f)
                w[u][f] = 4 * qd + u < nsteps
                              ? __builtin_nontemporal_load(
                                    reinterpret_cast<const u32x4*>(bq[f] + (int64_t)(4 * qd + u) * kWqStep))
                              : (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (4 * qd + u >= nsteps) break;
            const int64_t k0 = (int64_t)(4 * qd + u) * 128;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                u32x4 raw = {0u, 0u, 0u, 0u};
                if (k0 + 32 * q + 8 * s < p.K) raw = *reinterpret_cast<const u32x4*>(x + k0 + 8 * s);
                const auto a = __builtin_bit_cast(typename Op::type, raw);
#pragma unroll
                for (int f = 0; f < NB; ++f) {
                    const uint32_t code = (sf[f][u >> 1] >> (16 * (u & 1) + 8 * (s >> 1))) & 0xFFu;
                    acc[f] = Op::mfma(a, Op::dequant(w[u][f][s], code), acc[f]);
                }
            }
        }
    }
#pragma unroll
    for (int f = 0; f < NB; ++f) red[wave][f][lane] = acc[f];
    __syncthreads();
    // acc[i] of lane (c, q) is row 4q + i, column c
    const int per = GATED && p.alpha_stride > 1 ? 2 : 1;
    const float alpha = p.alpha[(int64_t)expert * per], alpha_up = p.alpha[(int64_t)expert * per + per - 1];
    for (int i = tid; i < 16 * rows; i += blockDim.x) {
        const int r = i >> 4, col = i & 15;
        float v[NB];
#pragma unroll
        for (int f = 0; f < NB; ++f) {
            v[f] = red[0][f][(r >> 2) * 16 + col][r & 3];
            for (int wv = 1; wv < waves; ++wv) v[f] += red[wv][f][(r >> 2) * 16 + col][r & 3];
        }
        float o = alpha * v[0];
        if constexpr (GATED) o = silu_mul(o, alpha_up * v[NB - 1]);
        static_cast<T*>(p.out)[(row0 + r) * 16 * blocks + nb * 16 + col] = from_f32<T>(o);
    }
}

}  // namespace

hipError_t launch_matvec(const MatvecParams& p, int dtype, hipStream_t s) {
    const int nquads = (int)((pitch_q(p.K) / 64 + 3) / 4);
    const int per = (nquads + kMaxWaves - 1) / kMaxWaves, waves = (nquads + per - 1) / per;
    const int64_t blocks = (p.gated ? p.N / 2 : p.N) / 16;
    const int64_t grid = matvec_tiles(p.M, p.offsets ? p.E : 0) * blocks;
    if (grid <= 0) return hipSuccess;
    auto run = [&](auto zero, auto gated) {
        matvec_kernel<decltype(zero), decltype(gated)::value><<<(unsigned)grid, 64 * waves, 0, s>>>(p);
    };
    if (dtype == kBf16) {
        if (p.gated) run((__bf16)0.0f, std::true_type()); else run((__bf16)0.0f, std::false_type());
    } else {
        if (p.gated) run((_Float16)0.0f, std::true_type()); else run((_Float16)0.0f, std::false_type());
    }
    return hipGetLastError();
}

}  // namespace nvfp4
