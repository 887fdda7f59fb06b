// A few rows times 4-bit weights with group scales (gfx950):
//
//   out[m][n] = alpha[e] * sum_k x[m][k] e2m1(code[k][n]) e4m3(scale[k / 16][n])
//
// with x in bf16 or float16, not quantized, against packed NVFP4 weights: one
// matrix for all rows, or one for each expert with the rows grouped by expert
// (offsets, as the token sort gives them). gated: the columns are [gate | up] and
// out = silu(gate) * up of the float32 sums, each with its alpha.
//
// Bound by the weights, read once (9/16 of a byte an element), so the kernel is
// built around their stream:
//
// * A work-group owns NB blocks of 16 columns (gated: a gate block and the matching
//   up block) of one tile of 4 RG rows; its waves share K in groups of four
//   128-element steps (quads), the unit that the scales are packed in, the next
//   quad's weights in flight while one is computed, and add their sums through LDS
//   in wave order. A lane loads 16 contiguous bytes of a step for its column: 32
//   values of K, two scale groups.
// * The products are 4x4x4 MFMAs, sixteen independent blocks of 4 lanes: a block's
//   sum runs over the four values that its own lanes hold, so a lane's sum over one
//   scale group is complete in that lane and the scale is one float32
//   multiply-add per row and group instead of two to four instructions a
//   weight. The 4-bit values enter as they are (exact in bf16 and float16).
// * A lane's 4 bits of position within 16 columns say which row and which quarter
//   of its 32 values of x it holds; the MFMA's broadcast (of one block to the four
//   that share K values) hands each quarter to all 16 columns. So x takes one 16-byte
//   load per step and 4 rows, straight from the caches for one group of rows. For
//   more, lanes that read different rows are a cache line each (64 cycles a load),
//   and x goes through LDS instead: rows as they lie in memory, swizzled by row so
//   that the four rows of a read lie in different banks.
//
// Measured, in a captured graph, weights not in the caches:
//   1 row of 6144 x 7168         7.7 us (24.8 MB; launch and first loads about 4)
//   16 rows of 6144 x 7168       13.0 us, of 7168 x 2048 6.6 us: issue of the MFMAs
//                                and of the scales' multiply-adds beside the stream
//   8 tokens' experts, gated     6.7 TB/s (37 experts of 4096 x 7168: 91 us)
//   32 tokens' experts, gated    154 to 170 us by the routing (47, 48 experts: 5.0, 4.7 TB/s)
// Scaling the weights before 16x16x32 MFMAs, 16 instructions for 8 of them in bf16,
// was slower at 1 row (11.3 us); for tiles of 16 rows alone it took 5 to 15 % less (16 x
// 28672 x 4096 23.1 against 26.6 us) and is not built in yet.
#include <type_traits>

#include "elements.hpp"

namespace nvfp4 {

namespace {

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// waves of a work-group at most: more rows and columns take more registers and LDS
template <int RG, int NB> constexpr int kMaxWaves = RG == 1 || NB == 1 ? 8 : 4;
constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kBeyond = 0x80000000u;   // an offset outside every buffer: reads zeros
constexpr int kStreamNT = 2;                // non-temporal: the weights are read once

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kRsrcWord3);
}

// Four weights (nibbles 4h .. 4h + 3 of word) as an operand of the 4x4x4 MFMA, and
// the MFMA whose x comes from lanes 4b .. 4b + 3 of each 16.
template <typename T> struct Operand;
template <> struct Operand<__bf16> {
    typedef short4_t type;
    template <int H>
    static __device__ __forceinline__ type weights(uint32_t word) {
        const u32x2 r = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, 1.0f, 2 * H)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, 1.0f, 2 * H + 1))};
        return __builtin_bit_cast(type, r);
    }
    template <int B>
    static __device__ __forceinline__ float4_t mfma(type a, type b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(a, b, c, 2, B, 0);
    }
};
template <> struct Operand<_Float16> {
    typedef half4_t type;
    template <int H>
    static __device__ __forceinline__ type weights(uint32_t word) {
        const u32x2 r = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, 1.0f, 2 * H)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, 1.0f, 2 * H + 1))};
        return __builtin_bit_cast(type, r);
    }
    template <int B>
    static __device__ __forceinline__ float4_t mfma(type a, type b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_4x4x4f16(a, b, c, 2, B, 0);
    }
};

// silu(g) * u by e^-|g|, which neither sign of g lets overflow (zero from |g| =
// 87.4 on: silu is then g or below 2^-119)
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float e = exp_split(fmaxf(-__builtin_fabsf(g), -200.0f));
    return g * ((g >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e)) * u;
}

// Tile `want` of the rows grouped by expert: tiles of TM rows, expert after expert.
// Each wave finds it by itself, 64 experts at a time. False: there is none.
template <int TM>
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

// One group of four K steps of a wave's NB column blocks: weights and scales.
template <int NB>
struct Quad {
    u32x4 w[4][NB];
    u32x2 s[NB];
};

// x of one step for RG groups of four rows: lane (c, q) holds of row c % 4 of each
// group the 8 values that dword c / 4 of the weights in quarter q meets.
template <int RG> struct Rows { u32x4 v[RG]; };

// x of a quad as it is loaded: RG 1, its four steps; else its rows, piece l (8
// values) in lane l, on the way to LDS
template <int RG> struct RowQuad { u32x4 v[4 * RG]; };
// LDS bytes of a wave: its x, and after the last step its sums
template <int RG, int NB> constexpr int kWaveLds = 1024 * RG * (RG > 1 ? 4 : NB);

// Column ranges that the work-groups of a tile take.
template <bool GATED, int NB>
__host__ __device__ inline int64_t column_ranges(int64_t N) {
    return GATED ? N / 32 : (N / 16 + NB - 1) / NB;
}

template <typename T, int RG, int NB>
__device__ __forceinline__ void add_step(const Rows<RG>& x, const u32x4 (&w)[NB], const u32x2 (&sf)[NB], int u,
                                         float4_t (&acc)[NB][RG]) {
    using Op = Operand<T>;
    using V = typename Op::type;
#pragma unroll
    for (int f = 0; f < NB; ++f) {
        const uint32_t codes = sf[f][u >> 1];
        float4_t sum[2][RG];                             // by scale group: dwords 0, 1 and 2, 3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < RG; ++g) sum[h][g] = (float4_t){0.f, 0.f, 0.f, 0.f};
        // one dword of either scale group at a time, so that no MFMA waits for the last
        auto dwords = [&](auto d) {
            constexpr int D = decltype(d)::value;
            const V a0 = Op::template weights<0>(w[f][D]), a1 = Op::template weights<1>(w[f][D]);
            const V b0 = Op::template weights<0>(w[f][D + 2]), b1 = Op::template weights<1>(w[f][D + 2]);
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const V x0 = __builtin_bit_cast(V, (u32x2){x.v[g][0], x.v[g][1]});
                sum[0][g] = Op::template mfma<D>(x0, a0, sum[0][g]);
                sum[1][g] = Op::template mfma<D + 2>(x0, b0, sum[1][g]);
            }
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const V x1 = __builtin_bit_cast(V, (u32x2){x.v[g][2], x.v[g][3]});
                sum[0][g] = Op::template mfma<D>(x1, a1, sum[0][g]);
                sum[1][g] = Op::template mfma<D + 2>(x1, b1, sum[1][g]);
            }
        };
        dwords(std::integral_constant<int, 0>());
        dwords(std::integral_constant<int, 1>());
        const float s0 = u & 1 ? __builtin_amdgcn_cvt_f32_fp8(codes, 2) : __builtin_amdgcn_cvt_f32_fp8(codes, 0);
        const float s1 = u & 1 ? __builtin_amdgcn_cvt_f32_fp8(codes, 3) : __builtin_amdgcn_cvt_f32_fp8(codes, 1);
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[f][g][i] = __builtin_fmaf(sum[1][g][i], s1, __builtin_fmaf(sum[0][g][i], s0, acc[f][g][i]));
    }
}

template <typename T, int RG, bool GATED, int NB>
__device__ __forceinline__ void matvec_tile(const MatvecParams& p, int expert, int64_t row0, int rows, int64_t nb,
                                            uint8_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x / 64;
    const int64_t blocks = (GATED ? p.N / 2 : p.N) / 16;         // column blocks of the output
    const int c = lane & 15, q = lane >> 4;
    const int64_t ldq = pitch_q(p.K), ldsf = pitch_wsf(p.K);
    const int nsteps = (int)(ldq / 64), nquads = (nsteps + 3) / 4;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.bq + (int64_t)expert * p.N * ldq, p.N * ldq);
    const __amdgpu_buffer_rsrc_t rsf = make_rsrc(p.bsf + (int64_t)expert * p.N * ldsf, p.N * ldsf);
    const __amdgpu_buffer_rsrc_t rx =
        make_rsrc(static_cast<const T*>(p.x) + row0 * p.K, (int64_t)rows * p.K * (int64_t)sizeof(T));
    // gated: a gate block and its up block; else NB blocks one after another (beyond
    // the last one: it again, not stored)
    uint32_t boff[NB], sfoff[NB];
#pragma unroll
    for (int f = 0; f < NB; ++f) {
        const int64_t n = (GATED ? nb + f * blocks : min(nb * NB + f, blocks - 1)) * 16 + c;
        boff[f] = (uint32_t)wq_off(n, ldq, 16 * q);
        sfoff[f] = (uint32_t)wsf_off(n, ldsf, 0, q);
    }
    // x of a quad, 1 KB a row. rows beyond the tile's read its last one; their sums
    // are not stored
    uint8_t* own = lds + wave * kWaveLds<RG, NB>;
    const int piece = c >> 2, kx = RG == 1 ? 32 * q + 8 * piece : 8 * lane;
    const uint32_t xrow = RG == 1 ? (uint32_t)min(c & 3, rows - 1) * (uint32_t)p.K * 2 : 0;
    auto load_x = [&](int qd, RowQuad<RG>& x) {
        const int k0 = 512 * qd;                                 // K <= 2^20
        if constexpr (RG == 1) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                x.v[u] = __builtin_amdgcn_raw_buffer_load_b128(
                    rx, k0 + 128 * u + kx < (int)p.K ? xrow + 2 * kx : kBeyond, 2 * (uint32_t)(k0 + 128 * u), 0);
        } else {
            const uint32_t at = k0 + kx < (int)p.K ? 2 * kx : kBeyond;
#pragma unroll
            for (int r = 0; r < 4 * RG; ++r)
                x.v[r] = __builtin_amdgcn_raw_buffer_load_b128(
                    rx, at, (uint32_t)min(r, rows - 1) * (uint32_t)p.K * 2 + 2 * (uint32_t)k0, 0);
        }
    };
    auto stage_x = [&](const RowQuad<RG>& x) {
        if constexpr (RG > 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int r = 0; r < 4 * RG; ++r)
                *reinterpret_cast<u32x4*>(own + r * 1024 + ((lane ^ ((r & 3) << 2)) << 4)) = x.v[r];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    };
    auto step_x = [&](int u, const RowQuad<RG>& x) {
        Rows<RG> r;
        if constexpr (RG == 1) {
            r.v[0] = x.v[u];
        } else {
            const int at = ((16 * u + 4 * q + piece) ^ ((c & 3) << 2)) << 4;
#pragma unroll
            for (int g = 0; g < RG; ++g) r.v[g] = *reinterpret_cast<const u32x4*>(own + (4 * g + (c & 3)) * 1024 + at);
        }
        return r;
    };

    auto load = [&](int qd, Quad<NB>& r) {
#pragma unroll
        for (int f = 0; f < NB; ++f)
            r.s[f] = __builtin_amdgcn_raw_buffer_load_b64(rsf, sfoff[f], (uint32_t)qd * kWsfQuad, kStreamNT);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // beyond the last step the last one again, which meets scales of zero
            const uint32_t kd = (uint32_t)min(4 * qd + u, nsteps - 1) * kWqStep;
#pragma unroll
            for (int f = 0; f < NB; ++f) r.w[u][f] = __builtin_amdgcn_raw_buffer_load_b128(rb, boff[f], kd, kStreamNT);
        }
    };
    float4_t acc[NB][RG];
#pragma unroll
    for (int f = 0; f < NB; ++f)
#pragma unroll
        for (int g = 0; g < RG; ++g) acc[f][g] = (float4_t){0.f, 0.f, 0.f, 0.f};
    // The weights one quad ahead, x (from the caches) when it is needed: loads return
    // in order, so x goes before the next weights. (x ahead too takes registers, and
    // with them waves, away: 16 rows of 6144 x 7168 14.4 against 12.6 us.)
    Quad<NB> cur, next;
    RowQuad<RG> x;
    auto compute = [&] {
        stage_x(x);
#pragma unroll
        for (int u = 0; u < 4; ++u) add_step<T, RG, NB>(step_x(u, x), cur.w[u], cur.s, u, acc);
    };
    int qd = wave;                                       // (waves <= nquads)
    load(qd, cur);
    for (; qd + waves < nquads; qd += waves) {
        load_x(qd, x);
        __builtin_amdgcn_sched_barrier(0);
        load(qd + waves, next);
        __builtin_amdgcn_sched_barrier(0);
        compute();
        cur = next;
    }
    load_x(qd, x);
    compute();
    // (over this wave's x)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float4_t* red = reinterpret_cast<float4_t*>(own);
#pragma unroll
    for (int f = 0; f < NB; ++f)
#pragma unroll
        for (int g = 0; g < RG; ++g) red[(f * RG + g) * 64 + lane] = acc[f][g];
    __syncthreads();
    // acc[g][i] of lane (c, q): row 4g + i, column c, the K values of quarter q
    const int per = GATED && p.alpha_stride > 1 ? 2 : 1;
    const float alpha = p.alpha[(int64_t)expert * per], alpha_up = p.alpha[(int64_t)expert * per + per - 1];
    constexpr int OB = GATED ? 1 : NB;                   // blocks of outputs
    for (int i = tid; i < 16 * OB * rows; i += blockDim.x) {
        const int r = i / (16 * OB), col = i % (16 * OB), blk = col >> 4;
        float v[GATED ? 2 : 1];
#pragma unroll
        for (int f = 0; f < (GATED ? 2 : 1); ++f) {
            v[f] = 0.0f;
            for (int wv = 0; wv < waves; ++wv)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    v[f] += reinterpret_cast<const float4_t*>(
                        lds + wv * kWaveLds<RG, NB>)[((blk + f) * RG + (r >> 2)) * 64 + 16 * h + (col & 15)][r & 3];
        }
        if (nb * OB + blk >= blocks) continue;
        float o = alpha * v[0];
        if constexpr (GATED) o = silu_mul(o, alpha_up * v[1]);
        static_cast<T*>(p.out)[(row0 + r) * 16 * blocks + nb * 16 * OB + col] = from_f32<T>(o);
    }
}

template <typename T, int RG, bool GATED, int NB>
__global__ __launch_bounds__((64 * kMaxWaves<RG, NB>)) __attribute__((amdgpu_waves_per_eu(2)))
void matvec_kernel(MatvecParams p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int TM = 4 * RG;
    const int lane = threadIdx.x & 63;
    const int64_t ranges = column_ranges<GATED, NB>(p.N);
    const int64_t tile = blockIdx.x / ranges, nb = blockIdx.x - tile * ranges;
    int expert = 0, rows;
    int64_t row0;
    if (p.offsets) {
        if (!find_tile<TM>(p.offsets, p.E, p.M, tile, lane, expert, row0, rows)) return;
        expert = __builtin_amdgcn_readfirstlane(expert);
        row0 = __builtin_amdgcn_readfirstlane((int)row0);
        rows = __builtin_amdgcn_readfirstlane(rows);
    } else {
        row0 = tile * TM;
        rows = (int)min((int64_t)TM, p.M - row0);
    }
    matvec_tile<T, RG, GATED, NB>(p, expert, row0, rows, nb, lds);
}

template <typename T, int RG, bool GATED, int NB>
hipError_t run(const MatvecParams& p, hipStream_t s) {
    const int64_t grid = matvec_tiles(p.M, p.offsets ? p.E : 0) * column_ranges<GATED, NB>(p.N);
    const int nquads = (int)((pitch_q(p.K) / 64 + 3) / 4);
    // Many work-groups stream best as 4 waves of two quads or more (8 experts of 4096
    // x 7168, 1024 work-groups: 24.0 against 27.5 us; 37 experts 91 against 106; 36 of
    // 7168 x 2048 as 2 waves 48 against 56); few want every wave (6144 x 7168, 384:
    // 7.8 against 8.2, 512 x 7168, 32: 4.9 against 5.7).
    const bool many = RG == 1 && grid >= 1024;
    const int most = many ? 4 : kMaxWaves<RG, NB>;
    int per = (nquads + most - 1) / most;
    if (many && per < 2) per = 2;
    const int waves = (nquads + per - 1) / per;
    const int lds = waves * kWaveLds<RG, NB>;
    static std::atomic<int> lds_set[kMaxDevices];
    if (lds > 65536) {
        const hipError_t e =
            ensure_dynamic_lds(reinterpret_cast<const void*>(&matvec_kernel<T, RG, GATED, NB>), lds, lds_set);
        if (e != hipSuccess) return e;
    }
    matvec_kernel<T, RG, GATED, NB><<<(unsigned)grid, 64 * waves, lds, s>>>(p);
    return hipGetLastError();
}

template <typename T, int RG, bool GATED>
hipError_t run(const MatvecParams& p, hipStream_t s) {
    if constexpr (GATED) {
        return run<T, RG, true, 2>(p, s);
    } else if constexpr (RG == 1) {
        return run<T, 1, false, 1>(p, s);
    } else {
        // x is read once for NB blocks, but one block fills more CUs: 16 rows of 4096 x
        // 7168 (256 blocks) 9.8 against 12.8 us, of 6144 x 7168 14.0 against 13.2, of
        // 28672 x 1024 12.3 against 9.8
        return matvec_tiles(p.M, p.offsets ? p.E : 0) * (p.N / 16) <= 256 ? run<T, RG, false, 1>(p, s)
                                                                          : run<T, RG, false, 2>(p, s);
    }
}

template <typename T, bool GATED>
hipError_t run(const MatvecParams& p, hipStream_t s) {
    const int tm = matvec_tile_rows(p.M, p.offsets ? p.E : 1);
    return tm == 4 ? run<T, 1, GATED>(p, s) : tm == 8 ? run<T, 2, GATED>(p, s) : run<T, 4, GATED>(p, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecParams& p, int dtype, hipStream_t s) {
    if (p.M <= 0) return hipSuccess;
    if (dtype == kBf16) return p.gated ? run<__bf16, true>(p, s) : run<__bf16, false>(p, s);
    return p.gated ? run<_Float16, true>(p, s) : run<_Float16, false>(p, s);
}

}  // namespace nvfp4
