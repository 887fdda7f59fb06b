// Low-rank adapters of many requests beside one shared NVFP4 projection:
//   out[m] = bf16(alpha * A[m] W + scale[a] (x[m] A_a^T) B_a^T),  a = ids[m]
// with A_a (R, K) and B_a (N, R) in bf16. The product with A_a ("shrink", here)
// gives v[m] = scale[a] x[m] A_a^T in float32; the product with B_a is added in
// the epilogue of the shared projection (gemm.hip), before its one rounding.
//
// Shrink. What has to move is x once and each adapter's A_a once; the
// arithmetic is small, so the split is made for bytes in flight. A work-group
// takes one tile of 64 rows, one adapter that occurs in it and one range of K,
// and gathers the tile's rows that have the adapter, so an adapter is read
// once per tile however its rows are scattered (a decode batch of 64 rows
// reads each adapter once; in a prefill batch a tile has one or two). Its 8
// waves interleave over the range in blocks of 64 K values, read straight from
// memory into v_mfma_f32_16x16x32_bf16 operands (a lane takes 32 contiguous
// bytes of a row, so a row's block is one 128-byte line), and join their sums
// in wave order through LDS. Ranges of K are separate partial sums, added in
// order by the reader. Nothing depends on scheduling.
#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int NT = 512;
constexpr int NW = NT / 64;
constexpr int kRankBlock = 64;      // ranks of a work-group (4 column blocks of 16)
constexpr int kSlots = 16;          // work-groups that share a tile's adapters

__global__ __launch_bounds__(NT) void lora_shrink_kernel(const uint16_t* __restrict__ x,
                                                         const uint16_t* __restrict__ wa,
                                                         const float* __restrict__ scale,
                                                         const int32_t* __restrict__ ids,
                                                         const int32_t* __restrict__ rank, int64_t M, int64_t K,
                                                         int L, int R, int planes, float* __restrict__ v) {
    __shared__ int list[kLoraRows];
    __shared__ __attribute__((aligned(16))) float red[NW][16][kRankBlock + 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kLoraRows;
    const int plane = blockIdx.z % planes, rb = blockIdx.z / planes;
    const int rbase = rb * kRankBlock;

    int id = m0 + lane < M ? ids[m0 + lane] : -1;
    if (id >= L) id = -1;
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    // blocks of 64 K values of this plane, dealt to the waves in turn
    const int nb = (int)((K + 63) / 64), per = (nb + planes - 1) / planes;
    const int b0 = plane * per, b1 = min(nb, b0 + per);

    // the tile's adapters in order of first appearance: this work-group takes
    // numbers y, y + gridDim.y, ...
    for (int d = 0; todo; ++d) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t rows = __builtin_amdgcn_ballot_w64(id == a);
        todo &= ~rows;
        if (d % (int)gridDim.y != (int)blockIdx.y) continue;
        const int rk = rank ? min(max(rank[a], 0), R) : R;
        const int n = __builtin_popcountll(rows);
        const float sc = scale[a];
        __syncthreads();                             // the previous adapter's readers are done
        if (wave == 0 && id == a) list[__builtin_popcountll(rows & ((1ull << lane) - 1))] = lane;
        __syncthreads();

        const int groups = (n + 15) / 16;            // 16-row groups of the gathered rows
        const int cols = min(max(rk - rbase, 0), kRankBlock);
        const uint16_t* xr[4];
        const uint16_t* ar[4];
        bool xok[4], aok[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            xok[g] = 16 * g + c < n;
            xr[g] = x + (m0 + (xok[g] ? list[16 * g + c] : 0)) * K + 16 * q;
            aok[g] = 16 * g + c < cols;
            ar[g] = wa + ((int64_t)a * R + rbase + (aok[g] ? 16 * g + c : 0)) * K + 16 * q;
        }
        float4_t acc[4][4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[g][f] = (float4_t){0.f, 0.f, 0.f, 0.f};
        const u32x4 zero = {0u, 0u, 0u, 0u};
        if (cols > 0) {
            for (int b = b0 + wave; b < b1; b += NW) {
                const int64_t k = (int64_t)b * 64;
                const bool kin = k + 16 * q < K;     // K % 16 == 0: a lane's 16 values are in or out together
                u32x4 fx[4][2], fw[4][2];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    fx[g][0] = fx[g][1] = fw[g][0] = fw[g][1] = zero;
                    if (kin && xok[g]) {
                        fx[g][0] = *reinterpret_cast<const u32x4*>(xr[g] + k);
                        fx[g][1] = *reinterpret_cast<const u32x4*>(xr[g] + k + 8);
                    }
                    if (kin && aok[g]) {
                        fw[g][0] = *reinterpret_cast<const u32x4*>(ar[g] + k);
                        fw[g][1] = *reinterpret_cast<const u32x4*>(ar[g] + k + 8);
                    }
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g >= groups) continue;
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        if (16 * f >= cols) continue;
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            acc[g][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, fx[g][t]), __builtin_bit_cast(bf16x8_t, fw[f][t]),
                                acc[g][f], 0, 0, 0);
                    }
                }
            }
        }
        // acc[g][f][i] = D[gathered row 16 g + 4 q + i][rank 16 f + c]
        const int store = min(R - rbase, kRankBlock);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if (g >= groups) continue;
            __syncthreads();
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[wave][4 * q + i][16 * f + c] = acc[g][f][i];
            __syncthreads();
            for (int e = tid; e < 16 * kRankBlock; e += NT) {
                const int r = e / kRankBlock, col = e % kRankBlock;
                if (16 * g + r >= n || col >= store) continue;
                float sum = red[0][r][col];
#pragma unroll
                for (int w = 1; w < NW; ++w) sum += red[w][r][col];
                v[((int64_t)plane * M + m0 + list[16 * g + r]) * R + rbase + col] = col < cols ? sc * sum : 0.0f;
            }
        }
    }
}

}  // namespace

// Work-groups of the shrink before K is split: tiles x the adapters a tile can
// hold x rank blocks; K ranges (at most 8, each at least 8 blocks of 64, one
// per wave) bring the launch to about one work-group per CU. Prefill tiles hold
// few adapters, which the host cannot know; counting one per tile is right for
// them and only costs partial sums where there are more.
int lora_planes(int64_t M, int64_t K, int64_t L, int64_t R) {
    const int64_t tiles = (M + kLoraRows - 1) / kLoraRows, rbs = (R + kRankBlock - 1) / kRankBlock;
    const int64_t here = tiles > 1 ? 1 : (M < L ? M : L);
    const int64_t nb = (K + 63) / 64;
    int64_t n = 256 / (tiles * rbs * here);
    if (n > nb / 8) n = nb / 8;
    if (n > 8) n = 8;
    if (n < 1) n = 1;
    const int64_t per = (nb + n - 1) / n;
    return (int)((nb + per - 1) / per);
}

hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const float* scale, const int32_t* ids,
                              const int32_t* rank, int64_t M, int64_t K, int64_t L, int64_t R, int planes, float* v,
                              hipStream_t s) {
    const int64_t tiles = (M + kLoraRows - 1) / kLoraRows, rbs = (R + kRankBlock - 1) / kRankBlock;
    int64_t slots = M < L ? M : L;
    if (slots > kSlots) slots = kSlots;
    const dim3 grid((unsigned)tiles, (unsigned)slots, (unsigned)(planes * rbs));
    lora_shrink_kernel<<<grid, NT, 0, s>>>(x, a, scale, ids, rank, M, K, (int)L, (int)R, planes, v);
    return hipGetLastError();
}

}  // namespace nvfp4
