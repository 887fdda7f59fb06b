// Low-rank adapters of many requests beside one shared NVFP4 projection:
//   out[m] = bf16(alpha * A[m] W + scale[a] (x[m] A_a^T) B_a^T),  a = ids[m]
// with A_a (R, K) and B_a (N, R) in bf16. The product with A_a ("shrink") gives
// v[m] = scale[a] x[m] A_a^T in float32; the product with B_a ("expand") is added
// to the projection before its one rounding. Per batch size:
//   up to 32 rows   shrink (beside it A laid out for streaming), then one kernel
//                   that streams the weights and adds the adapters
//   more rows       the rows are listed by adapter, shrink (beside it A's f16
//                   form), the tiled GEMM; the expand is in its epilogue, or,
//                   where K is cut into chunks, in the kernel that adds them
// A row's arithmetic does not depend on its place in a tile or on the other
// rows, so results depend neither on scheduling nor on the grouping.
//
// Shrink. What has to move is x once and each adapter's A_a once; the
// arithmetic is small, so the split is made for bytes in flight. A work-group
// takes one tile of 64 (listed) rows, one adapter that occurs in it and one
// range of K, and gathers the rows that have the adapter, so an adapter is read
// once per tile however its rows are scattered. Its 8 waves interleave over the
// range in blocks of 64 K values, read straight from memory into
// v_mfma_f32_16x16x32_bf16 operands (one load covers 64 contiguous bytes of 16
// rows; the next block's loads are issued before a block's products), and join
// their sums in wave order through LDS. Ranges of K are separate partial sums,
// added in order by the reader.
#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int NT = 512;
constexpr int NW = NT / 64;
constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr int kStreamNT = 2;        // buffer-load cache policy: non-temporal (read once)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kRsrcWord3);
}

constexpr int kRankBlock = 64;      // ranks of a work-group (4 column blocks of 16)

// A's exact f16 values, rows padded with zeros to whole steps (32-bit indices:
// M * pitch_h(K) is below 2^31).
__device__ void dequant_a(const uint8_t* __restrict__ aq, const uint8_t* __restrict__ asf, int64_t M, int64_t K,
                          uint8_t* __restrict__ ah, uint32_t first, uint32_t stride) {
    constexpr int B = 4;                // blocks of 16 in flight per thread
    const uint32_t groups = (uint32_t)(K / 16), ldh = (uint32_t)pitch_h(K), total = (uint32_t)M * groups;
    for (uint32_t b0 = first; b0 < total; b0 += B * stride) {
        u32x2 w[B];
        uint32_t sf[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const uint32_t b = b0 + j * stride;
            if (b < total) {
                w[j] = *reinterpret_cast<const u32x2*>(aq + (int64_t)b * 8);
                sf[j] = asf[b];
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const uint32_t b = b0 + j * stride;
            if (b >= total) continue;
            const uint32_t r = b / groups, g = b - r * groups;
            store_block_f16(ah + r * ldh + g * 32, w[j][0], w[j][1], sf[j]);
            if (g == groups - 1)
                for (uint32_t i = groups * 32; i < ldh; i += 16)
                    *reinterpret_cast<u32x4*>(ah + r * ldh + i) = (u32x4){0u, 0u, 0u, 0u};
        }
    }
}

// For the fused epilogue: A's exact f16 values, and the shrunk rows' partial
// sums joined into vs (the kernel's first work-groups).
__global__ __launch_bounds__(256) void lora_join_kernel(LoraParams p, int join_blocks, const uint8_t* __restrict__ aq,
                                                        const uint8_t* __restrict__ asf, uint8_t* __restrict__ ah) {
    if ((int)blockIdx.x >= join_blocks) {
        dequant_a(aq, asf, p.M, p.K, ah, (blockIdx.x - join_blocks) * 256 + threadIdx.x, (gridDim.x - join_blocks) * 256);
        return;
    }
    const int R8 = p.R / 8;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, pos = t / R8;
    const int k = 8 * (int)(t - pos * R8);
    if (pos >= p.M || p.ids[pos] < 0) return;
    u32x4 hi, low;
    lora_v_operand<8>(p, true, p.perm[pos], k, hi, low);
    uint16_t* dst = p.vs + pos * 2 * p.R + k;
    *reinterpret_cast<u32x4*>(dst) = hi;
    *reinterpret_cast<u32x4*>(dst + p.R) = low;
}

// A in the streaming kernel's layout, zero beyond M and K: data per 16-row
// block and 128-element step as one kilobyte (lane l = 16 q + c holds bytes
// [16 q, +16) of the step of row c), scales as the packed weights' (per group
// of four steps: row, pair q, step, two bytes).
__device__ void lay_out_a(const LoraParams& p, const uint8_t* __restrict__ aq, const uint8_t* __restrict__ asf,
                          uint8_t* __restrict__ aqp, uint8_t* __restrict__ asfp, int64_t first, int64_t stride) {
    const int steps = (int)(pitch_q(p.K) / 64), quads = (int)(pitch_wsf(p.K) / 32);
    const int mt = (int)((p.M + 15) / 16);
    const int64_t kb = p.K / 2, kg = p.K / 16;
    const int64_t nd = (int64_t)mt * steps * 64, nsf = (int64_t)mt * quads * 64;
    for (int64_t i = first; i < nd + nsf; i += stride) {
        if (i < nd) {
            const int lane = (int)(i & 63), st = (int)((i >> 6) % steps);
            const int64_t row = (i >> 6) / steps * 16 + (lane & 15), at = 64 * st + 16 * (lane >> 4);
            u32x2 lo = {0u, 0u}, hi = {0u, 0u};
            if (row < p.M && at < kb) lo = *reinterpret_cast<const u32x2*>(aq + row * kb + at);      // K / 2 % 8 == 0
            if (row < p.M && at + 8 < kb) hi = *reinterpret_cast<const u32x2*>(aq + row * kb + at + 8);
            *reinterpret_cast<u32x4*>(aqp + 16 * i) = (u32x4){lo[0], lo[1], hi[0], hi[1]};
        } else {
            const int64_t j = i - nd;
            const int t = (int)(j & 63), c = t >> 2, q = t & 3, quad = (int)((j >> 6) % quads);
            const int64_t row = (j >> 6) / quads * 16 + c;
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t g = 8 * (4 * quad + u) + 2 * q + e;
                    if (row < p.M && g < kg) w[u >> 1] |= (uint32_t)asf[row * kg + g] << (16 * (u & 1) + 8 * e);
                }
            *reinterpret_cast<u32x2*>(asfp + 8 * j) = (u32x2){w[0], w[1]};
        }
    }
}

__global__ __launch_bounds__(NT) void lora_shrink_kernel(LoraParams p, int tiles, int slots, int shrink_blocks,
                                                         bool rank_rows, int32_t* __restrict__ perm_out,
                                                         int32_t* __restrict__ sid_out,
                                                         const uint8_t* __restrict__ aq,
                                                         const uint8_t* __restrict__ asf, uint8_t* __restrict__ aqp,
                                                         uint8_t* __restrict__ asfp, uint8_t* __restrict__ ah) {
    if ((int)blockIdx.x >= shrink_blocks) {          // the launch's further work-groups: A's layout
        const uint32_t first = (blockIdx.x - shrink_blocks) * NT + threadIdx.x, stride = (gridDim.x - shrink_blocks) * NT;
        if (ah) dequant_a(aq, asf, p.M, p.K, ah, first, stride);
        else lay_out_a(p, aq, asf, aqp, asfp, first, stride);
        return;
    }
    constexpr int G = kLoraRows / 16, TR = kLoraRows;
    __shared__ int list[TR];
    __shared__ __attribute__((aligned(16))) float red[NW][16][kRankBlock + 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int slot = rest % slots, z = rest / slots;
    const int plane = z % p.planes, rb = z / p.planes;
    const int64_t m0 = (int64_t)tile * TR;
    const int rbase = rb * kRankBlock;
    const int64_t M = p.M, K = p.K;
    const int L = p.L, R = p.R, planes = p.planes;

    // the tile's rows and their adapters, by lane
    int id = -1, row_of = 0;
    const bool in = lane < TR && m0 + lane < M;
    if (rank_rows) {
        // a small batch is listed here: by (adapter, row), rows without one
        // last; every work-group finds the same order by counting
        __shared__ __attribute__((aligned(16))) int key[kLoraRankRows];
        __shared__ int order[kLoraRankRows];
        int mine = 0x7FFFFFFF;
        if (tid < kLoraRankRows) {
            if (tid < M) {
                const int a = p.ids[tid];
                mine = (a >= 0 && a < L ? a : L) * kLoraRankRows + tid;
            }
            key[tid] = mine;
        }
        __syncthreads();
        if (tid < M) {
            int pos = 0;
            for (int j = 0; j < (int)M; j += 4) {
                const u32x4 k = *reinterpret_cast<const u32x4*>(key + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) pos += (int)k[e] < mine;
            }
            order[pos] = mine;
        }
        __syncthreads();
        if (in) {
            row_of = order[m0 + lane] % kLoraRankRows;
            id = order[m0 + lane] / kLoraRankRows;
            if (id >= L) id = -1;
        }
        if (rest == 0 && wave == 0 && in) {
            perm_out[m0 + lane] = row_of;
            sid_out[m0 + lane] = id;
        }
    } else if (in) {
        id = p.ids[m0 + lane];
        if (id >= L) id = -1;
        row_of = p.perm ? p.perm[m0 + lane] : (int)(m0 + lane);
    }
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    // blocks of 64 K values of this plane, dealt to the waves in turn
    const int nb = (int)((K + 63) / 64), per = (nb + planes - 1) / planes;
    const int b0 = plane * per, b1 = min(nb, b0 + per);

    // the tile's adapters in order of first appearance: this work-group takes
    // numbers slot, slot + slots, ...
    for (int d = 0; todo; ++d) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t rows = __builtin_amdgcn_ballot_w64(id == a);
        todo &= ~rows;
        if (d % slots != slot) continue;
        const int rk = p.rank ? min(max(p.rank[a], 0), R) : R;
        const int n = __builtin_popcountll(rows);
        const float sc = p.scale[a];
        __syncthreads();                             // the previous adapter's readers are done
        if (wave == 0 && id == a) {
            const int at = __builtin_popcountll(rows & ((1ull << lane) - 1));
            list[at] = row_of;
        }
        __syncthreads();

        const int groups = (n + 15) / 16;            // 16-row groups of the gathered rows
        const int cols = min(max(rk - rbase, 0), kRankBlock);
        const uint16_t* xr[G];
        const uint16_t* ar[4];
        bool xok[G], aok[4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            xok[g] = 16 * g + c < n;
            xr[g] = p.x + (int64_t)(xok[g] ? list[16 * g + c] : 0) * K + 8 * q;
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            aok[f] = 16 * f + c < cols;
            ar[f] = p.a + ((int64_t)a * R + rbase + (aok[f] ? 16 * f + c : 0)) * K + 8 * q;
        }
        float4_t acc[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[g][f] = (float4_t){0.f, 0.f, 0.f, 0.f};
        struct Block {
            u32x4 x[G][2], a[4][2];
        };
        auto load = [&](int b, Block& r) {
            const int64_t k = (int64_t)b * 64;
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bool kin = k + 32 * t + 8 * q < K;     // K % 8 == 0: a lane's 8 values are in or out together
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    r.x[g][t] = zero;
                    if (kin && xok[g]) r.x[g][t] = *reinterpret_cast<const u32x4*>(xr[g] + k + 32 * t);
                }
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    r.a[f][t] = zero;
                    if (kin && aok[f]) r.a[f][t] = *reinterpret_cast<const u32x4*>(ar[f] + k + 32 * t);
                }
            }
        };
        auto compute = [&](const Block& r) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (g >= groups) continue;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    if (16 * f >= cols) continue;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        acc[g][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, r.x[g][t]), __builtin_bit_cast(bf16x8_t, r.a[f][t]),
                            acc[g][f], 0, 0, 0);
                }
            }
        };
        if (cols > 0 && b0 + wave < b1) {
            // (past the end a block that is there is loaded again and not used)
            Block even, odd;
            int b = b0 + wave;
            load(b, even);
            while (true) {
                load(min(b + NW, b1 - 1), odd);
                __builtin_amdgcn_sched_barrier(0);
                compute(even);
                if ((b += NW) >= b1) break;
                load(min(b + NW, b1 - 1), even);
                __builtin_amdgcn_sched_barrier(0);
                compute(odd);
                if ((b += NW) >= b1) break;
            }
        }
        // acc[g][f][i] = D[gathered row 16 g + 4 q + i][rank 16 f + c]
        const int store = min(R - rbase, kRankBlock);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g >= groups) continue;
            if (g > 0) __syncthreads();
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
                p.v[((int64_t)plane * M + list[16 * g + r]) * R + rbase + col] = col < cols ? sc * sum : 0.0f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Rows by adapter. One work-group counts, scans and places; the rows of one
// adapter come in no particular order (a row's result does not depend on its
// place). Where at least 16 lanes of a wave share an adapter, as in runs of
// rows, one of them counts for all: an LDS atomic takes one address at a time.
constexpr int ST = 1024;

__device__ __forceinline__ int count_id(int* bins, int bin, bool on) {
    const uint64_t act = __builtin_amdgcn_ballot_w64(on);
    if (!act) return 0;
    const int lane = threadIdx.x & 63;
    const int lead = __builtin_ctzll(act);
    const int b0 = __builtin_amdgcn_readlane(bin, lead);
    const uint64_t same = __builtin_amdgcn_ballot_w64(on && bin == b0);
    const int n = __builtin_popcountll(same);
    int pos = 0;
    if (n >= 16) {
        int base = 0;
        if (lane == lead) base = atomicAdd(&bins[b0], n);
        base = __builtin_amdgcn_readlane(base, lead);
        if (bin == b0) pos = base + __builtin_popcountll(same & ((1ull << lane) - 1));
        else if (on) pos = atomicAdd(&bins[bin], 1);
    } else if (on) {
        pos = atomicAdd(&bins[bin], 1);
    }
    return pos;
}

__global__ __launch_bounds__(ST) void lora_sort_kernel(const int32_t* __restrict__ ids, int M, int L,
                                                       int32_t* __restrict__ perm, int32_t* __restrict__ sid) {
    const int tid = threadIdx.x;
    __shared__ int bins[kLoraMaxAdapters + 1];       // the last used one: rows without an adapter
    __shared__ int wave_sum[ST / 64];
    for (int i = tid; i <= L; i += ST) bins[i] = 0;
    __syncthreads();
    auto bin_of = [&](int i) {
        const int id = i < M ? ids[i] : -1;
        return id >= 0 && id < L ? id : L;
    };
    // ids by rounds of one per thread; the first KEEP rounds stay in registers
    constexpr int KEEP = 8;
    const int rounds = (M + ST - 1) / ST;
    int kept[KEEP];
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (k < rounds) kept[k] = bin_of(k * ST + tid);
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (k < rounds) count_id(bins, kept[k], k * ST + tid < M);
    for (int k = KEEP; k < rounds; ++k) count_id(bins, bin_of(k * ST + tid), k * ST + tid < M);
    __syncthreads();
    // exclusive scan: each thread its share of consecutive bins
    const int share = (L + 1 + ST - 1) / ST, lo = min(tid * share, L + 1), hi = min(lo + share, L + 1);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += bins[i];
    int incl = sum;
    for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(incl, off, 64);
        if ((tid & 63) >= off) incl += up;
    }
    if ((tid & 63) == 63) wave_sum[tid >> 6] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < (tid >> 6); ++w) base += wave_sum[w];
    for (int i = lo; i < hi; ++i) {
        const int n = bins[i];
        bins[i] = base;
        base += n;
    }
    __syncthreads();
    auto place = [&](int k, int bin) {
        const int i = k * ST + tid;
        const int pos = count_id(bins, bin, i < M);
        if (i < M) {
            perm[pos] = i;
            sid[pos] = bin < L ? bin : -1;
        }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (k < rounds) place(k, kept[k]);
    for (int k = KEEP; k < rounds; ++k) place(k, bin_of(k * ST + tid));
}

// ---------------------------------------------------------------------------
// Expand into LDS: delta[r][n] = (v B_a^T) of row r of a tile of up to 64
// rows and 16 CB columns from n0. The tile's (adapter, 16 of its rows) pairs
// are dealt to the nw waves (a row has one adapter, so one wave writes it; the
// caller has zeroed delta). `lane`'s row of the tile has adapter id (-1: none)
// and is row row_of of v.
template <int CB, int LD, int UNROLL>
__device__ __forceinline__ void expand_tile(const LoraParams& p, int id, int row_of, int64_t n0, int wave, int nw,
                                            float (*delta)[LD]) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    int turn = 0;                       // number of the adapter's first pair
    while (todo) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t rows = __builtin_amdgcn_ballot_w64(id == a);
        todo &= ~rows;
        const int n = __builtin_popcountll(rows);
        const int first = turn;
        turn += (n + 15) / 16;
        // this wave's pairs among first .. turn - 1
        int pair = first + (wave - first % nw + nw) % nw;
        if (pair >= turn) continue;
        const int rank = p.rank ? min(max(p.rank[a], 0), p.R) : p.R;
        // lane i receives the adapter's i-th row: the lanes that have it push
        // theirs to 0 .. n - 1, the others to the rest
        const uint64_t below = (1ull << lane) - 1;
        const int to = id == a ? __builtin_popcountll(rows & below) : n + __builtin_popcountll(~rows & below);
        const int tile_row = __builtin_amdgcn_ds_permute(4 * to, lane);
        const int v_row = __builtin_amdgcn_ds_permute(4 * to, row_of);
        for (; pair < turn; pair += nw) {
            const int g = 16 * (pair - first);
            const int64_t row = __shfl(v_row, g + c, 64);
            float4_t acc[CB];
#pragma unroll
            for (int f = 0; f < CB; ++f) acc[f] = (float4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int k0 = 0; k0 < rank; k0 += 32) {
                const int k = k0 + 8 * q;
                u32x4 b[CB], hi, low;
#pragma unroll
                for (int f = 0; f < CB; ++f) {
                    const int64_t col = n0 + 16 * f + c;
                    b[f] = lora_b_operand(p, col < p.N, a, col, k, rank);
                }
                lora_v_operand<UNROLL>(p, g + c < n && k < rank, row, k, hi, low);
#pragma unroll
                for (int f = 0; f < CB; ++f) {
                    const bf16x8_t bf = __builtin_bit_cast(bf16x8_t, b[f]);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, hi), bf, acc[f], 0, 0, 0);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, low), bf, acc[f], 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = __shfl(tile_row, g + 4 * q + i, 64);
                if (g + 4 * q + i < n)
#pragma unroll
                    for (int f = 0; f < CB; ++f) delta[r][16 * f + c] = acc[f][i];
            }
        }
    }
}

// K chunks: out = bf16(alpha * (their sum, in order) + adapters), for one tile
// of 64 listed rows and 32 columns.
// (RT threads: 1024 for a batch that is one tile, which can hold up to 64
// adapters; else 256, as listed rows put few adapters into a tile and several
// work-groups share a CU)
template <int RT>
__global__ __launch_bounds__(RT) void lora_reduce_kernel(LoraParams p, int tiles, const float* __restrict__ partial,
                                                         int ksplit, const float* __restrict__ a_gs,
                                                         const float* __restrict__ b_alpha,
                                                         uint16_t* __restrict__ out) {
    constexpr int LD = 36;
    __shared__ __attribute__((aligned(16))) float delta[kLoraRows][LD];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)(blockIdx.x % tiles) * kLoraRows, n0 = (int64_t)(blockIdx.x / tiles) * 32;
    for (int i = tid; i < kLoraRows * LD; i += RT) (&delta[0][0])[i] = 0.0f;
    const bool in = m0 + lane < p.M;
    int id = in ? p.ids[m0 + lane] : -1;
    if (id >= p.L) id = -1;
    const int row_of = in ? (p.perm ? p.perm[m0 + lane] : (int)(m0 + lane)) : -1;
    // each thread: C columns of tile rows tid / (32 / C), + RT C / 32
    constexpr int C = RT == 1024 ? 2 : 4, TPR = 32 / C, NR = kLoraRows * TPR / RT;
    typedef float vec_t __attribute__((ext_vector_type(C)));
    const int col = C * (tid % TPR), r0 = tid / TPR;
    vec_t sum[NR];
    int row[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
        row[t] = __shfl(row_of, r0 + t * (RT / TPR), 64);
        if (n0 + col >= p.N) row[t] = -1;
        if (row[t] >= 0)
            sum[t] = sum_planes<8>(reinterpret_cast<const vec_t*>(partial + (int64_t)row[t] * p.N + n0 + col), ksplit, p.M * p.N / C);
    }
    __syncthreads();
    expand_tile<2, LD, 8>(p, id, row_of, n0, wave, RT / 64, delta);
    __syncthreads();
    const float alpha = a_gs[0] * b_alpha[0];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
        const int r = r0 + t * (RT / TPR);
        if (row[t] < 0) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(out + (int64_t)row[t] * p.N + n0 + col);
#pragma unroll
        for (int e = 0; e < C; e += 2)
            dst[e / 2] = pack_bf16x2_rne(alpha * sum[t][e] + delta[r][col + e], alpha * sum[t][e + 1] + delta[r][col + e + 1]);
    }
}

// ---------------------------------------------------------------------------
// Up to 32 rows: the projection as a weight stream. A work-group owns 16 CB
// columns and all rows; its first nk waves (up to 8) share K in whole groups
// of four 128-element steps, so every wave has a kilobyte per step and column
// block in flight, and nothing of the projection goes through memory again: the
// waves' sums meet in LDS (added in wave order), where the expand's are too.
// The adapters' pairs are dealt from the last wave on: it has no share of K
// (loads return in order: in a wave that streams, the adapters' operands
// arrive after its weights). With two row blocks and all eight waves streaming
// there is none: a ninth would leave them too few registers.
template <int MT> constexpr int kStreamWaves = MT == 1 ? NW + 1 : NW;
template <int MT, int CB>
__global__ __launch_bounds__(64 * kStreamWaves<MT>) __attribute__((amdgpu_waves_per_eu(MT == 1 ? 4 : 2)))
void lora_stream_kernel(LoraParams p, int nk, int per, const uint8_t* __restrict__ aqp,
                                                         const uint8_t* __restrict__ asfp,
                                                         const uint8_t* __restrict__ bq,
                                                         const uint8_t* __restrict__ bsf,
                                                         const float* __restrict__ a_gs,
                                                         const float* __restrict__ b_alpha,
                                                         uint16_t* __restrict__ out) {
    constexpr int LD = 16 * CB + 4;
    __shared__ __attribute__((aligned(16))) float delta[16 * MT][LD];
    __shared__ __attribute__((aligned(16))) float red[NW][16 * MT][LD];
    const int tid = threadIdx.x, lane = tid & 63, nthreads = blockDim.x, nw = nthreads / 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t ldq = pitch_q(p.K), ldwsf = pitch_wsf(p.K);
    const int steps = (int)(ldq / 64), quads = (int)(ldwsf / 32);
    const int64_t blk0 = (int64_t)blockIdx.x * CB;              // 16-column blocks
    const int64_t blocks = p.N / 16;

    struct Group {
        u32x4 w[CB][4], a[MT][4];
        u32x2 ws[CB], as[MT];
    };
    // buffer loads: one lane offset per operand, the rest in scalar offsets
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(bq, p.N * ldq), rws = make_rsrc(bsf, p.N * ldwsf);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(aqp, (int64_t)16 * MT * ldq), ras = make_rsrc(asfp, (int64_t)16 * MT * ldwsf);
    const uint32_t w_off = (q >> 1) * kWqHalf + c * 32 + (q & 1) * 16, sf_off = c * 32 + q * 8, a_off = lane * 16;
    auto load_w = [&](int g, Group& r) {
#pragma unroll
        for (int f = 0; f < CB; ++f) {
            const uint32_t blk = (uint32_t)(blk0 + f < blocks ? blk0 + f : blocks - 1);
            r.ws[f] = __builtin_amdgcn_raw_buffer_load_b64(rws, sf_off, blk * 16 * (uint32_t)ldwsf + (uint32_t)g * kWsfQuad, kStreamNT);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int st = min(4 * g + u, steps - 1);       // beyond the last step the scales are zero
                r.w[f][u] = __builtin_amdgcn_raw_buffer_load_b128(rw, w_off, blk * 16 * (uint32_t)ldq + (uint32_t)st * kWqStep, kStreamNT);
            }
        }
    };
    auto load_a = [&](int g, Group& r) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            r.as[m] = __builtin_amdgcn_raw_buffer_load_b64(ras, sf_off, (uint32_t)(m * quads + g) * 512, 0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int st = min(4 * g + u, steps - 1);
                r.a[m][u] = __builtin_amdgcn_raw_buffer_load_b128(ra, a_off, (uint32_t)(m * steps + st) * 1024, 0);
            }
        }
    };
    float4_t acc[MT][CB];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < CB; ++f) acc[m][f] = (float4_t){0.f, 0.f, 0.f, 0.f};
    // dword s of a step's 16 bytes: K values 32 q + 8 s .. + 7 in both operands,
    // in scale group 2 q + s / 2
    auto compute = [&](const Group& r) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int sh = 16 * (u & 1) + 8 * (s >> 1);
                half8_t ha[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) ha[m] = dequant8(r.a[m][u][s], scale_pair((r.as[m][u >> 1] >> sh) & 0xFFu));
#pragma unroll
                for (int f = 0; f < CB; ++f) {
                    const half8_t hb = dequant8(r.w[f][u][s], scale_pair((r.ws[f][u >> 1] >> sh) & 0xFFu));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ha[m], hb, acc[m][f], 0, 0, 0);
                }
            }
    };
    // two groups in flight (an index past the wave's last group loads it
    // again); A, which every work-group reads, follows from the L2
    const int g0 = wave * per, g1 = min(quads, g0 + per);
    const bool streams = wave < nk;
    int id = lane < p.M ? p.ids[lane] : -1;
    if (id >= p.L) id = -1;
    Group r0, r1;
    if (streams) {
        load_w(g0, r0);
        load_w(min(g0 + 1, g1 - 1), r1);
    }
    __builtin_amdgcn_sched_barrier(0);

    // the adapters while the first weights are on their way
    for (int i = tid; i < 16 * MT * LD; i += nthreads) (&delta[0][0])[i] = 0.0f;
    __syncthreads();
    expand_tile<CB, LD, 4>(p, id, lane, blk0 * 16, nw - 1 - wave, nw, delta);

    if (streams) {
    int g = g0;
    load_a(g0, r0);
    load_a(min(g0 + 1, g1 - 1), r1);
    for (; g + 2 < g1; g += 2) {
        compute(r0);
        load_w(g + 2, r0);
        load_a(g + 2, r0);
        compute(r1);
        load_w(min(g + 3, g1 - 1), r1);
        load_a(min(g + 3, g1 - 1), r1);
    }
    compute(r0);
    if (g + 1 < g1) compute(r1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < CB; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][16 * m + 4 * q + i][16 * f + c] = acc[m][f][i];
    }
    __syncthreads();
    const float alpha = a_gs[0] * b_alpha[0];
    for (int e = tid; e < 16 * MT * 8 * CB; e += nthreads) {
        const int r = e / (8 * CB), n = 2 * (e % (8 * CB));
        const int64_t col = blk0 * 16 + n;
        if (r >= p.M || col >= p.N) continue;
        float s0 = red[0][r][n], s1 = red[0][r][n + 1];
        for (int w = 1; w < nk; ++w) {
            s0 += red[w][r][n];
            s1 += red[w][r][n + 1];
        }
        *reinterpret_cast<uint32_t*>(out + (int64_t)r * p.N + col) =
            pack_bf16x2_rne(alpha * s0 + delta[r][n], alpha * s1 + delta[r][n + 1]);
    }
}

template <int MT, int CB>
hipError_t launch_stream(const LoraParams& p, const uint8_t* aqp, const uint8_t* asfp, const uint8_t* bq,
                         const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out, hipStream_t s) {
    const int quads = (int)(pitch_wsf(p.K) / 32), per = (quads + NW - 1) / NW, nk = (quads + per - 1) / per;
    const int64_t grid = (p.N / 16 + CB - 1) / CB;
    // waves beside the streaming ones: one, or what is left of eight
    const int nw = nk < NW ? NW : kStreamWaves<MT>;
    lora_stream_kernel<MT, CB><<<(unsigned)grid, 64 * nw, 0, s>>>(p, nk, per, aqp, asfp, bq, bsf, a_gs, b_alpha, out);
    return hipGetLastError();
}

}  // namespace

// Work-groups of the shrink before K is split: tiles x the adapters a tile can
// hold x rank blocks; K ranges (at most 8, each at least 8 blocks of 64, one
// per wave) bring the launch to about one work-group per CU. Listed tiles hold
// few adapters, which the host cannot know; counting one per tile is right for
// runs of rows and only costs partial sums where there are more.
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

hipError_t launch_lora_sort(const int32_t* ids, int64_t M, int64_t L, int32_t* perm, int32_t* sid, hipStream_t s) {
    lora_sort_kernel<<<1, ST, 0, s>>>(ids, (int)M, (int)L, perm, sid);
    return hipGetLastError();
}

hipError_t launch_lora_shrink(const LoraParams& p, LoraOrder order, int32_t* perm, int32_t* sid, const uint8_t* aq,
                              const uint8_t* asf, uint8_t* aqp, uint8_t* asfp, uint16_t* ah, hipStream_t s) {
    const int64_t tiles = (p.M + kLoraRows - 1) / kLoraRows, rbs = (p.R + kRankBlock - 1) / kRankBlock;
    // work-groups that share a tile's adapters: as many as it can hold when it
    // is the only tile; listed rows put few adapters into a tile
    int64_t slots = p.M < p.L ? p.M : p.L;
    if (order != kLoraAsIs && slots > 4) slots = 4;
    const int64_t blocks = tiles * slots * p.planes * rbs;
    const int64_t more = aqp  ? (lora_stream_aq_bytes(p.M, p.K) / 16 + lora_stream_asf_bytes(p.M, p.K) / 8 + NT - 1) / NT
                         : ah ? (p.M * (p.K / 16) + 4 * NT - 1) / (4 * NT)
                              : 0;
    lora_shrink_kernel<<<(unsigned)(blocks + more), NT, 0, s>>>(p, (int)tiles, (int)slots, (int)blocks,
                                                               order == kLoraRank, perm, sid, aq, asf, aqp, asfp,
                                                               reinterpret_cast<uint8_t*>(ah));
    return hipGetLastError();
}

hipError_t launch_lora_join(const LoraParams& p, const uint8_t* aq, const uint8_t* asf, uint16_t* ah, hipStream_t s) {
    const int64_t join = (p.M * (p.R / 8) + 255) / 256;
    int64_t more = (p.M * (p.K / 16) + 1023) / 1024;
    if (more > 4096) more = 4096;
    lora_join_kernel<<<(unsigned)(join + more), 256, 0, s>>>(p, (int)join, aq, asf, reinterpret_cast<uint8_t*>(ah));
    return hipGetLastError();
}

hipError_t launch_lora_reduce(const LoraParams& p, const float* partial, int ksplit, const float* a_gs,
                              const float* b_alpha, uint16_t* out, hipStream_t s) {
    const int64_t tiles = (p.M + kLoraRows - 1) / kLoraRows;
    const unsigned grid = (unsigned)(tiles * ((p.N + 31) / 32));
    if (tiles == 1)
        lora_reduce_kernel<1024><<<grid, 1024, 0, s>>>(p, 1, partial, ksplit, a_gs, b_alpha, out);
    else
        lora_reduce_kernel<256><<<grid, 256, 0, s>>>(p, (int)tiles, partial, ksplit, a_gs, b_alpha, out);
    return hipGetLastError();
}

hipError_t launch_lora_stream(const LoraParams& p, const uint8_t* aqp, const uint8_t* asfp, const uint8_t* bq,
                              const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out,
                              hipStream_t s) {
    if (p.M <= 16) return launch_stream<1, 1>(p, aqp, asfp, bq, bsf, a_gs, b_alpha, out, s);
    return launch_stream<2, 2>(p, aqp, asfp, bq, bsf, a_gs, b_alpha, out, s);
}

}  // namespace nvfp4
