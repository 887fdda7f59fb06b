// Low-rank adapters of many requests beside one shared NVFP4 projection:
//   out[m] = bf16(alpha * A[m] W + scale[a] (x[m] A_a^T) B_a^T),  a = ids[m]
// with A_a (R, K) and B_a (N, R) in bf16. The product with A_a ("shrink") gives
// v[m] = scale[a] x[m] A_a^T in float32; the product with B_a ("expand") is added
// to the projection before its one rounding. Per batch size:
//   up to 4 rows of small adapters (lora_is_token)
//                   everything in one launch
//   up to 64 rows, and up to 512 of narrow projections (lora_streams)
//                   shrink (beside it A laid out for streaming), then one kernel
//                   that streams the weights and adds the adapters
//   else            the rows are listed by adapter, shrink (beside it A's f16
//                   form), the tiled GEMM; the expand is in its epilogue, or,
//                   where K is cut into chunks, in the kernel that adds them
// A row's arithmetic does not depend on its place in a tile or on the other
// rows, so results depend neither on scheduling nor on the grouping.
//
// Shrink. What has to move is x once and each adapter's A_a once; the
// arithmetic is small, so the split is made for bytes in flight. A work-group
// takes one tile of 64 (listed) rows, one adapter that occurs in it and one
// range of K, and gathers the rows that have the adapter, so an adapter is read
// once per tile however its rows are scattered. x and A_a go to LDS by loads
// that write it directly, in a ring of stages of 64 K values (128 bytes of 64
// rows each), and from there to v_mfma_f32_16x16x32_bf16: reading the operands'
// fragments straight from memory has every lane in another row than its
// neighbours, 16 bytes an address, and ran at a quarter of the rate. Ranges of
// K are separate partial sums, added in order by the reader.
//
// What it measured (medians of a kernel trace; N 6144, K 7168; beside it the
// projection alone):
//   1 row,     L 8,  R 16   one launch, 14.8 us (see there); shrink and stream
//                           were 6.5 and 9.5
//   13 rows of 7168 x 2048, L 16, R 64   shrink 5.9, stream 10: latency
//   61 rows,   L 32, R 32   shrink 8.4 (15 MB of adapters, x and A), stream 19
//                           (25 MB of weights; their conversion and that of
//                           four row blocks of A: the vector units are active
//                           half the cycles, the matrix pipes a fifth, and 64
//                           CUs have no columns)
//   256 rows,  L 6,  R 16   shrink 9.4, tiled GEMM 27.5, chunks' sum and expand
//                           10.5 (nvfp4_gemm: 3.3, 27.8 and 6.3)
//   4093 rows, L 8,  R 64   sort 7, shrink 35 (59 MB of x and 16 MB of A read, 59
//                           MB of f16 written), join 5, GEMM with the expand 320
//                           (without it 297): the matrix cores
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int NT = 512;
constexpr int NW = NT / 64;
constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kBeyond = 0x80000000u;      // an offset outside every buffer: reads zeros
constexpr int kStreamNT = 2;        // buffer-load cache policy: non-temporal (read once)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, kRsrcWord3);
}

constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }
typedef __attribute__((address_space(3))) void lds_void;

// Work-group barrier for data in LDS: unlike __syncthreads() it does not wait
// for global loads and stores in flight.
__device__ __forceinline__ void lds_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

constexpr int kShrinkStage = 2 * 64 * 128;      // 64 rows of x and of A_a, 64 K values
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

// For the fused epilogue: the shrunk rows' partial sums joined into vs.
__global__ __launch_bounds__(256) void lora_join_kernel(LoraParams p) {
    const int R8 = p.R / 8;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, pos = t / R8;
    const int k = 8 * (int)(t - pos * R8);
    if (pos >= p.M || p.ids[pos] < 0) return;
    u32x4 hi, low;
    lora_v_operand(p, p.perm[pos], k, hi, low);
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

// NS stages, STEP of them between two barriers: 4 and 1 where two work-groups
// share a CU, 8 and 2 for small batches, which are bound by the time of a step
template <int NS, int STEP>
__global__ __launch_bounds__(NT) void lora_shrink_kernel(LoraParams p, int tiles, int rbs, int slots, int shrink_blocks,
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
    constexpr int TR = kLoraRows;
    extern __shared__ __attribute__((aligned(16))) uint8_t ring[];
    __shared__ int list[TR];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    // (the slots, which may have nothing to do, are the last work-groups)
    // Work-groups go to the eight XCDs in turn: each gets neighbouring tiles,
    // which mostly have the same adapter, so that its L2 serves it to them.
    const int rest = blockIdx.x / tiles, turn = blockIdx.x % tiles;
    const int per_xcd = tiles / 8, full = per_xcd * 8;
    const int tile = turn < full ? turn % 8 * per_xcd + turn / 8 : turn;
    const int plane = rest % p.planes, rb = rest / p.planes % rbs, slot = rest / (p.planes * rbs);
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
        // (two threads a row, each half of the keys; one took 1.5 us longer at 256
        // rows)
        static_assert(NT == 2 * kLoraRankRows, "two threads a row");
        __shared__ __attribute__((aligned(16))) int key[kLoraRankRows];
        __shared__ int below[kLoraRankRows], order[kLoraRankRows];
        const int r = tid % kLoraRankRows, part = tid / kLoraRankRows;
        int mine = 0x7FFFFFFF;
        if (r < M) {
            const int a = p.ids[r];
            mine = (a >= 0 && a < L ? a : L) * kLoraRankRows + r;
        }
        if (part == 0) key[r] = mine;
        lds_sync();
        int pos = 0;
        const int half = (int)((M + 7) / 8 * 4), j1 = part ? (int)M : half;
#pragma unroll 8
        for (int j = part * half; j < j1; j += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(key + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) pos += (int)k[e] < mine;
        }
        if (part == 0) below[r] = pos;
        lds_sync();
        if (part == 1 && r < M) order[pos + below[r]] = mine;
        lds_sync();
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
    // (by lane too: a scalar load of an adapter's would be waited for with the LDS)
    const float my_scale = id >= 0 ? p.scale[id] : 0.0f;
    const int my_rank = p.rank && id >= 0 ? min(max(p.rank[id], 0), R) : R;
    // blocks of 64 K values of this plane
    const int nb = (int)((K + 63) / 64), per = (nb + planes - 1) / planes;
    const int b0 = plane * per, b1 = min(nb, b0 + per);

    // the tile's adapters in order of first appearance: this work-group takes
    // numbers slot, slot + slots, ...
    for (int d = 0; todo; ++d) {
        const int lead = __builtin_ctzll(todo);
        const int a = __builtin_amdgcn_readlane(id, lead);
        const uint64_t rows = __builtin_amdgcn_ballot_w64(id == a);
        todo &= ~rows;
        if (d % slots != slot) continue;
        const int rk = __builtin_amdgcn_readlane(my_rank, lead);
        const int n = __builtin_popcountll(rows);
        lds_sync();                             // the previous adapter's readers are done
        if (wave == 0 && id == a) {
            const int at = __builtin_popcountll(rows & ((1ull << lane) - 1));
            list[at] = row_of;
        }
        lds_sync();

        // loads into LDS: wave w brings rows 8 w .. + 7 of x and of A_a of each
        // stage; lane l's 16 bytes are chunk l % 8 of row l / 8, stored swizzled
        // (chunk c of row r at c ^ ((r >> 1) & 7), so that the 16 rows of a
        // fragment read cover all banks). Rows, ranks and K values that are not
        // there have offsets beyond the buffers and read zeros (x is below 2 GiB,
        // as M * pitch_h(K) is).
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, M * K * 2), ra = make_rsrc(p.a + (int64_t)a * R * K, (int64_t)R * K * 2);
        const int cols = min(max(rk - rbase, 0), kRankBlock);
        const int lr = 8 * wave + (lane >> 3), ch = (lane & 7) ^ ((lr >> 1) & 7);
        const uint32_t x_off = lr < n ? (uint32_t)(((int64_t)list[lr] * K + 8 * ch) * 2) : kBeyond;
        const uint32_t a_off = lr < cols ? (uint32_t)(((int64_t)(rbase + lr) * K + 8 * ch) * 2) : kBeyond;
        auto issue = [&](int b) {                    // b past the range: zeros
            const uint32_t k = (uint32_t)b * 64;
            const uint32_t out = b < b1 && k + 8 * ch < (uint32_t)K ? 0u : kBeyond;
            uint8_t* at = ring + (b - b0) % NS * kShrinkStage + wave * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)at, 16, x_off | out, 2 * k, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(at + kShrinkStage / 2), 16, a_off | out, 2 * k, 0, 0);
        };
        // wave w: rows 16 (w % 4) .. + 15, ranks 32 (w / 4) .. + 31
        const int g = wave & 3, rh = wave >> 2;
        const bool busy = 16 * g < n && 32 * rh < cols;
        float4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const uint32_t sw = 16 * ((c >> 1) & 7);
        const uint32_t fx = (16 * g + c) * 128, fa = kShrinkStage / 2 + (32 * rh + c) * 128;
#pragma unroll
        for (int t = 0; t < NS - STEP; ++t) issue(b0 + t);
        for (int b = b0; b < b1; b += STEP) {
            // this wave's loads of the step's blocks are done when only later
            // ones are outstanding; after the barrier everyone's are, and the
            // blocks of the step before have been read by everyone: their stages
            // are refilled
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * (NS - 2 * STEP), 0));
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int t = 0; t < STEP; ++t) issue(b + NS - STEP + t);
            if (busy) {
#pragma unroll
                for (int t = 0; t < 2 * STEP; ++t) {
                    const uint8_t* st = ring + (b + t / 2 - b0) % NS * kShrinkStage;
                    const uint32_t at = (64 * (t & 1) + 16 * q) ^ sw;
                    const bf16x8_t vx = *reinterpret_cast<const bf16x8_t*>(st + fx + at);
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            vx, *reinterpret_cast<const bf16x8_t*>(st + fa + f * 2048 + at), acc[f], 0, 0, 0);
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));      // no load into LDS outlives its adapter
        const float sc = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_scale), lead));
        // acc[f][i] = D[gathered row 16 g + 4 q + i][rank 32 rh + 16 f + c]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * g + 4 * q + i;
            if (r >= n) continue;
            float* dst = p.v + ((int64_t)plane * M + list[r]) * R + rbase;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int col = 32 * rh + 16 * f + c;
                if (rbase + col < R) dst[col] = col < cols ? sc * acc[f][i] : 0.0f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Rows by adapter. One work-group counts, scans and places, about 1 us per thousand
// rows (7 us at 4093, 14 to 17 at 16384, 120 to 130 at 131072); the rows of one adapter come in no particular order (a
// row's result does not depend on its place). Where at least 16 lanes of a wave share an adapter, as in runs of
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
// rows and 16 CB columns from n0, in two parts.
//
// join_v: nthreads threads join the rows' partial sums of v into LDS as bf16
// hi + low (rows of 2 R values, lds_v_pitch(R) apart; row(r) < 0: none). v is
// read in order; a fragment of v straight from memory has every lane in
// another row than its neighbours, one address each.
__host__ __device__ inline int lds_v_pitch(int R) { return 2 * R + 8; }      // 16 bytes of skew between rows

template <typename F>
__device__ __forceinline__ void join_v(const LoraParams& p, int nrows, F row_of, int thread, int nthreads,
                                       uint16_t* __restrict__ lv) {
    const int R8 = p.R / 8, pitch = lds_v_pitch(p.R);
    for (int e = thread; e < nrows * R8; e += nthreads) {
        const int r = e / R8, k = 8 * (e - r * R8), row = row_of(r);
        if (row < 0) continue;
        u32x4 hi, low;
        lora_v_operand(p, row, k, hi, low);
        *reinterpret_cast<u32x4*>(lv + r * pitch + k) = hi;
        *reinterpret_cast<u32x4*>(lv + r * pitch + p.R + k) = low;
    }
}

// Expand: the tile's (adapter, 16 of its rows) pairs are dealt to nw waves (a
// row has one adapter, so one wave writes it; the caller has zeroed delta); a
// wave goes through its pairs 32 ranks at a time, with B_a of the next AHEAD
// steps on its way. The constructor asks for the first ones, run() (when lv is
// complete) does the work. `lane`'s row of the tile has adapter id (-1: none).
template <int CB, int LD>
struct Expand {
    static constexpr int AHEAD = 3;
    struct Step {
        bool on, first, last;           // a step; of its pair the first, the last
        int n, g, k0, rank, tile_row;
        u32x4 b[CB];
    };
    const LoraParams& p;
    const int64_t n0;
    const int id, wave, nw, lane, c, q;
    const int my_rank;                  // of the lane's row's adapter
    uint64_t todo, rows = 0;            // rows not looked at, rows of the adapter at hand
    int a = 0, rank = 0, n = 0;
    int turn = 0, first = 0, pair;      // pairs seen, the adapter's first one, this wave's
    int tile_row = 0, k0 = 0;
    bool fresh = true;                  // the next step starts a pair
    Step st[AHEAD + 1];

    __device__ __forceinline__ Expand(const LoraParams& p_, int id_, int64_t n0_, int wave_, int nw_)
        : p(p_), n0(n0_), id(id_), wave(wave_), nw(nw_), lane(threadIdx.x & 63), c(lane & 15), q(lane >> 4),
          my_rank(p_.rank && id_ >= 0 ? min(max(p_.rank[id_], 0), p_.R) : p_.R),
          todo(__builtin_amdgcn_ballot_w64(id_ >= 0)), pair(wave_ - nw_) {
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) next(st[t]);
    }
    __device__ __forceinline__ void next(Step& t) {
        t.first = fresh;
        if (fresh) {
            k0 = 0;
            pair += nw;
            while (pair >= turn && todo) {
                const int lead = __builtin_ctzll(todo);
                a = __builtin_amdgcn_readlane(id, lead);
                rank = __builtin_amdgcn_readlane(my_rank, lead);
                rows = __builtin_amdgcn_ballot_w64(id == a);
                todo &= ~rows;
                n = __builtin_popcountll(rows);
                first = turn;
                turn += (n + 15) / 16;
                if (pair < turn) {
                    // lane i receives the adapter's i-th row: the lanes that
                    // have it push theirs to 0 .. n - 1, the others to the rest
                    const uint64_t below = (1ull << lane) - 1;
                    const int to = id == a ? __builtin_popcountll(rows & below) : n + __builtin_popcountll(~rows & below);
                    tile_row = __builtin_amdgcn_ds_permute(4 * to, lane);
                }
            }
        } else {
            k0 += 32;
        }
        t.on = pair < turn;
        if (t.on) {
            t.last = fresh = k0 + 32 >= rank;
            t.n = n;
            t.g = 16 * (pair - first);
            t.k0 = k0;
            t.rank = rank;
            t.tile_row = tile_row;
        }
        // (buffer loads without a branch, so that the compiler's waits leave the
        // later steps' in flight: what is not there lies beyond the buffer)
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + ((int64_t)a * p.N + n0) * p.R, min((int64_t)16 * CB, p.N - n0) * p.R * 2);
        const int k = k0 + 8 * q;
#pragma unroll
        for (int f = 0; f < CB; ++f)
            t.b[f] = __builtin_amdgcn_raw_buffer_load_b128(
                rb, t.on && k < rank ? (uint32_t)((16 * f + c) * p.R + k) * 2 : kBeyond, 0, 0);
    }
    __device__ __forceinline__ void work(const Step& t, float4_t (&acc)[CB], const uint16_t* __restrict__ lv,
                                         float (*delta)[LD]) {
        if (t.first)
#pragma unroll
            for (int f = 0; f < CB; ++f) acc[f] = (float4_t){0.f, 0.f, 0.f, 0.f};
        const uint16_t* vr = lv + __shfl(t.tile_row, t.g + c, 64) * lds_v_pitch(p.R) + t.k0 + 8 * q;
        u32x4 hi = {0u, 0u, 0u, 0u}, low = {0u, 0u, 0u, 0u};
        if (t.g + c < t.n && t.k0 + 8 * q < t.rank) {
            hi = *reinterpret_cast<const u32x4*>(vr);
            low = *reinterpret_cast<const u32x4*>(vr + p.R);
        }
#pragma unroll
        for (int f = 0; f < CB; ++f) {
            u32x4 b = t.b[f];
            if (t.rank & 7) b = lora_mask_rank(b, t.k0 + 8 * q, t.rank);
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, hi),
                                                             __builtin_bit_cast(bf16x8_t, b), acc[f], 0, 0, 0);
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, low),
                                                             __builtin_bit_cast(bf16x8_t, lora_finite(b)), acc[f], 0, 0, 0);
        }
        if (!t.last) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = __shfl(t.tile_row, (t.g + 4 * q + i) & 63, 64);
            if (t.g + 4 * q + i < t.n)
#pragma unroll
                for (int f = 0; f < CB; ++f) delta[r][16 * f + c] = acc[f][i];
        }
    }
    __device__ __forceinline__ void run(const uint16_t* __restrict__ lv, float (*delta)[LD]) {
        float4_t acc[CB];
        while (true) {
#pragma unroll
            for (int t = 0; t <= AHEAD; ++t) {
                if (!st[t].on) return;
                next(st[(t + AHEAD) % (AHEAD + 1)]);
                work(st[t], acc, lv, delta);
            }
        }
    }
};

// K chunks: out = bf16(alpha * (their sum, in order) + adapters), for one tile
// of 64 listed rows and 32 columns. 10.5 us at 256 x 6144 and 5 chunks (31 MB of
// sums, held by the caches; the sum alone takes 6.6).
constexpr int RT = 256;
__global__ __launch_bounds__(RT) void lora_reduce_kernel(LoraParams p, int tiles, const float* __restrict__ partial,
                                                         int ksplit, const float* __restrict__ a_gs,
                                                         const float* __restrict__ b_alpha,
                                                         uint16_t* __restrict__ out) {
    constexpr int LD = 36;
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    uint16_t* lv = reinterpret_cast<uint16_t*>(dyn);
    __shared__ __attribute__((aligned(16))) float delta[kLoraRows][LD];
    __shared__ int rows[kLoraRows];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)(blockIdx.x % tiles) * kLoraRows, n0 = (int64_t)(blockIdx.x / tiles) * 32;
    const bool in = m0 + lane < p.M;
    const int id = in ? p.ids[m0 + lane] : -1;
    const int row_of = in ? p.perm[m0 + lane] : -1;
    if (wave == 0) rows[lane] = id >= 0 ? row_of : -1;
    for (int i = tid; i < kLoraRows * LD; i += RT) (&delta[0][0])[i] = 0.0f;
    lds_sync();
    // each thread: four columns of tile rows tid / 8 and tid / 8 + 32
    const int col = 4 * (tid & 7);
    int row[2];
    const float4_t* src[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        row[t] = __shfl(row_of, (tid >> 3) + 32 * t, 64);
        if (n0 + col >= p.N) row[t] = -1;
        src[t] = reinterpret_cast<const float4_t*>(row[t] >= 0 ? partial + (int64_t)row[t] * p.N + n0 + col : partial);
    }
    Expand<2, LD> expand(p, id, n0, wave, RT / 64);
    join_v(p, kLoraRows, [&](int r) { return rows[r]; }, tid, RT, lv);
    // the first chunks' sums arrive under the expand (loaded without a branch:
    // what is not there is chunk 0 again); before v they would hold it up
    constexpr int PL = 6;
    const int64_t plane = p.M * p.N / 4;
    float4_t part[2][PL];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < PL; ++k) part[t][k] = src[t][k < ksplit ? k * plane : 0];
    lds_sync();
    expand.run(lv, delta);
    float4_t sum[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        sum[t] = part[t][0];
#pragma unroll
        for (int k = 1; k < PL; ++k)
            if (k < ksplit) sum[t] += part[t][k];
        sum[t] = add_planes<8>(sum[t], src[t] + PL * plane, ksplit - PL, plane);
    }
    lds_sync();
    const float alpha = a_gs[0] * b_alpha[0];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (row[t] < 0) continue;
        const float* d = &delta[(tid >> 3) + 32 * t][col];
        *reinterpret_cast<u32x2*>(out + (int64_t)row[t] * p.N + n0 + col) =
            (u32x2){pack_bf16x2_rne(alpha * sum[t][0] + d[0], alpha * sum[t][1] + d[1]),
                    pack_bf16x2_rne(alpha * sum[t][2] + d[2], alpha * sum[t][3] + d[3])};
    }
}

// ---------------------------------------------------------------------------
// The projection as a weight stream. A work-group owns 16 CB columns and 16 MT
// rows (all of them up to 64; more are parts of 64 rows); its first nk waves share K in whole groups of four
// 128-element steps, so every wave has a kilobyte per step and column block in
// flight, and nothing of the projection goes through memory again: the waves'
// sums meet in LDS (added in wave order), where the expand's are too. The other
// waves do the expand meanwhile (loads return in order: in a wave that streams,
// the adapters' operands would arrive after its weights). 9.5 us for one row of
// 6144 x 7168 (24.8 MB of weights: 2.6 TB/s, most of it start and end), 19 us
// for 61 rows; the tiled form with its two further kernels took 49 us there.
template <int MT, int CB>
__global__ __launch_bounds__(MT == 4 ? NT + 256 : NT) __attribute__((amdgpu_waves_per_eu(MT == 1 ? 4 : MT == 4 ? 3 : 2)))
void lora_stream_kernel(LoraParams p, int parts, int nk, int per, const uint8_t* __restrict__ aqp,
                        const uint8_t* __restrict__ asfp, const uint8_t* __restrict__ bq,
                        const uint8_t* __restrict__ bsf, const float* __restrict__ a_gs,
                        const float* __restrict__ b_alpha, uint16_t* __restrict__ out) {
    constexpr int LD = 16 * CB + 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    float (*delta)[LD] = reinterpret_cast<float (*)[LD]>(dyn);                       // [16 MT]
    float (*red)[16 * MT][LD] = reinterpret_cast<float (*)[16 * MT][LD]>(dyn + 16 * MT * LD * 4);   // [nk]
    uint16_t* lv = reinterpret_cast<uint16_t*>(dyn + (1 + nk) * 16 * MT * LD * 4);
    const int tid = threadIdx.x, lane = tid & 63, nthreads = blockDim.x, nw = nthreads / 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t ldq = pitch_q(p.K), ldwsf = pitch_wsf(p.K);
    const int steps = (int)(ldq / 64), quads = (int)(ldwsf / 32);
    const int64_t blocks = p.N / 16;                            // 16-column blocks
    // the row parts of one column range follow each other on one XCD, whose L2
    // serves its weights to the second
    const int64_t blk0 = (int64_t)(blockIdx.x / (8 * parts) * 8 + blockIdx.x % 8) * CB;
    if (blk0 >= blocks) return;
    const int blk_a = (int)(blockIdx.x / 8 % parts) * MT;       // its first 16-row block
    const int row0 = 16 * blk_a, rows = min(16 * MT, (int)p.M - row0);

    struct Group {
        u32x4 w[CB][4];
        u32x2 ws[CB];
    };
    struct Half {                       // A of two of the group's steps
        u32x4 a[MT][2];
        uint32_t as[MT];
    };
    // buffer loads: one lane offset per operand, the rest in scalar offsets
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(bq, p.N * ldq), rws = make_rsrc(bsf, p.N * ldwsf);
    // (A has the row blocks that M has rows for; one further on, whose rows are
    // not used, is the last of them again)
    const int last = (int)((p.M - 1) / 16);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(aqp, (int64_t)16 * (last + 1) * ldq);
    const __amdgpu_buffer_rsrc_t ras = make_rsrc(asfp, (int64_t)16 * (last + 1) * ldwsf);
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
    auto load_a = [&](int g, int half, Half& r) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int mb = min(blk_a + m, last);
            r.as[m] = __builtin_amdgcn_raw_buffer_load_b32(ras, sf_off, (uint32_t)(mb * quads + g) * 512 + 4 * half, 0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int st = min(4 * g + 2 * half + u, steps - 1);
                r.a[m][u] = __builtin_amdgcn_raw_buffer_load_b128(ra, a_off, (uint32_t)(mb * steps + st) * 1024, 0);
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
    auto compute = [&](const Group& r, int half, const Half& x) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int sh = 16 * u + 8 * (s >> 1);
                half8_t ha[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) ha[m] = dequant8(x.a[m][u][s], scale_pair((x.as[m] >> sh) & 0xFFu));
#pragma unroll
                for (int f = 0; f < CB; ++f) {
                    const half8_t hb = dequant8(r.w[f][2 * half + u][s], scale_pair((r.ws[f][half] >> sh) & 0xFFu));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ha[m], hb, acc[m][f], 0, 0, 0);
                }
            }
    };
    // two groups of weights in flight; A, which every work-group reads, comes
    // from the L2
    const int g0 = wave * per, g1 = min(quads, g0 + per);
    // the expanding waves wait for each other on a counter in LDS (all waves of
    // a work-group run at the same time): a barrier would hold up the streams
    __shared__ int joined;
    if (tid == 0) joined = 0;
    lds_sync();
    if (wave < nk) {
        // (an index past the wave's last group loads it again)
        Group r0, r1;
        load_w(g0, r0);
        load_w(min(g0 + 1, g1 - 1), r1);
        // A of half a group at a time; with four row blocks three waves on a SIMD
        // hide its latency, and there are registers for one of them only
        constexpr int AB = MT == 4 ? 1 : 2;
        Half x[AB];
#pragma unroll
        for (int t = 0; t < AB; ++t) load_a(g0, t, x[t]);
        int g = g0;
        auto group = [&](const Group& r) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                compute(r, t, x[t % AB]);
                load_a(t + AB >= 2 ? min(g + 1, g1 - 1) : g, (t + AB) % 2, x[t % AB]);
            }
            ++g;
        };
        while (true) {
            group(r0);
            if (g >= g1) break;
            load_w(min(g + 1, g1 - 1), r0);
            group(r1);
            if (g >= g1) break;
            load_w(min(g + 1, g1 - 1), r1);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int f = 0; f < CB; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[wave][16 * m + 4 * q + i][16 * f + c] = acc[m][f][i];
    } else {
        // the few instructions of the expand go ahead of the streams' many
        __builtin_amdgcn_s_setprio(3);
        const int t = tid - 64 * nk, nt = 64 * (nw - nk);
        int id = lane < rows ? p.ids[row0 + lane] : -1;
        if (id >= p.L) id = -1;
        Expand<CB, LD> expand(p, id, blk0 * 16, wave - nk, nw - nk);
        // (rows without an adapter have no v: what is joined for them is not used)
        join_v(p, rows, [&](int r) { return row0 + r; }, t, nt, lv);
        for (int i = t; i < 16 * MT * LD; i += nt) (&delta[0][0])[i] = 0.0f;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
        if (lane == 0) __hip_atomic_fetch_add(&joined, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        while (__hip_atomic_load(&joined, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) < nw - nk) __builtin_amdgcn_s_sleep(1);
        asm volatile("" ::: "memory");
        expand.run(lv, delta);
    }
    lds_sync();
    const float alpha = a_gs[0] * b_alpha[0];
    for (int e = tid; e < 16 * MT * 8 * CB; e += nthreads) {
        const int r = e / (8 * CB), n = 2 * (e % (8 * CB));
        const int64_t col = blk0 * 16 + n;
        if (r >= rows || col >= p.N) continue;
        float s0 = red[0][r][n], s1 = red[0][r][n + 1];
        for (int w = 1; w < nk; ++w) {
            s0 += red[w][r][n];
            s1 += red[w][r][n + 1];
        }
        *reinterpret_cast<uint32_t*>(out + (int64_t)(row0 + r) * p.N + col) =
            pack_bf16x2_rne(alpha * s0 + delta[r][n], alpha * s1 + delta[r][n + 1]);
    }
}

// ---------------------------------------------------------------------------
// A few rows and small adapters (lora_is_token): everything in one launch. The
// weights are streamed as above by the first nk waves, with A laid out in LDS;
// the other eight waves of every work-group compute all of v again (M R K
// products, read from the L2: less than what a second launch and the trip of v
// through memory cost) while the weights arrive, and add the adapters.
// v = x A_a^T by rows: four ranks and one range of K per wave and turn, lanes
// along K, so that loads are whole rows; float32 sums, v is not rounded.
// One row of 6144 x 7168, R 16: 14 us. A is in LDS after 3.2, v known after 7.2,
// the first weights (which share the CU's loads with 230 KB of A_a and 60 KB of
// x) at 8.5, the last product at 11.
constexpr int kTokenWaves = 8;
constexpr int kTokenAhead = 4;      // B_a: chunks of 8 ranks loaded before v is known

// K ranges of v's sums: as many as keep the eight waves busy
__host__ __device__ inline int token_ranges(int M, int R) {
    const int groups = M * R / 4;
    return groups >= kTokenWaves ? 1 : kTokenWaves / groups;
}

template <int CB>
__global__ __launch_bounds__(2 * NT) __attribute__((amdgpu_waves_per_eu(4)))
void lora_token_kernel(LoraParams p, int nk, int per, const uint8_t* __restrict__ aq, const uint8_t* __restrict__ asf,
                       const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bsf,
                       const float* __restrict__ a_gs, const float* __restrict__ b_alpha, uint16_t* __restrict__ out) {
    constexpr int LD = 16 * CB + 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int M = (int)p.M, R = p.R, K = (int)p.K;
    const int ldq = (int)pitch_q(K), ldwsf = (int)pitch_wsf(K);
    const int steps = ldq / 64, quads = ldwsf / 32, ranges = token_ranges(M, R);
    uint8_t* la = dyn;                                                      // A: rows of ldq bytes, then their
    uint8_t* ls = la + M * ldq;                                             // scales in the weights' order
    float* lv = reinterpret_cast<float*>(ls + M * ldwsf);                   // v: [ranges][M][R]
    float (*red)[kLoraTokenRows][LD] = reinterpret_cast<float (*)[kLoraTokenRows][LD]>(lv + ranges * M * R);    // [nk]
    const int64_t blocks = p.N / 16, blk0 = (int64_t)blockIdx.x * CB;       // 16-column blocks

    if (wave < nk) {
        struct Group {
            u32x4 w[CB][4];
            u32x2 ws[CB];
        };
        const int g0 = wave * per, g1 = min(quads, g0 + per);
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(bq, p.N * ldq), rws = make_rsrc(bsf, p.N * ldwsf);
        const uint32_t w_off = (q >> 1) * kWqHalf + c * 32 + (q & 1) * 16, sf_off = c * 32 + q * 8;
        auto load_w = [&](int g, Group& r) {
            const bool on = g < g1;          // else zeros, and nothing is read
            if (!on) g = 0;
#pragma unroll
            for (int f = 0; f < CB; ++f) {
                const uint32_t blk = (uint32_t)(blk0 + f < blocks ? blk0 + f : blocks - 1);
                r.ws[f] = __builtin_amdgcn_raw_buffer_load_b64(rws, on ? sf_off : kBeyond, blk * 16 * (uint32_t)ldwsf + (uint32_t)g * kWsfQuad, kStreamNT);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int st = min(4 * g + u, steps - 1);       // beyond the last step the scales are zero
                    r.w[f][u] = __builtin_amdgcn_raw_buffer_load_b128(rw, on ? w_off : kBeyond, blk * 16 * (uint32_t)ldq + (uint32_t)st * kWqStep, kStreamNT);
                }
            }
        };
        // A's groups of 16, zero beyond K: thread by thread, its loads before the
        // weights' (loads return in order)
        const int nt = 64 * nk, per_row = quads * 32;
        constexpr int AHEAD = 4;
        auto stage = [&](int i0, bool first, Group* r0, Group* r1, int g0, int g1) {
            u32x2 a[AHEAD];
            uint32_t sf[AHEAD];
            const __amdgpu_buffer_rsrc_t ra = make_rsrc(aq, (int64_t)M * K / 2), rs = make_rsrc(asf, (int64_t)M * K / 16);
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) {
                const int i = i0 + t * nt, row = i / per_row, g = i - row * per_row;
                const bool on = row < M && 16 * g < K;
                a[t] = __builtin_amdgcn_raw_buffer_load_b64(ra, on ? (uint32_t)(row * (K / 2) + 8 * g) : kBeyond, 0, 0);
                sf[t] = __builtin_amdgcn_raw_buffer_load_b8(rs, on ? (uint32_t)(row * (K / 16) + g) : kBeyond, 0, 0);
            }
            if (first) {
                load_w(g0, *r0);
                load_w(g1, *r1);
            }
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) {
                const int i = i0 + t * nt, row = i / per_row, g = i - row * per_row;
                if (row >= M) continue;
                if (8 * g < ldq) *reinterpret_cast<u32x2*>(la + row * ldq + 8 * g) = a[t];
                ls[row * ldwsf + (g >> 5) * 32 + ((g >> 1) & 3) * 8 + ((g >> 3) & 3) * 2 + (g & 1)] = (uint8_t)sf[t];
            }
        };
        Group r0, r1;
        stage(tid, true, &r0, &r1, g0, g0 + 1);
        for (int i = tid + AHEAD * nt; i < M * per_row; i += AHEAD * nt) stage(i, false, nullptr, nullptr, 0, 0);
        lds_sync();
        float4_t acc[CB];
#pragma unroll
        for (int f = 0; f < CB; ++f) acc[f] = (float4_t){0.f, 0.f, 0.f, 0.f};
        // (rows beyond M are the last one again, and not used)
        const int row = min(c, M - 1);
        const uint8_t* ar = la + row * ldq + 16 * q;
        const uint8_t* sr = ls + row * ldwsf + 8 * q;
        auto compute = [&](int g, const Group& r) {
            const u32x2 as = *reinterpret_cast<const u32x2*>(sr + 32 * g);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(ar + 64 * min(4 * g + u, steps - 1));
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int sh = 16 * (u & 1) + 8 * (s >> 1);
                    const half8_t ha = dequant8(a[s], scale_pair((as[u >> 1] >> sh) & 0xFFu));
#pragma unroll
                    for (int f = 0; f < CB; ++f)
                        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            ha, dequant8(r.w[f][u][s], scale_pair((r.ws[f][u >> 1] >> sh) & 0xFFu)), acc[f], 0, 0, 0);
                }
            }
        };
        for (int g = g0;;) {
            compute(g, r0);
            if (++g >= g1) break;
            load_w(g + 1, r0);
            compute(g, r1);
            if (++g >= g1) break;
            load_w(g + 1, r1);
        }
        if (q == 0) {
#pragma unroll
            for (int f = 0; f < CB; ++f)
#pragma unroll
                for (int i = 0; i < kLoraTokenRows; ++i) red[wave][i][16 * f + c] = acc[f][i];
        }
        lds_sync();
        return;
    }

    // one output per thread: row orow, column n of the work-group's
    const int t = tid - 64 * nk, tw = wave - nk;
    const int orow = t / (16 * CB), n = t - orow * 16 * CB;
    const int64_t col = blk0 * 16 + n;
    int oid = -1, rank = 0;
    if (orow < M && col < p.N) oid = p.ids[orow];
    if (oid >= p.L) oid = -1;
    if (oid >= 0) rank = p.rank ? min(max(p.rank[oid], 0), R) : R;
    const uint16_t* brow = oid >= 0 ? p.b + ((int64_t)oid * p.N + col) * R : p.b;
    const float scale = oid >= 0 ? p.scale[oid] : 0.0f;
    u32x4 b[kTokenAhead];
#pragma unroll
    for (int j = 0; j < kTokenAhead; ++j) b[j] = *reinterpret_cast<const u32x4*>(brow + (8 * j < R ? 8 * j : 0));

    // v
    const int R4 = R / 4, units = M * R4 * ranges, slabs = (K + 511) / 512, span = (slabs + ranges - 1) / ranges;
    for (int u = tw; u < units; u += kTokenWaves) {
        const int range = u / (M * R4), rest = u - range * M * R4, row = rest / R4, j0 = 4 * (rest - row * R4);
        const int id = p.ids[row];
        if (id < 0 || id >= p.L) continue;                  // its v is not used
        const int rk = p.rank ? min(max(p.rank[id], 0), R) : R;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + (int64_t)row * K, (int64_t)K * 2);
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (int64_t)id * R * K, (int64_t)R * K * 2);
        const int s0 = range * span, s1 = min(slabs, s0 + span);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int U = 4;                                // slabs of 512 K values in flight
        for (int s = s0; s < s1; s += U) {
            u32x4 x[U], a[U][4];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = 512 * (s + k) + 8 * lane;
                const bool on = s + k < s1 && at < K;
                x[k] = __builtin_amdgcn_raw_buffer_load_b128(rx, on ? (uint32_t)at * 2 : kBeyond, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[k][j] = __builtin_amdgcn_raw_buffer_load_b128(
                        ra, on && j0 + j < rk ? (uint32_t)((j0 + j) * K + at) * 2 : kBeyond, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x0 = bf16_to_f32(x[k][e] & 0xFFFFu), x1 = bf16_to_f32(x[k][e] >> 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum[j] = __builtin_fmaf(x0, bf16_to_f32(a[k][j][e] & 0xFFFFu), sum[j]);
                        sum[j] = __builtin_fmaf(x1, bf16_to_f32(a[k][j][e] >> 16), sum[j]);
                    }
                }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int off = 32; off; off >>= 1) sum[j] += __shfl_xor(sum[j], off, 64);
            if (lane == 0) lv[(range * M + row) * R + j0 + j] = j0 + j < rk ? sum[j] : 0.0f;
        }
    }
    lds_sync();         // A is in place (the streaming waves')
    lds_sync();         // red and v are
    if (orow >= M || col >= p.N) return;
    float delta = 0.0f;
    auto add = [&](u32x4 w, int j0) {
        w = lora_mask_rank(w, j0, rank);
        const float* v = lv + orow * R + j0;
        for (int r = 0; r < ranges; ++r, v += M * R) {
            const float4_t v0 = *reinterpret_cast<const float4_t*>(v), v1 = *reinterpret_cast<const float4_t*>(v + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                delta = __builtin_fmaf(e < 4 ? v0[e & 3] : v1[e & 3], bf16_to_f32(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu), delta);
        }
    };
#pragma unroll
    for (int j = 0; j < kTokenAhead; ++j)
        if (8 * j < rank) add(b[j], 8 * j);
    for (int j0 = 8 * kTokenAhead; j0 < rank; j0 += 8) add(*reinterpret_cast<const u32x4*>(brow + j0), j0);
    float part[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) part[w] = red[w < nk ? w : 0][orow][n];
    float sum = part[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += w < nk ? part[w] : 0.0f;
    const float y = a_gs[0] * b_alpha[0] * sum + (rank > 0 ? scale * delta : 0.0f);
    out[(int64_t)orow * p.N + col] = (uint16_t)pack_bf16x2_rne(y, 0.0f);
}

template <int MT, int CB>
hipError_t launch_stream(const LoraParams& p, const uint8_t* aqp, const uint8_t* asfp, const uint8_t* bq,
                         const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out, hipStream_t s) {
    // waves that stream and waves that expand: eight in all where two
    // work-groups share a CU, else four and up to eight
    const int expand = p.M <= 2 ? 1 : 4, most = MT == 4 ? NW : NW - expand;
    const int quads = (int)(pitch_wsf(p.K) / 32), per = (quads + most - 1) / most, nk = (quads + per - 1) / per;
    const int64_t cols = (p.N / 16 + CB - 1) / CB, parts = (p.M + 16 * MT - 1) / (16 * MT);
    const int64_t grid = parts == 1 ? cols : (cols + 7) / 8 * 8 * parts;
    const int rows = (int)(p.M < 16 * MT ? p.M : 16 * MT);
    const int lds = (1 + nk) * 16 * MT * (16 * CB + 4) * 4 + rows * lds_v_pitch(p.R) * 2;
    static std::atomic<int> lds_set[kMaxDevices];
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&lora_stream_kernel<MT, CB>), lds, lds_set);
    if (e != hipSuccess) return e;
    lora_stream_kernel<MT, CB><<<(unsigned)grid, 64 * (nk + expand), lds, s>>>(p, (int)parts, nk, per, aqp, asfp, bq, bsf, a_gs,
                                                                              b_alpha, out);
    return hipGetLastError();
}

}  // namespace

// Work-groups of the shrink before K is split: tiles x the adapters a tile can
// hold x rank blocks; K ranges (at most 8, each at least 4 blocks of 64) bring
// the launch to about two work-groups per CU. Listed tiles hold few adapters,
// which the host cannot know; counting one per tile, with room for the tiles
// where two meet, is right for runs of rows. A streamed tile's rows are not
// listed: each may have its own. The two counts are not sharp: with anything from
// 256 to 1024 the whole operator took the same time within 2 % at 7 to 4093 rows;
// with 128 it took 7 % longer at 61 rows (29.2 us against 27.2) and 3 % at 1500.
int lora_planes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    const int64_t tiles = (M + kLoraRows - 1) / kLoraRows, rbs = (R + kRankBlock - 1) / kRankBlock;
    const int64_t rows = M < kLoraRows ? M : kLoraRows;
    const bool listed = !lora_streams(M, N, K, L, R);
    const int64_t here = listed ? 1 : rows < L ? rows : L;
    const int64_t nb = (K + 63) / 64;
    int64_t n = (listed ? 416 : 512) / (tiles * rbs * here);
    if (n > nb / 4) n = nb / 4;
    if (n > kLoraMaxPlanes) n = kLoraMaxPlanes;
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
    // work-groups that share a tile's adapters: as many as it can hold; listed
    // rows put few adapters into a tile
    int64_t slots = p.M < kLoraRows ? p.M : kLoraRows;
    if (slots > p.L) slots = p.L;
    const int64_t most = tiles <= 4 ? 8 : tiles <= 16 ? 4 : tiles <= 64 ? 2 : 1;
    if (order != kLoraAsIs && slots > most) slots = most;
    const int64_t blocks = tiles * slots * p.planes * rbs;
    const int64_t more = aqp  ? (lora_stream_aq_bytes(p.M, p.K) / 16 + lora_stream_asf_bytes(p.M, p.K) / 8 + NT - 1) / NT
                              : (p.M * (p.K / 16) + 4 * NT - 1) / (4 * NT);
    auto launch = [&](auto ns, auto step) {
        constexpr int NS = decltype(ns)::value, STEP = decltype(step)::value, lds = NS * kShrinkStage;
        static std::atomic<int> lds_set[kMaxDevices];
        hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&lora_shrink_kernel<NS, STEP>), lds, lds_set);
        if (e != hipSuccess) return e;
        lora_shrink_kernel<NS, STEP><<<(unsigned)(blocks + more), NT, lds, s>>>(
            p, (int)tiles, (int)rbs, (int)slots, (int)blocks, order == kLoraRank, perm, sid, aq, asf, aqp, asfp,
            reinterpret_cast<uint8_t*>(ah));
        return hipGetLastError();
    };
    return tiles <= 4 ? launch(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{})
                      : launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
}

hipError_t launch_lora_join(const LoraParams& p, hipStream_t s) {
    lora_join_kernel<<<(unsigned)((p.M * (p.R / 8) + 255) / 256), 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_lora_reduce(const LoraParams& p, const float* partial, int ksplit, const float* a_gs,
                              const float* b_alpha, uint16_t* out, hipStream_t s) {
    const int64_t tiles = (p.M + kLoraRows - 1) / kLoraRows;
    const int lds = kLoraRows * lds_v_pitch(p.R) * 2;
    static std::atomic<int> lds_set[kMaxDevices];
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&lora_reduce_kernel), lds, lds_set);
    if (e != hipSuccess) return e;
    lora_reduce_kernel<<<(unsigned)(tiles * ((p.N + 31) / 32)), RT, lds, s>>>(p, (int)tiles, partial, ksplit, a_gs,
                                                                              b_alpha, out);
    return hipGetLastError();
}

hipError_t launch_lora_stream(const LoraParams& p, const uint8_t* aqp, const uint8_t* asfp, const uint8_t* bq,
                              const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out,
                              hipStream_t s) {
    if (p.M <= 16) return launch_stream<1, 1>(p, aqp, asfp, bq, bsf, a_gs, b_alpha, out, s);
    if (p.M <= 32) return launch_stream<2, 2>(p, aqp, asfp, bq, bsf, a_gs, b_alpha, out, s);
    return launch_stream<4, 2>(p, aqp, asfp, bq, bsf, a_gs, b_alpha, out, s);
}

hipError_t launch_lora_token(const LoraParams& p, const uint8_t* aq, const uint8_t* asf, const uint8_t* bq,
                             const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out,
                             hipStream_t s) {
    const int quads = (int)(pitch_wsf(p.K) / 32), per = (quads + NW - 1) / NW, nk = (quads + per - 1) / per;
    const int64_t blocks = p.N / 16;
    const int cb = blocks <= 256 ? 1 : 2;
    const int lds = (int)(p.M * (pitch_q(p.K) + pitch_wsf(p.K))) + token_ranges((int)p.M, p.R) * (int)p.M * p.R * 4 +
                    nk * kLoraTokenRows * (16 * cb + 4) * 4;
    auto launch = [&](auto width) {
        constexpr int CB = decltype(width)::value;
        static std::atomic<int> lds_set[kMaxDevices];
        hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&lora_token_kernel<CB>), lds, lds_set);
        if (e != hipSuccess) return e;
        lora_token_kernel<CB><<<(unsigned)((blocks + CB - 1) / CB), 64 * (nk + kTokenWaves), lds, s>>>(
            p, nk, per, aq, asf, bq, bsf, a_gs, b_alpha, out);
        return hipGetLastError();
    };
    return cb == 1 ? launch(std::integral_constant<int, 1>{}) : launch(std::integral_constant<int, 2>{});
}

}  // namespace nvfp4
