// Gated feed-forward block in bf16: act = silu(x Wg) * (x Wu) with
// w13 = [Wg | Wu] (H, 2I), and its backward pass. The dense (or shared) expert
// beside the routed ones: its weights stay in bf16 and may be trained.
//
//   forward   g = x Wg, u = x Wu (float32 sums), act = bf16(g / (1 + e^-g) * u),
//             optionally gate_up = [bf16(g) | bf16(u)] for the backward pass
//   backward  s = 1 / (1 + e^-g);  dg = d u s (1 + g (1 - s));  du = d g s
//             dx = [dg | du] w13^T,  dw13 = x^T [dg | du]
//
// All three products run through one tile routine (below) on
// v_mfma_f32_32x32x16_bf16. The two directions a reduction can lie in are
// handled at the LDS read: an operand whose rows are contiguous along K
// (x in the forward; [dg | du] and w13 in dx) is staged as its rows and
// read with 16-byte loads; one whose rows are contiguous along M or N (w13 in
// the forward; both operands of dw13) is staged as K rows and read with the
// transposing LDS load (ds_read_b64_tr_b16: 16 lanes read 4 K rows of 16
// columns and each lane receives the 4 K values of its column). Nothing is
// transposed in memory and no weight is repacked, which training could not
// keep up to date for free.
//
// Tile. A work-group of 8 waves (two per SIMD) computes 64 MI x 256 outputs;
// wave w owns rows 32 MI (w / 4) .. and columns 64 (w % 4) .. +64. In the
// forward a wave's 64 columns are 32 gate columns and the matching 32 up
// columns, so both projections of an output meet in one lane and the
// activation and the product are its epilogue. Stages of 32 or 64 K elements
// move from memory to LDS by buffer loads that write LDS directly, into a ring
// of stages. Every load is issued with either an offset inside the operand or
// one beyond the buffer (which reads zeros): K tails, rows beyond M and columns
// beyond N are zeros in both operands, so nothing else (a NaN beside the tile)
// enters a sum.
//
// Few tiles: K is cut into chunks that fill the GPU, each work-group writes
// float32 partial sums, and a second kernel adds them in chunk order (the
// result does not depend on scheduling) before the one rounding.
//
// What bounds it, and what it measured (medians; H 7168, I 2048 but for the last
// line):
//   T 1, 23      the weights, 58.7 MB once: 12.2 us (4.8 TB/s) and 13.5 us, and
//                4 us for the chunks' sums
//   T 301        the caches: every stage of a tile is 24 KB for 1/2 us of matrix
//                work; 26 us + 6 us for the chunks' sums
//   T 4096       the matrix cores at the clock that they get under load, 2.0 GHz:
//                forward 192 to 202 us in calls back to back (1.2 PFLOP/s; no LDS
//                bank conflicts, the matrix pipes busy 59 % of the cycles), both
//                products of the backward 405 to 414 us (1.17 PFLOP/s)
//   1001 rows, H 4112, I 1360   the ends: 499 tiles of unequal lengths on 256 CUs,
//                and both widths end 16 columns into a tile; products 57 to 61 us
// Four waves of 128 x 128 outputs, which read LDS less often, were slower (218
// us against 194 for the forward: one wave per SIMD leaves no one to issue while
// it waits).
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef short short8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) short4_t lds_short4;

constexpr int NT = 512;                     // 8 waves
constexpr int BN = kGatedBN;                // tile columns
constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kBeyond = 0x80000000u;   // an offset outside every buffer: reads zeros
constexpr int kWaves = NT / 64;

// K elements per stage: 64 where both operands are contiguous along K, whose
// rows are then read 128 bytes at a time (64 bytes a row and stage cost dx 5 to
// 20 %); else 32, which leaves room for more stages in flight (4 % of the forward
// at 4096 rows)
template <int MODE> constexpr int kKS = MODE == kGatedDx ? 64 : 32;
template <int MODE, int MI> constexpr int kABytes = 64 * MI * kKS<MODE> * 2;
template <int MODE, int MI> constexpr int kStage = kABytes<MODE, MI> + BN * kKS<MODE> * 2;
// ring depth: 120 to 144 KB
template <int MODE, int MI> constexpr int kStages = MODE == kGatedDx ? (MI == 4 ? 2 : 3) : (MI == 4 ? 4 : MI == 2 ? 5 : 6);
template <int MODE, int MI> constexpr int kLds = kStages<MODE, MI> * kStage<MODE, MI>;

constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A buffer whose valid offsets are the ones the callers form (all below 2^31);
// kBeyond lies outside.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7FFFFFFF, kRsrcWord3);
}

// e^-|g|, at most 1, so neither sign of g overflows. It is zero from |g| = 87.4 on
// (no subnormal results: silu there is below 2^-119 of u); exp_split's own steps
// overflow beyond about 2^127.
__device__ __forceinline__ float exp_neg_abs(float g) { return exp_split(fmaxf(-__builtin_fabsf(g), -200.0f)); }

// 1 / (1 + e^-g) by e^-|g|, and silu(g) * u, in float32.
__device__ __forceinline__ float sigmoid_f32(float g) {
    const float e = exp_neg_abs(g);
    return (g >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
}
__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid_f32(g) * u; }

// Transposing LDS load. The restrict argument gives the access alias
// information; without any, the compiler drains every outstanding load into
// LDS before it (the waits that order them are the main loop's own).
__device__ __forceinline__ short4_t lds_read_tr(lds_short4* __restrict__ q) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(q);
}

// 4 x 4 transpose inside each quad of lanes: lane m of a quad gives v[r] = row
// r of column m and receives row m of columns 0..3.
__device__ __forceinline__ void quad_transpose(float (&v)[4], int lane) {
    const bool odd = lane & 1, upper = lane & 2;
    auto swap1 = [](float x) {       // quad_perm(1,0,3,2)
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, false));
    };
    auto swap2 = [](float x) {       // quad_perm(2,3,0,1)
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x4E, 0xF, 0xF, false));
    };
    const float a = swap1(odd ? v[0] : v[1]), b = swap1(odd ? v[2] : v[3]);
    if (odd) { v[0] = a; v[2] = b; } else { v[1] = a; v[3] = b; }
    const float c = swap2(upper ? v[0] : v[2]), d = swap2(upper ? v[1] : v[3]);
    if (upper) { v[0] = c; v[1] = d; } else { v[2] = c; v[3] = d; }
}

// Work-group b -> tile (m, n) and K chunk. Work-groups go to the eight XCDs
// round-robin, so XCD b % 8 gets a contiguous range of tile numbers, and tile
// numbers run over blocks of 4 row tiles, so that an XCD's tiles share
// operand rows in its L2.
struct TileId { int m, n, chunk; };
__device__ __forceinline__ TileId map_tile(int b, int total, int mt, int ntn) {
    const int x = b & 7, q = total >> 3, rem = total & 7;
    const int id = x * q + min(x, rem) + (b >> 3);
    const int tiles = mt * ntn;
    const int chunk = id / tiles, t = id - chunk * tiles;
    constexpr int GM = 4;
    const int g = t / (GM * ntn), r = t - g * GM * ntn;
    const int gm = min(GM, mt - g * GM);
    return {g * GM + r % gm, r / gm, chunk};
}

// One operand of a tile. KSTRIDED = false: `rows` rows (from base), each
// contiguous along K, ld elements apart; true: K rows, contiguous along the
// tile's W columns (column ranges given per 8-column chunk by `off`).
//
// LDS layout of a stage of KS K elements. K-contiguous: rows of 2 KS bytes,
// 16-byte chunk c of row r stored at c ^ ((r >> 1) & 7) (KS = 64; c ^ ((r >> 2) &
// 3) for 32), so the 16 rows a 16-lane group reads cover all 64 banks. K-strided:
// KS K rows of 2 W bytes; 16-byte chunk c of row k at c ^ swz(k), so the 4 K rows
// x 64 bytes that 32 lanes of a transposing load read cover all banks.
template <int W> __device__ __forceinline__ int kstrided_swz(int k) {
    return W >= 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}

template <int MODE, int MI>
__device__ __forceinline__ void gated_tile(const GatedGemm& p, int block, uint8_t* smem) {
    constexpr bool A_KS = MODE == kGatedDw;              // A contiguous along M
    constexpr bool B_KS = MODE != kGatedDx;              // B contiguous along N
    constexpr int AW = 64 * MI;                          // tile rows
    constexpr int KS = kKS<MODE>, SUB = KS / 16;         // substeps of a stage: one MFMA deep
    constexpr int NS = kStages<MODE, MI>;
    constexpr int STAGE = kStage<MODE, MI>, A_BYTES = kABytes<MODE, MI>;
    // loads per wave and stage (a 64-row tile of 32 K has 4 KB of A: waves 4..7
    // load what waves 0..3 do)
    constexpr int AI = A_BYTES / 1024, NA = AI < kWaves ? 1 : AI / kWaves, NB = BN * KS * 2 / 1024 / kWaves, NL = NA + NB;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ntn = (int)((p.ncols + p.tile_cols - 1) / p.tile_cols);
    const int mt = (int)((p.M + AW - 1) / AW);
    const TileId id = map_tile(block, mt * ntn * p.ksplit, mt, ntn);
    const int64_t m0 = (int64_t)id.m * AW, n0 = (int64_t)id.n * p.tile_cols;
    const int rows = (int)min((int64_t)AW, p.M - m0);

    // K range of this work-group, in stages; kend bounds every load
    const int nk_all = (int)((p.K + KS - 1) / KS);
    const int kper = (nk_all + p.ksplit - 1) / p.ksplit;
    const int kb = id.chunk * kper;
    const int nk = min(nk_all, kb + kper) - kb;
    const int kend = (int)min(p.K, (int64_t)(kb + nk) * KS);

    // K-contiguous rows of a stage: 16-byte chunks, rows of a load, swizzle
    constexpr int kChunks = KS / 8, kRows = 64 / kChunks;
    auto row_swz = [](int r) { return KS == 64 ? (r >> 1) & 7 : (r >> 2) & 3; };

    // ---- per-lane load offsets (bytes from the stage's base) and K position ----
    const uint16_t* abase = p.a + (A_KS ? m0 : m0 * p.lda);
    const uint16_t* bbase = p.b + (MODE == kGatedDx ? n0 * p.ldb : MODE == kGatedDw ? n0 : 0);
    uint32_t a_off[NA], b_off[NB];
    int a_k[NA], b_k[NB];
#pragma unroll
    for (int t = 0; t < NA; ++t) {
        const int u = (NA * wave + t) % AI;
        if (A_KS) {
            constexpr int CH = AW / 8;                   // chunks per K row
            const int k = u * (64 / CH) + lane / CH, pc = lane % CH;
            const int c = pc ^ kstrided_swz<AW>(k);
            a_k[t] = k;
            a_off[t] = 8 * c < rows ? (uint32_t)(k * p.lda * 2 + 16 * c) : kBeyond;
        } else {
            const int r = u * kRows + lane / kChunks;
            const int c = (lane % kChunks) ^ row_swz(r);
            a_k[t] = 8 * c;
            a_off[t] = r < rows ? (uint32_t)(r * p.lda * 2 + 16 * c) : kBeyond;
        }
    }
#pragma unroll
    for (int t = 0; t < NB; ++t) {
        const int u = NB * wave + t;
        if (B_KS) {
            const int k = 2 * u + (lane >> 5), pc = lane & 31;
            const int c = pc ^ kstrided_swz<BN>(k);
            b_k[t] = k;
            int64_t col;
            bool ok;
            if (MODE == kGatedFwd) {                     // chunk c: 4 chunks gate, 4 chunks up per wave
                const int64_t a = n0 + 32 * (c >> 3) + 8 * (c & 3);
                ok = a < p.I;
                col = (c & 4) ? p.I + a : a;
            } else {
                col = 8 * c;
                ok = n0 + col < p.ncols;
            }
            b_off[t] = ok ? (uint32_t)((k * p.ldb + col) * 2) : kBeyond;
        } else {
            const int r = u * kRows + lane / kChunks;
            const int c = (lane % kChunks) ^ row_swz(r);
            b_k[t] = 8 * c;
            b_off[t] = n0 + r < p.ncols ? (uint32_t)(r * p.ldb * 2 + 16 * c) : kBeyond;
        }
    }
    const int64_t a_step = A_KS ? (int64_t)KS * p.lda : KS;       // elements per stage
    const int64_t b_step = B_KS ? (int64_t)KS * p.ldb : KS;

    // running state of the refills: the next stage's bases and how many K
    // elements are left from there
    const uint16_t* pa = abase + (int64_t)kb * a_step;
    const uint16_t* pb = bbase + (int64_t)kb * b_step;
    int left = kend - kb * KS;
    auto issue = [&](int st) {
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(pa), rb = make_rsrc(pb);
        uint8_t* base = smem + st * STAGE;
#pragma unroll
        for (int t = 0; t < NA; ++t) {
            const int u = (NA * wave + t) % AI;
            const uint32_t off = a_k[t] < left ? a_off[t] : kBeyond;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + u * 1024), 16, off, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const uint32_t off = b_k[t] < left ? b_off[t] : kBeyond;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + A_BYTES + (NB * wave + t) * 1024), 16,
                                                     off, 0, 0, 0);
        }
        pa += a_step;
        pb += b_step;
        left -= KS;
    };

    // ---- fragments ---------------------------------------------------------------
    // Lane l serves row / column l % 32 and, of a 16-element substep, K values
    // 8 h .. 8 h + 7 with h = l / 32, in both operands.
    const int wm = wave >> 2, wn = wave & 3;
    const int l32 = lane & 31, h = lane >> 5;
    const int tk = 8 * h + ((lane & 15) >> 2);                     // transposing loads: K row
    const int tc = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);      // chunk inside a 32-column block
    uint32_t fa_off[MI], fb_off[2], fc_a, fc_b;
    fc_a = (uint32_t)(16 * (h ^ row_swz(l32)));                // K-contiguous: chunk of substep 0
    fc_b = fc_a;
#pragma unroll
    for (int i = 0; i < MI; ++i)
        fa_off[i] = A_KS ? (uint32_t)(tk * AW * 2 + 16 * ((4 * (wm * MI + i) + tc) ^ kstrided_swz<AW>(tk)) + 8 * (lane & 1))
                         : (uint32_t)((wm * 32 * MI + 32 * i + l32) * 2 * KS);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        fb_off[j] = A_BYTES +
                    (B_KS ? (uint32_t)(tk * BN * 2 + 16 * ((4 * (wn * 2 + j) + tc) ^ kstrided_swz<BN>(tk)) + 8 * (lane & 1))
                          : (uint32_t)((wn * 64 + 32 * j + l32) * 2 * KS));

    auto read_tr = [&](uint32_t off, int ldw, int s) -> bf16x8_t {
        const uint8_t* q = smem + off + s * 16 * ldw;
        const short4_t lo = lds_read_tr((lds_short4*)q);
        const short4_t hi = lds_read_tr((lds_short4*)(q + 4 * ldw));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read_row = [&](uint32_t off, uint32_t fc, int s) -> bf16x8_t {
        return *reinterpret_cast<const bf16x8_t*>(smem + off + (fc ^ (uint32_t)(32 * s)));
    };
    bf16x8_t fa[2][MI], fb[2][2];
    auto read = [&](int st, int s, int d) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            fb[d][j] = B_KS ? read_tr(st * STAGE + fb_off[j], BN * 2, s) : read_row(st * STAGE + fb_off[j], fc_b, s);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            fa[d][i] = A_KS ? read_tr(st * STAGE + fa_off[i], AW * 2, s) : read_row(st * STAGE + fa_off[i], fc_a, s);
    };

    float16_t acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    auto mfma = [&](int d) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[d][i], fb[d][j], acc[i][j], 0, 0, 0);
    };

    // ---- main loop ------------------------------------------------------------------
    // Step r: substep 0's fragments are in registers. Each next substep's are
    // read under a substep's MFMAs; before the last substep's MFMAs this wave's
    // loads of stage r + 1 are waited for (those of the NS - 2 later stages stay
    // in flight), the barrier makes everyone's visible and says that everyone
    // has read stage r, whose buffer stage r + NS refills. Loads past the last stage read
    // zeros, so the count of outstanding loads is the same in every step.
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 1) * NL, 0));
    lds_barrier();
    // A wave whose rows or columns all lie outside the matrix only brings its
    // share of the stages: the tile's other waves have the matrix cores alone
    // (301 rows: 31.9 -> 31.2 us; 1001 x 4112 x 1360 backward: 63.3 -> 62.6).
    if (wm * 32 * MI >= rows || n0 + wn * (MODE == kGatedFwd ? 32 : 64) >= p.ncols) {
        for (int r = 0, st = 0; r < nk; ++r, st = st + 1 == NS ? 0 : st + 1) {
            __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * NL, 0));
            lds_barrier();
            issue(st);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        return;
    }
    read(0, 0, 0);
    // LDS reads of one substep, spread over its first MFMAs (one instruction
    // group each), so that the matrix core starts at once and the reads land
    // under the rest
    constexpr int NR = (A_KS ? 2 : 1) * MI + (B_KS ? 2 : 1) * 2;
    constexpr int NM = 2 * MI;                                   // MFMAs of a substep
    constexpr int SPREAD = NM > 2 ? NM - 2 : 1;
    constexpr int PER = (NR + SPREAD - 1) / SPREAD;
    auto step = [&](int st) {
#pragma unroll
        for (int t = 0; t + 1 < SUB; ++t) {
            read(st, t + 1, (t + 1) & 1);
            mfma(t & 1);
#pragma unroll
            for (int k = 0; k < NM; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);       // one MFMA
                __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);     // its share of the LDS reads
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * NL, 0));
        lds_barrier();
        read(st + 1 == NS ? 0 : st + 1, 0, 0);
        issue(st);
        mfma((SUB - 1) & 1);
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
            __builtin_amdgcn_sched_group_barrier(0x010, (NL + NM - 1) / NM, 0);     // loads into LDS
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int r = 0;
    for (; r + NS <= nk; r += NS) {
#pragma unroll
        for (int s = 0; s < NS; ++s) step(s);
    }
    for (int s = 0; r + s < nk; ++s) step(s);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));      // no load into LDS outlives the work-group

    // ---- epilogue -------------------------------------------------------------------
    // acc[i][j][r] = D[row 32 i + 8 (r / 4) + 4 h + r % 4][column 32 j + l32] of
    // the wave's part; after a transpose inside each quad of lanes, lane 4 c +
    // m holds columns 4 c .. 4 c + 3 of row m of each group of four rows
    const int m4 = lane & 3, c4 = l32 & ~3;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int local = wm * 32 * MI + 32 * i + 8 * g + 4 * h + m4;
            const int64_t row = m0 + local;
            float v[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j][k] = acc[i][j][4 * g + k];
                quad_transpose(v[j], lane);
            }
            if (MODE == kGatedFwd) {
                const int64_t col = n0 + wn * 32 + c4;       // I % 16 == 0: four columns are in or out together
                if (local >= rows || col >= p.I) continue;
                if (p.ksplit > 1) {
                    float* dst = p.partial + ((int64_t)id.chunk * p.M + row) * 2 * p.I + col;
                    *reinterpret_cast<float4_t*>(dst) = (float4_t){v[0][0], v[0][1], v[0][2], v[0][3]};
                    *reinterpret_cast<float4_t*>(dst + p.I) = (float4_t){v[1][0], v[1][1], v[1][2], v[1][3]};
                    continue;
                }
                float a[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] = silu_mul(v[0][k], v[1][k]);
                *reinterpret_cast<u32x2*>(p.out + row * p.I + col) =
                    (u32x2){pack_bf16x2_rne(a[0], a[1]), pack_bf16x2_rne(a[2], a[3])};
                if (p.gate_up) {
                    uint16_t* gu = p.gate_up + row * 2 * p.I + col;
                    *reinterpret_cast<u32x2*>(gu) =
                        (u32x2){pack_bf16x2_rne(v[0][0], v[0][1]), pack_bf16x2_rne(v[0][2], v[0][3])};
                    *reinterpret_cast<u32x2*>(gu + p.I) =
                        (u32x2){pack_bf16x2_rne(v[1][0], v[1][1]), pack_bf16x2_rne(v[1][2], v[1][3])};
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t col = n0 + wn * 64 + 32 * j + c4;
                    if (local >= rows || col >= p.ncols) continue;
                    if (p.ksplit > 1)
                        *reinterpret_cast<float4_t*>(p.partial + ((int64_t)id.chunk * p.M + row) * p.ncols + col) =
                            (float4_t){v[j][0], v[j][1], v[j][2], v[j][3]};
                    else
                        *reinterpret_cast<u32x2*>(p.out + row * p.ncols + col) =
                            (u32x2){pack_bf16x2_rne(v[j][0], v[j][1]), pack_bf16x2_rne(v[j][2], v[j][3])};
                }
            }
        }
    }
}

template <int MODE, int MI>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gated_kernel(GatedGemm p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    gated_tile<MODE, MI>(p, blockIdx.x, smem);
}

// The backward's two products in one launch (they only share inputs): their
// work-groups fill the GPU together, and neither waits for the other's last
// ones. The product with the longer tiles comes first. (129 rows, H 2048, I 1408:
// 31 -> 26 us for the whole backward; the same at 4096 rows.)
template <int MODE>
__device__ __forceinline__ void gated_any_tile(const GatedGemm& p, int block, uint8_t* smem) {
    if (p.mi == 4) gated_tile<MODE, 4>(p, block, smem);
    else if (p.mi == 2) gated_tile<MODE, 2>(p, block, smem);
    else gated_tile<MODE, 1>(p, block, smem);
}
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gated_backward_kernel(GatedGemm gx, GatedGemm gw, int nx, int nw, bool dx_first) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int b = blockIdx.x;
    if (dx_first ? b < nx : b >= nw) gated_any_tile<kGatedDx>(gx, dx_first ? b : b - nw, smem);
    else gated_any_tile<kGatedDw>(gw, dx_first ? b - nx : b, smem);
}

// Partial sums of the forward, in chunk order, then the epilogue of the tile
// routine. One thread per 4 columns: 3.9 us up to 23 rows (latency), 5.8 us at
// 301 (25 MB of sums, which the caches still hold).
constexpr int kReduceThreads = 64;
__global__ __launch_bounds__(kReduceThreads) void gated_reduce_kernel(GatedGemm p) {
    const int64_t I4 = p.I / 4, n = p.M * I4, plane = p.M * 2 * p.I;
    for (int64_t t = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x; t < n; t += (int64_t)gridDim.x * kReduceThreads) {
        const int64_t row = t / I4, col = 4 * (t - row * I4);
        // up to 16 loads in flight (gate and up of 8 chunks): a small batch has few
        // threads here and is bound by their latency
        const float* src = p.partial + row * 2 * p.I + col;
        float4_t g = *reinterpret_cast<const float4_t*>(src), u = *reinterpret_cast<const float4_t*>(src + p.I);
        for (int c0 = 1; c0 < p.ksplit; c0 += 8) {
            float4_t vg[8], vu[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < p.ksplit) {
                    vg[j] = *reinterpret_cast<const float4_t*>(src + (c0 + j) * plane);
                    vu[j] = *reinterpret_cast<const float4_t*>(src + (c0 + j) * plane + p.I);
                }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < p.ksplit) {
                    g += vg[j];
                    u += vu[j];
                }
        }
        float a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = silu_mul(g[k], u[k]);
        *reinterpret_cast<u32x2*>(p.out + row * p.I + col) =
            (u32x2){pack_bf16x2_rne(a[0], a[1]), pack_bf16x2_rne(a[2], a[3])};
        if (p.gate_up) {
            uint16_t* gu = p.gate_up + row * 2 * p.I + col;
            *reinterpret_cast<u32x2*>(gu) = (u32x2){pack_bf16x2_rne(g[0], g[1]), pack_bf16x2_rne(g[2], g[3])};
            *reinterpret_cast<u32x2*>(gu + p.I) = (u32x2){pack_bf16x2_rne(u[0], u[1]), pack_bf16x2_rne(u[2], u[3])};
        }
    }
}

// out = bf16(sum of the chunks' partial sums, in chunk order), 4 columns a
// thread: 3.9 us at 129 x 2048 (latency).
__global__ __launch_bounds__(256) void gated_sum_kernel(const float* __restrict__ partial, int ksplit, int64_t n4,
                                                        uint16_t* __restrict__ out) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n4; t += (int64_t)gridDim.x * 256) {
        const float4_t v = sum_planes<8>(reinterpret_cast<const float4_t*>(partial) + t, ksplit, n4);
        *reinterpret_cast<u32x2*>(out + 4 * t) = (u32x2){pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
    }
}

// [dg | du] from the saved bf16 gate | up and d_act. It is rounded to bf16,
// the matrix cores' operand type: independent relative errors of at most 2^-8
// per element, which a sum over them carries as one such error, the size of
// the outputs' own rounding. 8 columns a thread: 3 reads and 2 writes of 16
// bytes, nothing to reuse, bound by memory: 16 us at T 4096, I 2048 (84 MB,
// 5.2 TB/s).
__global__ __launch_bounds__(256) void gated_dgu_kernel(const uint16_t* __restrict__ d_act,
                                                        const uint16_t* __restrict__ gate_up, int64_t T, int64_t I,
                                                        uint16_t* __restrict__ dgu) {
    const int64_t I8 = I / 8, n = T * I8;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256) {
        const int64_t row = t / I8, col = 8 * (t - row * I8);
        const u32x4 d = *reinterpret_cast<const u32x4*>(d_act + row * I + col);
        const u32x4 g = *reinterpret_cast<const u32x4*>(gate_up + row * 2 * I + col);
        const u32x4 u = *reinterpret_cast<const u32x4*>(gate_up + row * 2 * I + I + col);
        u32x4 og, ou;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float dg[2], du[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float dv = bf16_to_f32((d[k] >> (16 * b)) & 0xFFFFu), gv = bf16_to_f32((g[k] >> (16 * b)) & 0xFFFFu);
                const float uv = bf16_to_f32((u[k] >> (16 * b)) & 0xFFFFu);
                // 1 - s = sigmoid(-g): formed without cancellation
                const float e = exp_neg_abs(gv), q = __builtin_amdgcn_rcpf(1.0f + e);
                const float s = gv >= 0.0f ? q : e * q, s1 = gv >= 0.0f ? e * q : q;
                du[b] = dv * (gv * s);
                dg[b] = dv * uv * (s * (1.0f + gv * s1));
            }
            og[k] = pack_bf16x2_rne(dg[0], dg[1]);
            ou[k] = pack_bf16x2_rne(du[0], du[1]);
        }
        *reinterpret_cast<u32x4*>(dgu + row * 2 * I + col) = og;
        *reinterpret_cast<u32x4*>(dgu + row * 2 * I + I + col) = ou;
    }
}

__global__ __launch_bounds__(256) void zero_kernel(u32x4* p, int64_t n) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256)
        p[t] = (u32x4){0u, 0u, 0u, 0u};
}

unsigned grid_for(int64_t n) {
    const int64_t g = (n + 255) / 256;
    return (unsigned)(g < 1 ? 1 : g < 2048 ? g : 2048);
}

int64_t work_groups(const GatedGemm& p) {
    return (p.M + 64 * p.mi - 1) / (64 * p.mi) * ((p.ncols + p.tile_cols - 1) / p.tile_cols) * p.ksplit;
}

template <int MODE>
int lds_of(int mi) { return mi == 4 ? kLds<MODE, 4> : mi == 2 ? kLds<MODE, 2> : kLds<MODE, 1>; }

template <int MODE, int MI>
hipError_t launch_tiles(const GatedGemm& p, hipStream_t s) {
    const int64_t grid = work_groups(p);
    static std::atomic<int> lds_set[kMaxDevices];
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&gated_kernel<MODE, MI>), kLds<MODE, MI>, lds_set);
    if (e != hipSuccess) return e;
    gated_kernel<MODE, MI><<<(unsigned)grid, NT, kLds<MODE, MI>, s>>>(p);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_mode(const GatedGemm& p, hipStream_t s) {
    switch (p.mi) {
        case 1: return launch_tiles<MODE, 1>(p, s);
        case 2: return launch_tiles<MODE, 2>(p, s);
        default: return launch_tiles<MODE, 4>(p, s);
    }
}

// microseconds of one work-group of a product, the whole launch keeping a
// share f of the CUs busy (see the plans below)
double tile_us(int mi, double f, int64_t k32) {
    const double stage = mi == 4 ? 0.25 + 0.60 * f : mi == 2 ? 0.21 + 0.24 * f : 0.25 + 0.13 * f;
    return k32 * stage + 2.5;
}

}  // namespace

// Tile height and K chunks of a product: the pair with the smallest estimate, in
// microseconds, of the last work-group's end plus the partial sums' kernel and
// traffic. A stage takes longer the more CUs are at work (they share the
// caches and the power); its times are fits to sweeps over tile heights and
// chunks at 1 to 4096 rows, where the choice is within a few percent of the
// best one. (Wide layers too: H 4096 or 5120, I 13824 to 17920, 1 to 4096 rows,
// forward and backward: within 2 % of the best of a sweep.)
namespace {

struct Shape { int64_t M, ncols, tile_cols, outcols, K; int kstage; };

// Visits (tile height, K chunks, work-groups, stages of 32 K of one, cost of the
// partial sums) of a product.
template <typename F>
void each_plan(const Shape& s, int max_chunks, F f) {
    const int64_t nk = (s.K + s.kstage - 1) / s.kstage, ntn = (s.ncols + s.tile_cols - 1) / s.tile_cols;
    for (int mi = 4; mi >= 1; mi /= 2) {
        const int64_t tiles = (s.M + 64 * mi - 1) / (64 * mi) * ntn;
        for (int64_t ks = 1; ks <= max_chunks && ks <= nk && (ks == 1 || tiles * ks <= 256); ++ks) {
            const int64_t per = (nk + ks - 1) / ks;
            if ((nk + per - 1) / per != ks) continue;        // no empty chunk
            f(GatedPlan{mi, (int)ks}, tiles * ks, per * (s.kstage / 32),
              ks > 1 ? 2.5 + (double)ks * s.M * s.outcols * 4 * 2 / 8e6 : 0.0);
        }
    }
}

// End of n1 jobs of w1 and then n2 of w2 <= w1, dealt in this order to 256 CUs as
// they get free.
double makespan(int64_t n1, double w1, int64_t n2, double w2) {
    const int64_t q = n1 / 256, r = n1 % 256;               // r CUs are one job ahead
    if (n2 == 0) return (q + (r > 0)) * w1;
    const double a = q * w1, b = a + (r ? w1 : 0.0);        // when the CUs get free: 256 - r at a, r at b
    const double even = (a * (256 - r) + b * r + n2 * w2) / 256;
    double t = even > b ? even : b;                         // no CU does better than the even share
    for (;; t += w2 / 4) {
        const int64_t fits = (256 - r) * (int64_t)((t - a) / w2 + 1e-9) + r * (int64_t)((t - b) / w2 + 1e-9);
        if (fits >= n2) return t;
    }
}

}  // namespace

GatedPlan gated_forward_plan(int64_t T, int64_t H, int64_t I) {
    GatedPlan best = {4, 1};
    double best_t = 1e30;
    each_plan({T, I, kGatedBN / 2, 2 * I, H, kKS<kGatedFwd>}, 32, [&](GatedPlan g, int64_t n, int64_t k32, double extra) {
        const double t = makespan(n, tile_us(g.mi, n < 256 ? n / 256.0 : 1.0, k32), 0, 0.0) + extra;
        if (t < best_t) {
            best_t = t;
            best = g;
        }
    });
    return best;
}

void gated_backward_plan(int64_t T, int64_t H, int64_t I, GatedPlan& px, GatedPlan& pw, bool& dx_first) {
    // dx and dw13 share a launch: the pair whose work-groups, the longer ones
    // first, fill the CUs best
    const Shape sx = {T, H, kGatedBN, H, 2 * I, kKS<kGatedDx>}, sw = {H, 2 * I, kGatedBN, 2 * I, T, kKS<kGatedDw>};
    double best_t = 1e30;
    each_plan(sx, 8, [&](GatedPlan gx, int64_t nx, int64_t kx, double ex) {
        each_plan(sw, 4, [&](GatedPlan gw, int64_t nw, int64_t kw, double ew) {
            const double f = nx + nw < 256 ? (nx + nw) / 256.0 : 1.0;
            const double wx = tile_us(gx.mi, f, kx), ww = tile_us(gw.mi, f, kw);
            const double t = (wx >= ww ? makespan(nx, wx, nw, ww) : makespan(nw, ww, nx, wx)) + ex + ew;
            if (t < best_t) {
                best_t = t;
                px = gx;
                pw = gw;
                dx_first = wx >= ww;
            }
        });
    });
}

hipError_t launch_gated_forward(const GatedGemm& p, hipStream_t s) { return launch_mode<kGatedFwd>(p, s); }

hipError_t launch_gated_backward(const GatedGemm* gx, const GatedGemm* gw, bool dx_first, hipStream_t s) {
    if (!gw) return launch_mode<kGatedDx>(*gx, s);
    if (!gx) return launch_mode<kGatedDw>(*gw, s);
    const int lx = lds_of<kGatedDx>(gx->mi), lw = lds_of<kGatedDw>(gw->mi), lds = lx > lw ? lx : lw;
    const int64_t nx = work_groups(*gx), nw = work_groups(*gw);
    static std::atomic<int> lds_set[kMaxDevices];
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(&gated_backward_kernel), lds, lds_set);
    if (e != hipSuccess) return e;
    gated_backward_kernel<<<(unsigned)(nx + nw), NT, lds, s>>>(*gx, *gw, (int)nx, (int)nw, dx_first);
    return hipGetLastError();
}

hipError_t launch_gated_reduce(const GatedGemm& p, hipStream_t s) {
    const int64_t g = (p.M * p.I / 4 + kReduceThreads - 1) / kReduceThreads;
    gated_reduce_kernel<<<(unsigned)(g < 16384 ? g : 16384), kReduceThreads, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_gated_sum(const float* partial, int ksplit, int64_t n, uint16_t* out, hipStream_t s) {
    gated_sum_kernel<<<grid_for(n / 4), 256, 0, s>>>(partial, ksplit, n / 4, out);
    return hipGetLastError();
}

hipError_t launch_gated_dgu(const uint16_t* d_act, const uint16_t* gate_up, int64_t T, int64_t I, uint16_t* dgu,
                            hipStream_t s) {
    gated_dgu_kernel<<<grid_for(T * I / 8), 256, 0, s>>>(d_act, gate_up, T, I, dgu);
    return hipGetLastError();
}

hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t s) {
    zero_kernel<<<grid_for(bytes / 16), 256, 0, s>>>(static_cast<u32x4*>(p), bytes / 16);
    return hipGetLastError();
}

}  // namespace nvfp4
