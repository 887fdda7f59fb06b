// Host-side launchers of the NVFP4 kernels. Each returns hipSuccess or the
// launch error; none synchronizes and none allocates.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace nvfp4 {

// Raise a kernel's dynamic-LDS limit to at least `bytes` on the current
// device. The attribute belongs to the (kernel, device) pair, so the largest
// value set so far is remembered per device (one cache per kernel, indexed by
// device); concurrent callers may both set it, which is harmless, and the
// remembered maximum only grows.
constexpr int kMaxDevices = 64;
inline hipError_t ensure_dynamic_lds(const void* kernel, int bytes, std::atomic<int> (&done)[kMaxDevices]) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire) >= bytes) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess || dev < 0 || dev >= kMaxDevices) return e;
    int cur = done[dev].load(std::memory_order_relaxed);
    while (cur < bytes && !done[dev].compare_exchange_weak(cur, bytes, std::memory_order_release)) {
    }
    return hipSuccess;
}

// Tile descriptor of the grouped GEMMs: rows [row_start, row_start + row_count)
// of the sorted slot order, all routed to `expert`.
struct Tile {
    int32_t expert;
    int32_t row_start;
    int32_t row_count;
    int32_t pad;
};

constexpr int kGemmBM = 256;      // rows per GEMM tile
constexpr int kGemmBN = 256;      // B columns per GEMM tile (L1: 128 gate + 128 up)
constexpr int kRouteThreads = 1024;
constexpr int kMaxExperts = 512;

// zero `n` 32-bit words
hipError_t launch_zero_u32(uint32_t* p, int n, hipStream_t s);

// amax over `n` bf16 values (n % 8 == 0, 16-byte aligned) into *slot as float
// bits (atomic max; *slot must hold 0 or a smaller value).
hipError_t launch_amax_bf16(const uint16_t* x, int64_t n, uint32_t* slot, hipStream_t s);

// Per-matrix amax of E matrices of `per` bf16 values each into slots[e].
hipError_t launch_amax_bf16_batched(const uint16_t* x, int64_t E, int64_t per, uint32_t* slots,
                                    hipStream_t s);

// Row pitches of the GEMM operand layout: packed data padded to whole
// 128-element K steps, scales to whole 8-byte steps; the exact f16 form of a
// quantized activation (e2m1 * e4m3 per element, the global scale left out)
// has the same padded length, 2 bytes per element.
__host__ __device__ inline int64_t pitch_q(int64_t K) { return (K / 2 + 63) / 64 * 64; }
__host__ __device__ inline int64_t pitch_sf(int64_t K) { return (K / 16 + 7) / 8 * 8; }
__host__ __device__ inline int64_t pitch_h(int64_t K) { return 4 * pitch_q(K); }

// Row-block quantization of x (M, K) with amax taken from *amax_slot, or with
// the global scale *gs_in when gs_in is not null. Rows at or beyond *m_dev
// (when m_dev is not null) are left untouched. gs_out receives gs.
// Output rows are ldq bytes (q) and ldsf bytes (sf) apart; when h is not null
// the dequantized f16 values (without gs) go to rows of pitch_h(K) bytes too.
hipError_t launch_quant_rows(const uint16_t* x, int64_t M, int64_t K, const int32_t* m_dev,
                             const uint32_t* amax_slot, uint8_t* q, int64_t ldq, uint8_t* sf,
                             int64_t ldsf, float* gs_out, hipStream_t s,
                             const float* gs_in = nullptr, uint16_t* h = nullptr);

// Quantized rows (M, K/2) + (M, K/16), K % 16 == 0, unpadded -> their exact
// f16 values in rows of pitch_h(K) bytes, zero padded.
hipError_t launch_dequant_rows_f16(const uint8_t* q, const uint8_t* sf, int64_t M, int64_t K,
                                   uint16_t* h, hipStream_t s);

// Packed weight layout. A weight matrix is N rows (one per output column) of
// pitch_q(K) bytes, K-packed; rows are grouped in blocks of 16, and inside a
// block the 32 bytes of one 64-element half of a K step of all 16 rows are
// stored together (512 bytes), half step after half step. So one half step of
// a 16-row block, the unit a GEMM stage holds, is contiguous, and so is one
// whole 128-element K step (1 KB, the unit a streaming load covers).
// Scales: per block, groups of four K steps (512 bytes): row c (0..15), pair q
// (0..3: groups 2q, 2q+1 of a step), step u of the four, then the two bytes.
// The two scale bytes a streaming lane needs for four consecutive steps are
// thus one 8-byte piece, and a wave reads 512 contiguous bytes at once.
constexpr int kWqStep = 16 * 64;      // bytes of one K step of a 16-row block
constexpr int kWqHalf = 16 * 32;      // bytes of one half step of a 16-row block
constexpr int kWsfQuad = 16 * 32;     // scale bytes of four K steps of a block
// offset of byte kh (0..pitch_q - 1) of packed row n
__host__ __device__ inline int64_t wq_off(int64_t n, int64_t ldq, int64_t kh) {
    return (n >> 4) * 16 * ldq + (kh >> 5) * kWqHalf + (n & 15) * 32 + (kh & 31);
}
// scale row pitch of the packed weights: whole groups of four K steps
__host__ __device__ inline int64_t pitch_wsf(int64_t K) { return (pitch_q(K) / 64 + 3) / 4 * 32; }
// offset of scale pair q of K step st of row n (two bytes: groups 8st + 2q, +1)
__host__ __device__ inline int64_t wsf_off(int64_t n, int64_t ldsf, int64_t st, int q) {
    return (n >> 4) * 16 * ldsf + (st >> 2) * kWsfQuad + (n & 15) * 32 + q * 8 + (st & 3) * 2;
}

// Canonical (R, C) byte matrices (E of them, R = K-packed rows, C = N) into
// the packed layout: element (r, c) goes to row c, byte r of a row of pitch
// ldo; scales (scale_layout) in the four-step groups above, data in steps of
// 64 bytes. Padding bytes are 0.
hipError_t launch_pack_weights(const uint8_t* in, int64_t E, int64_t R, int64_t C, uint8_t* out,
                               int64_t ldo, bool scale_layout, hipStream_t s);

// Per-part amax of E weight matrices (E, K, N), each split along N into
// `parts` equal column ranges (N / parts % 8 == 0), into slots[e * parts + p].
hipError_t launch_amax_cols(const uint16_t* w, int64_t E, int64_t K, int64_t N, int parts,
                            uint32_t* slots, hipStream_t s);

// Column-block quantization of E weight matrices (E, K, N), one amax (and one
// alpha out) per column part: amax_slots / alpha [e * parts + p].
hipError_t launch_quant_cols(const uint16_t* w, int64_t E, int64_t K, int64_t N, int parts,
                             const uint32_t* amax_slots, uint8_t* q, uint8_t* sf, float* alpha,
                             hipStream_t s);

// Quantization of the activation done inside the routing launch by extra
// work-groups, concurrently with the routing work-groups: each takes the
// global scale from gs_in (static), else from the maximum of the pre-pass's
// partial maxima, else reduces the whole amax itself (small inputs), then
// quantizes its share of the 16-element blocks.
struct SmallQuant {
    const uint16_t* x;
    const float* gs_in;      // static global scale, or null
    const uint32_t* amax_partials;  // partial maxima (bf16 magnitude bits) of x, or null
    int n_partials;
    int64_t M, K;
    uint8_t* q;
    int64_t ldq;
    uint8_t* sf;
    int64_t ldsf;
    float* gs;
    uint16_t* h;             // exact f16 values, rows of pitch_h(K) bytes, or null
};
constexpr int64_t kSmallQuantMax = 1 << 17;   // elements: larger inputs take the two-kernel path

// Routing in chunks: up to kRouteChunk slots take one routing work-group
// (which counts them itself); more take one work-group per chunk of
// route_chunk(S) slots (at most kRouteMaxChunks chunks), whose counts the
// pre-pass provides.
constexpr int64_t kRouteChunk = 4096;
constexpr int64_t kRouteMaxChunks = 64;
constexpr int kRouteMaxPartials = 1024;
int64_t route_chunk(int64_t S);
// number of partial maxima the pre-pass writes for n activation values
int route_amax_partials(int64_t n);

// Pre-pass of the routing launch: when x is not null, the partial maxima of
// its n bf16 values (route_amax_partials(n) words into `partial`); when S >
// kRouteChunk, the per-expert counts of every chunk of slots into wg_counts
// (chunks x E int32).
hipError_t launch_route_prepass(const uint16_t* x, int64_t n, uint32_t* partial, const int32_t* ids,
                                int64_t S, int E, int32_t* wg_counts, hipStream_t s);

// Routing tables and the tile list, plus the quantization of *xq when xq is
// not null (further work-groups of the same launch). Also zeroes `zero_slots`
// (n_zero words) before anything else in the layer runs. wg_counts: the
// pre-pass's chunk counts (used when S > kRouteChunk).
hipError_t launch_route(const int32_t* ids, int64_t S, int topk, int E, int BM, const int32_t* wg_counts,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_slot, int32_t* slot_row, Tile* tiles,
                        int32_t* num_tiles, uint32_t* zero_slots, int n_zero, const SmallQuant* xq,
                        hipStream_t s);

// Top-k router: ids (T, k) = the k largest logits of each row of (T, E)
// (ties: smaller expert first), weights (T, k) = softmax over the selected
// logits. E <= kMaxExperts, 1 <= k <= E.
hipError_t launch_route_topk(const float* logits, int64_t T, int E, int k, int32_t* ids,
                             float* weights, hipStream_t s);

// y[t] = bf16(sum_j w[t][j] * o2[slot_row[t*topk+j]]) for rows that exist.
hipError_t launch_combine(const float* o2, const int32_t* slot_row, const float* weights,
                          int64_t T, int topk, int64_t H, uint16_t* y, hipStream_t s);

enum GemmMode { kGemmDense = 0, kGemmL1 = 1, kGemmL2 = 2, kGemmLora = 3 };

// Low-rank adapters of the rows of a dense GEMM (lora.hip). The shrunk rows
// scale[a] * x A_a^T are written only for rows that have an adapter and are
// zero from the adapter's rank on: v, `planes` partial sums (planes, M, R) in
// float32, and for the fused epilogue vs (M, 2R) bf16 in the listed order: the
// rounding of each sum, then the rounding of what is left (2^-17 together). b is
// (L, N, R) bf16. perm / ids list the rows grouped by adapter: row perm[i] has
// adapter ids[i] (-1: none); perm null: the rows in order, and ids (M) the
// caller's (outside [0, L): none).
struct LoraParams {
    const uint16_t* x;         // (M, K)
    const uint16_t* a;         // (L, R, K)
    const float* scale;        // (L)
    float* v;
    uint16_t* vs;
    int planes;
    const uint16_t* b;
    const int32_t* perm;
    const int32_t* ids;
    const int32_t* rank;       // (L) or null: R for all
    int64_t M, K, N;
    int L, R;
};
constexpr int64_t kLoraMaxRank = 256;
constexpr int64_t kLoraMaxAdapters = 8192;
constexpr int kLoraRows = 64;     // rows of a tile of the adapters' kernels
constexpr int kLoraStreamRows = 512;
constexpr int kLoraMaxPlanes = 8;
// How the rows are listed by adapter: streamed batches not at all (each tile
// gathers its rows), small ones by the shrink's own work-groups, larger ones by
// a launch of its own.
enum LoraOrder { kLoraAsIs = 0, kLoraRank = 1, kLoraSort = 2 };
constexpr int kLoraRankRows = 256;
// Whether M rows take the weight-streaming kernel (then A is laid out by
// launch_lora_shrink) or the tiled GEMM. Work-groups stream 32 columns for 64
// rows, one on a CU: up to two of them a CU it is faster (128 rows of 2048 x
// 4096, 128 work-groups: 21 us against 35; of 6144 x 7168, 384: 41.7 against
// 44; 512 rows of 2048 x 2048, 512: 19 to 22 against 34), with three it is not
// (160 rows of 6144 x 7168, 576: 59 against 44). Its rows are not listed by
// adapter, so each 64 rows may read every adapter again: where that is more
// than 2^25 values it costs more than it saves (rows at random, L 48: 300 rows
// of 1024 x 2048, R 128, 25 M: 34 us against 38; 512 rows of 2048 x 2048, R 64,
// 44 M: 55 against 42).
inline bool lora_streams(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    const int64_t parts = (M + kLoraRows - 1) / kLoraRows;
    return parts <= 1 || (M <= kLoraStreamRows && parts * ((N + 31) / 32) <= 512 &&
                          (parts - 1) * (L < kLoraRows ? L : kLoraRows) * R * K <= (int64_t)1 << 25);
}
constexpr int kLoraTokenRows = 4;
// Whether one launch does it all: a few rows of small adapters (every
// work-group reads their A_a: at most half a megabyte, and four turns of its
// eight waves), one round of work-groups. One row of 6144 x 7168, R 8 to 32: 14
// to 16.5 us, in two launches 16 to 17.5; twice as many turns (4 rows of R 64)
// 20 against 17, two rounds (N 12288, K 4096) 18.4 against 17.3.
inline bool lora_is_token(int64_t M, int64_t N, int64_t K, int64_t R) {
    return M <= kLoraTokenRows && N <= 8192 && M * R <= 128 && M * R * K <= 262144;
}
// bytes of the streaming kernel's A operand: rows padded to 16, K to whole
// groups of four steps for the scales
inline int64_t lora_stream_aq_bytes(int64_t M, int64_t K) { return (M + 15) / 16 * 16 * pitch_q(K); }
inline int64_t lora_stream_asf_bytes(int64_t M, int64_t K) { return (M + 15) / 16 * 16 * pitch_wsf(K); }
// number of partial sums (K ranges) of the shrink into v
int lora_planes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R);
// perm (M), sid (M) from the caller's ids (kLoraSort)
hipError_t launch_lora_sort(const int32_t* ids, int64_t M, int64_t L, int32_t* perm, int32_t* sid, hipStream_t s);
// p.v. order kLoraRank: also perm and sid (p.ids are the caller's, and
// p.perm is not read). Beside it A, in the streaming kernel's layout (aqp, asfp)
// or in its exact f16 form (ah); the others null.
hipError_t launch_lora_shrink(const LoraParams& p, LoraOrder order, int32_t* perm, int32_t* sid, const uint8_t* aq,
                              const uint8_t* asf, uint8_t* aqp, uint8_t* asfp, uint16_t* ah, hipStream_t s);
// For the fused epilogue: p.vs from p.v.
hipError_t launch_lora_join(const LoraParams& p, hipStream_t s);
// out = bf16(alpha * sum over chunks of partial[c] (M, N) + adapters)
hipError_t launch_lora_reduce(const LoraParams& p, const float* partial, int ksplit, const float* a_gs,
                              const float* b_alpha, uint16_t* out, hipStream_t s);
// out = bf16(alpha * A W + adapters) for lora_streams
hipError_t launch_lora_stream(const LoraParams& p, const uint8_t* aqp, const uint8_t* asfp, const uint8_t* bq,
                              const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out,
                              hipStream_t s);

// out = bf16(alpha * A W + adapters) for lora_is_token
hipError_t launch_lora_token(const LoraParams& p, const uint8_t* aq, const uint8_t* asf, const uint8_t* bq,
                             const uint8_t* bsf, const float* a_gs, const float* b_alpha, uint16_t* out,
                             hipStream_t s);

struct GemmParams {
    int mode;
    // A: rows of quantized activations, pitches pitch_q(K) / pitch_sf(K)
    // (weight-streaming kernel), or their exact f16 values, pitch pitch_h(K)
    // (tiled kernel)
    const uint8_t* aq;
    const uint8_t* asf;
    const uint16_t* ah;
    int64_t M;                 // dense: rows of A
    int64_t a_rows;            // rows in the A tensor (bounds of the buffer loads)
    const int32_t* a_gather;   // L1: sorted row -> slot index; token = slot / topk
    int topk;
    // B: per-expert weights, one K-packed row per output column (N rows of
    // pitch_q(K) bytes, scales N rows of pitch_wsf(K) bytes, packed layout)
    const uint8_t* bq;
    const uint8_t* bsf;
    int64_t N;                 // columns of B
    int64_t K;
    const float* a_gs;         // device scalar
    const float* b_alpha;      // device, alpha_stride per expert
    int alpha_stride;          // L1: 2 = (gate, up) per expert, else 1
    // grouped tiles
    const Tile* tiles;
    const int32_t* num_tiles;
    int64_t max_tiles;
    // outputs
    uint16_t* out_bf16;        // dense: (M, N); L1: act (S, I)
    float* out_f32;            // L2: (S, N)
    int64_t I;                 // L1: act columns (N = 2I)
    uint32_t* amax_slot;       // L1: act amax (atomic max of float bits)
    uint16_t* gu_tap;          // L1: null, or (rows, 2I) bf16 gate | up values out
    // dense with ksplit > 1: the K steps are cut into ksplit chunks, each
    // summed by its own work-groups into partial[chunk] (M, N) float32 (no
    // alpha); launch_splitk_reduce then forms out_bf16
    int ksplit;
    float* partial;
    // kGemmLora: the dense GEMM over the rows grouped by adapter, whose
    // epilogue adds the adapters (one K chunk)
    LoraParams lora;
};

hipError_t launch_gemm(const GemmParams& p, hipStream_t s);

// Number of K chunks of the dense GEMM: 1 when its tiles fill half the GPU,
// else as many as keep (tiles x chunks) within one work-group per CU, each
// chunk at least 4 K steps and none empty.
int dense_ksplit(int64_t M, int64_t N, int64_t K);

// Rows per dense GEMM tile: 128 when 256-row tiles would fill less than half
// the GPU (the split-K regime: half-height tiles double the tiles and halve
// the K chunks, and with them the partial sums written and read back), else 256.
__host__ __device__ inline int64_t dense_tile_rows(int64_t M, int64_t N) {
    const int64_t t256 = (M + kGemmBM - 1) / kGemmBM * ((N + kGemmBN - 1) / kGemmBN);
    return t256 < 128 ? kGemmBM / 2 : kGemmBM;
}

// out[m][n] = bf16((a_gs[0] * b_alpha[0]) * sum over chunks c, in order, of
// partial[c][m][n]) for (M, N), N % 4 == 0.
hipError_t launch_splitk_reduce(const float* partial, int ksplit, int64_t M, int64_t N, const float* a_gs,
                                const float* b_alpha, uint16_t* out, hipStream_t s);

// Weight-streaming variant for tiles of at most kSkinnyBM rows (L1 / L2 only).
// It stages the tile's A rows whole in LDS: skinny_lds_bytes(K) must not
// exceed kSkinnyMaxLds (K up to about 17,000).
constexpr int kSkinnyBM = 16;
constexpr int64_t kSkinnyMaxLds = 150 * 1024;
__host__ __device__ inline int64_t skinny_lds_bytes(int64_t K) {
    return (int64_t)kSkinnyBM * (pitch_q(K) + 16 + pitch_sf(K));
}
hipError_t launch_skinny(const GemmParams& p, hipStream_t s);

// Gated feed-forward block in bf16 (gated.hip). One product C = A B of a tile
// routine: M rows, `ncols` columns in tiles of tile_cols, reduction length K.
//   kGatedFwd  A = x (T, H), B = w13 (H, 2I): M = T, K = H, ncols = I act
//              columns (tile_cols = 128: as many gate as up columns a tile)
//   kGatedDx   A = dgu (T, 2I), B = w13 (H, 2I): M = T, K = 2I, ncols = H
//   kGatedDw   A = x (T, H), B = dgu (T, 2I): M = H, K = T, ncols = 2I
enum GatedMode { kGatedFwd = 0, kGatedDx = 1, kGatedDw = 2 };
constexpr int kGatedBN = 256;
struct GatedGemm {
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb;
    int64_t M, K, ncols, tile_cols, I;
    uint16_t* out;             // act (T, I), dx (T, H) or dw13 (H, 2I)
    uint16_t* gate_up;         // forward: null, or (T, 2I)
    int mi, ksplit;            // tiles of 64 mi rows, K chunks; with ksplit > 1 chunk
    float* partial;            // c writes partial[c] instead (rows as out's;
                               // forward: (T, 2I))
};
struct GatedPlan { int mi, ksplit; };   // tiles of 64 mi rows, K chunks
GatedPlan gated_forward_plan(int64_t T, int64_t H, int64_t I);
// (dx_first: the order in which one launch has the two products' work-groups)
void gated_backward_plan(int64_t T, int64_t H, int64_t I, GatedPlan& dx, GatedPlan& dw13, bool& dx_first);
hipError_t launch_gated_forward(const GatedGemm& p, hipStream_t s);
// dx and dw13 in one launch, or (the other null) one of them
hipError_t launch_gated_backward(const GatedGemm* gx, const GatedGemm* gw, bool dx_first, hipStream_t s);
// forward with ksplit > 1: sums, activation and stores
hipError_t launch_gated_reduce(const GatedGemm& p, hipStream_t s);
// out = bf16(sum over chunks of partial[c][0 .. n)), n % 4 == 0
hipError_t launch_gated_sum(const float* partial, int ksplit, int64_t n, uint16_t* out, hipStream_t s);
// gradients of gate | up (T, 2I), bf16
hipError_t launch_gated_dgu(const uint16_t* d_act, const uint16_t* gate_up, int64_t T, int64_t I, uint16_t* dgu,
                            hipStream_t s);
// zero `bytes` bytes (a multiple of 16, 16-byte aligned)
hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t s);

// Element types (enum nvfp4_dtype).
enum Dtype { kBf16 = 0, kF16 = 1, kF32 = 2 };

// Tokens sorted by expert and back (tokens.hip). slot_row (T, k): the sorted row of
// each slot; entries outside [0, R) have none.
struct SortParams {
    const void* x;             // (T, H)
    const int32_t* ids;        // (T, k)
    int64_t T, H;
    int E, k;
    void* rows;                // (T k, H)
    int32_t* offsets;          // (E + 1)
    int32_t* slot_row;         // (T, k)
    // set by launch_sort_tokens
    const int32_t* counts;     // (chunks, E)
    const int32_t* ranks;      // (T, k)
    int chunks, C, TW, parts;
};
// How the slots are ranked. Small batches: every work-group counts all ids by itself.
// Then a launch counts chunks of 256 slots and every work-group adds up the counts.
// Then the layer's routing kernels, and launch_place_rows. Measured (H 512, top 8; us,
// in this order): 48 experts, 4096 slots 6.9 in one launch; 6144 8.8, 8.6, 14.7; 16384
// 17.5, 12.1, 17.4; 65536 -, 25.1, 29.3; 256 experts, 6144 9.4, 13.0, 16.8; 16384 16.7,
// 24.1, 19.6; 32768 26.5, 38.0, 24.2; 128 experts, 24576 (12288 counts) 22.1, 20.9, 20.2.
// At the border in experts, 8192, 12288 and 16384 slots: 97 experts 11.2, 12.7, 17.7 in
// one launch, 11.3, 12.0, 14.6 in two; 128 experts 11.6, 12.8, 18.0 and 12.1, 12.9, 16.4:
// the larger border costs 97 to 128 experts up to 3 us at 16384 slots and gives 256 7.
inline bool sort_small(int64_t S, int64_t E) { return S <= (E > 96 ? 16384 : 6144); }
inline bool sort_by_counts(int64_t S, int64_t E, int64_t k) {
    return !sort_small(S, E) && k <= 256 && (S + 255) / 256 * E <= 12288;
}
inline int64_t sort_counts_bytes(int64_t S, int64_t E) { return (S + 255) / 256 * E * 4; }
// sort_small, or sort_by_counts (which takes memory for the chunks' counts, and for
// the slots' ranks: S values)
hipError_t launch_sort_tokens(int dtype, SortParams p, int32_t* counts, int32_t* ranks, hipStream_t s);
// rows[slot_row[t][j]] = x[t] for entries from 0 on
hipError_t launch_place_rows(int dtype, const void* x, const int32_t* slot_row, int64_t T, int64_t H, int k, void* rows,
                             hipStream_t s);
// y[t] = sum over j of w[t][j] (null: 1) rows[slot_row[t][j]]
hipError_t launch_gather_rows(int dtype, const void* rows, const int32_t* slot_row, const float* w, int64_t T,
                              int64_t H, int k, int64_t R, void* y, hipStream_t s);
// d_rows and dw, or one of them (the other null)
hipError_t launch_unsort_backward(int dtype, const void* dy, const void* rows, const int32_t* slot_row, const float* w,
                                  int64_t T, int64_t H, int k, int64_t R, void* d_rows, float* dw, hipStream_t s);
hipError_t launch_route_topk_backward(const float* dw, const int32_t* ids, const float* w, int64_t T, int E, int k,
                                      float* dl, hipStream_t s);

// A few rows times packed weights (matvec.hip).
struct MatvecParams {
    const void* x;             // (M, K) bf16 or f16
    const uint8_t* bq;         // E matrices of N columns, packed
    const uint8_t* bsf;
    const float* alpha;        // E, or 2 E (gate, up)
    int alpha_stride;
    const int32_t* offsets;    // (E + 1), or null: one matrix
    int64_t M, N, K;
    int E;
    bool gated;
    void* out;                 // (M, N), gated (M, N / 2)
};
// Rows of a tile: 4, 8 or 16, by the rows that a matrix has in the mean (48 experts,
// gated 4096 x 7168, tiles of 4, 8, 16 rows: mean 2.7 125, 141, 201 us; 4.0 146,
// 137, 201; 5.3 184, 155, 208; 8.0 245, 196, 216; 10.7 303, 243, 232). One matrix and
// experts share the border of 4, which fills one matrix's tile; experts with just 4
// rows in the mean would take 6 % less in tiles of 8. The host knows M alone, which
// counts rows behind the last expert's too: a share of the experts, whose rows are
// mostly those, gets larger tiles than it fills (16 of 48 experts, top 8, with the
// rows behind and without them: 16 tokens 50, 53 us; 24 74, 53; 32 81, 63; 64 79, 66).
inline int matvec_tile_rows(int64_t M, int64_t E) { return M <= 4 * E ? 4 : M <= 8 * E ? 8 : 16; }
// tiles: all there can be (E = 0: one matrix)
inline int64_t matvec_tiles(int64_t M, int64_t E) {
    const int64_t tm = matvec_tile_rows(M, E ? E : 1);
    return E ? M / tm + (E < M ? E : M) : (M + tm - 1) / tm;
}
hipError_t launch_matvec(const MatvecParams& p, int dtype, hipStream_t s);

// Dropout of n elements (dropout.hip); residual may be null; rng: seed, offset.
hipError_t launch_dropout(int dtype, const void* x, const void* residual, int64_t n, double p, const int64_t* rng,
                          void* y, hipStream_t s);

}  // namespace nvfp4
