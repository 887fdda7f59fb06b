// Tokens sorted by expert and back (gfx950): the permutation of the expert layer
// on rows of bf16, float16 or float32 values, with its gradients, and the
// router's gradient. With row(t, j) = slot_row[t][j], the sorted row of choice j
// of token t (outside [0, R): none):
//
//   sort      rows[row(t, j)] = x[t]
//             dx[t] = sum_j d_rows[row(t, j)]
//   unsort    y[t] = sum_j w[t][j] rows[row(t, j)]
//             d_rows[row(t, j)] = w[t][j] dy[t],  dw[t][j] = <dy[t], rows[row(t, j)]>
//   router    dl[t][e] = sum over j with id(t, j) = e of w_j (dw_j - sum_i w_i dw_i)
//
// Every sum is float32 in the order of j (the dot products over H: per thread, then
// over the work-group in a fixed order) and is rounded once. Nothing is added by
// atomics, so results do not depend on scheduling.
//
// All of it moves memory: a thread holds 16 bytes of one token's row, so that the sort
// reads a token once and writes its copies from registers (the gradients of the way
// back read dy once for every 8 choices), and all loads of a thread are in flight
// together. Measured, top 8 of 48 experts, H 7168 in bf16 (in
// a captured graph; floor: the bytes at the 4.9 TB/s of a copy):
//   8 tokens       sort 5.0 us, way back 3.9, both gradients 6.5 (latency)
//   1024 tokens    sort 26, way back 21, gradients 40 (partly from the last cache)
//   4096 tokens    sort 101 (108), way back 91 (108), gradients 187 (203): the
//                  memory's rate, which is higher for reads than for a copy
// Rows start at any element (odd H).
#include <algorithm>
#include <type_traits>

#include "elements.hpp"

namespace nvfp4 {

namespace {

constexpr int NT = 256;

// The token and column piece of this thread: pieces of all tokens one after
// another, C a token.
struct Piece { int64_t t; int c; };
__device__ __forceinline__ Piece piece_of(int64_t blk, int C) {
    const int64_t p0 = blk * NT, t0 = p0 / C;
    const int c = (int)(p0 - t0 * C) + (int)threadIdx.x, d = c / C;
    return {t0 + d, c - d * C};
}

// A thread a piece of one token, written to each of its rows.
template <typename T, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(NT) void place_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ slot_row,
                                                        int64_t T_, int64_t H, int k, int C, int64_t nblk,
                                                        T* __restrict__ rows) {
    const RowPieces<T, WHOLE> rp{H};
    for (int64_t b = blockIdx.x; b < nblk; b += gridDim.x) {
        const Piece p = piece_of(b, C);
        if (p.t >= T_) return;
        const int64_t at = rp.start(p.c);
        const Vec<T> v = __builtin_bit_cast(Vec<T>, rp.load(x + p.t * H + at));
        for (int j0 = 0; j0 < k; j0 += 8) {
            int32_t row[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) row[u] = j0 + u < k ? slot_row[p.t * k + j0 + u] : -1;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0) rp.template store<STREAM>(rows + (int64_t)row[u] * H + at, v);
        }
    }
}

// Ranks of a chunk of NT slots: ranks[s] = the slots of the chunk before s with its
// expert, counts[chunk][e] = all that have expert e.
__global__ __launch_bounds__(NT) void sort_count_kernel(const int32_t* __restrict__ ids, int64_t S, int E, int nbits,
                                                        int32_t* __restrict__ ranks, int32_t* __restrict__ counts) {
    extern __shared__ int32_t wave_count[];               // [NT / 64][E]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t s = (int64_t)blockIdx.x * NT + tid;
    for (int i = tid; i < NT / 64 * E; i += NT) wave_count[i] = 0;
    const int e = s < S ? ids[s] : -1;
    const bool valid = e >= 0 && e < E;
    uint64_t match = __ballot(valid);                     // lanes of this wave with the same expert
    for (int b = 0; b < nbits; ++b) {
        const bool bit = valid && ((e >> b) & 1);
        const uint64_t bl = __ballot(bit);
        match &= bit ? bl : ~bl;
    }
    int rank = __popcll(match & ~(~0ull << lane));
    __syncthreads();
    if (valid && rank == 0) wave_count[wave * E + e] = __popcll(match);
    __syncthreads();
    for (int v = 0; v < wave; ++v)
        if (valid) rank += wave_count[v * E + e];
    if (s < S) ranks[s] = rank;
    for (int i = tid; i < E; i += NT) {
        int sum = 0;
#pragma unroll
        for (int v = 0; v < NT / 64; ++v) sum += wave_count[v * E + i];
        counts[(int64_t)blockIdx.x * E + i] = sum;
    }
}

// TW tokens of a work-group (their slots lie in two chunks at most), of which it
// moves one of `parts` ranges of pieces. It finds its slots' rows by itself: the
// experts' totals, and of each expert the slots before its first one, from all ids
// (SMALL) or from the chunks' counts. The first work-group writes offsets, those of
// the first range slot_row. The counts are added up by atomics in LDS, so slots that
// all name one expert meet at one address: 4096 slots of 48 experts, H 512, 16.9 us
// (SMALL) where evenly drawn ones take 6.5, and as many where only one choice of each
// token is the same (6.7); 16384 slots, by counts of chunks, 12.1 either way.
template <typename T, bool STREAM, bool SMALL, bool WHOLE>
__global__ __launch_bounds__(NT) void sort_rows_kernel(SortParams p) {
    extern __shared__ int32_t lds[];
    int32_t* first = lds;                                 // [E + 1]: the totals, then each expert's first row
    int32_t* before = first + p.E + 1;                    // [E]
    int32_t* row = before + p.E;                          // [TW k]
    int32_t* id = row + p.TW * p.k;                       // [TW k]
    const int tid = threadIdx.x, lane = tid & 63, E = p.E;
    const int64_t group = blockIdx.x / p.parts;
    const int part = (int)(blockIdx.x - group * p.parts);
    const int64_t t0 = group * p.TW, s0 = t0 * p.k;
    const int tokens = (int)min((int64_t)p.TW, p.T - t0), slots = tokens * p.k;
    const int64_t g0 = s0 / NT;
    for (int i = tid; i < 2 * E + 1; i += NT) first[i] = 0;
    for (int i = tid; i < slots; i += NT) {
        const int e = p.ids[s0 + i];
        id[i] = e >= 0 && e < E ? e : -1;
    }
    __syncthreads();
    constexpr int U = 8;                                  // loads in flight
    const int n = SMALL ? (int)(p.T * p.k) : p.chunks * E;
    for (int i0 = tid; i0 < n; i0 += U * NT) {
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) at[u] = i0 + u * NT < n ? (SMALL ? p.ids : p.counts)[i0 + u * NT] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NT;
            if (SMALL) {
                if (at[u] < 0 || at[u] >= E) continue;
                atomicAdd(&first[at[u]], 1);
                if (i < s0) atomicAdd(&before[at[u]], 1);
            } else if (at[u] > 0) {
                const int h = i / E, e = i - h * E;
                atomicAdd(&first[e], at[u]);
                if (h < g0) atomicAdd(&before[e], at[u]);
            }
        }
    }
    __syncthreads();
    if (tid < 64) {                                       // exclusive scan, 64 experts at a time
        int sum = 0;
        for (int e0 = 0; e0 <= E; e0 += 64) {
            const int c = e0 + lane < E ? first[e0 + lane] : 0;
            int inc = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(inc, d);
                if (lane >= d) inc += up;
            }
            if (e0 + lane <= E) first[e0 + lane] = sum + inc - c;
            sum += __shfl(inc, 63);
        }
    }
    __syncthreads();
    for (int i = tid; i < slots; i += NT) {
        const int e = id[i];
        int r = -1;
        if (e >= 0) {
            r = first[e] + before[e];
            if (SMALL) {
                for (int u = 0; u < i; ++u) r += id[u] == e;
            } else {
                r += p.ranks[s0 + i];
                if ((s0 + i) / NT > g0) r += p.counts[g0 * E + e];
            }
        }
        row[i] = r;
    }
    __syncthreads();
    if (part == 0)
        for (int i = tid; i < slots; i += NT) p.slot_row[s0 + i] = row[i];
    if (blockIdx.x == 0)
        for (int i = tid; i <= E; i += NT) p.offsets[i] = first[i];

    // pieces, four of them in flight (beyond the last: it again, not written)
    const RowPieces<T, WHOLE> rp{p.H};
    const T* x = static_cast<const T*>(p.x);
    T* rows = static_cast<T*>(p.rows);
    const int per = (p.C + p.parts - 1) / p.parts, c0 = part * per, width = min(per, p.C - c0);
    if (width <= 0) return;
    const int pieces = tokens * width;
    constexpr int P = 4;
    for (int i0 = tid; i0 < pieces; i0 += P * NT) {
        u32x4 v[P];
        int64_t at[P];
        int token[P];
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int i = min(i0 + u * NT, pieces - 1);
            token[u] = i / width;
            at[u] = rp.start(c0 + i - token[u] * width);
            v[u] = rp.load(x + (t0 + token[u]) * p.H + at[u]);
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            if (i0 + u * NT >= pieces) break;
            for (int j = 0; j < p.k; ++j) {
                const int r = row[token[u] * p.k + j];
                if (r >= 0) rp.template store<STREAM>(rows + (int64_t)r * p.H + at[u], __builtin_bit_cast(Vec<T>, v[u]));
            }
        }
    }
}

// The sum over a token's rows, with weights or (w null) without.
template <typename T, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(NT) void gather_rows_kernel(const T* __restrict__ rows,
                                                         const int32_t* __restrict__ slot_row,
                                                         const float* __restrict__ w, int64_t T_, int64_t H, int k,
                                                         int64_t R, int C, int64_t nblk, T* __restrict__ y) {
    constexpr int V = kVec<T>;
    const RowPieces<T, WHOLE> rp{H};
    for (int64_t b = blockIdx.x; b < nblk; b += gridDim.x) {
        const Piece p = piece_of(b, C);
        if (p.t >= T_) return;
        const int64_t at = rp.start(p.c);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < k; j0 += 8) {
            int32_t row[8];
            float wj[8];
            u32x4 raw[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                row[u] = j0 + u < k ? slot_row[p.t * k + j0 + u] : -1;
                wj[u] = w && j0 + u < k ? w[p.t * k + j0 + u] : 1.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0 && row[u] < R) raw[u] = rp.template load<STREAM>(rows + (int64_t)row[u] * H + at);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0 && row[u] < R) {
                    const Vec<T> v = __builtin_bit_cast(Vec<T>, raw[u]);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(wj[u], to_f32(v.v[i]), acc[i]);
                }
        }
        Vec<T> out;
#pragma unroll
        for (int i = 0; i < V; ++i) out.v[i] = from_f32<T>(acc[i]);
        rp.store(y + p.t * H + at, out);
    }
}

// Sums over the wave's lanes of eight values, in a fixed order: of value lane / 8 in
// each lane (ten exchanges, where eight sums alone take 48).
__device__ __forceinline__ float wave_sum8(const float (&d)[8], int lane) {
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (lane & 32 ? d[i + 4] : d[i]) + __shfl_xor(lane & 32 ? d[i] : d[i + 4], 32, 64);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (lane & 16 ? a[i + 2] : a[i]) + __shfl_xor(lane & 16 ? a[i] : a[i + 2], 16, 64);
    c = (lane & 8 ? b[1] : b[0]) + __shfl_xor(lane & 8 ? b[0] : b[1], 8, 64);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) c += __shfl_xor(c, off, 64);
    return c;
}

// One work-group a token: d_rows (null: not wanted) and dw (null: not wanted). The
// token's rows are the same for the whole work-group, so their addresses and the
// branches on them are scalar.
template <typename T, bool STREAM, bool WHOLE, int TB>
__global__ __launch_bounds__(TB) void unsort_backward_kernel(const T* __restrict__ dy, const T* __restrict__ rows,
                                                             const int32_t* __restrict__ slot_row,
                                                             const float* __restrict__ w, int64_t T_, int64_t H, int k,
                                                             int64_t R, int C, T* __restrict__ d_rows,
                                                             float* __restrict__ dw) {
    constexpr int V = kVec<T>, J = 8;                     // choices at a time
    __shared__ float red[TB / 64][J];
    const RowPieces<T, WHOLE> rp{H};
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
        for (int j0 = 0; j0 < k; j0 += J) {
            int32_t row[J];
            float wj[J], dot[J];
#pragma unroll
            for (int u = 0; u < J; ++u) {
                const int32_t r = j0 + u < k ? __builtin_amdgcn_readfirstlane(slot_row[t * k + j0 + u]) : -1;
                row[u] = r < R ? r : -1;
                wj[u] = d_rows && j0 + u < k ? w[t * k + j0 + u] : 0.0f;
                dot[u] = 0.0f;
            }
            for (int c = tid; c < C; c += TB) {
                const int64_t at = rp.start(c);
                const u32x4 graw = rp.load(dy + t * H + at);
                u32x4 raw[J];
                if (dw) {
#pragma unroll
                    for (int u = 0; u < J; ++u)
                        if (row[u] >= 0) raw[u] = rp.template load<STREAM>(rows + (int64_t)row[u] * H + at);
                }
                const Vec<T> g = __builtin_bit_cast(Vec<T>, graw);
                if (dw) {
                    // the last piece's first elements, which the piece before counts, do not count
                    const int skip = WHOLE ? (int)((int64_t)c * V - at) : 0;
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        if (row[u] < 0) continue;
                        const Vec<T> v = __builtin_bit_cast(Vec<T>, raw[u]);
                        if (skip == 0) {
#pragma unroll
                            for (int i = 0; i < V; ++i) dot[u] = __builtin_fmaf(to_f32(g.v[i]), to_f32(v.v[i]), dot[u]);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                if (i >= skip) dot[u] = __builtin_fmaf(to_f32(g.v[i]), to_f32(v.v[i]), dot[u]);
                        }
                    }
                }
                if (d_rows) {
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        if (row[u] < 0) continue;
                        Vec<T> o;
#pragma unroll
                        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(wj[u] * to_f32(g.v[i]));
                        rp.template store<STREAM>(d_rows + (int64_t)row[u] * H + at, o);
                    }
                }
            }
            if (dw) {
                const float mine = wave_sum8(dot, lane);
                if ((lane & 7) == 0) red[wave][lane >> 3] = mine;
                __syncthreads();
                if (tid < J && j0 + tid < k) {
                    float s = red[0][tid];
#pragma unroll
                    for (int v = 1; v < TB / 64; ++v) s += red[v][tid];
                    dw[t * k + j0 + tid] = s;
                }
                __syncthreads();
            }
        }
    }
}

// TB tokens of a work-group: their gradients are put together in LDS, a thread for
// each choice, and written as they lie. An expert that a token names more than once
// has the sum over its choices in order, made by the first of them.
__global__ __launch_bounds__(NT) void route_topk_backward_kernel(const float* __restrict__ dw,
                                                                 const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ w, int64_t T_, int E, int k,
                                                                 int TB, float* __restrict__ dl) {
    extern __shared__ __attribute__((aligned(16))) float out[];      // [TB][E], then the choices' weights, dw and ids
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * TB;
    const int tokens = (int)min((int64_t)TB, T_ - t0), n = tokens * E, m = tokens * k;
    float* lw = out + (TB * E + 3) / 4 * 4;
    float* ld = lw + TB * k;
    int32_t* lid = reinterpret_cast<int32_t*>(ld + TB * k);
    for (int i = tid; i < m; i += NT) {
        lw[i] = w[t0 * k + i];
        ld[i] = dw[t0 * k + i];
        lid[i] = ids[t0 * k + i];
    }
    for (int i = 4 * tid; i < n; i += 4 * NT) *reinterpret_cast<float4_t*>(out + i) = (float4_t){0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    for (int i = tid; i < m; i += NT) {
        const int t = i / k, j = i - t * k, id = lid[i];
        const float *tw = lw + t * k, *td = ld + t * k;
        float s = 0.0f;
        bool first = id >= 0 && id < E;
        for (int u = 0; u < k; ++u) {
            s = __builtin_fmaf(tw[u], td[u], s);
            if (u < j && lid[t * k + u] == id) first = false;
        }
        if (!first) continue;
        float v = tw[j] * (td[j] - s);
        for (int u = j + 1; u < k; ++u)
            if (lid[t * k + u] == id) v += tw[u] * (td[u] - s);
        out[t * E + id] = v;
    }
    __syncthreads();
    float* to = dl + t0 * E;
    for (int i = 4 * tid; i < n; i += 4 * NT) {
        Vec<float> v;
        __builtin_memcpy(&v, out + i, 16);
        if (n - i >= 4) store_vec(to + i, v);
        else store_part(to + i, v, n - i);
    }
}

constexpr int64_t kMaxGrid = (int64_t)1 << 22;             // work-groups (a launch has fewer than 2^32 threads)

template <typename T>
struct Pieces {
    int C;
    int64_t nblk;
    unsigned grid;
    Pieces(int64_t T_, int64_t H) {
        C = (int)((H + kVec<T> - 1) / kVec<T>);
        nblk = (T_ * C + NT - 1) / NT;
        grid = (unsigned)(nblk < kMaxGrid ? nblk : kMaxGrid);
    }
};

// Whether rows of so many bytes in all (slots without a row counted in: the host does
// not know them) pass by the caches: those that do not fit the last one (256 MB), where they push out what follows (4096 tokens of 7168, top 8, 448
// MB: sort 101 against 117 us, its way back 90 against 103, both gradients 187 against
// 201). Smaller ones are found there by whoever reads them next (1024 tokens, 112 MB:
// the four calls one after another 136 against 106 us).
bool streams(int64_t bytes) { return bytes >= (int64_t)256 << 20; }

// Tokens of a work-group, about 1024 of those; for few tokens ranges of its pieces
// down to one a thread (8 tokens of 896 pieces: 2 ranges 6.1 us, 4 5.0, 8 5.0).
void sort_plan(SortParams& p) {
    int64_t tw = (p.T + 1023) / 1024;
    tw = std::min<int64_t>(tw, NT / p.k > 0 ? NT / p.k : 1);
    p.TW = (int)std::max<int64_t>(tw, 1);
    const int64_t groups = (p.T + p.TW - 1) / p.TW;
    int parts = 1;
    while (groups * parts < 512 && (int64_t)p.TW * p.C / (2 * parts) >= NT / 2) parts *= 2;
    p.parts = parts;
}

template <typename F>
void with_flag(bool on, F&& f) {
    if (on) f(std::true_type());
    else f(std::false_type());
}

}  // namespace

hipError_t launch_sort_tokens(int dtype, SortParams p, int32_t* counts, int32_t* ranks, hipStream_t s) {
    const int64_t S = p.T * p.k;
    const bool small = sort_small(S, p.E);
    p.chunks = (int)((S + NT - 1) / NT);
    p.counts = counts;
    p.ranks = ranks;
    if (!small) {
        int nbits = 1;
        while ((1 << nbits) < p.E) ++nbits;
        sort_count_kernel<<<(unsigned)p.chunks, NT, sizeof(int32_t) * (NT / 64) * p.E, s>>>(p.ids, S, p.E, nbits,
                                                                                         ranks, counts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        p.C = (int)((p.H + kVec<V> - 1) / kVec<V>);
        sort_plan(p);
        const int64_t grid = (p.T + p.TW - 1) / p.TW * p.parts;
        const size_t lds = sizeof(int32_t) * (2 * (size_t)p.E + 1 + 2 * (size_t)p.TW * p.k);
        with_flag(streams(S * p.H * (int64_t)sizeof(V)), [&](auto stream) {
            with_flag(small, [&](auto sm) {
                with_flag(p.H >= kVec<V>, [&](auto whole) {
                    sort_rows_kernel<V, decltype(stream)::value, decltype(sm)::value, decltype(whole)::value>
                        <<<(unsigned)grid, NT, lds, s>>>(p);
                });
            });
        });
    });
}

hipError_t launch_place_rows(int dtype, const void* x, const int32_t* slot_row, int64_t T, int64_t H, int k, void* rows,
                             hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        with_flag(streams(T * k * H * (int64_t)sizeof(V)), [&](auto stream) {
            with_flag(H >= kVec<V>, [&](auto whole) {
                place_rows_kernel<V, decltype(stream)::value, decltype(whole)::value><<<p.grid, NT, 0, s>>>(
                    static_cast<const V*>(x), slot_row, T, H, k, p.C, p.nblk, static_cast<V*>(rows));
            });
        });
    });
}

hipError_t launch_gather_rows(int dtype, const void* rows, const int32_t* slot_row, const float* w, int64_t T,
                              int64_t H, int k, int64_t R, void* y, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        with_flag(streams(T * k * H * (int64_t)sizeof(V)), [&](auto stream) {
            with_flag(H >= kVec<V>, [&](auto whole) {
                gather_rows_kernel<V, decltype(stream)::value, decltype(whole)::value><<<p.grid, NT, 0, s>>>(
                    static_cast<const V*>(rows), slot_row, w, T, H, k, R, p.C, p.nblk, static_cast<V*>(y));
            });
        });
    });
}

hipError_t launch_unsort_backward(int dtype, const void* dy, const void* rows, const int32_t* slot_row, const float* w,
                                  int64_t T, int64_t H, int k, int64_t R, void* d_rows, float* dw, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        with_flag(streams(T * k * H * (int64_t)sizeof(V) * (d_rows && dw ? 2 : 1)), [&](auto stream) {
            // A piece a thread for few tokens (8 of 7168 bf16 values, 896 pieces: 256 threads
            // 9.4 us, 512 6.9, 1024 6.4; of 2048, 256 pieces: 64 threads 8.5, 256 4.9), no
            // idle ones for short rows (4096 tokens of 512: 64 threads 13.8, 256 16.7, 512
            // 23.1; of 2048: 70, 55, 55), and more work-groups than 1024 threads leave room
            // for (1024 tokens of 4096: 512 threads 23.8, 1024 28.3).
            auto run = [&](auto threads, auto whole) {
                constexpr int TB = decltype(threads)::value;
                unsort_backward_kernel<V, decltype(stream)::value, decltype(whole)::value, TB>
                    <<<(unsigned)std::min(T, kMaxGrid / 4), TB, 0, s>>>(static_cast<const V*>(dy),
                                                                        static_cast<const V*>(rows), slot_row, w, T, H,
                                                                        k, R, p.C, static_cast<V*>(d_rows), dw);
            };
            const std::true_type whole;
            if (H < kVec<V>) run(std::integral_constant<int, 64>(), std::false_type());
            else if (p.C <= 64) run(std::integral_constant<int, 64>(), whole);
            else if (p.C <= 256) run(std::integral_constant<int, 256>(), whole);
            else if (p.C <= 512 || T > 256) run(std::integral_constant<int, 512>(), whole);
            else run(std::integral_constant<int, 1024>(), whole);
        });
    });
}

hipError_t launch_route_topk_backward(const float* dw, const int32_t* ids, const float* w, int64_t T, int E, int k,
                                      float* dl, hipStream_t s) {
    // tokens of a work-group: what fills 32 KB of LDS, but 512 work-groups
    int64_t tb = 8192 / (E + 3 * k);
    tb = std::max<int64_t>(1, std::min<int64_t>(tb, (T + 511) / 512));
    const size_t lds = sizeof(float) * ((size_t)(tb * E + 3) / 4 * 4 + 3 * (size_t)(tb * k));
    route_topk_backward_kernel<<<(unsigned)((T + tb - 1) / tb), NT, lds, s>>>(dw, ids, w, T, E, k, (int)tb, dl);
    return hipGetLastError();
}

}  // namespace nvfp4
