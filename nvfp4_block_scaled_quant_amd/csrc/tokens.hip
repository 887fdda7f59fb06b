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
// All of it moves memory: a thread holds 16 bytes of one token's row, so that a
// token is read once and its copies are written from registers. Rows start at
// any element (odd H): the loads and stores are declared at the element's
// alignment, which global memory instructions of 16 bytes allow.
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
template <typename T, bool STREAM>
__global__ __launch_bounds__(NT) void place_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ slot_row,
                                                        int64_t T_, int64_t H, int k, int C, int64_t nblk,
                                                        T* __restrict__ rows) {
    constexpr int V = kVec<T>;
    for (int64_t b = blockIdx.x; b < nblk; b += gridDim.x) {
        const Piece p = piece_of(b, C);
        if (p.t >= T_) return;
        const int n = (int)min((int64_t)V, H - (int64_t)p.c * V);
        const Vec<T> v = load_vec(x + p.t * H + (int64_t)p.c * V, n);
        for (int j0 = 0; j0 < k; j0 += 8) {
            int32_t row[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) row[u] = j0 + u < k ? slot_row[p.t * k + j0 + u] : -1;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0) store_vec<T, STREAM>(rows + (int64_t)row[u] * H + (int64_t)p.c * V, v, n);
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
// the first range slot_row.
template <typename T, bool STREAM, bool SMALL>
__global__ __launch_bounds__(NT) void sort_rows_kernel(SortParams p) {
    constexpr int V = kVec<T>;
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

    // pieces, four of them in flight
    const T* x = static_cast<const T*>(p.x);
    T* rows = static_cast<T*>(p.rows);
    const int per = (p.C + p.parts - 1) / p.parts, c0 = part * per, width = min(per, p.C - c0);
    if (width <= 0) return;
    const int pieces = tokens * width;
    constexpr int P = 4;
    for (int i0 = tid; i0 < pieces; i0 += P * NT) {
        Vec<T> v[P];
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int i = i0 + u * NT, tt = i / width;
            const int64_t c = (int64_t)(c0 + i - tt * width) * V;
            if (i < pieces) v[u] = load_vec(x + (t0 + tt) * p.H + c, (int)min((int64_t)V, p.H - c));
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
            const int i = i0 + u * NT, tt = i / width;
            const int64_t c = (int64_t)(c0 + i - tt * width) * V;
            if (i >= pieces) break;
            for (int j = 0; j < p.k; ++j) {
                const int r = row[tt * p.k + j];
                if (r >= 0) store_vec<T, STREAM>(rows + (int64_t)r * p.H + c, v[u], (int)min((int64_t)V, p.H - c));
            }
        }
    }
}

// The sum over a token's rows, with weights or (w null) without.
template <typename T, bool STREAM>
__global__ __launch_bounds__(NT) void gather_rows_kernel(const T* __restrict__ rows,
                                                         const int32_t* __restrict__ slot_row,
                                                         const float* __restrict__ w, int64_t T_, int64_t H, int k,
                                                         int64_t R, int C, int64_t nblk, T* __restrict__ y) {
    constexpr int V = kVec<T>;
    for (int64_t b = blockIdx.x; b < nblk; b += gridDim.x) {
        const Piece p = piece_of(b, C);
        if (p.t >= T_) return;
        const int n = (int)min((int64_t)V, H - (int64_t)p.c * V);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < k; j0 += 8) {
            int32_t row[8];
            float wj[8];
            Vec<T> v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                row[u] = j0 + u < k ? slot_row[p.t * k + j0 + u] : -1;
                wj[u] = w && j0 + u < k ? w[p.t * k + j0 + u] : 1.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0 && row[u] < R) v[u] = load_vec<T, STREAM>(rows + (int64_t)row[u] * H + (int64_t)p.c * V, n);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (row[u] >= 0 && row[u] < R) {
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(wj[u], to_f32(v[u].v[i]), acc[i]);
                }
        }
        Vec<T> out;
#pragma unroll
        for (int i = 0; i < V; ++i) out.v[i] = from_f32<T>(acc[i]);
        store_vec(y + p.t * H + (int64_t)p.c * V, out, n);
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
template <typename T, bool STREAM, int TB>
__global__ __launch_bounds__(TB) void unsort_backward_kernel(const T* __restrict__ dy, const T* __restrict__ rows,
                                                             const int32_t* __restrict__ slot_row,
                                                             const float* __restrict__ w, int64_t T_, int64_t H, int k,
                                                             int64_t R, int C, T* __restrict__ d_rows,
                                                             float* __restrict__ dw) {
    constexpr int V = kVec<T>, J = 8;                     // choices at a time
    __shared__ float red[TB / 64][J];
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
                const int n = (int)min((int64_t)V, H - (int64_t)c * V);
                const Vec<T> g = load_vec(dy + t * H + (int64_t)c * V, n);
                Vec<T> v[J];
                if (dw) {
#pragma unroll
                    for (int u = 0; u < J; ++u)
                        if (row[u] >= 0) v[u] = load_vec<T, STREAM>(rows + (int64_t)row[u] * H + (int64_t)c * V, n);
                }
                if (d_rows) {
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        if (row[u] < 0) continue;
                        Vec<T> o;
#pragma unroll
                        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(wj[u] * to_f32(g.v[i]));
                        store_vec<T, STREAM>(d_rows + (int64_t)row[u] * H + (int64_t)c * V, o, n);
                    }
                }
                if (dw) {
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        if (row[u] < 0) continue;
#pragma unroll
                        for (int i = 0; i < V; ++i) dot[u] = __builtin_fmaf(to_f32(g.v[i]), to_f32(v[u].v[i]), dot[u]);
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
        store_vec(to + i, v, n - i);
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

// Whether rows of so many bytes in all pass by the caches: those that do not fit the
// last one (256 MB), where they push out what follows (4096 tokens, 448 MB: sort 104
// against 115 us, both gradients of the way back 222 against 239). Smaller ones are
// found there by whoever reads them next (1024 tokens, 112 MB: the four calls one
// after another 157 against 127 us).
bool streams(int64_t bytes) { return bytes >= (int64_t)256 << 20; }

// Tokens of a work-group and ranges of its pieces: about 1024 work-groups, and four
// pieces a thread.
void sort_plan(SortParams& p) {
    int64_t tw = (p.T + 1023) / 1024;
    tw = std::min<int64_t>(tw, NT / p.k > 0 ? NT / p.k : 1);
    p.TW = (int)std::max<int64_t>(tw, 1);
    const int64_t groups = (p.T + p.TW - 1) / p.TW;
    int parts = 1;
    while (groups * parts < 512 && (int64_t)p.TW * p.C / (2 * parts) >= NT) parts *= 2;
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
                sort_rows_kernel<V, decltype(stream)::value, decltype(sm)::value><<<(unsigned)grid, NT, lds, s>>>(p);
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
            place_rows_kernel<V, decltype(stream)::value>
                <<<p.grid, NT, 0, s>>>(static_cast<const V*>(x), slot_row, T, H, k, p.C, p.nblk, static_cast<V*>(rows));
        });
    });
}

hipError_t launch_gather_rows(int dtype, const void* rows, const int32_t* slot_row, const float* w, int64_t T,
                              int64_t H, int k, int64_t R, void* y, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        with_flag(streams(T * k * H * (int64_t)sizeof(V)), [&](auto stream) {
            gather_rows_kernel<V, decltype(stream)::value><<<p.grid, NT, 0, s>>>(
                static_cast<const V*>(rows), slot_row, w, T, H, k, R, p.C, p.nblk, static_cast<V*>(y));
        });
    });
}

hipError_t launch_unsort_backward(int dtype, const void* dy, const void* rows, const int32_t* slot_row, const float* w,
                                  int64_t T, int64_t H, int k, int64_t R, void* d_rows, float* dw, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        with_flag(streams(T * k * H * (int64_t)sizeof(V) * (d_rows && dw ? 2 : 1)), [&](auto stream) {
            // a piece a thread while the tokens do not fill the GPU (8 tokens of 7168: 256
            // threads 17.7 us, 512 12.0, 1024 10.3), then 512 threads (1024 tokens: 44, 47
            // and 54 us, 4096: 230, 222 and 225)
            auto run = [&](auto threads) {
                constexpr int TB = decltype(threads)::value;
                unsort_backward_kernel<V, decltype(stream)::value, TB>
                    <<<(unsigned)std::min(T, kMaxGrid / 4), TB, 0, s>>>(static_cast<const V*>(dy),
                                                                        static_cast<const V*>(rows), slot_row, w, T, H,
                                                                        k, R, p.C, static_cast<V*>(d_rows), dw);
            };
            if (p.C <= 64) run(std::integral_constant<int, 64>());
            else if (p.C <= 512 || T > 256) run(std::integral_constant<int, 512>());
            else run(std::integral_constant<int, 1024>());
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
