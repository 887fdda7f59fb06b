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

template <typename T>
__global__ __launch_bounds__(NT) void sort_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ slot_row,
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
                if (row[u] >= 0) store_vec(rows + (int64_t)row[u] * H + (int64_t)p.c * V, v, n);
        }
    }
}

// The sum over a token's rows, with weights or (w null) without.
template <typename T>
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
                if (row[u] >= 0 && row[u] < R) v[u] = load_vec(rows + (int64_t)row[u] * H + (int64_t)p.c * V, n);
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

// Sum over the wave's lanes, the same in every lane and in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// One work-group a token: d_rows (null: not wanted) and dw (null: not wanted).
template <typename T>
__global__ __launch_bounds__(NT) void unsort_backward_kernel(const T* __restrict__ dy, const T* __restrict__ rows,
                                                             const int32_t* __restrict__ slot_row,
                                                             const float* __restrict__ w, int64_t T_, int64_t H, int k,
                                                             int64_t R, int C, T* __restrict__ d_rows,
                                                             float* __restrict__ dw) {
    constexpr int V = kVec<T>;
    __shared__ float red[NT / 64][8];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
        for (int j0 = 0; j0 < k; j0 += 8) {
            int32_t row[8];
            float wj[8], dot[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int32_t r = j0 + u < k ? slot_row[t * k + j0 + u] : -1;
                row[u] = r < R ? r : -1;
                wj[u] = j0 + u < k ? w[t * k + j0 + u] : 0.0f;
                dot[u] = 0.0f;
            }
            for (int c = tid; c < C; c += NT) {
                const int n = (int)min((int64_t)V, H - (int64_t)c * V);
                const Vec<T> g = load_vec(dy + t * H + (int64_t)c * V, n);
                Vec<T> v[8];
                if (dw) {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (row[u] >= 0) v[u] = load_vec(rows + (int64_t)row[u] * H + (int64_t)c * V, n);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (row[u] < 0) continue;
                    if (dw) {
#pragma unroll
                        for (int i = 0; i < V; ++i) dot[u] = __builtin_fmaf(to_f32(g.v[i]), to_f32(v[u].v[i]), dot[u]);
                    }
                    if (d_rows) {
                        Vec<T> o;
#pragma unroll
                        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(wj[u] * to_f32(g.v[i]));
                        store_vec(d_rows + (int64_t)row[u] * H + (int64_t)c * V, o, n);
                    }
                }
            }
            if (dw) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float s = wave_sum(dot[u]);
                    if (lane == 0) red[wave][u] = s;
                }
                __syncthreads();
                if (tid < 8 && j0 + tid < k) {
                    float s = red[0][tid];
#pragma unroll
                    for (int v = 1; v < NT / 64; ++v) s += red[v][tid];
                    dw[t * k + j0 + tid] = s;
                }
                __syncthreads();
            }
        }
    }
}

// One wave a token, a lane for every 64th choice and every 64th expert. An
// expert's value is the sum over the choices that have it, in order (one at
// most, as the router gives them).
constexpr int kGradWaves = 4;
__global__ __launch_bounds__(64 * kGradWaves) void route_topk_backward_kernel(
    const float* __restrict__ dw, const int32_t* __restrict__ ids, const float* __restrict__ w, int64_t T_, int E,
    int k, float* __restrict__ dl) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kGradWaves + (threadIdx.x >> 6);
    if (t >= T_) return;                      // uniform per wave
    float s = 0.0f;
    for (int j = lane; j < k; j += 64) s = __builtin_fmaf(w[t * k + j], dw[t * k + j], s);
    s = wave_sum(s);
    float acc[kMaxExperts / 64];
#pragma unroll
    for (int i = 0; i < kMaxExperts / 64; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 64) {
        const int j = j0 + lane;
        const int id = j < k ? ids[t * k + j] : -1;
        const float v = j < k ? w[t * k + j] * (dw[t * k + j] - s) : 0.0f;
        const int m = min(64, k - j0);
        for (int u = 0; u < m; ++u) {
            const int e = __builtin_amdgcn_readlane(id, u);
            const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), u));
#pragma unroll
            for (int i = 0; i < kMaxExperts / 64; ++i) acc[i] += e == 64 * i + lane ? d : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < kMaxExperts / 64; ++i)
        if (64 * i + lane < E) dl[t * E + 64 * i + lane] = acc[i];
}

constexpr int64_t kMaxGrid = (int64_t)1 << 30;

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

}  // namespace

hipError_t launch_sort_rows(int dtype, const void* x, const int32_t* slot_row, int64_t T, int64_t H, int k, void* rows,
                            hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        sort_rows_kernel<V><<<p.grid, NT, 0, s>>>(static_cast<const V*>(x), slot_row, T, H, k, p.C, p.nblk,
                                                  static_cast<V*>(rows));
    });
}

hipError_t launch_gather_rows(int dtype, const void* rows, const int32_t* slot_row, const float* w, int64_t T,
                              int64_t H, int k, int64_t R, void* y, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        gather_rows_kernel<V><<<p.grid, NT, 0, s>>>(static_cast<const V*>(rows), slot_row, w, T, H, k, R, p.C, p.nblk,
                                                    static_cast<V*>(y));
    });
}

hipError_t launch_unsort_backward(int dtype, const void* dy, const void* rows, const int32_t* slot_row, const float* w,
                                  int64_t T, int64_t H, int k, int64_t R, void* d_rows, float* dw, hipStream_t s) {
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const Pieces<V> p(T, H);
        unsort_backward_kernel<V><<<(unsigned)T, NT, 0, s>>>(static_cast<const V*>(dy), static_cast<const V*>(rows),
                                                             slot_row, w, T, H, k, R, p.C, static_cast<V*>(d_rows), dw);
    });
}

hipError_t launch_route_topk_backward(const float* dw, const int32_t* ids, const float* w, int64_t T, int E, int k,
                                      float* dl, hipStream_t s) {
    const int64_t grid = (T + kGradWaves - 1) / kGradWaves;
    route_topk_backward_kernel<<<(unsigned)grid, 64 * kGradWaves, 0, s>>>(dw, ids, w, T, E, k, dl);
    return hipGetLastError();
}

}  // namespace nvfp4
