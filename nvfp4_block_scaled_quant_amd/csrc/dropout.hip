// Dropout from a counter-based generator (gfx950): y = x / (1 - p) where an
// element is kept, zero where it is not, optionally added to a residual. The
// gradient is the same function of dy: the mask is computed again from the
// element's index and never stored.
//
// The generator is Philox4x32 (Salmon, Moraes, Dror, Shaw: Parallel random
// numbers: as easy as 1, 2, 3, SC 2011) in seven rounds, the fewest that the
// authors found to pass all of their statistical tests: element i takes word i % 4
// of the counter offset + i / 4 under the key `seed`, and is kept where that word
// is at least p 2^32.
//
// Bound by memory: the generator's 14 64-bit products for four elements run while
// other waves' loads are in flight. 4096 x 7168 in bf16 20.8 us (a copy: 19.0), with
// the residual 28.3 (6.2 TB/s); 2^28 float32 348 us (a copy: 431).
#include <type_traits>

#include "elements.hpp"

namespace nvfp4 {

namespace {

constexpr int NT = 256;
constexpr int kRounds = 7;

__device__ __forceinline__ void philox(uint64_t counter, uint64_t seed, uint32_t (&w)[4]) {
    uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// least = p 2^32; none: p = 1, nothing is kept.
template <typename T>
__global__ __launch_bounds__(NT) void dropout_kernel(const T* x, const T* residual, int64_t n,
                                                     uint32_t least, bool none, float scale,
                                                     const int64_t* __restrict__ rng, T* y) {
    constexpr int V = kVec<T>;
    const uint64_t seed = (uint64_t)rng[0], offset = (uint64_t)rng[1];
    for (int64_t i = ((int64_t)blockIdx.x * NT + threadIdx.x) * V; i < n; i += (int64_t)gridDim.x * NT * V) {
        const int m = (int)min((int64_t)V, n - i);
        auto piece = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
            const Vec<T> v = W ? load_vec(x + i) : load_part(x + i, m);
            Vec<T> r, out;
            if (residual) r = W ? load_vec(residual + i) : load_part(residual + i, m);
#pragma unroll
            for (int h = 0; h < V / 4; ++h) {
                uint32_t w[4];
                philox(offset + (uint64_t)(i / 4 + h), seed, w);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool keep = w[u] >= least && !none;
                    float f = keep ? to_f32(v.v[4 * h + u]) * scale : 0.0f;
                    if (residual) f = to_f32(r.v[4 * h + u]) + f;
                    out.v[4 * h + u] = from_f32<T>(f);
                }
            }
            if (W) store_vec(y + i, out);
            else store_part(y + i, out, m);
        };
        if (m == V) piece(std::true_type());
        else piece(std::false_type());
    }
}

}  // namespace

hipError_t launch_dropout(int dtype, const void* x, const void* residual, int64_t n, double p, const int64_t* rng,
                          void* y, hipStream_t s) {
    const double words = p * 4294967296.0;
    const bool none = words >= 4294967295.5;
    const uint32_t least = none ? 0u : (uint32_t)(words + 0.5);
    const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.0f;
    return with_type(dtype, [&](auto zero) {
        using V = decltype(zero);
        const int64_t nblk = (n + NT * kVec<V> - 1) / (NT * kVec<V>);
        const int64_t grid = nblk < (1 << 22) ? nblk : 1 << 22;
        dropout_kernel<V><<<(unsigned)grid, NT, 0, s>>>(static_cast<const V*>(x), static_cast<const V*>(residual), n,
                                                        least, none, scale, rng, static_cast<V*>(y));
    });
}

}  // namespace nvfp4
