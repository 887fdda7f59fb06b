// Elements of the operators that take bf16, float16 or float32 (gfx950): 16-byte
// pieces of rows that start at any element, and conversions.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace nvfp4 {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);   // elements of a piece
template <typename T>
struct Vec {
    T v[kVec<T>];
};

__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }
// nearest-even, the type's infinity beyond its range
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    return (T)v;
}

// The first n elements (at most a piece) at p, which is aligned to its element
// alone; the others are zero. STREAM: read or written once, past the caches.
template <typename T, bool STREAM = false>
__device__ __forceinline__ Vec<T> load_vec(const T* __restrict__ p, int n) {
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { u32x4 v; };
    Vec<T> r;
    if (n >= kVec<T>) {
        const Raw* q = reinterpret_cast<const Raw*>(p);
        r = __builtin_bit_cast(Vec<T>, STREAM ? __builtin_nontemporal_load(&q->v) : q->v);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) r.v[i] = i < n ? p[i] : (T)0.0f;
    }
    return r;
}
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_vec(T* __restrict__ p, const Vec<T>& r, int n) {
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { u32x4 v; };
    if (n >= kVec<T>) {
        Raw* q = reinterpret_cast<Raw*>(p);
        if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, r), &q->v);
        else q->v = __builtin_bit_cast(u32x4, r);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (i < n) p[i] = r.v[i];
    }
}

// f(a value of the type that `dtype` (enum nvfp4_dtype) names), then the launch's error.
template <typename F>
hipError_t with_type(int dtype, F&& f) {
    switch (dtype) {
        case kBf16: f((__bf16)0.0f); break;
        case kF16: f((_Float16)0.0f); break;
        case kF32: f(0.0f); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace nvfp4
