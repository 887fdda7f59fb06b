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

// A piece at p, which is aligned to its element alone (a global memory instruction
// of 16 bytes takes any alignment). STREAM: read or written once, past the caches.
template <bool STREAM = false, typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* __restrict__ p) {
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { u32x4 v; };
    const Raw* q = reinterpret_cast<const Raw*>(p);
    return __builtin_bit_cast(Vec<T>, STREAM ? __builtin_nontemporal_load(&q->v) : q->v);
}
template <bool STREAM = false, typename T>
__device__ __forceinline__ void store_vec(T* __restrict__ p, const Vec<T>& r) {
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { u32x4 v; };
    Raw* q = reinterpret_cast<Raw*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, r), &q->v);
    else q->v = __builtin_bit_cast(u32x4, r);
}
// Its first n elements alone; the others are zero.
template <typename T>
__device__ __forceinline__ Vec<T> load_part(const T* __restrict__ p, int n) {
    Vec<T> r;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) r.v[i] = i < n ? p[i] : (T)0.0f;
    return r;
}
template <typename T>
__device__ __forceinline__ void store_part(T* __restrict__ p, const Vec<T>& r, int n) {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
        if (i < n) p[i] = r.v[i];
}

// The pieces of rows of H elements. Where H is no multiple of a piece, the last one
// starts so that it ends with the row, over elements that the piece before has too:
// both threads write the same values there. So every access is a whole piece (a
// branch around each would make the compiler wait for one load before the next).
// WHOLE = false: rows shorter than a piece, element by element.
template <typename T, bool WHOLE>
struct RowPieces {
    int64_t H;
    __device__ __forceinline__ int64_t start(int c) const { return WHOLE ? min((int64_t)c * kVec<T>, H - kVec<T>) : 0; }
    // (as bits: a value that is only loaded under a condition stays four words, which
    // nothing unpacks, and so waits for, before it is used)
    template <bool STREAM = false>
    __device__ __forceinline__ u32x4 load(const T* __restrict__ p) const {
        return __builtin_bit_cast(u32x4, WHOLE ? load_vec<STREAM>(p) : load_part(p, (int)H));
    }
    template <bool STREAM = false>
    __device__ __forceinline__ void store(T* __restrict__ p, const Vec<T>& r) const {
        if (WHOLE) store_vec<STREAM>(p, r);
        else store_part(p, r, (int)H);
    }
};

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
