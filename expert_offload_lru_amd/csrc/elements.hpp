// 16-byte pieces of a row of fp32, fp16 or bf16 elements, read and written as fp32 values.
//
// Rows need no alignment beyond their element's: the loads and stores are 16-byte memory
// instructions all the same (global memory takes them at any element's address), and only the last,
// partial piece of a row goes element by element.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

typedef _Float16 f16;
typedef __bf16 bf16;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);   // elements of a piece

__device__ inline float widen(float v) { return v; }
__device__ inline float widen(f16 v) { return (float)v; }
__device__ inline float widen(bf16 v) { return (float)v; }
// one rounding, to nearest
template <typename T>
__device__ inline T narrow(float v) { return (T)v; }

// The n <= kVec<T> elements at p, zeros behind them.
template <typename T>
__device__ inline uint4 load_piece(const T *p, int n) {
    uint4 r = {0, 0, 0, 0};
    if (n >= kVec<T>) {
        __builtin_memcpy(&r, p, 16);
    } else {
        T e[kVec<T>];
        __builtin_memcpy(e, &r, 16);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (i < n) e[i] = p[i];
        __builtin_memcpy(&r, e, 16);
    }
    return r;
}

template <typename T>
__device__ inline void store_piece(T *p, uint4 v, int n) {
    if (n >= kVec<T>) {
        __builtin_memcpy(p, &v, 16);
    } else {
        T e[kVec<T>];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (i < n) p[i] = e[i];
    }
}

template <typename T>
__device__ inline void unpack(uint4 v, float (&f)[kVec<T>]) {
    T e[kVec<T>];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) f[i] = widen(e[i]);
}

template <typename T>
__device__ inline uint4 pack(const float (&f)[kVec<T>]) {
    T e[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) e[i] = narrow<T>(f[i]);
    uint4 r;
    __builtin_memcpy(&r, e, 16);
    return r;
}

}  // namespace moe
