// 8 columns of a row: as fp32 values, and as codes of rows kept in 8 bits.
#pragma once

#include <algorithm>

#include "rows8.hpp"

namespace moe {

// Values at p, the first n of them, past the caches where they are whole: what a product writes is as large as what it
// reads, and would push that out of L2 (gradients of 65536 rows 745 -> 700 us).
template <typename T>
__device__ inline void stream_piece(T *p, uint4 v, int n) {
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    if (n >= kVec<T>) __builtin_nontemporal_store(words{v.x, v.y, v.z, v.w}, reinterpret_cast<words *>(p));
    else store_piece(p, v, n);
}
__device__ inline void stream4(float *p, float a, float b, float c, float d, int n) { stream_piece(p, pack<float>({a, b, c, d}), n); }
template <typename T>
__device__ inline void stream8(T *p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        stream4(p, f[0], f[1], f[2], f[3], n);
        stream4(p + 4, f[4], f[5], f[6], f[7], n - 4);
    } else {
        stream_piece(p, pack<T>(f), n);
    }
}

// 8 values at p, the first n of them
template <typename T>
__device__ inline void store8(T *p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        store_piece(p, pack<T>({f[0], f[1], f[2], f[3]}), min(n, 4));
        store_piece(p + 4, pack<T>({f[4], f[5], f[6], f[7]}), min(n - 4, 4));
    } else {
        store_piece(p, pack<T>(f), n);
    }
}
template <typename T>
__device__ inline void load8(const T *p, float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        float a[4], b[4];
        unpack<T>(load_piece(p, n), a);
        unpack<T>(load_piece(p + 4, n - 4), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
        unpack<T>(load_piece(p, n), f);
    }
}
__device__ inline uint2 load_codes(const int8_t *p, int n) {
    uint2 c = {0, 0};
    if (n >= 8) {
        __builtin_memcpy(&c, p, 8);
    } else {
        int8_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : 0;
        __builtin_memcpy(&c, e, 8);
    }
    return c;
}
__device__ inline void store_codes(int8_t *p, uint2 c, int n) {
    if (n >= 8) {
        __builtin_memcpy(p, &c, 8);
    } else {
        int8_t e[8];
        __builtin_memcpy(e, &c, 8);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = e[i];
    }
}

// Codes of 8 columns of a row; the 4 lanes of a block of 32 (lanes 4j .. 4j+3) share its scale.  Columns
// from n on count as zeros.
__device__ inline uint2 encode8(const float (&f)[8], int n, int &scale) {
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = i < n ? f[i] : 0.f;
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);   // NaN is the largest
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    scale = block_scale(__uint_as_float(top));
    uint32_t b[8];
    if ((unsigned)(scale - 6) < 248u) {   // 2^(133 - scale) is a normal number, and no code leaves the range
        // added to 1.5 * 2^23, a value becomes a whole number, rounded to nearest, ties to even: the low byte is the code
        const float to = __uint_as_float((uint32_t)(127 + kScaleBias - scale) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(v[i], to, 12582912.f));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = scale == kScaleNaN ? 0u : (uint32_t)encode1(v[i], scale);
    }
    auto four = [&](int i) {
        const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0c0c0400u);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    };
    return {four(0), four(4)};
}

}  // namespace moe
