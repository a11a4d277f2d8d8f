// 8 columns of a row: as fp32 values, and as codes of rows kept in 8 bits.
#pragma once

#include <algorithm>

#include "rows8.hpp"

namespace moe {

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
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, i < n ? __float_as_uint(f[i]) & 0x7FFFFFFFu : 0u);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    scale = block_scale(__uint_as_float(top));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n && scale != kScaleNaN) w[i >> 2] |= (uint32_t)(uint8_t)(int8_t)encode1(f[i], scale) << (8 * (i & 3));
    return {w[0], w[1]};
}

}  // namespace moe
