// Rows kept in 8 bits: blocks of 32 columns, int8 codes and a shared power of two.
//
// value = code * 2^e, e = scale - 133 from -133 to 121.  e is the least of these for which the block's largest size, over
// 2^e and rounded, is 127 or less (121 where none is), so from a largest size of 2^-127 on the largest code is 64 .. 127
// and a value is off by at most 2^(e-1) (2^e at 121); blocks below have e = -133 and smaller codes.
// A power of two makes the codes exact values of fp32 and bf16: code * 2^e has 7 bits and is no less than bf16's least
// step, so reading a row back rounds nothing (a product with a scale of 24 bits would round again), and x / 2^e is
// exact.  fp16 takes the values that are within its range and not below its least step as they are.
#pragma once

#include <type_traits>

#include "elements.hpp"

namespace moe {

constexpr int kScaleBias = 133, kScaleNaN = 255;
constexpr int kMinExp = -133, kMaxExp = 121;

// The scale of a block whose largest size is amax (inf or NaN: kScaleNaN).
__device__ inline int block_scale(float amax) {
    if (!(amax <= 3.402823466e38f)) return kScaleNaN;
    if (amax == 0.f) return 0;
    int e = __builtin_amdgcn_frexp_expf(amax) - 7;   // amax / 2^e in [64, 128)
    if (__builtin_rintf(__builtin_ldexpf(amax, -e)) > 127.f) ++e;
    return min(max(e, kMinExp), kMaxExp) + kScaleBias;
}

__device__ inline int encode1(float v, int scale) {
    const float q = __builtin_rintf(__builtin_ldexpf(v, kScaleBias - scale));
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// values of 8 columns from their codes and their block's scale, within T's finite range
template <typename T>
__device__ inline void decode8(uint2 q, int scale, float (&f)[8]) {
    // fast: 2^(scale - 133) and 128 of it are normal numbers, and 127 of it is within f16's range
    constexpr unsigned kFast = std::is_same_v<T, f16> ? 142 - 7 : 254 - 7;
    if ((unsigned)(scale - 7) < kFast) {
        const float s = __uint_as_float((uint32_t)(scale - 6) << 23), less = -128.f * s;
        const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};   // codes + 128
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fmaf((float)((w[i >> 2] >> (8 * (i & 3))) & 0xFFu), s, less);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = i < 4 ? q.x : q.y;
        const float v = __builtin_ldexpf((float)(int8_t)(w >> (8 * (i & 3))), scale - kScaleBias);
        // beyond the other types' range there is one value, -128 * 2^121 (rows that were encoded hold no -128)
        constexpr float kMost = std::is_same_v<T, f16> ? 65504.f : std::is_same_v<T, bf16> ? 3.3895313892515355e38f : 3.4028234663852886e38f;
        f[i] = scale == kScaleNaN ? __builtin_nanf("") : fminf(fmaxf(v, -kMost), kMost);
    }
}

}  // namespace moe
