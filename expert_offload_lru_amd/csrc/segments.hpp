// Rows of experts from device offsets: every workgroup finds its own tile, so no launch has to lay out a
// table first.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kSegPerLane = 16;   // 1024 experts over 64 lanes

__device__ inline int wave_max_scan(int v) {   // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}
__device__ inline int wave_sum_scan(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

struct Tile {
    int e, row, end;   // expert; the tile's first row and the expert's end
};

// Tile `index` of the experts' rows in tiles of `per` rows, experts in order; total: how many there are.
// False if there is no such tile.  index(total) may choose the tile by the total.  Every wave does it by itself.
// An offset counts as at least the ones before it and as 0 .. R.
template <typename Index>
__device__ inline bool find_tile(const int32_t *offsets, int E, int R, int per, Index index, Tile &t) {
    const int lane = threadIdx.x & 63;
    const int n = (E + 63) >> 6, first = lane * n;
    int most = 0;   // of the offsets up to the end of the lane's last expert
    int o[kSegPerLane + 1];
#pragma unroll
    for (int i = 0; i <= kSegPerLane; ++i) {
        o[i] = 0;
        if (i <= n && first + i <= E) o[i] = min(max(offsets[first + i], 0), R);
        most = max(most, o[i]);
    }
    int before = __shfl_up(wave_max_scan(most), 1);
    if (lane == 0) before = 0;
    int run = max(before, o[0]), tiles = 0;
#pragma unroll
    for (int i = 0; i < kSegPerLane; ++i)
        if (i < n && first + i < E) {
            const int next = max(run, o[i + 1]);
            tiles += (next - run + per - 1) / per;
            run = next;
        }
    const int upto = wave_sum_scan(tiles), total = __builtin_amdgcn_readlane(upto, 63);
    const int at = index(total);
    if (at < 0 || at >= total) return false;
    const uint64_t has = __ballot(upto > at);
    const int who = __ffsll((unsigned long long)has) - 1;
    // the lane that holds it walks its experts again
    int e = 0, row = 0, end = 0, left = at - (upto - tiles);
    run = max(before, o[0]);
    bool found = false;
#pragma unroll
    for (int i = 0; i < kSegPerLane; ++i)
        if (i < n && first + i < E && !found) {
            const int next = max(run, o[i + 1]);
            const int c = (next - run + per - 1) / per;
            if (left < c) {
                e = first + i;
                row = run + left * per;
                end = next;
                found = true;
            }
            left -= c;
            run = next;
        }
    t.e = __builtin_amdgcn_readfirstlane(__shfl(e, who));
    t.row = __builtin_amdgcn_readfirstlane(__shfl(row, who));
    t.end = __builtin_amdgcn_readfirstlane(__shfl(end, who));
    return true;
}

// Rows of expert e: begin and end.
__device__ inline void rows_of(const int32_t *offsets, int e, int R, int &begin, int &end) {
    int m = 0;
    for (int i = threadIdx.x & 63; i <= e; i += 64) m = max(m, min(max(offsets[i], 0), R));
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, __shfl_xor(m, d));
    begin = __builtin_amdgcn_readfirstlane(m);
    end = max(begin, __builtin_amdgcn_readfirstlane(min(max(offsets[e + 1], 0), R)));
}

}  // namespace moe
