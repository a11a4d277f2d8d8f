// Rows of experts from device offsets: every workgroup finds its own tile, so no launch has to lay out a
// table first.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

// Inclusive scans over a wave of values from 0 on.
template <typename Op>
__device__ inline int wave_scan(int v, Op op) {
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));   // row_shr:1 .. 8: within 16 lanes
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));   // row_bcast:15, to rows 1 and 3
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));   // row_bcast:31, to rows 2 and 3
}

struct Tile {
    int e, row, end;   // expert; the tile's first row and the expert's end
};

// find_tile for up to 64 N experts, n a lane.
template <int N, typename Index>
__device__ inline bool find_tile_n(const int32_t *offsets, int E, int R, int per, int n, Index index, Tile &t) {
    const int lane = threadIdx.x & 63, first = lane * n;
    int o[N + 1], most = 0;   // most: of the offsets up to the end of the lane's last expert
#pragma unroll
    for (int i = 0; i <= N; ++i) {
        o[i] = 0;
        if (i <= n && first + i <= E) o[i] = offsets[first + i];
    }
#pragma unroll
    for (int i = 0; i <= N; ++i) {
        o[i] = min(max(o[i], 0), R);
        most = max(most, o[i]);
    }
    const int before = __builtin_amdgcn_update_dpp(0, wave_scan(most, [](int a, int b) { return max(a, b); }), 0x138, 0xf,
                                                   0xf, false);   // wave_shr:1
    int run = max(before, o[0]), tiles = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n && first + i < E) {
            const int next = max(run, o[i + 1]);
            tiles += (next - run + per - 1) / per;
            run = next;
        }
    const int upto = wave_scan(tiles, [](int a, int b) { return a + b; }), total = __builtin_amdgcn_readlane(upto, 63);
    const int at = index(total);
    if (at < 0 || at >= total) return false;
    const int who = __ffsll((unsigned long long)__ballot(upto > at)) - 1;
    // the lane that holds it walks its experts again
    int e = 0, row = 0, end = 0, left = at - (upto - tiles);
    run = max(before, o[0]);
    bool found = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
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
    t.e = __builtin_amdgcn_readlane(e, who);
    t.row = __builtin_amdgcn_readlane(row, who);
    t.end = __builtin_amdgcn_readlane(end, who);
    return true;
}

// Tile `index` of the experts' rows in tiles of `per` rows (a power of two), experts in order; total: how many there
// are.  False if there is no such tile.  index(total) may choose the tile by the total.  Every wave does it by
// itself.  An offset counts as at least the ones before it and as 0 .. R.
template <typename Index>
__device__ inline bool find_tile(const int32_t *offsets, int E, int R, int per, Index index, Tile &t) {
    const int n = (E + 63) >> 6;
    if (n <= 2) return find_tile_n<2>(offsets, E, R, per, n, index, t);
    return find_tile_n<16>(offsets, E, R, per, n, index, t);   // 1024 experts at most
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
