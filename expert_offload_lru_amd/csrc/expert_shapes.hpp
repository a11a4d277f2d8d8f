// Tiles of the products over experts' rows, and how work is dealt to them.
#pragma once

namespace moe {

// A workgroup's tile: 2 waves along m and NW along n, each FM x FN pieces of 32 x 32; S steps in LDS at a time.
template <int FM_, int FN_, int NW, int S>
struct Shape {
    static constexpr int FM = FM_, FN = FN_, STAGES = S, WM = FM * 32, WN = FN * 32;   // WM, WN: a wave's columns and rows
    static constexpr int BM = 2 * WM, BN = NW * WN, WAVES = 2 * NW, THREADS = WAVES * 64;
};
// 256 x 256: 8 waves, 128 KB of LDS, one workgroup a CU.
using Wide = Shape<4, 2, 4, 4>;
// 128 x 128: 4 waves, 64 KB, two workgroups a CU; for few tiles, and for loads through registers.
using Mid = Shape<2, 2, 2, 4>;
#ifndef MID_BELOW
#define MID_BELOW 128
#endif

inline int tiles(int n, int per) { return (n + per - 1) / per; }

// A weights' gradient: its tile, and runs of an expert's rows that are summed apart.
struct GradPlan {
    bool wide;
    int splits;
};

}  // namespace moe
