// Tiles of the products over experts' rows, and how work is dealt to them.
#pragma once

namespace moe {

// A workgroup's tile: MW waves along m and NW along n, each FM x FN pieces of 32 x 32; S steps in LDS at a time.
template <int FM_, int FN_, int MW_, int NW, int S>
struct Shape {
    static constexpr int FM = FM_, FN = FN_, MW = MW_, STAGES = S, WM = FM * 32, WN = FN * 32;   // WM, WN: a wave's columns, rows
    static constexpr int BM = MW * WM, BN = NW * WN, WAVES = MW * NW, THREADS = WAVES * 64;
};
// 256 x 256: 8 waves, 128 KB of LDS, one workgroup a CU.
using Wide = Shape<4, 2, 2, 4, 4>;
// 128 x 128: 4 waves, 64 KB, two workgroups a CU; for few tiles, and for loads through registers.
using Mid = Shape<2, 2, 2, 2, 4>;
// 64 x 64: 2 waves, 64 KB; for few rows and small products, where there are not enough of the others for every CU, and
// what counts are the loads on their way: seven steps of them.
using Small = Shape<2, 1, 1, 2, 8>;

inline int tiles(int n, int per) { return (n + per - 1) / per; }

// A weights' gradient: its tile, and runs of an expert's rows that are summed apart.
struct GradPlan {
    bool wide;
    int splits;
};

}  // namespace moe
