// Launchers of the token-order and adapter kernels (include/moe_tokens.h); the arguments have been
// checked by the C entry points.
#pragma once

#include "kernels.hpp"

namespace moe {

enum Elem { T_F32 = 0, T_F16 = 1, T_BF16 = 2 };
constexpr int kMaxPicks = 16;        // picks of a token
constexpr int kMaxSegments = 1024;   // experts of a dispatch, adapters of a backward call
constexpr int kMaxRank = 256;

struct DispatchArgs {
    const void *x;        // null: only the order
    void *rows;
    int64_t ld_x, ld_rows;
    const int32_t *ids;   // [T x k]
    int32_t *offsets, *pos, *src, *expert;   // pos and expert may be null
    int T, H, k, E;
};
size_t dispatch_workspace(int T, int k, int E);
hipError_t launch_dispatch(int dtype, const DispatchArgs &a, void *workspace, hipStream_t stream);

struct CombineRowsArgs {
    const void *rows;
    int64_t ld_rows, n_rows;
    const int32_t *pos;   // [T x k]
    const float *gate;    // [T x k], null: every weight is 1
    const void *base;     // null: zeros
    void *out;
    int64_t ld_base, ld_out;
    int T, H, k;
};
hipError_t launch_combine_rows(int dtype, const CombineRowsArgs &a, hipStream_t stream);

struct CombineBackArgs {
    const void *d_out, *rows;
    void *d_rows;
    int64_t ld_d_out, ld_rows, ld_d_rows, n_rows;
    const int32_t *pos;
    const float *gate;
    float *d_gate;
    int T, H, k;
};
hipError_t launch_combine_back(int dtype, const CombineBackArgs &a, hipStream_t stream);

struct AdapterArgs {
    const void *x, *base;
    void *out;
    int64_t ld_x, ld_base, ld_out;
    const int32_t *adapter;
    const void *a, *b;       // [n x r x inner], [n x outer x r]
    const float *scale;
    int T, inner, outer, n, r;
};
// Bytes of workspace; copies: with room for copies of matrices whose rows are not aligned.
size_t adapters_forward_workspace(int T, int inner, int outer, int n, int r, bool copies);
hipError_t launch_adapters(int dtype, int wtype, const AdapterArgs &a, void *workspace, size_t bytes, hipStream_t stream);

struct AdapterBackArgs {
    const void *d_out, *x, *dx_base;
    void *d_x;
    int64_t ld_d_out, ld_x, ld_dx_base, ld_d_x;
    const int32_t *adapter;
    const void *a, *b;
    const float *scale;
    float *d_a, *d_b;
    int T, inner, outer, n, r;
};
size_t adapters_workspace(int T, int inner, int outer, int n, int r, bool copies);
hipError_t launch_adapters_back(int dtype, int wtype, const AdapterBackArgs &a, void *workspace, size_t bytes, hipStream_t stream);

}  // namespace moe
