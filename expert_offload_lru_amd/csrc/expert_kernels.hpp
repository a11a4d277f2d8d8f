// Launchers of the experts' feed-forward, 8-bit rows and block norms (include/moe_experts.h); the
// arguments have been checked by the C entry points.
#pragma once

#include "moe_experts.h"
#include "token_kernels.hpp"

namespace moe {

constexpr int kBlock = 32;   // columns that share a scale in 8-bit rows

// A matrix by rows, in memory.
struct Rows {
    const void *p;
    int64_t ld;   // elements
};
struct RowsOut {
    void *p;
    int64_t ld;
};
struct Codes {
    const int8_t *q;
    int64_t ld;
    const uint8_t *s;
    int64_t ld_s;
};
struct CodesOut {
    int8_t *q;
    int64_t ld;
    uint8_t *s;
    int64_t ld_s;
};

hipError_t launch_encode(int dtype, Rows x, CodesOut c, int n_rows, int cols, hipStream_t stream);
hipError_t launch_decode(int dtype, Codes c, RowsOut x, int n_rows, int cols, hipStream_t stream);

// A product over the rows of each expert.  M: columns of the result.
struct ExpertArgs {
    Rows x;                   // [R x K]
    const void *w;            // hidden: [E x 2M x K]; product: [E x M x K]; backward: [E x K x M]
    const int32_t *offsets;   // [E + 1]
    int E, R, K, M;
    int act;
    RowsOut out;              // hidden, product, d_x: [R x M]; hidden_backward: hidden [R x M]
    RowsOut pre;              // hidden: [R x 2M]; hidden_backward: d_pre [R x 2M]
    CodesOut kept;            // hidden
    Rows pre_in;              // hidden_backward
    Codes kept_in;
};
hipError_t launch_hidden(int dtype, const ExpertArgs &a, hipStream_t stream);
hipError_t launch_product(int dtype, const ExpertArgs &a, hipStream_t stream);
hipError_t launch_hidden_back(int dtype, const ExpertArgs &a, hipStream_t stream);
hipError_t launch_product_back(int dtype, const ExpertArgs &a, hipStream_t stream);

// d_w [E x N x M] fp32 = sum over an expert's rows of d_out [R x N] and x [R x M].
struct ExpertGradArgs {
    Rows d_out, x;
    Codes codes;   // x in 8 bits, where x.p is null
    const int32_t *offsets;
    int E, R, M, N;
    float *d_w;
};
size_t expert_grad_workspace(int R, int M, int N, int E);
hipError_t launch_expert_grad(int dtype, const ExpertGradArgs &a, void *workspace, hipStream_t stream);

struct NormArgs {
    Rows x, y;   // y null: the first norm alone
    const float *w_post, *gate, *alpha, *w_pre;
    int T, H, per_gate;
    float eps;
    RowsOut out, normed;
    float *stats;
};
hipError_t launch_norm(int dtype, const NormArgs &a, hipStream_t stream);

struct NormBackArgs {
    Rows d_out, d_normed, x, y;
    const float *w_post, *gate, *alpha, *w_pre, *stats;
    int T, H, per_gate;
    RowsOut d_x, d_y;
    float *d_w_post, *d_gate, *d_alpha, *d_w_pre;
};
size_t norm_workspace(int T, int H, int per_gate);
hipError_t launch_norm_back(int dtype, const NormBackArgs &a, void *workspace, hipStream_t stream);

}  // namespace moe
