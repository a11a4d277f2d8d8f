// Products over the rows of experts (include/moe_experts.h): the launches by type, and the joining of partial sums.
#include <algorithm>

#include "expert_kernels.hpp"
#include "expert_shapes.hpp"
#include "pieces8.hpp"

namespace moe {

#define MOE_DECLARE(NAME)                                                                              \
    hipError_t hidden_##NAME(const ExpertArgs &a, hipStream_t s);                                       \
    hipError_t product_##NAME(const ExpertArgs &a, hipStream_t s);                                      \
    hipError_t hidden_back_##NAME(const ExpertArgs &a, hipStream_t s);                                  \
    hipError_t product_back_##NAME(const ExpertArgs &a, hipStream_t s);                                 \
    hipError_t grad_##NAME(const ExpertGradArgs &a, const GradPlan &p, float *parts, hipStream_t s);
MOE_DECLARE(f32)
MOE_DECLARE(f16)
MOE_DECLARE(bf16)

namespace {

// Sum of the runs, in order.
__global__ __launch_bounds__(256) void k_grad_join(const float *parts, float *d_w, int64_t n, int splits) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int m = (int)min((int64_t)4, n - i);
    float s[4] = {0, 0, 0, 0}, f[4];
    for (int k = 0; k < splits; ++k) {
        unpack<float>(load_piece(parts + k * n + i, m), f);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += f[j];
    }
    store_piece(d_w + i, pack<float>(s), m);
}

// The larger tile from 128 rows an expert on where there are at least four rounds of it, or from 1024 rows on (128 experts,
// 768 x 2048: 64 rows each 144 us against the smaller's 139, 128 rows 174 / 214, 512 rows 309 / 400; 8 experts, 2048 x 1536,
// one and a half rounds: 512 rows 46 / 40, 2048 rows 113 / 133).  Widths that are not whole pieces go through
// registers, in the smaller one (so do rows at other addresses, with the runs of the larger one if it was chosen: the plan
// and the workspace go by sizes).  Runs of an expert's rows, 512 and more, until there is a workgroup a CU (two of the
// smaller ones): a run's partial sums are written and read once more.
GradPlan grad_plan(int R, int M, int N, int E) {
    const int64_t wide = (int64_t)tiles(M, Wide::BM) * tiles(N, Wide::BN) * E, mid = (int64_t)tiles(M, Mid::BM) * tiles(N, Mid::BN) * E;
    const int each = R / E;
    const bool use = M % 8 == 0 && N % 8 == 0 && each >= 128 && (wide >= 1024 || each >= 1024);
    const int64_t s = std::min<int64_t>({use ? 256 / wide : 512 / mid, each / 512, 16});
    return {use, (int)std::max<int64_t>(1, s)};
}

}  // namespace

#define MOE_BY_TYPE(FN, ...) \
    (dtype == T_F32 ? FN##_f32(__VA_ARGS__) : dtype == T_F16 ? FN##_f16(__VA_ARGS__) : FN##_bf16(__VA_ARGS__))

hipError_t launch_hidden(int dtype, const ExpertArgs &a, hipStream_t stream) { return MOE_BY_TYPE(hidden, a, stream); }
hipError_t launch_product(int dtype, const ExpertArgs &a, hipStream_t stream) { return MOE_BY_TYPE(product, a, stream); }
hipError_t launch_hidden_back(int dtype, const ExpertArgs &a, hipStream_t stream) { return MOE_BY_TYPE(hidden_back, a, stream); }
hipError_t launch_product_back(int dtype, const ExpertArgs &a, hipStream_t stream) { return MOE_BY_TYPE(product_back, a, stream); }

size_t expert_grad_workspace(int R, int M, int N, int E) {
    const int s = grad_plan(R, M, N, E).splits;
    return s == 1 ? 0 : (size_t)s * E * M * N * sizeof(float);
}

hipError_t launch_expert_grad(int dtype, const ExpertGradArgs &a, void *workspace, hipStream_t stream) {
    const GradPlan plan = grad_plan(a.R, a.M, a.N, a.E);
    float *parts = static_cast<float *>(workspace);
    const hipError_t e = MOE_BY_TYPE(grad, a, plan, parts, stream);
    if (e != hipSuccess || plan.splits == 1) return e;
    const int64_t size = (int64_t)a.E * a.M * a.N;
    return launch(k_grad_join, dim3((unsigned)((size + 1023) / 1024)), dim3(256), stream, nullptr, nullptr,
                  static_cast<const float *>(parts), a.d_w, size, plan.splits);
}

}  // namespace moe
