// C entry points of include/moe_experts.h: argument checks, then the launches.
#include <algorithm>
#include <cmath>

#include "expert_kernels.hpp"
#include "moe_experts.h"
#include "token_checks.hpp"

namespace moe {
namespace {

constexpr int kMaxHidden = 16384;              // of a block norm
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 4096;   // a launch holds fewer than 2^32; grids are rounded up by 7 workgroups

int check_size(int n_rows, std::initializer_list<int> widths) {
    if (n_rows < 0) return invalid("n_rows is negative");
    for (int w : widths)
        if (w < 1) return invalid("sizes must be positive");
    for (int w : widths)
        if (w >= kMaxTokenCount) return unsupported("a width of 2^24 or more");
    return n_rows >= kMaxTokenCount ? unsupported("n_rows >= 2^24") : MOE_OK;
}

int check_experts(int dtype, int n_rows, int inner, int outer, int n_experts) {
    if (!known(dtype)) return invalid("unknown type");
    if (n_experts < 1) return invalid("sizes must be positive");
    MOE_TRY(check_size(n_rows, {inner, outer}));
    if (n_experts > kMaxSegments) return unsupported("n_experts > 1024");
    // Workgroups of the smallest tiles that such widths meet: 128 rows x 64 columns by 256 threads (hidden's), or 64 x 32 by
    // 128; the weights' gradients 128 x 128 by 256.
    const bool tiny = std::min(inner, outer) < 8;
    const int64_t br = tiny ? 64 : 128, bc = tiny ? 32 : 64, threads = tiny ? 128 : 256, c = std::max(inner, outer);
    const int64_t rows = (n_rows / br + std::min(n_rows, n_experts)) * ((c + bc - 1) / bc);
    const int64_t grads = (int64_t)((inner + 127) / 128) * ((outer + 127) / 128) * n_experts;
    if (rows * threads >= kMaxThreads || grads * 256 >= kMaxThreads) return unsupported("more than one launch holds");
    return MOE_OK;
}

int64_t blocks(int cols) { return (cols + kBlock - 1) / kBlock; }

bool same(const void *a, int64_t ld_a, const void *b, int64_t ld_b) { return a == b && ld_a == ld_b; }

int check_codes(const void *codes, int64_t ld, const void *scales, int64_t ld_s, int64_t cols, int64_t n_blocks) {
    if (!codes != !scales) return invalid("codes and scales go together");
    MOE_TRY(check_ld("codes", codes, ld, cols));
    return check_ld("scales", scales, ld_s, n_blocks);
}

int check_activation(int a) {
    return a == MOE_ACT_SILU || a == MOE_ACT_GELU ? MOE_OK : invalid("unknown activation");
}

int check_workspace(const void *p, size_t given, size_t need) {
    if (need && (!p || given < need || reinterpret_cast<uintptr_t>(p) % 16))
        return invalid("the workspace is too small or not aligned");
    return MOE_OK;
}

int check_norm(int dtype, int n_rows, int hidden, const void *gate, int rows_per_gate) {
    if (!known(dtype)) return invalid("unknown type");
    MOE_TRY(check_size(n_rows, {hidden}));
    if (hidden > kMaxHidden) return unsupported("hidden > 16384");
    if (hidden > kMaxHidden / 2 && n_rows >= kMaxTokenCount / 2) return unsupported("n_rows >= 2^23 with hidden > 8192");
    if (gate && rows_per_gate < 1) return invalid("rows_per_gate must be positive");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_rows_encode(const void *x, int64_t ld_x, int dtype, int n_rows, int cols, int8_t *codes, int64_t ld_codes,
                    uint8_t *scales, int64_t ld_scales, void *stream) {
    if (!known(dtype)) return invalid("unknown type");
    MOE_TRY(check_size(n_rows, {cols}));
    if (n_rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("x", x, ld_x, cols));
    MOE_TRY(check_codes(codes, ld_codes, scales, ld_scales, cols, blocks(cols)));
    MOE_TRY(check_overlap({matrix("codes", codes, n_rows, cols, ld_codes, 1),
                           matrix("scales", scales, n_rows, blocks(cols), ld_scales, 1)},
                          {matrix("x", x, n_rows, cols, ld_x, elem_size(dtype))}));
    return finish(launch_encode(dtype, {x, ld_x}, {codes, ld_codes, scales, ld_scales}, n_rows, cols,
                                static_cast<hipStream_t>(stream)));
}

int moe_rows_decode(const int8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales, int dtype,
                    int n_rows, int cols, void *x, int64_t ld_x, void *stream) {
    if (!known(dtype)) return invalid("unknown type");
    MOE_TRY(check_size(n_rows, {cols}));
    if (n_rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("x", x, ld_x, cols));
    MOE_TRY(check_codes(codes, ld_codes, scales, ld_scales, cols, blocks(cols)));
    MOE_TRY(check_overlap({matrix("x", x, n_rows, cols, ld_x, elem_size(dtype))},
                          {matrix("codes", codes, n_rows, cols, ld_codes, 1),
                           matrix("scales", scales, n_rows, blocks(cols), ld_scales, 1)}));
    return finish(launch_decode(dtype, {codes, ld_codes, scales, ld_scales}, {x, ld_x}, n_rows, cols,
                                static_cast<hipStream_t>(stream)));
}

int moe_experts_hidden(const void *x, int64_t ld_x, int dtype, int n_rows, int inner, int inter, const int32_t *offsets,
                       int n_experts, const void *w, int activation, void *hidden, int64_t ld_hidden, void *pre,
                       int64_t ld_pre, int8_t *codes, int64_t ld_codes, uint8_t *scales, int64_t ld_scales,
                       void *stream) {
    MOE_TRY(check_experts(dtype, n_rows, inner, inter, n_experts));
    MOE_TRY(check_activation(activation));
    if (inter >= kMaxTokenCount / 2) return unsupported("2 * inter >= 2^24");
    if (n_rows == 0) return MOE_OK;
    if (!x || !offsets || !w || !hidden) return invalid("a tensor is NULL");
    if (pre && codes) return invalid("pre and codes do not go together");
    const int64_t two = 2 * (int64_t)inter, nb = 2 * blocks(inter);
    MOE_TRY(check_ld("x", x, ld_x, inner));
    MOE_TRY(check_ld("hidden", hidden, ld_hidden, inter));
    MOE_TRY(check_ld("pre", pre, ld_pre, two));
    MOE_TRY(check_codes(codes, ld_codes, scales, ld_scales, two, nb));
    const size_t z = elem_size(dtype);
    MOE_TRY(check_overlap({matrix("hidden", hidden, n_rows, inter, ld_hidden, z), matrix("pre", pre, n_rows, two, ld_pre, z),
                           matrix("codes", codes, n_rows, two, ld_codes, 1), matrix("scales", scales, n_rows, nb, ld_scales, 1)},
                          {matrix("x", x, n_rows, inner, ld_x, z), array("offsets", offsets, n_experts + 1),
                           array("w", w, n_experts * two * inner, z)}));
    ExpertArgs a{};
    a.x = {x, ld_x};
    a.w = w;
    a.offsets = offsets;
    a.E = n_experts;
    a.R = n_rows;
    a.K = inner;
    a.M = inter;
    a.act = activation;
    a.out = {hidden, ld_hidden};
    a.pre = {pre, ld_pre};
    a.kept = {codes, ld_codes, scales, ld_scales};
    return finish(launch_hidden(dtype, a, static_cast<hipStream_t>(stream)));
}

int moe_experts_hidden_backward(const void *d_out, int64_t ld_d_out, int dtype, int n_rows, int outer, int inter,
                                const int32_t *offsets, int n_experts, const void *w, int activation, const void *pre,
                                int64_t ld_pre, const int8_t *codes, int64_t ld_codes, const uint8_t *scales,
                                int64_t ld_scales, void *d_pre, int64_t ld_d_pre, void *hidden, int64_t ld_hidden,
                                void *stream) {
    MOE_TRY(check_experts(dtype, n_rows, outer, inter, n_experts));
    MOE_TRY(check_activation(activation));
    if (inter >= kMaxTokenCount / 2) return unsupported("2 * inter >= 2^24");
    if (n_rows == 0) return MOE_OK;
    if (!d_out || !offsets || !w || !d_pre) return invalid("a tensor is NULL");
    if (!pre == !codes) return invalid("either pre or codes is wanted");
    const int64_t two = 2 * (int64_t)inter, nb = 2 * blocks(inter);
    MOE_TRY(check_ld("d_out", d_out, ld_d_out, outer));
    MOE_TRY(check_ld("pre", pre, ld_pre, two));
    MOE_TRY(check_codes(codes, ld_codes, scales, ld_scales, two, nb));
    MOE_TRY(check_ld("d_pre", d_pre, ld_d_pre, two));
    MOE_TRY(check_ld("hidden", hidden, ld_hidden, inter));
    const size_t z = elem_size(dtype);
    MOE_TRY(check_overlap({matrix("d_pre", d_pre, n_rows, two, ld_d_pre, z),
                           matrix("hidden", hidden, n_rows, inter, ld_hidden, z)},
                          {matrix("d_out", d_out, n_rows, outer, ld_d_out, z), array("offsets", offsets, n_experts + 1),
                           array("w", w, (int64_t)n_experts * outer * inter, z), matrix("pre", pre, n_rows, two, ld_pre, z),
                           matrix("codes", codes, n_rows, two, ld_codes, 1),
                           matrix("scales", scales, n_rows, nb, ld_scales, 1)}));
    ExpertArgs a{};
    a.x = {d_out, ld_d_out};
    a.w = w;
    a.offsets = offsets;
    a.E = n_experts;
    a.R = n_rows;
    a.K = outer;
    a.M = inter;
    a.act = activation;
    a.out = {hidden, ld_hidden};
    a.pre = {d_pre, ld_d_pre};
    a.pre_in = {pre, ld_pre};
    a.kept_in = {codes, ld_codes, scales, ld_scales};
    return finish(launch_hidden_back(dtype, a, static_cast<hipStream_t>(stream)));
}

int moe_experts_product(const void *x, int64_t ld_x, int dtype, int n_rows, int inner, int outer, const int32_t *offsets,
                        int n_experts, const void *w, void *out, int64_t ld_out, void *stream) {
    MOE_TRY(check_experts(dtype, n_rows, inner, outer, n_experts));
    if (n_rows == 0) return MOE_OK;
    if (!x || !offsets || !w || !out) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("x", x, ld_x, inner));
    MOE_TRY(check_ld("out", out, ld_out, outer));
    const size_t z = elem_size(dtype);
    MOE_TRY(check_overlap({matrix("out", out, n_rows, outer, ld_out, z)},
                          {matrix("x", x, n_rows, inner, ld_x, z), array("offsets", offsets, n_experts + 1),
                           array("w", w, (int64_t)n_experts * outer * inner, z)}));
    ExpertArgs a{};
    a.x = {x, ld_x};
    a.w = w;
    a.offsets = offsets;
    a.E = n_experts;
    a.R = n_rows;
    a.K = inner;
    a.M = outer;
    a.out = {out, ld_out};
    return finish(launch_product(dtype, a, static_cast<hipStream_t>(stream)));
}

size_t moe_experts_product_workspace(int n_rows, int inner, int outer, int n_experts) {
    if (check_experts(MOE_T_F32, n_rows, inner, outer, n_experts) != MOE_OK) return 0;
    return expert_grad_workspace(n_rows, inner, outer, n_experts);
}

int moe_experts_product_backward(const void *d_out, int64_t ld_d_out, int dtype, int n_rows, int inner, int outer,
                                 const int32_t *offsets, int n_experts, const void *w, const void *x, int64_t ld_x,
                                 const int8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales,
                                 void *d_x, int64_t ld_d_x, float *d_w, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    MOE_TRY(check_experts(dtype, n_rows, inner, outer, n_experts));
    if (n_rows == 0) d_x = nullptr;
    if (!offsets && (d_x || d_w)) return invalid("a tensor is NULL");
    if ((d_x || d_w) && n_rows > 0 && !d_out) return invalid("a tensor is NULL");
    if (d_x && !w) return invalid("d_x needs w");
    if (!d_x) w = nullptr;
    if (!d_w) {
        x = codes = nullptr;
        scales = nullptr;
    } else if (n_rows > 0 && !x == !codes) {
        return invalid("d_w needs either x or codes");
    }
    MOE_TRY(check_ld("d_out", d_out, ld_d_out, outer));
    MOE_TRY(check_ld("x", x, ld_x, inner));
    MOE_TRY(check_codes(codes, ld_codes, scales, ld_scales, inner, blocks(inner)));
    MOE_TRY(check_ld("d_x", d_x, ld_d_x, inner));
    const size_t z = elem_size(dtype), need = d_w ? expert_grad_workspace(n_rows, inner, outer, n_experts) : 0;
    MOE_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t nw = (int64_t)n_experts * outer * inner;
    MOE_TRY(check_overlap({matrix("d_x", d_x, n_rows, inner, ld_d_x, z), array("d_w", d_w, nw),
                           array("workspace", workspace, need, 1)},
                          {matrix("d_out", d_out, n_rows, outer, ld_d_out, z), array("offsets", offsets, n_experts + 1),
                           array("w", w, nw, z), matrix("x", x, n_rows, inner, ld_x, z),
                           matrix("codes", codes, n_rows, inner, ld_codes, 1),
                           matrix("scales", scales, n_rows, blocks(inner), ld_scales, 1)}));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (d_x) {
        ExpertArgs a{};
        a.x = {d_out, ld_d_out};
        a.w = w;
        a.offsets = offsets;
        a.E = n_experts;
        a.R = n_rows;
        a.K = outer;
        a.M = inner;
        a.out = {d_x, ld_d_x};
        MOE_TRY(finish(launch_product_back(dtype, a, s)));
    }
    if (!d_w) return MOE_OK;
    ExpertGradArgs a{};
    a.d_out = {d_out, ld_d_out};
    a.x = {x, ld_x};
    a.codes = {codes, ld_codes, scales, ld_scales};
    a.offsets = offsets;
    a.E = n_experts;
    a.R = n_rows;
    a.M = inner;
    a.N = outer;
    a.d_w = d_w;
    return finish(launch_expert_grad(dtype, a, workspace, s));
}

int moe_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, int dtype, int n_rows, int hidden,
                   const float *w_post, const float *gate, int rows_per_gate, const float *alpha, const float *w_pre,
                   float eps, void *out, int64_t ld_out, void *normed, int64_t ld_normed, float *stats, void *stream) {
    MOE_TRY(check_norm(dtype, n_rows, hidden, gate, rows_per_gate));
    if (!(eps >= 0.f) || std::isinf(eps)) return invalid("eps is negative or not finite");
    if (!w_pre != !normed && n_rows > 0) return invalid("w_pre and normed go together");
    if (!y && n_rows > 0 && (w_post || gate || alpha || out)) return invalid("w_post, gate, alpha and out go with y");
    if (n_rows == 0) return MOE_OK;
    if (!x || (!out && !normed && !stats)) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("x", x, ld_x, hidden));
    MOE_TRY(check_ld("y", y, ld_y, hidden));
    MOE_TRY(check_ld("out", out, ld_out, hidden));
    MOE_TRY(check_ld("normed", normed, ld_normed, hidden));
    const size_t z = elem_size(dtype);
    const int64_t gates = gate ? (n_rows + (int64_t)rows_per_gate - 1) / rows_per_gate : 0;
    const Span params[] = {array("w_post", w_post, hidden), array("gate", gate, gates * hidden), array("alpha", alpha, hidden),
                           array("w_pre", w_pre, hidden)};
    const Span s_out = matrix("out", out, n_rows, hidden, ld_out, z), s_normed = matrix("normed", normed, n_rows, hidden, ld_normed, z);
    const Span s_stats = array("stats", stats, 2 * (int64_t)n_rows), s_x = matrix("x", x, n_rows, hidden, ld_x, z);
    const Span s_y = matrix("y", y, n_rows, hidden, ld_y, z), none{};
    MOE_TRY(check_overlap({s_out, s_normed, s_stats}, {params[0], params[1], params[2], params[3]}));
    // a row is read before it is written, each element by the same thread
    MOE_TRY(check_overlap({s_out}, {same(out, ld_out, x, ld_x) ? none : s_x, same(out, ld_out, y, ld_y) ? none : s_y}));
    MOE_TRY(check_overlap({s_normed}, {same(normed, ld_normed, x, ld_x) ? none : s_x, same(normed, ld_normed, y, ld_y) ? none : s_y}));
    MOE_TRY(check_overlap({s_stats}, {s_x, s_y}));
    NormArgs a{{x, ld_x}, {y, ld_y}, w_post, gate, alpha, w_pre, n_rows, hidden, gate ? rows_per_gate : 1, eps,
               {out, ld_out}, {normed, ld_normed}, stats};
    return finish(launch_norm(dtype, a, static_cast<hipStream_t>(stream)));
}

size_t moe_block_norm_workspace(int n_rows, int hidden, int rows_per_gate) {
    if (check_norm(MOE_T_F32, n_rows, hidden, nullptr, 0) != MOE_OK) return 0;
    return norm_workspace(n_rows, hidden, std::max(1, rows_per_gate));
}

int moe_block_norm_backward(const void *d_out, int64_t ld_d_out, const void *d_normed, int64_t ld_d_normed,
                            const void *x, int64_t ld_x, const void *y, int64_t ld_y, int dtype, int n_rows, int hidden,
                            const float *w_post, const float *gate, int rows_per_gate, const float *alpha,
                            const float *w_pre, const float *stats, void *d_x, int64_t ld_d_x, void *d_y,
                            int64_t ld_d_y, float *d_w_post, float *d_gate, float *d_alpha, float *d_w_pre,
                            void *workspace, size_t workspace_bytes, void *stream) {
    MOE_TRY(check_norm(dtype, n_rows, hidden, gate, rows_per_gate));
    if ((d_w_post && !w_post) || (d_gate && !gate) || (d_alpha && !alpha) || (d_w_pre && !w_pre))
        return invalid("a gradient of a parameter that is not there");
    if (n_rows > 0 && !y && (w_post || gate || alpha || d_y)) return invalid("w_post, gate, alpha and d_y go with y");
    if (n_rows > 0 && (!x || (!d_out && !d_normed) || ((w_post || w_pre) && !stats))) return invalid("a tensor is NULL");
    if (n_rows > 0 && d_normed && !w_pre) return invalid("d_normed goes with w_pre");
    MOE_TRY(check_ld("d_out", d_out, ld_d_out, hidden));
    MOE_TRY(check_ld("d_normed", d_normed, ld_d_normed, hidden));
    MOE_TRY(check_ld("x", x, ld_x, hidden));
    MOE_TRY(check_ld("y", y, ld_y, hidden));
    MOE_TRY(check_ld("d_x", d_x, ld_d_x, hidden));
    MOE_TRY(check_ld("d_y", d_y, ld_d_y, hidden));
    const size_t z = elem_size(dtype);
    const bool params = d_w_post || d_gate || d_alpha || d_w_pre;
    // the kernel finds a row's gate by this: a gate of more rows than there are is one of all rows
    const int per_gate = gate ? std::min(rows_per_gate, std::max(n_rows, 1)) : 1;
    const size_t need = params ? norm_workspace(n_rows, hidden, per_gate) : 0;
    MOE_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t gates = gate ? (n_rows + (int64_t)per_gate - 1) / per_gate : 0;
    const Span none{};
    const Span s_dx = matrix("d_x", d_x, n_rows, hidden, ld_d_x, z), s_dy = matrix("d_y", d_y, n_rows, hidden, ld_d_y, z);
    const Span rows[] = {matrix("d_out", d_out, n_rows, hidden, ld_d_out, z), matrix("d_normed", d_normed, n_rows, hidden, ld_d_normed, z),
                         matrix("x", x, n_rows, hidden, ld_x, z), matrix("y", y, n_rows, hidden, ld_y, z)};
    const int64_t lds[] = {ld_d_out, ld_d_normed, ld_x, ld_y};
    const Span g[] = {array("d_w_post", d_w_post, hidden), array("d_gate", d_gate, gates * hidden), array("d_alpha", d_alpha, hidden),
                      array("d_w_pre", d_w_pre, hidden), array("workspace", workspace, need, 1)};
    MOE_TRY(check_overlap({s_dx, s_dy, g[0], g[1], g[2], g[3], g[4]},
                          {array("w_post", w_post, hidden), array("gate", gate, gates * hidden), array("alpha", alpha, hidden),
                           array("w_pre", w_pre, hidden), array("stats", stats, 2 * (int64_t)n_rows)}));
    MOE_TRY(check_overlap({g[0], g[1], g[2], g[3], g[4]}, {rows[0], rows[1], rows[2], rows[3]}));
    for (int i = 0; i < 4; ++i) {
        MOE_TRY(check_overlap({s_dx}, {same(d_x, ld_d_x, rows[i].p, lds[i]) ? none : rows[i]}));
        MOE_TRY(check_overlap({s_dy}, {same(d_y, ld_d_y, rows[i].p, lds[i]) ? none : rows[i]}));
    }
    NormBackArgs a{{d_out, ld_d_out}, {d_normed, ld_d_normed}, {x, ld_x}, {y, ld_y}, w_post, gate, alpha, w_pre, stats,
                   n_rows, hidden, per_gate, {d_x, ld_d_x}, {d_y, ld_d_y}, d_w_post, d_gate, d_alpha, d_w_pre};
    if (n_rows == 0 && !params) return MOE_OK;
    return finish(launch_norm_back(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
