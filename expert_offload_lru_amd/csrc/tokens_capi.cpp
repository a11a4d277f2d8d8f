// C entry points of include/moe_tokens.h: argument checks, then the launches.
#include <algorithm>
#include <initializer_list>

#include "errors.hpp"
#include "moe_offload.h"
#include "moe_tokens.h"
#include "token_kernels.hpp"

namespace moe {
namespace {

constexpr int kMaxTokenCount = 1 << 24;   // grids of one workgroup of 256 a token stay under 2^32 threads

// A caller's matrix of `rows` rows of `cols` elements.
struct Span {
    const char *name;
    const void *p;
    size_t bytes;
};

size_t elem_size(int dtype) { return dtype == MOE_T_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == MOE_T_F32 || dtype == MOE_T_F16 || dtype == MOE_T_BF16; }

Span matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size) {
    return {name, p, p && rows > 0 ? (size_t)((rows - 1) * ld + cols) * size : 0};
}
Span array(const char *name, const void *p, int64_t n, size_t size = 4) { return {name, p, p ? (size_t)n * size : 0}; }

bool overlap(const Span &a, const Span &b) {
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

int invalid(const std::string &msg) { return set_error(MOE_ERR_INVALID, msg); }
int unsupported(const std::string &msg) { return set_error(MOE_ERR_UNSUPPORTED, msg); }

// No output overlaps an input or another output.
int check_overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (auto o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (overlap(*o, i)) return invalid(std::string(o->name) + " overlaps " + i.name);
        for (auto p = o + 1; p != outputs.end(); ++p)
            if (overlap(*o, *p)) return invalid(std::string(o->name) + " overlaps " + p->name);
    }
    return MOE_OK;
}

int check_ld(const char *name, const void *p, int64_t ld, int64_t cols) {
    if (p && (ld < cols || ld > ((int64_t)1 << 40))) return invalid(std::string("ld of ") + name + " is out of range");
    return MOE_OK;
}

int finish(hipError_t e) {
    return e == hipSuccess ? MOE_OK : set_error(MOE_ERR_HIP, std::string("launch: ") + hipGetErrorString(e));
}

int check_tokens(int n_tokens, int top_k, int n_experts) {
    if (n_tokens < 0 || top_k < 1 || n_experts < 1) return invalid("sizes must be positive");
    if (top_k > kMaxPicks || n_experts > kMaxSegments) return unsupported("top_k > 16 or n_experts > 1024");
    if (n_tokens >= kMaxTokenCount) return unsupported("n_tokens >= 2^24");
    return MOE_OK;
}

int check_rows(int dtype, int n_tokens, int hidden, int top_k, int64_t n_rows) {
    if (!known(dtype)) return invalid("unknown type");
    if (hidden < 1) return invalid("hidden must be positive");
    if (hidden >= kMaxTokenCount) return unsupported("hidden >= 2^24");
    if (n_rows < 0 || n_rows > ((int64_t)1 << 31)) return invalid("n_rows is out of range");
    return check_tokens(n_tokens, top_k, 1);
}

int check_adapters(int dtype, int wtype, int n_rows, int inner, int outer, int n_adapters, int rank) {
    if (!known(dtype) || !known(wtype)) return invalid("unknown type");
    if (wtype != dtype && dtype != MOE_T_F32) return invalid("adapters of another type go with fp32 activations only");
    if (n_rows < 0 || inner < 1 || outer < 1 || n_adapters < 1 || rank < 1) return invalid("sizes must be positive");
    if (rank > kMaxRank) return unsupported("rank > 256");
    if (n_rows >= kMaxTokenCount || inner >= kMaxTokenCount || outer >= kMaxTokenCount)
        return unsupported("a size of 2^24 or more");
    return MOE_OK;
}

size_t forward_bytes(int n_rows, int inner, int outer, int n_adapters, int rank, bool copies) {
    if (check_adapters(MOE_T_F32, MOE_T_F32, n_rows, inner, outer, n_adapters, rank) != MOE_OK) return 0;
    return adapters_forward_workspace(n_rows, inner, outer, n_adapters, rank, copies);
}

size_t backward_bytes(int n_rows, int inner, int outer, int n_adapters, int rank, bool copies) {
    if (check_adapters(MOE_T_F32, MOE_T_F32, n_rows, inner, outer, n_adapters, rank) != MOE_OK) return 0;
    return n_adapters > kMaxSegments ? 0 : adapters_workspace(n_rows, inner, outer, n_adapters, rank, copies);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_TRY(call)                  \
    do {                               \
        const int rc_ = (call);        \
        if (rc_ != MOE_OK) return rc_; \
    } while (0)

extern "C" {

size_t moe_tokens_workspace(int n_tokens, int top_k, int n_experts) {
    if (check_tokens(n_tokens, top_k, n_experts) != MOE_OK) return 0;
    return dispatch_workspace(n_tokens, top_k, n_experts);
}

int moe_tokens_dispatch(const void *x, int64_t ld_x, int dtype, int n_tokens, int hidden, const int32_t *ids, int top_k,
                        int n_experts, void *rows, int64_t ld_rows, int32_t *offsets, int32_t *pos, int32_t *src,
                        int32_t *expert, void *workspace, size_t workspace_bytes, void *stream) {
    if (!known(dtype)) return invalid("unknown type");
    MOE_TRY(check_tokens(n_tokens, top_k, n_experts));
    const int64_t picks = (int64_t)n_tokens * top_k;
    if (!offsets || (picks > 0 && (!ids || !pos || !src || !expert))) return invalid("ids or an index output is NULL");
    if (picks > 0 && !x != !rows) return invalid("x and rows go together");
    if (x && rows) {
        if (hidden < 1) return invalid("hidden must be positive");
        if (hidden >= kMaxTokenCount) return unsupported("hidden >= 2^24");
        MOE_TRY(check_ld("x", x, ld_x, hidden));
        MOE_TRY(check_ld("rows", rows, ld_rows, hidden));
    }
    const size_t need = dispatch_workspace(n_tokens, top_k, n_experts), z = elem_size(dtype);
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 4))
        return invalid("the workspace is too small or not aligned");
    MOE_TRY(check_overlap({matrix("rows", x ? rows : nullptr, picks, hidden, ld_rows, z),
                           array("offsets", offsets, n_experts + 1), array("pos", pos, picks), array("src", src, picks),
                           array("expert", expert, picks), array("workspace", workspace, need, 1)},
                          {matrix("x", rows ? x : nullptr, n_tokens, hidden, ld_x, z), array("ids", ids, picks)}));
    DispatchArgs a{};
    const bool data = x && rows;
    a.x = data ? x : nullptr;
    a.rows = data ? rows : nullptr;
    a.ld_x = ld_x;
    a.ld_rows = ld_rows;
    a.ids = ids;
    a.offsets = offsets;
    a.pos = pos;
    a.src = src;
    a.expert = expert;
    a.T = n_tokens;
    a.H = data ? hidden : 1;
    a.k = top_k;
    a.E = n_experts;
    return finish(launch_dispatch(dtype, a, workspace, static_cast<hipStream_t>(stream)));
}

int moe_tokens_dispatch_backward(const void *d_rows, int64_t ld_rows, int64_t n_rows, int dtype, int n_tokens, int hidden,
                                 const int32_t *pos, int top_k, void *d_x, int64_t ld_x, void *stream) {
    MOE_TRY(check_rows(dtype, n_tokens, hidden, top_k, n_rows));
    if (n_tokens == 0) return MOE_OK;
    if (!pos || !d_x || (!d_rows && n_rows > 0)) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("d_rows", d_rows, ld_rows, hidden));
    MOE_TRY(check_ld("d_x", d_x, ld_x, hidden));
    const size_t z = elem_size(dtype);
    MOE_TRY(check_overlap({matrix("d_x", d_x, n_tokens, hidden, ld_x, z)},
                          {matrix("d_rows", d_rows, n_rows, hidden, ld_rows, z),
                           array("pos", pos, (int64_t)n_tokens * top_k)}));
    CombineRowsArgs a{d_rows, ld_rows, n_rows, pos, nullptr, nullptr, d_x, 0, ld_x, n_tokens, hidden, top_k};
    return finish(launch_combine_rows(dtype, a, static_cast<hipStream_t>(stream)));
}

int moe_tokens_combine(const void *rows, int64_t ld_rows, int64_t n_rows, int dtype, int n_tokens, int hidden,
                       const int32_t *pos, const float *gate, int top_k, const void *base, int64_t ld_base, void *out,
                       int64_t ld_out, void *stream) {
    MOE_TRY(check_rows(dtype, n_tokens, hidden, top_k, n_rows));
    if (n_tokens == 0) return MOE_OK;
    if (!pos || !gate || !out || (!rows && n_rows > 0)) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("rows", rows, ld_rows, hidden));
    MOE_TRY(check_ld("base", base, ld_base, hidden));
    MOE_TRY(check_ld("out", out, ld_out, hidden));
    const size_t z = elem_size(dtype);
    const int64_t picks = (int64_t)n_tokens * top_k;
    const bool in_place = base == out && ld_base == ld_out;
    MOE_TRY(check_overlap({matrix("out", out, n_tokens, hidden, ld_out, z)},
                          {matrix("rows", rows, n_rows, hidden, ld_rows, z), array("pos", pos, picks),
                           array("gate", gate, picks),
                           matrix("base", in_place ? nullptr : base, n_tokens, hidden, ld_base, z)}));
    CombineRowsArgs a{rows, ld_rows, n_rows, pos, gate, base, out, ld_base, ld_out, n_tokens, hidden, top_k};
    return finish(launch_combine_rows(dtype, a, static_cast<hipStream_t>(stream)));
}

int moe_tokens_combine_backward(const void *d_out, int64_t ld_d_out, const void *rows, int64_t ld_rows, int64_t n_rows,
                                int dtype, int n_tokens, int hidden, const int32_t *pos, const float *gate, int top_k,
                                void *d_rows, int64_t ld_d_rows, float *d_gate, void *stream) {
    MOE_TRY(check_rows(dtype, n_tokens, hidden, top_k, n_rows));
    if (n_tokens == 0) return MOE_OK;
    if (!d_out || !pos || !gate || !d_gate || (n_rows > 0 && (!rows || !d_rows))) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("d_out", d_out, ld_d_out, hidden));
    MOE_TRY(check_ld("rows", rows, ld_rows, hidden));
    MOE_TRY(check_ld("d_rows", d_rows, ld_d_rows, hidden));
    const size_t z = elem_size(dtype);
    const int64_t picks = (int64_t)n_tokens * top_k;
    MOE_TRY(check_overlap({matrix("d_rows", d_rows, n_rows, hidden, ld_d_rows, z), array("d_gate", d_gate, picks)},
                          {matrix("d_out", d_out, n_tokens, hidden, ld_d_out, z),
                           matrix("rows", rows, n_rows, hidden, ld_rows, z), array("pos", pos, picks),
                           array("gate", gate, picks)}));
    CombineBackArgs a{d_out, rows, d_rows, ld_d_out, ld_rows, ld_d_rows, n_rows, pos, gate, d_gate, n_tokens, hidden,
                      top_k};
    return finish(launch_combine_back(dtype, a, static_cast<hipStream_t>(stream)));
}

size_t moe_adapters_forward_workspace(int n_rows, int inner, int outer, int n_adapters, int rank) {
    return forward_bytes(n_rows, inner, outer, n_adapters, rank, false);
}

size_t moe_adapters_forward_workspace_strided(int n_rows, int inner, int outer, int n_adapters, int rank) {
    return forward_bytes(n_rows, inner, outer, n_adapters, rank, true);
}

int moe_adapters_forward(const void *x, int64_t ld_x, const void *base, int64_t ld_base, int dtype, int n_rows, int inner,
                         int outer, const int32_t *adapter, const void *a, const void *b, int wtype, const float *scale,
                         int n_adapters, int rank, void *out, int64_t ld_out, void *workspace, size_t workspace_bytes,
                         void *stream) {
    MOE_TRY(check_adapters(dtype, wtype, n_rows, inner, outer, n_adapters, rank));
    if (n_rows == 0) return MOE_OK;
    if (!x || !adapter || !a || !b || !scale || !out) return invalid("a tensor is NULL");
    MOE_TRY(check_ld("x", x, ld_x, inner));
    MOE_TRY(check_ld("base", base, ld_base, outer));
    MOE_TRY(check_ld("out", out, ld_out, outer));
    const size_t z = elem_size(dtype), zw = elem_size(wtype);
    const bool in_place = base == out && ld_base == ld_out;
    const size_t need = adapters_forward_workspace(n_rows, inner, outer, n_adapters, rank, false);
    const size_t most = std::min(workspace_bytes, adapters_forward_workspace(n_rows, inner, outer, n_adapters, rank, true));
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
        return invalid("the workspace is too small or not aligned");
    MOE_TRY(check_overlap({matrix("out", out, n_rows, outer, ld_out, z), array("workspace", workspace, most, 1)},
                          {matrix("x", x, n_rows, inner, ld_x, z),
                           matrix("base", in_place ? nullptr : base, n_rows, outer, ld_base, z),
                           array("adapter", adapter, n_rows), array("a", a, (int64_t)n_adapters * rank * inner, zw),
                           array("b", b, (int64_t)n_adapters * rank * outer, zw), array("scale", scale, n_adapters)}));
    AdapterArgs g{x, base, out, ld_x, ld_base, ld_out, adapter, a, b, scale, n_rows, inner, outer, n_adapters, rank};
    return finish(launch_adapters(dtype, wtype, g, workspace, most, static_cast<hipStream_t>(stream)));
}

size_t moe_adapters_workspace(int n_rows, int inner, int outer, int n_adapters, int rank) {
    return backward_bytes(n_rows, inner, outer, n_adapters, rank, false);
}

size_t moe_adapters_workspace_strided(int n_rows, int inner, int outer, int n_adapters, int rank) {
    return backward_bytes(n_rows, inner, outer, n_adapters, rank, true);
}

int moe_adapters_backward(const void *d_out, int64_t ld_d_out, const void *x, int64_t ld_x, const void *dx_base,
                          int64_t ld_dx_base, int dtype, int n_rows, int inner, int outer, const int32_t *adapter,
                          const void *a, const void *b, int wtype, const float *scale, int n_adapters, int rank, void *d_x,
                          int64_t ld_d_x, float *d_a, float *d_b, void *workspace, size_t workspace_bytes, void *stream) {
    MOE_TRY(check_adapters(dtype, wtype, n_rows, inner, outer, n_adapters, rank));
    if (n_adapters > kMaxSegments) return unsupported("n_adapters > 1024");
    if (!a || !b || !scale || !d_a || !d_b || (n_rows > 0 && (!d_out || !x || !adapter || !d_x)))
        return invalid("a tensor is NULL");
    MOE_TRY(check_ld("d_out", d_out, ld_d_out, outer));
    MOE_TRY(check_ld("x", x, ld_x, inner));
    MOE_TRY(check_ld("dx_base", dx_base, ld_dx_base, inner));
    MOE_TRY(check_ld("d_x", d_x, ld_d_x, inner));
    const size_t need = adapters_workspace(n_rows, inner, outer, n_adapters, rank, false);
    const size_t most = std::min(workspace_bytes, adapters_workspace(n_rows, inner, outer, n_adapters, rank, true));
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16))
        return invalid("the workspace is too small or not aligned");
    const size_t z = elem_size(dtype), zw = elem_size(wtype);
    const int64_t na = (int64_t)n_adapters * rank * inner, nb = (int64_t)n_adapters * rank * outer;
    const bool in_place = dx_base == d_x && ld_dx_base == ld_d_x;
    MOE_TRY(check_overlap({matrix("d_x", d_x, n_rows, inner, ld_d_x, z), array("d_a", d_a, na), array("d_b", d_b, nb),
                           array("workspace", workspace, most, 1)},
                          {matrix("d_out", d_out, n_rows, outer, ld_d_out, z), matrix("x", x, n_rows, inner, ld_x, z),
                           matrix("dx_base", in_place ? nullptr : dx_base, n_rows, inner, ld_dx_base, z),
                           array("adapter", adapter, n_rows), array("a", a, na, zw), array("b", b, nb, zw),
                           array("scale", scale, n_adapters)}));
    AdapterBackArgs g{d_out, x, dx_base, d_x, ld_d_out, ld_x, ld_dx_base, ld_d_x, adapter, a, b, scale, d_a, d_b, n_rows,
                      inner, outer, n_adapters, rank};
    return finish(launch_adapters_back(dtype, wtype, g, workspace, most, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
