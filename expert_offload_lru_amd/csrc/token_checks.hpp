// Argument checks of the C entry points on caller tensors (include/moe_tokens.h, include/moe_experts.h).
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "errors.hpp"
#include "moe_offload.h"
#include "moe_tokens.h"

#define MOE_TRY(call)                  \
    do {                               \
        const int rc_ = (call);        \
        if (rc_ != MOE_OK) return rc_; \
    } while (0)

namespace moe {

constexpr int kMaxTokenCount = 1 << 24;   // grids of one workgroup of 256 a token stay under 2^32 threads

// A caller's matrix of `rows` rows of `cols` elements.
struct Span {
    const char *name;
    const void *p;
    size_t bytes;
};

inline size_t elem_size(int dtype) { return dtype == MOE_T_F32 ? 4 : 2; }
inline bool known(int dtype) { return dtype == MOE_T_F32 || dtype == MOE_T_F16 || dtype == MOE_T_BF16; }

inline Span matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size) {
    return {name, p, p && rows > 0 ? (size_t)((rows - 1) * ld + cols) * size : 0};
}
inline Span array(const char *name, const void *p, int64_t n, size_t size = 4) { return {name, p, p ? (size_t)n * size : 0}; }

inline bool overlap(const Span &a, const Span &b) {
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

inline int invalid(const std::string &msg) { return set_error(MOE_ERR_INVALID, msg); }
inline int unsupported(const std::string &msg) { return set_error(MOE_ERR_UNSUPPORTED, msg); }

// No output overlaps an input or another output.
inline int check_overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (auto o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (overlap(*o, i)) return invalid(std::string(o->name) + " overlaps " + i.name);
        for (auto p = o + 1; p != outputs.end(); ++p)
            if (overlap(*o, *p)) return invalid(std::string(o->name) + " overlaps " + p->name);
    }
    return MOE_OK;
}

inline int check_ld(const char *name, const void *p, int64_t ld, int64_t cols) {
    if (p && (ld < cols || ld > ((int64_t)1 << 40))) return invalid(std::string("ld of ") + name + " is out of range");
    return MOE_OK;
}

inline int finish(hipError_t e) {
    return e == hipSuccess ? MOE_OK : set_error(MOE_ERR_HIP, std::string("launch: ") + hipGetErrorString(e));
}

}  // namespace moe
