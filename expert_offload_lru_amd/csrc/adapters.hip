// Low-rank adapters (include/moe_tokens.h): out = base + scale B (A x) with a row's own A and B, and
// the gradients.
#include <algorithm>

#include "elements.hpp"
#include "token_kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;

// n <= 8 elements at p as fp32, zeros behind them.
template <typename T>
__device__ inline void load8(const T *p, int n, float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
        unpack<T>(load_piece(p, n), f);
    } else {
        float lo[4], hi[4];
        unpack<T>(load_piece(p, n), lo);
        unpack<T>(load_piece(p + 4, n - 4), hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = lo[i];
            f[4 + i] = hi[i];
        }
    }
}

__device__ inline float wave_total(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// v[q] = <a's row q, x> for q < r: a wave per row of a.
template <typename TX, typename TW>
__device__ inline void shrink_row(const TX *x, const TW *a, int inner, int r, float *v) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int q = wave; q < r; q += kThreads / 64) {
        float s = 0.f;
        for (int c = lane * 8; c < inner; c += 512) {
            float fx[8], fa[8];
            load8(x + c, inner - c, fx);
            load8(a + (size_t)q * inner + c, inner - c, fa);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(fx[i], fa[i], s);
        }
        s = wave_total(s);
        if (lane == 0) v[q] = s;
    }
}

template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void k_adapters_row(AdapterArgs g) {
    __shared__ float v[kMaxRank];
    const int row = blockIdx.x, e = g.adapter[row];
    const bool has = (unsigned)e < (unsigned)g.n;
    if (has)
        shrink_row(static_cast<const TX *>(g.x) + row * g.ld_x, static_cast<const TW *>(g.a) + (size_t)e * g.r * g.inner,
                   g.inner, g.r, v);
    __syncthreads();
    const float scale = has ? g.scale[e] : 0.f;
    const TX *base = static_cast<const TX *>(g.base);
    TX *out = static_cast<TX *>(g.out) + row * g.ld_out;
    for (int o = threadIdx.x; o < g.outer; o += kThreads) {
        float s = 0.f;
        if (has) {
            const TW *b = static_cast<const TW *>(g.b) + ((size_t)e * g.outer + o) * g.r;
            for (int q = 0; q < g.r; ++q) s = fmaf(widen(b[q]), v[q], s);
            s *= scale;
        }
        out[o] = base ? narrow<TX>(widen(base[row * g.ld_base + o]) + s) : narrow<TX>(s);
    }
}

// v and u of a row to memory, and its d_x.
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void k_back_row(AdapterBackArgs g, float *gv, float *gu) {
    __shared__ float v[kMaxRank], u[kMaxRank];
    const int row = blockIdx.x, e = g.adapter[row], lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool has = (unsigned)e < (unsigned)g.n;
    const TW *a = static_cast<const TW *>(g.a) + (has ? (size_t)e * g.r * g.inner : 0);
    const TX *dy = static_cast<const TX *>(g.d_out) + row * g.ld_d_out;
    if (has) {
        shrink_row(static_cast<const TX *>(g.x) + row * g.ld_x, a, g.inner, g.r, v);
        const TW *b = static_cast<const TW *>(g.b) + (size_t)e * g.outer * g.r;
        const float scale = g.scale[e];
        for (int q = wave; q < g.r; q += kThreads / 64) {
            float s = 0.f;
            for (int o = lane; o < g.outer; o += 64) s = fmaf(widen(dy[o]), widen(b[(size_t)o * g.r + q]), s);
            s = wave_total(s);
            if (lane == 0) u[q] = s * scale;
        }
    }
    __syncthreads();
    if (has)
        for (int q = threadIdx.x; q < g.r; q += kThreads) {
            gv[(size_t)row * g.r + q] = v[q];
            gu[(size_t)row * g.r + q] = u[q];
        }
    const TX *base = static_cast<const TX *>(g.dx_base);
    TX *dx = static_cast<TX *>(g.d_x) + row * g.ld_d_x;
    for (int c = threadIdx.x; c < g.inner; c += kThreads) {
        float s = 0.f;
        if (has)
            for (int q = 0; q < g.r; ++q) s = fmaf(widen(a[(size_t)q * g.inner + c]), u[q], s);
        dx[c] = base ? narrow<TX>(widen(base[row * g.ld_dx_base + c]) + s) : narrow<TX>(s);
    }
}

// d_a and d_b of one adapter, 64 columns and 16 ranks a workgroup; four threads a column take every
// fourth of the adapter's rows each.
template <typename TX>
__global__ __launch_bounds__(kThreads) void k_back_weights(AdapterBackArgs g, const int32_t *offsets, const int32_t *order,
                                                           const float *gv, const float *gu) {
    __shared__ float part[3][64][17];
    const int e = blockIdx.z, q0 = blockIdx.y * 16, tiles_a = (g.inner + 63) / 64;
    const bool is_b = (int)blockIdx.x >= tiles_a;
    const int tile = is_b ? blockIdx.x - tiles_a : blockIdx.x;
    const int cols = is_b ? g.outer : g.inner, c = tile * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
    const TX *m = static_cast<const TX *>(is_b ? g.d_out : g.x);
    const int64_t ld = is_b ? g.ld_d_out : g.ld_x;
    const float *left = is_b ? gv : gu;
    float acc[16] = {};
    if (c < cols)
        for (int i = offsets[e] + w; i < offsets[e + 1]; i += 4) {
            const int row = order[i];
            const float f = widen(m[row * ld + c]);
#pragma unroll
            for (int q = 0; q < 16; ++q)
                if (q0 + q < g.r) acc[q] = fmaf(left[(size_t)row * g.r + q0 + q], f, acc[q]);
        }
    if (w > 0)
#pragma unroll
        for (int q = 0; q < 16; ++q) part[w - 1][threadIdx.x & 63][q] = acc[q];
    __syncthreads();
    if (w > 0 || c >= cols) return;
    const float scale = is_b ? g.scale[e] : 1.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const float s = (acc[q] + part[0][threadIdx.x][q] + part[1][threadIdx.x][q] + part[2][threadIdx.x][q]) * scale;
        if (q0 + q >= g.r) continue;
        if (is_b)
            g.d_b[((size_t)e * g.outer + c) * g.r + q0 + q] = s;
        else
            g.d_a[((size_t)e * g.r + q0 + q) * g.inner + c] = s;
    }
}

// Workspace of a backward call.
struct BackSpace {
    size_t offsets, order, sort, v, u, bytes;
};
BackSpace back_space(int T, int n, int r) {
    auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    BackSpace s;
    s.offsets = 0;
    s.order = up((size_t)(n + 1) * 4);
    s.sort = s.order + up((size_t)T * 4);
    s.v = s.sort + up(dispatch_workspace(T, 1, n));
    s.u = s.v + up((size_t)T * r * 4);
    s.bytes = s.u + up((size_t)T * r * 4);
    return s;
}

template <typename TX, typename TW>
hipError_t forward(const AdapterArgs &g, hipStream_t stream) {
    return launch(k_adapters_row<TX, TW>, dim3(g.T), dim3(kThreads), stream, nullptr, nullptr, g);
}

template <typename TX, typename TW>
hipError_t backward(int dtype, const AdapterBackArgs &g, void *workspace, hipStream_t stream) {
    const BackSpace s = back_space(g.T, g.n, g.r);
    char *ws = static_cast<char *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + s.offsets), *order = reinterpret_cast<int32_t *>(ws + s.order);
    float *v = reinterpret_cast<float *>(ws + s.v), *u = reinterpret_cast<float *>(ws + s.u);
    DispatchArgs d{};
    d.ids = g.adapter;
    d.offsets = offsets;
    d.src = order;
    d.T = g.T;
    d.H = 1;
    d.k = 1;
    d.E = g.n;
    hipError_t err = launch_dispatch(dtype, d, ws + s.sort, stream);
    if (err == hipSuccess && g.T > 0)
        err = launch(k_back_row<TX, TW>, dim3(g.T), dim3(kThreads), stream, nullptr, nullptr, g, v, u);
    if (err == hipSuccess) {
        const dim3 grid((g.inner + 63) / 64 + (g.outer + 63) / 64, (g.r + 15) / 16, g.n);
        err = launch(k_back_weights<TX>, grid, dim3(kThreads), stream, nullptr, nullptr, g,
                     static_cast<const int32_t *>(offsets), static_cast<const int32_t *>(order),
                     static_cast<const float *>(v), static_cast<const float *>(u));
    }
    return err;
}

}  // namespace

size_t adapters_workspace(int T, int, int, int n, int r) { return back_space(T, n, r).bytes; }

hipError_t launch_adapters(int dtype, int wtype, const AdapterArgs &g, hipStream_t stream) {
    if (g.T == 0) return hipSuccess;
    if (dtype == T_F16) return forward<f16, f16>(g, stream);
    if (dtype == T_BF16) return forward<bf16, bf16>(g, stream);
    if (wtype == T_F16) return forward<float, f16>(g, stream);
    if (wtype == T_BF16) return forward<float, bf16>(g, stream);
    return forward<float, float>(g, stream);
}

hipError_t launch_adapters_back(int dtype, int wtype, const AdapterBackArgs &g, void *workspace, hipStream_t stream) {
    if (dtype == T_F16) return backward<f16, f16>(dtype, g, workspace, stream);
    if (dtype == T_BF16) return backward<bf16, bf16>(dtype, g, workspace, stream);
    if (wtype == T_F16) return backward<float, f16>(dtype, g, workspace, stream);
    if (wtype == T_BF16) return backward<float, bf16>(dtype, g, workspace, stream);
    return backward<float, float>(dtype, g, workspace, stream);
}

}  // namespace moe
