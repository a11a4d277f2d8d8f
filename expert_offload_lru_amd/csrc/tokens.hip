// Tokens sorted by expert and back (include/moe_tokens.h): a stable counting sort of the picks fused
// with the copy of the rows, the weighted sum of a token's rows, and its gradients.
//
// All of it is bound by memory (at most three flops an element), so every kernel reads each input
// row once and writes each output row once, in 16-byte pieces, and the small index work rides along.
// Measured rates stand beside a copy's on the same card: 5.4 TB/s at 0.5 GB of traffic, 5.2 at 2 GB.
#include <algorithm>

#include "elements.hpp"
#include "order.hpp"

namespace moe {
namespace {

// Up to here every workgroup counts all picks itself, above it sums the counts of slices that a launch
// before has made.  8192 picks with rows of 2048 bf16: 13.4 us so, 14.1 with slices; 16384: 20.3 and 18.9
// (the order alone: 10.9 and 10.4).
constexpr int kDirectPicks = 8192;
// 64 slices at most, and more only where a slice would be over 32768 picks: a workgroup reads every
// slice's counts and half a slice's picks.  2^21 picks: 64 slices; 2^23: 374 us with 256, 483 with 64.
constexpr int kSlicePicks = 2048;     // picks of a histogram slice above, at least
constexpr int kMaxSlices = 64;
constexpr int kLongSlice = 32768, kMostSlices = 512;
// Workgroups of a dispatch that copies rows: four a CU.  8192 tokens of 2048 bf16: 70 us, 72 with 512
// and 68 with 2048; 32768 tokens of 64: 19.5 us, 21.9 and 21.3.
constexpr int kWgTarget = 1024;

int slices_of(int N) {
    if (N <= kDirectPicks) return 0;
    return std::max(std::min(kMaxSlices, (N + kSlicePicks - 1) / kSlicePicks), std::min(kMostSlices, N / kLongSlice));
}
int per_slice(int N, int slices) { return (N + slices - 1) / slices; }

__global__ __launch_bounds__(kThreads) void k_slice_counts(const int32_t *ids, int N, int per, int E, int32_t *counts) {
    __shared__ int hist[kMaxSegments * kCopies];
    for (int i = threadIdx.x; i < E * kCopies; i += kThreads) hist[i] = 0;
    __syncthreads();
    const int p0 = blockIdx.x * per;
    count(ids, p0, min(N, p0 + per), E, hist);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) counts[(size_t)blockIdx.x * E + e] = total_of(hist, e);
}

// The order of the picks (order_picks), then the rows of the workgroup's tokens: read once, written once a
// pick.  The first four tokens' pieces are requested before the order is made.
// 8192 tokens of 2048 bf16, 8 picks each: 302 MB in 65 us, 4.6 TB/s (k_slice_counts before it 4 us);
// one token 6.2 us, the steps of the order one after another.
template <typename T, int EM>
__global__ __launch_bounds__(kThreads) void k_dispatch(DispatchArgs a, int tokens, int lanes_log2, const int32_t *counts,
                                                       int slices, int per) {
    __shared__ OrderSpace<EM> o;
    const int tid = threadIdx.x, t0 = blockIdx.x * tokens, t1 = min(a.T, t0 + tokens);
    const int L = 1 << lanes_log2, groups = kThreads >> lanes_log2, l = tid & (L - 1);
    const int first = t0 + (tid >> lanes_log2), pieces = (a.H + kVec<T> - 1) / kVec<T>;
    const T *x = static_cast<const T *>(a.x);
    auto request = [&](uint4 (&v)[4], int t, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (t + u * groups < t1) v[u] = load_piece(x + (int64_t)(t + u * groups) * a.ld_x + c * kVec<T>, a.H - c * kVec<T>);
    };
    uint4 ahead[4];
    if (x && l < pieces) request(ahead, first, l);
    order_picks<EM>(a, blockIdx.x, tokens, counts, slices, per, o);
    if (!x) return;
    __syncthreads();

    for (int c = l; c < pieces; c += L) {
        const int n = a.H - c * kVec<T>;
        T *rows = static_cast<T *>(a.rows) + c * kVec<T>;
        for (int t = first; t < t1; t += 4 * groups) {
            uint4 v[4];
            if (c == l && t == first)
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = ahead[u];
            else
                request(v, t, c);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (t + u * groups >= t1) break;
                for (int j = 0; j < a.k; ++j) {
                    const int row = o.row_of[(t + u * groups - t0) * a.k + j];
                    if (row >= 0) store_piece(rows + (int64_t)row * a.ld_rows, v[u], n);
                }
            }
        }
    }
}

// L lanes a token (a whole workgroup for wide rows); each lane sums its pieces over the picks in
// order, eight rows' loads in flight.  4096 tokens of 2048 columns, 8 picks each: bf16 with base 160 MB in
// 34 us, 4.7 TB/s; fp32 302 MB in 65 us; four tokens 5.6 us, the latency of position, gate and row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_combine_rows(CombineRowsArgs a, int lanes_log2) {
    const int L = 1 << lanes_log2;
    const int t = (blockIdx.x << (8 - lanes_log2)) + ((int)threadIdx.x >> lanes_log2);
    if (t >= a.T) return;
    const int pieces = (a.H + kVec<T> - 1) / kVec<T>;
    const T *rows = static_cast<const T *>(a.rows);
    for (int c = threadIdx.x & (L - 1); c < pieces; c += L) {
        const int n = a.H - c * kVec<T>;
        float sum[kVec<T>] = {};
        uint4 base = {0, 0, 0, 0};
        if (a.base) base = load_piece(static_cast<const T *>(a.base) + (int64_t)t * a.ld_base + c * kVec<T>, n);
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            uint4 v[8];
            float g[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int j = j0 + u;
                const int row = j < a.k ? a.pos[(int64_t)t * a.k + j] : -1;
                v[u] = uint4{0, 0, 0, 0};
                g[u] = 0.f;
                if (row >= 0 && row < a.n_rows) {
                    v[u] = load_piece(rows + (int64_t)row * a.ld_rows + c * kVec<T>, n);
                    g[u] = a.gate ? a.gate[(int64_t)t * a.k + j] : 1.f;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float f[kVec<T>];
                unpack<T>(v[u], f);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) sum[i] = fmaf(g[u], f[i], sum[i]);
            }
        }
        float f[kVec<T>];
        unpack<T>(base, f);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum[i] += f[i];
        store_piece(static_cast<T *>(a.out) + (int64_t)t * a.ld_out + c * kVec<T>, pack<T>(sum), n);
    }
}

// L lanes a token: d_out's piece is read once and serves every pick's gradient row and dot product.
// KM: picks held in registers (8 or 16).  8192 tokens of 2048 bf16, 8 picks each: 571 MB in 116 us,
// 4.9 TB/s; 333 tokens 7.7 us.
template <typename T, int KM>
__global__ __launch_bounds__(kThreads) void k_combine_back(CombineBackArgs a, int lanes_log2) {
    __shared__ float part[kThreads / 64][KM];
    const int L = 1 << lanes_log2, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = (blockIdx.x << (8 - lanes_log2)) + (tid >> lanes_log2);
    const bool live = t < a.T;
    const int pieces = live ? (a.H + kVec<T> - 1) / kVec<T> : 0;
    const T *rows = static_cast<const T *>(a.rows);
    int row[KM];
    float gate[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        row[j] = live && j < a.k ? a.pos[(int64_t)t * a.k + j] : -1;
        if (row[j] >= a.n_rows) row[j] = -1;
        gate[j] = row[j] >= 0 ? a.gate[(int64_t)t * a.k + j] : 0.f;
        dot[j] = 0.f;
    }
    for (int c = tid & (L - 1); c < pieces; c += L) {
        const int n = a.H - c * kVec<T>;
        float d[kVec<T>];
        uint4 v[KM];
        unpack<T>(load_piece(static_cast<const T *>(a.d_out) + (int64_t)t * a.ld_d_out + c * kVec<T>, n), d);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            v[j] = uint4{0, 0, 0, 0};
            if (row[j] >= 0) v[j] = load_piece(rows + (int64_t)row[j] * a.ld_rows + c * kVec<T>, n);
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            if (row[j] < 0) continue;
            float f[kVec<T>], s = 0.f;
            unpack<T>(v[j], f);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                s = fmaf(d[i], f[i], s);
                f[i] = gate[j] * d[i];
            }
            dot[j] += s;
            store_piece(static_cast<T *>(a.d_rows) + (int64_t)row[j] * a.ld_d_rows + c * kVec<T>, pack<T>(f), n);
        }
    }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        for (int d = min(L, 64) >> 1; d > 0; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
    if (L <= 64) {
        if (live && (tid & (L - 1)) == 0)
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (j < a.k) a.d_gate[(int64_t)t * a.k + j] = dot[j];
        return;
    }
    if (lane == 0)
#pragma unroll
        for (int j = 0; j < KM; ++j) part[wave][j] = dot[j];
    __syncthreads();
    if (live && tid < a.k) a.d_gate[(int64_t)t * a.k + tid] = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
}

// Lanes that share a token: as many as its row has pieces, 8 .. 64, or the whole workgroup of 256.
int lanes_for(int H, int vec) {
    const int pieces = (H + vec - 1) / vec;
    int log2 = 3;
    while (log2 < 6 && (1 << log2) < pieces) ++log2;
    return pieces > 64 ? 8 : log2;
}
int vec_of(int dtype) { return dtype == T_F32 ? 4 : 8; }

template <typename T>
hipError_t dispatch(const DispatchArgs &a, int32_t *counts, hipStream_t stream) {
    const int N = a.T * a.k;
    const int slices = slices_of(N), per = slices ? per_slice(N, slices) : 1;
    if (slices) {
        const hipError_t e = launch(k_slice_counts, dim3(slices), dim3(kThreads), stream, nullptr, nullptr, a.ids, N, per,
                                    a.E, counts);
        if (e != hipSuccess) return e;
    }
    // without rows to copy, as many tokens a workgroup as it can rank
    const int tokens = std::max(1, a.x ? std::min((a.T + kWgTarget - 1) / kWgTarget, kWgPicks / a.k) : kWgPicks / a.k);
    const dim3 grid(std::max(1, (a.T + tokens - 1) / tokens)), block(kThreads);
    const int32_t *from = slices ? counts : nullptr;
    const int lanes = lanes_for(a.H, kVec<T>);
    return a.E <= 256 ? launch(k_dispatch<T, 256>, grid, block, stream, nullptr, nullptr, a, tokens, lanes, from, slices, per)
                      : launch(k_dispatch<T, kMaxSegments>, grid, block, stream, nullptr, nullptr, a, tokens, lanes, from,
                               slices, per);
}

}  // namespace

size_t dispatch_workspace(int T, int k, int E) { return (size_t)slices_of(T * k) * E * sizeof(int32_t); }

hipError_t launch_dispatch(int dtype, const DispatchArgs &a, void *workspace, hipStream_t stream) {
    int32_t *counts = static_cast<int32_t *>(workspace);
    if (dtype == T_F32) return dispatch<float>(a, counts, stream);
    if (dtype == T_F16) return dispatch<f16>(a, counts, stream);
    return dispatch<bf16>(a, counts, stream);
}

hipError_t launch_combine_rows(int dtype, const CombineRowsArgs &a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int log2 = lanes_for(a.H, vec_of(dtype)), per = kThreads >> log2;
    const dim3 grid((a.T + per - 1) / per), block(kThreads);
    if (dtype == T_F32) return launch(k_combine_rows<float>, grid, block, stream, nullptr, nullptr, a, log2);
    if (dtype == T_F16) return launch(k_combine_rows<f16>, grid, block, stream, nullptr, nullptr, a, log2);
    return launch(k_combine_rows<bf16>, grid, block, stream, nullptr, nullptr, a, log2);
}

template <typename T>
static hipError_t combine_back(const CombineBackArgs &a, hipStream_t stream) {
    const int log2 = lanes_for(a.H, kVec<T>), per = kThreads >> log2;
    const dim3 grid((a.T + per - 1) / per), block(kThreads);
    return a.k <= 8 ? launch(k_combine_back<T, 8>, grid, block, stream, nullptr, nullptr, a, log2)
                    : launch(k_combine_back<T, 16>, grid, block, stream, nullptr, nullptr, a, log2);
}

hipError_t launch_combine_back(int dtype, const CombineBackArgs &a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    if (dtype == T_F32) return combine_back<float>(a, stream);
    if (dtype == T_F16) return combine_back<f16>(a, stream);
    return combine_back<bf16>(a, stream);
}

}  // namespace moe
