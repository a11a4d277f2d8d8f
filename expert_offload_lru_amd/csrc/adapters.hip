// Low-rank adapters (include/moe_tokens.h): out = base + scale B (A x) with a row's own A and B, and
// the gradients.
#include <algorithm>
#include <type_traits>

#include "elements.hpp"
#include "token_kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kTileElements = 1 << 30;   // an adapter's matrix in a block kernel: 32-bit offsets
constexpr int kRowCalls = 256;   // rows of a call that takes a workgroup a row

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

// ------------------------------------------------------------------ blocks of rows, matrix cores

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / 64;

// The 16x16 products of one lane's chunk of kChunk reduction elements per operand: 16-bit types
// multiply as they are (v_mfma_f32_16x16x32), fp32 activations in fp32 (four v_mfma_f32_16x16x4,
// the weights widened).  Lane l holds row l%16 of either operand; which reduction elements its
// quarter l/16 holds is free as long as both operands agree.  Result: lane l, value i is
// element (4 (l/16) + i) of the left rows with row l%16 of the right.
template <typename TX>
struct Mma {
    static constexpr int kChunk = 8;
    typedef f16x8 Frag;
    __device__ static f32x4 mul(Frag a, Frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};
template <>
struct Mma<bf16> {
    static constexpr int kChunk = 8;
    typedef bf16x8 Frag;
    __device__ static f32x4 mul(Frag a, Frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Mma<float> {
    static constexpr int kChunk = 4;
    typedef f32x4 Frag;
    __device__ static f32x4 mul(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// The chunk at p, n elements of it (zeros behind).  EVEN: n is 0 or less, or the whole chunk, and no
// code for a part of one is made (it would cost the registers that keep loads in flight).
template <typename TX, bool EVEN, typename T>
__device__ __forceinline__ typename Mma<TX>::Frag load_chunk(const T *p, int n) {
    typedef typename Mma<TX>::Frag Frag;
    constexpr int C = Mma<TX>::kChunk;
    if constexpr (sizeof(TX) == 2 || sizeof(T) == 4) {
        if constexpr (EVEN) return n > 0 ? __builtin_bit_cast(Frag, load_piece(p, C)) : Frag{};
        return __builtin_bit_cast(Frag, load_piece(p, n));
    } else {   // four 16-bit weights beside fp32 activations
        T e[4] = {};
        if (EVEN ? n > 0 : n >= 4) {
            __builtin_memcpy(e, p, 8);
        } else if constexpr (!EVEN) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) e[i] = p[i];
        }
        return f32x4{widen(e[0]), widen(e[1]), widen(e[2]), widen(e[3])};
    }
}

// Two parts of v whose sum is v to 16 bits or more; an infinity is all in the first.
template <typename T>
__device__ inline void split(float v, T &hi, T &lo) {
    hi = narrow<T>(v);
    const float rest = v - widen(hi);
    lo = narrow<T>(__builtin_isfinite(rest) ? rest : 0.f);
}

// Where a lane's 16 rows x NT x MT work sits: lane l has row l%16 of each of the MT sixteens.
struct Lane {
    int l16, quad, wave;
    __device__ Lane()
        : l16(threadIdx.x & 15), quad((threadIdx.x >> 4) & 3), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {}
};

// The first product of a block of 16 MT rows: v = m w^T.  A wave takes every eighth run of 128 bytes
// of the rows, two chunks a lane, so that a row's cache line is read by one wave at once.
template <typename TX, int MT, bool EVEN>
struct Rows {
    typedef Mma<TX> M;
    static constexpr int C = M::kChunk, kRun = 8 * C;
    const TX *row[MT];   // the lane's rows, from the lane's first chunk on
    int cols;

    // part[wave][row][q] = the wave's share of sum_k m[row, k] w[q0 + q, k].  `then` is called once,
    // behind the first loads: what it requests arrives while these are multiplied and joined.
    template <typename TW, int NT, typename F>
    __device__ __forceinline__ void shrink(const Lane &l, const TW *w, int q0, int r, float *part, F then) const {
        const int full = cols / kRun;
        f32x4 acc[NT][MT] = {};
        unsigned wr[NT];   // r * cols is under 2^30
#pragma unroll
        for (int i = 0; i < NT; ++i) wr[i] = (unsigned)min(q0 + 16 * i + l.l16, r - 1) * cols + 2 * l.quad * C;
        auto run = [&](int d, auto count, auto whole, auto first) __attribute__((always_inline)) {
            constexpr int N = decltype(count)::value;
            typename M::Frag x[N][MT][2], a[N][NT][2];
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = (d + u * kTileWaves) * kRun + s * C;
                    const int n = decltype(whole)::value ? C : cols - k - 2 * l.quad * C;
#pragma unroll
                    for (int j = 0; j < MT; ++j) x[u][j][s] = load_chunk<TX, EVEN || decltype(whole)::value>(row[j] + k, n);
#pragma unroll
                    for (int i = 0; i < NT; ++i) a[u][i][s] = load_chunk<TX, EVEN || decltype(whole)::value>(w + k + wr[i], n);
                }
            if constexpr (decltype(first)::value) {
                __builtin_amdgcn_sched_barrier(0);
                then();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < MT; ++j) acc[i][j] = M::mul(a[u][i][s], x[u][j][s], acc[i][j]);
        };
        constexpr int U = NT == 1 ? 4 / MT : NT == 2 ? 2 : 1;
        int d = l.wave;
        if (d + (U - 1) * kTileWaves < full) {
            run(d, std::integral_constant<int, U>{}, std::true_type{}, std::true_type{});
            for (d += U * kTileWaves; d + (U - 1) * kTileWaves < full; d += U * kTileWaves)
                run(d, std::integral_constant<int, U>{}, std::true_type{}, std::false_type{});
        } else {
            then();
        }
        for (; d < full; d += kTileWaves) run(d, std::integral_constant<int, 1>{}, std::true_type{}, std::false_type{});
        if (full * kRun < cols && full % kTileWaves == l.wave)
            run(full, std::integral_constant<int, 1>{}, std::false_type{}, std::false_type{});
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                *reinterpret_cast<f32x4 *>(part + ((l.wave * MT + j) * 16 + l.l16) * (16 * NT) + 16 * i + 4 * l.quad) =
                    acc[i][j];
    }
};

// v[row][q0 + q] = scale * (sum of the waves' parts), zeros from rank r up to the next multiple of 32.
template <int NT, int MT, int RP>
__device__ inline void join_parts(const float *part, float *v, int q0, int r, float scale) {
    if (NT == 1)
        for (int i = threadIdx.x; i < 16 * MT * 16; i += kTileThreads) v[i / 16 * RP + 16 + i % 16] = 0.f;
    for (int i = threadIdx.x; i < 16 * MT * 16 * NT; i += kTileThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) s += part[w * 16 * MT * 16 * NT + i];
        const int row = i / (16 * NT), q = q0 + i % (16 * NT);
        v[row * RP + q] = q < r ? s * scale : 0.f;
    }
}

// v's operand for the second product: fp32 as it is, 16-bit types in two parts; fp16, whose range
// v may exceed, after a power of two per row.
template <typename TX>
struct Left {
    typename Mma<TX>::Frag hi, lo;
};
template <typename TX>
__device__ inline Left<TX> left_of(const float *v, int exponent) {
    Left<TX> f;
    if constexpr (sizeof(TX) == 4) {
        f.hi = *reinterpret_cast<const f32x4 *>(v);
        f.lo = f.hi;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = std::is_same_v<TX, f16> ? ldexpf(v[i], -exponent) : v[i];
            TX hi, lo;
            split(x, hi, lo);
            f.hi[i] = hi;
            f.lo[i] = lo;
        }
    }
    return f;
}

// The second product: out[row, c] = base[row, c] + sum_q v[row][q] w[c, q] for the columns c0 .. c1.
// A wave takes every eighth group of 64 columns; a lane gets 16 consecutive ones of its row.  hold()
// requests the base of its first kHeld groups ahead of time.
template <typename TX, int MT, bool EVEN>
struct Columns {
    typedef Mma<TX> M;
    static constexpr int C = M::kChunk, kBlock = 4 * C, kPieces = 16 / kVec<TX>, kHeld = 4 / kPieces / MT;
    const TX *base[MT];
    TX *out[MT];
    uint4 held[kHeld][MT][kPieces];
    int cols, c0, c1;

    __device__ __forceinline__ uint4 base_piece(int j, int c) const {
        const int left = cols - c;
        if (!base[j] || left <= 0) return uint4{0, 0, 0, 0};
        return load_piece(base[j] + c, EVEN ? kVec<TX> : left);
    }
    __device__ __forceinline__ void hold(const Lane &l, const bool (&mine)[MT]) {
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int g = c0 + (l.wave + u * kTileWaves) * 64;
            if (g < c1)
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int p = 0; p < kPieces; ++p)
                        held[u][j][p] = mine[j] ? base_piece(j, g + 16 * l.quad + p * kVec<TX>) : uint4{0, 0, 0, 0};
        }
    }
    // kBlocks: blocks of ranks whose split values stay in registers
    template <typename TW, int RP, int kBlocks>
    __device__ __forceinline__ void expand(const Lane &l, const float *v, const TW *w, int r, const bool (&mine)[MT]) const {
        const int blocks = (r + kBlock - 1) / kBlock;
        int exponent[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            exponent[j] = 0;
            if constexpr (std::is_same_v<TX, f16>) {
                float most = 0.f;
                for (int b = 0; b < blocks; ++b)
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        const float a = fabsf(v[(16 * j + l.l16) * RP + b * kBlock + l.quad * C + i]);
                        most = a < __builtin_inff() ? fmaxf(most, a) : most;
                    }
                most = fmaxf(most, __shfl_xor(most, 16));
                most = fmaxf(most, __shfl_xor(most, 32));
                if (most > 0.f) frexpf(most, &exponent[j]);
            }
        }
        Left<TX> left[kBlocks][MT];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            if (b < blocks)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    left[b][j] = left_of<TX>(v + (16 * j + l.l16) * RP + b * kBlock + l.quad * C, exponent[j]);

        auto group = [&](int g, const uint4 (&from)[MT][kPieces]) __attribute__((always_inline)) {
            f32x4 acc[4][MT] = {};
            auto block = [&](int b, const Left<TX> (&f)[MT]) __attribute__((always_inline)) {
                typename M::Frag a[4] = {};
                const int q = b * kBlock + l.quad * C;
                if (q < r)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int c = min(g + 16 * (l.l16 >> 2) + 4 * t + (l.l16 & 3), cols - 1);
                        a[t] = load_chunk<TX, EVEN>(w + ((unsigned)c * r + q), r - q);
                    }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        if constexpr (sizeof(TX) == 2) acc[t][j] = M::mul(a[t], f[j].lo, acc[t][j]);
                        acc[t][j] = M::mul(a[t], f[j].hi, acc[t][j]);
                    }
            };
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                if (b < blocks) block(b, left[b]);
            for (int b = kBlocks; b < blocks; ++b) {
                Left<TX> f[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    f[j] = left_of<TX>(v + (16 * j + l.l16) * RP + b * kBlock + l.quad * C, exponent[j]);
                block(b, f);
            }
            const int c = g + 16 * l.quad;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (!mine[j]) continue;
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    const int left_cols = cols - (c + p * kVec<TX>);
                    if (left_cols <= 0) continue;
                    float sum[kVec<TX>];
                    unpack<TX>(from[j][p], sum);
#pragma unroll
                    for (int i = 0; i < kVec<TX>; ++i) {
                        const int at = p * kVec<TX> + i;
                        float s = acc[at / 4][j][at % 4];
                        if constexpr (std::is_same_v<TX, f16>) s = ldexpf(s, exponent[j]);
                        sum[i] += s;
                    }
                    store_piece(out[j] + c + p * kVec<TX>, pack<TX>(sum), EVEN ? kVec<TX> : left_cols);
                }
            }
        };
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int g = c0 + (l.wave + u * kTileWaves) * 64;
            if (g < c1) group(g, held[u]);
        }
        for (int g = c0 + (l.wave + kHeld * kTileWaves) * 64; g < c1; g += kTileWaves * 64) {
            uint4 from[MT][kPieces];
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int p = 0; p < kPieces; ++p) from[j][p] = base_piece(j, g + 16 * l.quad + p * kVec<TX>);
            group(g, from);
        }
    }
    // Keeps the compiler from computing every address of a turn ahead of the loop over a block's adapters
    // (it spilled registers for them): what they start from becomes unknown here.
    __device__ __forceinline__ void renew(Lane &l, int &r) {
        asm volatile("" : "+s"(r), "+s"(cols), "+s"(c0), "+v"(l.l16), "+v"(l.quad));
    }
    // base (or zeros) to out for the rows without an adapter
    __device__ __forceinline__ void pass(const Lane &l, const bool (&none)[MT]) const {
        for (int g = c0 + l.wave * 64; g < c1; g += kTileWaves * 64)
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (!none[j] || base[j] == out[j]) continue;
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    const int c = g + 16 * l.quad + p * kVec<TX>;
                    if (c < cols) store_piece(out[j] + c, base_piece(j, c), EVEN ? kVec<TX> : cols - c);
                }
            }
    }
};

// The smallest adapter number left among a block's rows (e < 0: done or none), the same in every
// lane of every wave; -1 if there is none.
template <int MT>
__device__ inline int next_adapter(const int (&e)[MT]) {
    unsigned now = ~0u;
#pragma unroll
    for (int j = 0; j < MT; ++j) now = min(now, (unsigned)e[j]);   // a negative number is a large one
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) now = min(now, (unsigned)__shfl_xor((int)now, d));
    return max(__builtin_amdgcn_readfirstlane((int)now), -1);
}

// 16 MT rows a workgroup, for each adapter among them: v = x A^T with the reduction split over the
// waves and joined in LDS, then out = base + v B^T, the columns split over the waves.  Bound by
// memory: x and base are read and out written once, the adapters' matrices come from L2.  Several
// workgroups may share a block of rows (blockIdx.y), each for its own columns, with v computed by each.
// NT: tiles of 16 ranks a pass; RM: ranks that v has room for.
// EVEN: inner, outer and the rank are multiples of a lane's chunk.
template <typename TX, typename TW, int NT, int RM, int MT, bool EVEN>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(EVEN ? 4 : 2))) void k_adapters_tile(AdapterArgs g,
                                                                                                   int slice_cols) {
    constexpr int RP = RM + 4;
    __shared__ __align__(16) float part[kTileWaves * 16 * MT * 16 * NT];
    __shared__ __align__(16) float v[16 * MT * RP];
    Lane l;
    Rows<TX, MT, EVEN> x;
    Columns<TX, MT, EVEN> y;
    x.cols = g.inner;
    y.cols = g.outer;
    y.c0 = blockIdx.y * slice_cols;
    y.c1 = min(g.outer, y.c0 + slice_cols);
    int e[MT];
    bool none[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int row = (blockIdx.x * MT + j) * 16 + l.l16, at = min(row, g.T - 1);
        x.row[j] = static_cast<const TX *>(g.x) + at * g.ld_x + 2 * l.quad * Mma<TX>::kChunk;
        y.base[j] = g.base ? static_cast<const TX *>(g.base) + at * g.ld_base : nullptr;
        y.out[j] = static_cast<TX *>(g.out) + at * g.ld_out;
        const int id = g.adapter[at];
        const bool valid = (unsigned)id < (unsigned)g.n;
        none[j] = row < g.T && !valid;
        e[j] = row < g.T && valid ? id : -1;
    }
    for (int now = next_adapter(e); now >= 0; now = next_adapter(e)) {
        int r = g.r;
        y.renew(l, r);
        const TW *a = static_cast<const TW *>(g.a) + (size_t)now * r * g.inner;
        const TW *b = static_cast<const TW *>(g.b) + (size_t)now * r * g.outer;
        const float scale = g.scale[now];
        bool mine[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            mine[j] = e[j] == now;
            if (mine[j]) e[j] = -1;
        }
        x.template shrink<TW, NT>(l, a, 0, r, part, [&]() __attribute__((always_inline)) { y.hold(l, mine); });
        __syncthreads();
        join_parts<NT, MT, RP>(part, v, 0, r, scale);
        for (int q0 = 16 * NT; q0 < r; q0 += 16 * NT) {
            __syncthreads();
            x.template shrink<TW, NT>(l, a, q0, r, part, [] {});
            __syncthreads();
            join_parts<NT, MT, RP>(part, v, q0, r, scale);
        }
        __syncthreads();
        y.template expand<TW, RP, (RM >= 64 ? 64 : 32) / (4 * Mma<TX>::kChunk)>(l, v, b, r, mine);
    }
    y.pass(l, none);
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

template <typename TX, typename TW, int NT, int RM, bool EVEN>
hipError_t forward_tile(const AdapterArgs &g, hipStream_t stream) {
    constexpr int MT = 1;
    const int tiles = (g.T + 16 * MT - 1) / (16 * MT);
    const int groups = (g.outer + 63) / 64;
    const int slices = std::max(1, std::min(groups / kTileWaves, 512 / tiles));
    const int cols = (groups + slices - 1) / slices * 64;
    return launch(k_adapters_tile<TX, TW, NT, RM, MT, EVEN>, dim3(tiles, (g.outer + cols - 1) / cols), dim3(kTileThreads), stream,
                  nullptr, nullptr, g, cols);
}

template <typename TX, typename TW>
hipError_t forward(const AdapterArgs &g, hipStream_t stream) {
    if (g.T > kRowCalls && (int64_t)g.r * std::max(g.inner, g.outer) < kTileElements) {
        constexpr int C = Mma<TX>::kChunk;
        if (g.inner % C || g.outer % kVec<TX> || g.r % C)
            return g.r <= 64 ? forward_tile<TX, TW, 4, 64, false>(g, stream)
                             : forward_tile<TX, TW, 4, kMaxRank, false>(g, stream);
        if (g.r <= 16) return forward_tile<TX, TW, 1, 32, true>(g, stream);
        if (g.r <= 32) return forward_tile<TX, TW, 2, 32, true>(g, stream);
        if (g.r <= 64) return forward_tile<TX, TW, 4, 64, true>(g, stream);
        return forward_tile<TX, TW, 4, kMaxRank, true>(g, stream);
    }
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
