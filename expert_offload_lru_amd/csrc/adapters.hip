// Low-rank adapters (include/moe_tokens.h): out = base + scale B (A x) with a row's own A and B, and
// the gradients.
#include <algorithm>
#include <type_traits>

#include "elements.hpp"
#include "token_kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRowCalls = 256;    // rows of a call that takes a workgroup a row
constexpr int kRowTarget = 512;   // workgroups of such a call: two a CU

// Eight elements at p (n of them there, zeros behind), as loaded and as fp32.
template <typename T>
struct Eight {
    static constexpr int kPieces = sizeof(T) / 2;
    uint4 raw[kPieces];
    __device__ __forceinline__ void load(const T *p, int n) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) raw[i] = load_piece(p + i * kVec<T>, n - i * kVec<T>);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float e[kVec<T>];
            unpack<T>(raw[i], e);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) f[i * kVec<T> + k] = e[k];
        }
    }
};

__device__ inline float wave_total(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// v[q] = <a's row q, x> for q < r: four rows of a at a time a wave, their loads in flight together.
template <typename TX, typename TW>
__device__ inline void shrink_row(const TX *x, const TW *a, int inner, int r, float *v) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int q0 = wave * 4; q0 < r; q0 += kThreads / 64 * 4) {
        float s[4] = {};
#pragma unroll 2
        for (int c = lane * 8; c < inner; c += 512) {
            Eight<TX> ex;
            Eight<TW> ea[4];
            ex.load(x + c, inner - c);
#pragma unroll
            for (int i = 0; i < 4; ++i) ea[i].load(a + (size_t)min(q0 + i, r - 1) * inner + c, inner - c);
            float fx[8];
            ex.get(fx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float fa[8];
                ea[i].get(fa);
#pragma unroll
                for (int k = 0; k < 8; ++k) s[i] = fmaf(fx[k], fa[k], s[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = wave_total(s[i]);
            if (lane == 0 && q0 + i < r) v[q0 + i] = s[i];
        }
    }
}

// A workgroup a row and slice of the columns: v by dot products (each slice makes its own), then a
// thread a column.  For calls of few rows, whose time is the chain of loads: the first column's share
// of b and base is requested before v is made.
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void k_adapters_row(AdapterArgs g, int slice_cols) {
    __shared__ __align__(16) float v[kMaxRank];
    const int row = blockIdx.x, e = g.adapter[row];
    const int o0 = blockIdx.y * slice_cols + threadIdx.x, o1 = min(g.outer, (int)(blockIdx.y + 1) * slice_cols);
    const bool has = (unsigned)e < (unsigned)g.n;
    const TX *base = g.base ? static_cast<const TX *>(g.base) + row * g.ld_base : nullptr;
    TX *out = static_cast<TX *>(g.out) + row * g.ld_out;
    const TW *b = static_cast<const TW *>(g.b) + (has ? (size_t)e * g.outer * g.r : 0);
    Eight<TW> ahead[2];
    float scale = 0.f, from = 0.f;
    if (o0 < o1) {
        if (has)
#pragma unroll
            for (int i = 0; i < 2; ++i) ahead[i].load(b + (size_t)o0 * g.r + 8 * i, g.r - 8 * i);
        if (base) from = widen(base[o0]);
    }
    if (has) {
        scale = g.scale[e];
        shrink_row(static_cast<const TX *>(g.x) + row * g.ld_x, static_cast<const TW *>(g.a) + (size_t)e * g.r * g.inner,
                   g.inner, g.r, v);
        if (threadIdx.x >= (unsigned)g.r && threadIdx.x < ((g.r + 7) & ~7u)) v[threadIdx.x] = 0.f;
    }
    __syncthreads();
    auto dot = [&](const Eight<TW> &eb, int q, float s) __attribute__((always_inline)) {
        float f[8];
        eb.get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(f[k], v[q + k], s);
        return s;
    };
    for (int o = o0; o < o1; o += kThreads) {
        float s = 0.f;
        if (has) {
            if (o != o0)
#pragma unroll
                for (int i = 0; i < 2; ++i) ahead[i].load(b + (size_t)o * g.r + 8 * i, g.r - 8 * i);
            s = dot(ahead[0], 0, 0.f);
            if (g.r > 8) s = dot(ahead[1], 8, s);
            for (int q = 16; q < g.r; q += 8) {
                Eight<TW> eb;
                eb.load(b + (size_t)o * g.r + q, g.r - q);
                s = dot(eb, q, s);
            }
            s *= scale;
        }
        const float add = o == o0 ? from : base ? widen(base[o]) : 0.f;
        out[o] = narrow<TX>(add + s);
    }
}

// ------------------------------------------------------------------ blocks of rows, matrix cores
//
// For sizes that 16-byte pieces divide.  All loads and stores of the block kernels are buffer
// instructions whose lanes with nothing to do carry an offset out of range (a load gives zeros, a store
// does nothing): without branches around them the compiler keeps them in flight together.

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / 64;
constexpr int kTileRows = 16;
constexpr unsigned kNowhere = 0x80000000u;                   // an offset out of every buffer's range
constexpr int64_t kBufferBytes = (int64_t)kNowhere - 65536;   // a buffer's size at most

typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void *p, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, p ? (int)bytes : 0, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, unsigned at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0));
}
__device__ __forceinline__ void store16(Buffer b, unsigned at, u32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(v, b, (int)at, 0, 0);
}

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

// A chunk as it is loaded, and as the product takes it (16-bit weights beside fp32 activations are
// widened there).
template <typename TX, typename T>
struct Chunk {
    static constexpr bool kWide = sizeof(TX) == 4 && sizeof(T) == 2;
    typename std::conditional<kWide, uint2, u32x4>::type raw;
    __device__ __forceinline__ void load(Buffer b, unsigned at) {
        if constexpr (kWide)
            raw = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(b, (int)at, 0, 0));
        else
            raw = load16(b, at);
    }
    __device__ __forceinline__ typename Mma<TX>::Frag frag() const {
        if constexpr (kWide) {
            T e[4];
            __builtin_memcpy(e, &raw, 8);
            return f32x4{widen(e[0]), widen(e[1]), widen(e[2]), widen(e[3])};
        } else {
            return __builtin_bit_cast(typename Mma<TX>::Frag, raw);
        }
    }
};

// Two parts of v whose sum is v to 16 bits or more; an infinity is all in the first.
template <typename T>
__device__ inline void split(float v, T &hi, T &lo) {
    hi = narrow<T>(v);
    const float rest = v - widen(hi);
    lo = narrow<T>(__builtin_isfinite(rest) ? rest : 0.f);
}

// A lane's place: row l16 of the block, quarter quad of the reduction (or of a piece's 64 bytes).
struct Lane {
    int l16, quad, wave;
    __device__ Lane()
        : l16(threadIdx.x & 15), quad((threadIdx.x >> 4) & 3), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {}
    // The same, unknown to the compiler: addresses are computed again from it where they are used, and
    // not all ahead of the loop over a block's adapters (which spilled 60 registers and more).
    __device__ __forceinline__ Lane again() const {
        Lane l = *this;
        asm volatile("" : "+s"(l.wave), "+v"(l.l16), "+v"(l.quad));
        return l;
    }
};

// The first product of a block's rows: v = m w^T.  A wave takes every eighth run of 128 bytes of the
// rows, two chunks a lane, so that a row's cache line is read by one wave at once, 64 bytes of a row in
// an instruction.  NT: tiles of 16 ranks at a time.
template <typename TX, typename TW, int NT>
struct Shrink {
    typedef Mma<TX> M;
    static constexpr int C = M::kChunk, kRun = 8 * C;
    static constexpr int U = NT == 1 ? 4 : NT == 2 ? 2 : 1;   // runs in flight
    Buffer m, w;
    unsigned row;   // the lane's row in m, bytes
    int cols;

    // part[wave][row][q] = the wave's share of sum_k m[row, k] w[q0 + q, k].  `then` is called once,
    // behind the first loads: what it requests arrives while these are multiplied and joined.
    template <typename F>
    __device__ __forceinline__ void run(const Lane &lane, int q0, int r, float *part, F then) const {
        const Lane l = lane.again();
        f32x4 acc[NT] = {};
        unsigned wr[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int q = q0 + 16 * i + l.l16;
            wr[i] = q < r ? (unsigned)q * cols : kNowhere / sizeof(TW);
        }
        const int runs = (cols + kRun - 1) / kRun;
        auto batch = [&](int d, auto first) __attribute__((always_inline)) {
            Chunk<TX, TX> x[U][2];
            Chunk<TX, TW> a[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = (d + u * kTileWaves) * kRun + 4 * s * C + l.quad * C;
                    const bool in = k < cols;
                    x[u][s].load(m, in ? row + k * (unsigned)sizeof(TX) : kNowhere);
#pragma unroll
                    for (int i = 0; i < NT; ++i) a[u][i][s].load(w, in ? (wr[i] + k) * (unsigned)sizeof(TW) : kNowhere);
                }
            if constexpr (decltype(first)::value) {
                __builtin_amdgcn_sched_barrier(0);
                then();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < NT; ++i) acc[i] = M::mul(a[u][i][s].frag(), x[u][s].frag(), acc[i]);
        };
        batch(l.wave, std::true_type{});
        for (int d = U * kTileWaves; d < runs; d += U * kTileWaves) batch(d + l.wave, std::false_type{});
#pragma unroll
        for (int i = 0; i < NT; ++i)
            *reinterpret_cast<f32x4 *>(part + (l.wave * 16 + l.l16) * (16 * NT) + 16 * i + 4 * l.quad) = acc[i];
    }
};

// v[row][q0 + q] = scale * (sum of the waves' parts), zeros from rank r up to the next multiple of 32.
template <int NT, int RP>
__device__ __forceinline__ void join_parts(const float *part, float *v, int q0, int r, float scale) {
    if (NT == 1)
        for (int i = threadIdx.x; i < 256; i += kTileThreads) v[i / 16 * RP + 16 + i % 16] = 0.f;
    for (int i = threadIdx.x; i < 256 * NT; i += kTileThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) s += part[w * 256 * NT + i];
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
__device__ __forceinline__ Left<TX> left_of(const float *v, int exponent) {
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
// A wave takes every eighth group of 64 columns, a lane 16 of its row's, in pieces of 16 bytes: the
// four lanes of a row have 64 bytes of it in each piece, which the memory reads and writes faster than
// 16 bytes here and there.  kTiles: products of 16x16 that make a piece.  kHeld pieces of base are requested
// ahead (half of it behind the first product's own loads, half behind that product) with the first two
// groups' weights, the results replace the base in its registers, and all are stored at the end: a load
// that waits behind a store waits for the store too.
template <typename TX, typename TW, int kHeld>
struct Expand {
    typedef Mma<TX> M;
    static constexpr int C = M::kChunk, kBlock = 4 * C, V = kVec<TX>, kPieces = 16 / V, kTiles = V / 4;
    static constexpr int kRing = kHeld / kPieces, kEarly = (kRing + 1) / 2, kStep = kTileWaves * 64;
    Buffer base, out, w;
    unsigned base_row, out_row;   // the lane's row, bytes; kNowhere or above: not its turn
    int c0, c1;                   // c1: at most the columns of w
    u32x4 held[kRing][kPieces];
    Chunk<TX, TW> ahead[2][4];

    __device__ __forceinline__ unsigned at(const Lane &l, unsigned row, int g, int p) const {
        const int c = g + p * 4 * V + l.quad * V;
        return c < c1 ? row + c * (unsigned)sizeof(TX) : kNowhere;
    }
    __device__ __forceinline__ void load_base(const Lane &l, int u, int g) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) held[u][p] = load16(base, at(l, base_row, g, p));
    }
    __device__ __forceinline__ void load_weights(const Lane &l, Chunk<TX, TW> (&a)[4], int r, int g, int b) const {
        const int q = b * kBlock + l.quad * C;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = g + t / kTiles * 4 * V + (l.l16 >> 2) * V + 4 * (t % kTiles) + (l.l16 & 3);
            a[t].load(w, c < c1 && q < r ? ((unsigned)c * r + q) * (unsigned)sizeof(TW) : kNowhere);
        }
    }
    __device__ __forceinline__ void early(const Lane &lane) {
        const Lane l = lane.again();
#pragma unroll
        for (int u = 0; u < kEarly; ++u) load_base(l, u, c0 + l.wave * 64 + u * kStep);
    }
    __device__ __forceinline__ void late(const Lane &lane, int r, int g, bool all) {
        const Lane l = lane.again();
#pragma unroll
        for (int u = 0; u < 2 && u < kRing; ++u) load_weights(l, ahead[u], r, g + u * kStep, 0);
        if (all)
#pragma unroll
            for (int u = 0; u < kEarly; ++u) load_base(l, u, g + u * kStep);
#pragma unroll
        for (int u = kEarly; u < kRing; ++u) load_base(l, u, g + u * kStep);
    }
    // kBlocks: blocks of ranks whose split values stay in registers
    template <int RP, int kBlocks>
    __device__ __forceinline__ void run(const Lane &lane, const float *v, int r) {
        const Lane l = lane.again();
        const int blocks = (r + kBlock - 1) / kBlock;
        const float *mine = v + l.l16 * RP + l.quad * C;
        int exponent = 0;
        if constexpr (std::is_same_v<TX, f16>) {
            float most = 0.f;
            for (int b = 0; b < blocks; ++b)
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const float a = fabsf(mine[b * kBlock + i]);
                    most = a < __builtin_inff() ? fmaxf(most, a) : most;
                }
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            if (most > 0.f) frexpf(most, &exponent);
        }
        Left<TX> left[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) left[b] = left_of<TX>(mine + b * kBlock, exponent);
        for (int g0 = c0 + l.wave * 64; g0 < c1; g0 += kRing * kStep) {
            if (g0 != c0 + l.wave * 64) late(l, r, g0, true);
#pragma unroll
            for (int u = 0; u < kRing; ++u) {
                const int g = g0 + u * kStep;
                f32x4 acc[4] = {};
                auto multiply = [&](const Chunk<TX, TW> (&a)[4], const Left<TX> &f) __attribute__((always_inline)) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if constexpr (sizeof(TX) == 2) acc[t] = M::mul(a[t].frag(), f.lo, acc[t]);
                        acc[t] = M::mul(a[t].frag(), f.hi, acc[t]);
                    }
                };
                multiply(ahead[u & 1], left[0]);
                if (u + 2 < kRing) load_weights(lane.again(), ahead[u & 1], r, g + 2 * kStep, 0);
                if constexpr (kBlocks > 1) {
#pragma unroll
                    for (int b = 1; b < kBlocks; ++b)
                        if (b < blocks) {
                            Chunk<TX, TW> a[4];
                            load_weights(l, a, r, g, b);
                            multiply(a, left[b]);
                        }
                    for (int b = kBlocks; b < blocks; ++b) {
                        Chunk<TX, TW> a[4];
                        load_weights(l, a, r, g, b);
                        multiply(a, left_of<TX>(mine + b * kBlock, exponent));
                    }
                }
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    float sum[V];
                    unpack<TX>(__builtin_bit_cast(uint4, held[u][p]), sum);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float s = acc[(p * V + i) / 4][i % 4];
                        if constexpr (std::is_same_v<TX, f16>) s = ldexpf(s, exponent);
                        sum[i] += s;
                    }
                    held[u][p] = __builtin_bit_cast(u32x4, pack<TX>(sum));
                }
                __builtin_amdgcn_sched_barrier(0);   // one group's products at a time: registers
            }
            const Lane o = lane.again();
#pragma unroll
            for (int u = 0; u < kRing; ++u)
#pragma unroll
                for (int p = 0; p < kPieces; ++p) store16(out, at(o, out_row, g0 + u * kStep, p), held[u][p]);
        }
    }
    // base (or zeros) to out
    __device__ __forceinline__ void pass(const Lane &l) const {
        for (int g = c0 + l.wave * 64; g < c1; g += kStep)
#pragma unroll
            for (int p = 0; p < kPieces; ++p) store16(out, at(l, out_row, g, p), load16(base, at(l, base_row, g, p)));
    }
};

// The smallest adapter number left among a block's rows (e < 0: done or none), the same in every
// lane of every wave; -1 if there is none.
__device__ __forceinline__ int next_adapter(int e) {
    unsigned now = (unsigned)e;   // a negative number is a large one
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) now = min(now, (unsigned)__shfl_xor((int)now, d));
    return max(__builtin_amdgcn_readfirstlane((int)now), -1);
}

// Rows row0 .. row0 + 15 of a matrix, as a buffer.
template <typename T>
__device__ __forceinline__ Buffer rows_of(const void *p, int64_t ld, int row0, int rows, int cols) {
    return buffer(p ? static_cast<const T *>(p) + row0 * ld : nullptr,
                  ((size_t)(min(rows - row0, kTileRows) - 1) * ld + cols) * sizeof(T));
}

// 16 rows a workgroup, for each adapter among them: v = x A^T with the reduction split over the
// waves and joined in LDS, then out = base + v B^T, the columns split over the waves.  Bound by
// memory: x and base are read and out written once, the adapters' matrices come from L2.  Several
// workgroups may share a block of rows, each for its own slice of the columns, with v computed by each;
// and a block's adapters are dealt to `turns` workgroups, the first adapter's behind all others, so that
// a block with several of them does not end a whole turn after the rest (a workgroup without an adapter
// ends when it has seen the numbers).
// Workgroups go to the 8 XCDs in turn by index: a block's workgroups have one index modulo 8, and follow
// each other there, so that they share its rows in that XCD's cache.
// RM: ranks that v has room for.
template <typename TX, typename TW, int NT, int RM>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(4))) void k_adapters_tile(
    AdapterArgs g, int slice_cols, int slices, int turns) {
    constexpr int RP = RM + 4;
    __shared__ __align__(16) float part[kTileWaves * 256 * NT];
    __shared__ __align__(16) float v[16 * RP];
    const int of = blockIdx.x >> 3, block = of / slices * 8 + (blockIdx.x & 7), turn = turns - 1 - blockIdx.y;
    const int row0 = block * kTileRows;
    if (row0 >= g.T) return;
    Lane l;
    const int row = row0 + l.l16;
    const int id = g.adapter[min(row, g.T - 1)];
    const bool valid = (unsigned)id < (unsigned)g.n;
    const bool none = row < g.T && !valid;
    int e = row < g.T && valid ? id : -1;
    Shrink<TX, TW, NT> x;
    Expand<TX, TW, NT == 4 && sizeof(TX) == 2 ? 2 : 4> y;
    x.m = rows_of<TX>(g.x, g.ld_x, row0, g.T, g.inner);
    x.row = l.l16 * (unsigned)g.ld_x * sizeof(TX);
    x.cols = g.inner;
    y.base = rows_of<TX>(g.base, g.ld_base, row0, g.T, g.outer);
    y.out = rows_of<TX>(g.out, g.ld_out, row0, g.T, g.outer);
    y.c0 = of % slices * slice_cols;
    y.c1 = min(g.outer, y.c0 + slice_cols);
    const unsigned base_row = l.l16 * (unsigned)g.ld_base * sizeof(TX), out_row = l.l16 * (unsigned)g.ld_out * sizeof(TX);
    int seen = 0;
    for (int now = next_adapter(e); now >= 0; now = next_adapter(e)) {
        const bool mine = e == now;
        if (mine) e = -1;
        if (seen++ % turns != turn) continue;
        int r = g.r;
        asm volatile("" : "+s"(r));
        const size_t of_a = (size_t)now * r * g.inner, of_b = (size_t)now * r * g.outer;
        x.w = buffer(static_cast<const TW *>(g.a) + of_a, (size_t)r * g.inner * sizeof(TW));
        y.w = buffer(static_cast<const TW *>(g.b) + of_b, (size_t)r * g.outer * sizeof(TW));
        y.base_row = mine ? base_row : kNowhere;
        y.out_row = mine ? out_row : kNowhere;
        const float scale = g.scale[now];
        const int g0 = y.c0 + l.wave * 64;
        x.run(l, 0, r, part, [&]() __attribute__((always_inline)) { y.early(l); });
        __builtin_amdgcn_sched_barrier(0);
        if (RM <= 16 * NT || NT == 1) y.late(l, r, g0, false);
        __syncthreads();
        join_parts<NT, RP>(part, v, 0, r, scale);
        if constexpr (RM > 64) {
            for (int q0 = 16 * NT; q0 < r; q0 += 16 * NT) {
                __syncthreads();
                x.run(l, q0, r, part, []() __attribute__((always_inline)) {});
                __syncthreads();
                join_parts<NT, RP>(part, v, q0, r, scale);
            }
            y.late(l, r, g0, false);
        }
        __syncthreads();
        y.template run<RP, (RM >= 64 ? 64 : 32) / (4 * Mma<TX>::kChunk)>(l, v, r);
    }
    if (turn == 0 && __ballot(none) && !(g.base == g.out && g.ld_base == g.ld_out)) {
        y.base_row = none ? base_row : kNowhere;
        y.out_row = none ? out_row : kNowhere;
        y.pass(l);
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

// ------------------------------------------------------------------ gradients, blocks of rows
//
// d_x is the forward's two products with the matrices transposed, so a call first lays them out that
// way (ranks padded to a multiple of 8); v and u go to memory on the way, and the weights' gradients
// are products over the rows of one adapter at a time, in the order of a counting sort.

// at[e][c][q] = a[e][q][c], bt[e][q][o] = b[e][o][q], zeros in the padding; and where inner is padded,
// ap[e][q][c] = a[e][q][c].  32 ranks by 64 columns a workgroup.
template <typename TW>
__global__ __launch_bounds__(kThreads) void k_back_layout(const TW *a, const TW *b, TW *at, TW *bt, TW *ap, int inner,
                                                          int outer, int ip, int op, int r, int rp) {
    __shared__ TW tile[32][65];
    const int tiles_a = (ip + 63) / 64, e = blockIdx.z, q0 = blockIdx.y * 32;
    const bool is_b = (int)blockIdx.x >= tiles_a;
    const int c0 = (is_b ? blockIdx.x - tiles_a : blockIdx.x) * 64;
    const int cols = is_b ? outer : inner, padded = is_b ? op : ip;
    const size_t ea = (size_t)e * r * inner, eb = (size_t)e * r * outer;
    for (int i = threadIdx.x; i < 32 * 64; i += kThreads) {
        const int q = is_b ? i % 32 : i / 64, c = is_b ? i / 32 : i % 64;
        TW v = narrow<TW>(0.f);
        if (q0 + q < r && c0 + c < cols)
            v = is_b ? b[eb + (size_t)(c0 + c) * r + q0 + q] : a[ea + (size_t)(q0 + q) * inner + c0 + c];
        tile[q][c] = v;
        if (!is_b && ap && q0 + q < r && c0 + c < padded) ap[((size_t)e * r + q0 + q) * ip + c0 + c] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 64; i += kThreads) {
        const int q = is_b ? i / 64 : i % 32, c = is_b ? i % 64 : i / 32;
        if (q0 + q >= rp || c0 + c >= padded) continue;
        if (is_b)
            bt[((size_t)e * rp + q0 + q) * op + c0 + c] = tile[q][c];
        else
            at[((size_t)e * ip + c0 + c) * rp + q0 + q] = tile[q][c];
    }
}

// Up to three matrices copied row by row to another row distance and width: zeros behind the narrower
// source (and for a missing one).
struct Reshape {
    const void *from[3];
    void *to[3];
    int64_t ld_from[3], ld_to[3];
    int cols_from[3], cols_to[3];
};
template <typename TX>
__global__ __launch_bounds__(kThreads) void k_back_reshape(Reshape g, int rows) {
    const int m = blockIdx.y;
    for (int row = blockIdx.x * 4 + ((int)threadIdx.x >> 6); row < rows; row += gridDim.x * 4) {
        const TX *from = static_cast<const TX *>(g.from[m]) + row * g.ld_from[m];
        TX *to = static_cast<TX *>(g.to[m]) + row * g.ld_to[m];
        for (int c = (threadIdx.x & 63) * kVec<TX>; c < g.cols_to[m]; c += 64 * kVec<TX>) {
            const uint4 v = g.from[m] && c < g.cols_from[m] ? load_piece(from + c, g.cols_from[m] - c) : uint4{0, 0, 0, 0};
            store_piece(to + c, v, g.cols_to[m] - c);
        }
    }
}

// What the block kernels of a backward call read and write: as AdapterBackArgs, or padded copies.
struct BackBlocks {
    const void *x, *d_out, *dx_base;
    void *d_x;
    int64_t ld_x, ld_d_out, ld_dx_base, ld_d_x;
    const void *a, *at, *bt;          // [n x r x ip], [n x ip x rp], [n x rp x op]
    const int32_t *adapter;
    const float *scale;
    float *v, *u;                     // [T x r]: scale * (A x), scale * (B^T d_out)
    int T, ip, op, n, r, rp;
};

// d_x = dx_base + u A of 16 rows a workgroup, and u; built as k_adapters_tile.  v is the work of one more
// workgroup a block (the last slice), which shares nothing with the others but the adapters' numbers.
template <typename TX, typename TW, int NT, int RM>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(std::is_same_v<TX, f16> && NT == 4 ? 2 : 4))) void k_back_tile(
    BackBlocks g, int slice_cols, int slices, int turns) {
    constexpr int RP = RM + 4;
    __shared__ __align__(16) float part[kTileWaves * 256 * NT];
    __shared__ __align__(16) float u[16 * RP];
    const int of = blockIdx.x >> 3, block = of / (slices + 1) * 8 + (blockIdx.x & 7), turn = turns - 1 - blockIdx.y;
    const int row0 = block * kTileRows, slice = of % (slices + 1);
    if (row0 >= g.T) return;
    Lane l;
    const int row = row0 + l.l16;
    const int id = g.adapter[min(row, g.T - 1)];
    const bool valid = (unsigned)id < (unsigned)g.n;
    const bool none = row < g.T && !valid;
    int e = row < g.T && valid ? id : -1;
    Shrink<TX, TW, NT> x, dy;
    Expand<TX, TW, sizeof(TX) == 2 ? 2 : 4> y;
    x.m = rows_of<TX>(g.x, g.ld_x, row0, g.T, g.ip);
    x.row = l.l16 * (unsigned)g.ld_x * sizeof(TX);
    x.cols = g.ip;
    dy.m = rows_of<TX>(g.d_out, g.ld_d_out, row0, g.T, g.op);
    dy.row = l.l16 * (unsigned)g.ld_d_out * sizeof(TX);
    dy.cols = g.op;
    y.base = rows_of<TX>(g.dx_base, g.ld_dx_base, row0, g.T, g.ip);
    y.out = rows_of<TX>(g.d_x, g.ld_d_x, row0, g.T, g.ip);
    y.c0 = slice * slice_cols;
    y.c1 = min(g.ip, y.c0 + slice_cols);
    const unsigned base_row = l.l16 * (unsigned)g.ld_dx_base * sizeof(TX), out_row = l.l16 * (unsigned)g.ld_d_x * sizeof(TX);
    int seen = 0;
    for (int now = next_adapter(e); now >= 0; now = next_adapter(e)) {
        const bool mine = e == now;
        if (mine) e = -1;
        if (seen++ % turns != turn) continue;
        const unsigned rows = (unsigned)__ballot(mine) & 0xFFFFu;
        int r = g.r;
        asm volatile("" : "+s"(r));
        x.w = buffer(static_cast<const TW *>(g.a) + (size_t)now * r * g.ip, (size_t)r * g.ip * sizeof(TW));
        dy.w = buffer(static_cast<const TW *>(g.bt) + (size_t)now * g.rp * g.op, (size_t)g.rp * g.op * sizeof(TW));
        y.w = buffer(static_cast<const TW *>(g.at) + (size_t)now * g.rp * g.ip, (size_t)g.rp * g.ip * sizeof(TW));
        y.base_row = mine ? base_row : kNowhere;
        y.out_row = mine ? out_row : kNowhere;
        const float scale = g.scale[now];
        const int g0 = y.c0 + l.wave * 64;
        auto keep = [&](float *to) __attribute__((always_inline)) {
            for (int i = threadIdx.x; i < 16 * r; i += kTileThreads) {
                const int k = i / r, q = i - k * r;
                if ((rows >> k) & 1) to[(size_t)(row0 + k) * r + q] = u[k * RP + q];
            }
        };
        if (slice == slices) {
            for (int q0 = 0; q0 < r; q0 += 16 * NT) {
                x.run(l, q0, r, part, []() __attribute__((always_inline)) {});
                __syncthreads();
                join_parts<NT, RP>(part, u, q0, r, scale);
                __syncthreads();
            }
            keep(g.v);
            __syncthreads();
            continue;
        }
        for (int q0 = 0; q0 < r; q0 += 16 * NT) {
            if (q0) __syncthreads();
            dy.run(l, q0, r, part, []() __attribute__((always_inline)) {});
            __syncthreads();
            join_parts<NT, RP>(part, u, q0, r, scale);
        }
        y.early(l);
        y.late(l, g.rp, g0, false);
        __syncthreads();
        if (slice == 0) keep(g.u);
        y.template run<RP, (RM >= 64 ? 64 : 32) / (4 * Mma<TX>::kChunk)>(l, u, g.rp);
        __syncthreads();
    }
    if (turn == 0 && slice < slices && __ballot(none) && !(g.dx_base == g.d_x && g.ld_dx_base == g.ld_d_x)) {
        y.base_row = none ? base_row : kNowhere;
        y.out_row = none ? out_row : kNowhere;
        y.pass(l);
    }
}

// An adapter's rows, in their sorted order, are cut into pieces of `rows`; pieces are numbered through.
struct Piece {
    int e, first, begin, end, count;   // adapter, its first piece, the piece's rows, its pieces
};
constexpr int kPieceCols = 128;

// Piece p, found by every workgroup from the offsets (four adapters a thread); e < 0: there is none.
__device__ inline Piece find_piece(const int32_t *offsets, int n, int rows, int p) {
    __shared__ int wave_sum[kThreads / 64];
    __shared__ Piece found;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) found.e = -1;
    int count[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * threadIdx.x + i;
        count[i] = e < n ? (offsets[e + 1] - offsets[e] + rows - 1) / rows : 0;
        mine += count[i];
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    int start = upto - mine;
    for (int w = 0; w < wave; ++w) start += wave_sum[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (p >= start && p < start + count[i]) {
            const int e = 4 * threadIdx.x + i;
            found.e = e;
            found.first = start;
            found.begin = offsets[e] + (p - start) * rows;
            found.end = min(offsets[e + 1], found.begin + rows);
            found.count = count[i];
        }
        start += count[i];
    }
    __syncthreads();
    return found;
}

// Calls of up to this many rows: an adapter is one piece, its rows are found by the workgroups themselves,
// and there is neither a sort nor a join.
constexpr int kSmallBack = 512;

struct BackWeights {
    const int32_t *adapter;
    const void *x, *d_out;
    int64_t ld_x, ld_d_out;
    const int32_t *offsets, *order;
    const float *v, *u;
    float *partial;      // [piece][r][ip + op]
    float *d_a, *d_b;
    int T, inner, outer, ip, op, n, r, piece_rows;
};

__device__ __forceinline__ void store_grad(const BackWeights &g, int e, bool is_b, int q, int c, float s) {
    if (is_b)
        g.d_b[((size_t)e * g.outer + c) * g.r + q] = s;
    else
        g.d_a[((size_t)e * g.r + q) * g.inner + c] = s;
}

// d_a and d_b of one piece: 128 columns and 16 NT ranks a workgroup, 32 rows a wave at a time.
// left[q][col] = sum over rows of (u or v)[row][q] (x or d_out)[row][col], the rows being the reduction:
// a lane loads 16 bytes of 8 rows, and for bf16 turns them into the eight columns' operands, pairs of
// rows a dword (v_perm), with u and v in two parts of 16 bits together; other types multiply in fp32,
// whose operand is one element.
template <typename TX, int NT, bool SMALL>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(NT == 4 && sizeof(TX) == 4 ? 1 : 2))) void k_back_pieces(BackWeights g) {
    constexpr bool kPairs = std::is_same_v<TX, bf16>;
    constexpr int kLoads = sizeof(TX) == 4 ? 2 : 1;   // of 16 bytes for a lane's 8 columns of a row
    __shared__ __align__(16) f32x4 part[kThreads / 64][8][64];
    Piece p;
    const int32_t *order;
    if constexpr (SMALL) {
        __shared__ int32_t list[kSmallBack];
        __shared__ int found;
        if (threadIdx.x < 64) {
            int at = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x < g.T; i += 64) {
                const bool is = i < g.T && g.adapter[i] == (int)blockIdx.y;
                const unsigned long long m = __ballot(is);
                if (is) list[at + __popcll(m & ((1ull << threadIdx.x) - 1))] = i;
                at += __popcll(m);
            }
            if (threadIdx.x == 0) found = at;
        }
        __syncthreads();
        p = Piece{(int)blockIdx.y, 0, 0, found, 1};
        order = list;
    } else {
        p = find_piece(g.offsets, g.n, g.piece_rows, blockIdx.y);
        if (p.e < 0) return;
        order = g.order;
    }
    const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4, wave = threadIdx.x >> 6;
    const int tiles_a = (g.ip + kPieceCols - 1) / kPieceCols;
    const bool is_b = (int)blockIdx.x >= tiles_a;
    const int c0 = (is_b ? blockIdx.x - tiles_a : blockIdx.x) * kPieceCols, cols = is_b ? g.op : g.ip;
    const int q0 = blockIdx.z * 16 * NT;
    const TX *m = static_cast<const TX *>(is_b ? g.d_out : g.x);
    const int64_t ld = is_b ? g.ld_d_out : g.ld_x;
    const float *left = is_b ? g.v : g.u;
    // the lane's first column of a load; beyond the matrix its last piece (the results are dropped)
    int at[kLoads], rank[NT];
#pragma unroll
    for (int h = 0; h < kLoads; ++h) at[h] = min(c0 + h * 64 + l16 * kVec<TX>, cols - kVec<TX>);
#pragma unroll
    for (int i = 0; i < NT; ++i) rank[i] = min(q0 + 16 * i + l16, g.r - 1);
    f32x4 acc[NT][8] = {};
    for (int b = p.begin + wave * 32; b < p.end; b += 32 * (kThreads / 64)) {
        uint4 x[8][kLoads];
        float f[NT][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // rows 8 quad + j of the 32 (bf16: a lane's chunk of the reduction), or 4 j + quad
            const int i = b + (kPairs ? 8 * quad + j : 4 * j + quad);
            const int row = order[min(i, p.end - 1)];
#pragma unroll
            for (int h = 0; h < kLoads; ++h) x[j][h] = load_piece(m + row * ld + at[h], kVec<TX>);
#pragma unroll
            for (int k = 0; k < NT; ++k) f[k][j] = left[(size_t)row * g.r + rank[k]];
        }
        if (b + 32 > p.end) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (b + (kPairs ? 8 * quad + j : 4 * j + quad) >= p.end) {
#pragma unroll
                    for (int h = 0; h < kLoads; ++h) x[j][h] = uint4{0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < NT; ++k) f[k][j] = 0.f;
                }
        }
        if constexpr (kPairs) {
            bf16x8 hi[NT], lo[NT];
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    bf16 h, w;
                    split(f[k][j], h, w);
                    hi[k][j] = h;
                    lo[k][j] = w;
                }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u32x4 pairs;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const u32x4 r0 = __builtin_bit_cast(u32x4, x[2 * d][0]), r1 = __builtin_bit_cast(u32x4, x[2 * d + 1][0]);
                    pairs[d] = __builtin_amdgcn_perm(r1[t / 2], r0[t / 2], t % 2 ? 0x07060302u : 0x05040100u);
                }
                const bf16x8 right = __builtin_bit_cast(bf16x8, pairs);
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    acc[k][t] = Mma<bf16>::mul(lo[k], right, acc[k][t]);
                    acc[k][t] = Mma<bf16>::mul(hi[k], right, acc[k][t]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float w[8];
#pragma unroll
                for (int h = 0; h < kLoads; ++h) {
                    float e[kVec<TX>];
                    unpack<TX>(x[j][h], e);
#pragma unroll
                    for (int i = 0; i < kVec<TX>; ++i) w[h * kVec<TX> + i] = e[i];
                }
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < NT; ++k)
                        acc[k][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[k][j], w[t], acc[k][t], 0, 0, 0);
            }
        }
    }
    // the waves' sums, joined in order; each wave writes two of the eight column tiles
    const int real = is_b ? g.outer : g.inner;
    const size_t width = g.ip + g.op;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
        if (k) __syncthreads();
#pragma unroll
        for (int t = 0; t < 8; ++t) part[wave][t][lane] = acc[k][t];
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int t = 2 * wave + s;
            const int c = c0 + (kLoads == 2 ? 64 * (t / 4) + 4 * l16 + t % 4 : 8 * l16 + t);
            f32x4 sum = part[0][t][lane];
#pragma unroll
            for (int w = 1; w < kThreads / 64; ++w) sum += part[w][t][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = q0 + 16 * k + 4 * quad + i;
                if (q >= g.r || c >= real) continue;
                if (p.count == 1)
                    store_grad(g, p.e, is_b, q, c, sum[i]);
                else
                    g.partial[((size_t)blockIdx.y * g.r + q) * width + (is_b ? g.ip : 0) + c] = sum[i];
            }
        }
    }
}

// The sum of an adapter's pieces, in order, or zeros where it has no rows.
__global__ __launch_bounds__(kThreads) void k_back_join(BackWeights g) {
    const int e = blockIdx.z, q = blockIdx.y, c0 = blockIdx.x * kThreads + threadIdx.x;
    // pieces of the adapters before, and of this one
    __shared__ int sums[kThreads / 64];
    int before = 0;
    for (int i = threadIdx.x; i < e; i += kThreads) before += (g.offsets[i + 1] - g.offsets[i] + g.piece_rows - 1) / g.piece_rows;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = before;
    __syncthreads();
    const int first = sums[0] + sums[1] + sums[2] + sums[3];
    const int count = (g.offsets[e + 1] - g.offsets[e] + g.piece_rows - 1) / g.piece_rows;
    if (count == 1 || c0 >= g.inner + g.outer) return;
    const bool is_b = c0 >= g.inner;
    const int c = is_b ? c0 - g.inner : c0;
    const size_t width = g.ip + g.op, at = (is_b ? g.ip : 0) + c;
    float s = 0.f;
    for (int p = 0; p < count; ++p) s += g.partial[((size_t)(first + p) * g.r + q) * width + at];
    store_grad(g, e, is_b, q, c, s);
}

// Sizes of a backward call and where its workspace holds what (element sizes as for fp32: the entry
// point does not ask for the types).
struct BackSpace {
    int ip, op, rp, piece_rows, max_pieces;
    bool padded;   // rows are copied to whole pieces of 8 elements
    size_t offsets, order, sort, v, u, at, bt, ap, partial, x, d_out, d_x, bytes;
};
BackSpace back_space(int T, int inner, int outer, int n, int r) {
    BackSpace s;
    s.ip = (inner + 7) / 8 * 8;
    s.op = (outer + 7) / 8 * 8;
    s.rp = (r + 7) / 8 * 8;
    s.padded = s.ip != inner || s.op != outer;
    // pieces such that their workgroups are about two and a half rounds of the chip's CUs
    const int64_t tiles = (s.ip + kPieceCols - 1) / kPieceCols + (s.op + kPieceCols - 1) / kPieceCols;
    s.piece_rows = (int)std::min<int64_t>(1 << 24, std::max<int64_t>(128, (T * tiles / 640 + 127) / 128 * 128));
    s.max_pieces = T / s.piece_rows + std::min(n, T);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    const size_t row = T, adapters = n;
    s.offsets = take((adapters + 1) * 4);
    s.order = take(row * 4);
    s.sort = take(dispatch_workspace(T, 1, n));
    s.v = take(row * r * 4);
    s.u = take(row * r * 4);
    s.at = take(adapters * s.ip * s.rp * 4);
    s.bt = take(adapters * s.op * s.rp * 4);
    s.partial = take((size_t)s.max_pieces * r * (s.ip + s.op) * 4);
    s.ap = take(s.padded ? adapters * r * s.ip * 4 : 0);
    s.x = take(s.padded ? row * s.ip * 4 : 0);
    s.d_out = take(s.padded ? row * s.op * 4 : 0);
    s.d_x = take(s.padded ? row * s.ip * 4 : 0);
    s.bytes = at;
    return s;
}

template <typename TX, typename TW, int NT, int RM>
hipError_t forward_tile(const AdapterArgs &g, hipStream_t stream) {
    const int tiles = (g.T + kTileRows - 1) / kTileRows;
    const int groups = (g.outer + 63) / 64;
    const int slices = std::max(1, std::min(groups / kTileWaves, 512 / tiles));
    const int cols = (groups + slices - 1) / slices * 64, used = (g.outer + cols - 1) / cols;
    const int turns = std::min(g.n, std::max(2, std::min(16, 1024 / (tiles * slices))));
    return launch(k_adapters_tile<TX, TW, NT, RM>, dim3((tiles + 7) / 8 * 8 * used, turns), dim3(kTileThreads), stream,
                  nullptr, nullptr, g, cols, used, turns);
}

// Whether a matrix can be read by the block kernels: rows of whole, aligned 16-byte pieces, sixteen of
// them within a buffer.
bool piecewise(const void *p, int64_t ld, int cols, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && cols * size % 16 == 0 &&
           (15 * ld + cols) * (int64_t)size < kBufferBytes;
}
bool piecewise_adapters(const void *a, const void *b, int inner, int outer, int r, int chunk, size_t size) {
    return (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % (chunk * size) == 0 && r % chunk == 0 &&
           inner % chunk == 0 && outer % chunk == 0 && (int64_t)r * std::max(inner, outer) * (int64_t)size < kBufferBytes;
}

template <typename TX, typename TW>
hipError_t forward(const AdapterArgs &g, hipStream_t stream) {
    constexpr size_t z = sizeof(TX);
    if (g.T > kRowCalls && piecewise(g.x, g.ld_x, g.inner, z) && piecewise(g.out, g.ld_out, g.outer, z) &&
        (!g.base || piecewise(g.base, g.ld_base, g.outer, z)) &&
        piecewise_adapters(g.a, g.b, g.inner, g.outer, g.r, Mma<TX>::kChunk, sizeof(TW))) {
        if (g.r <= 16) return forward_tile<TX, TW, 1, 32>(g, stream);
        if (g.r <= 32) return forward_tile<TX, TW, 2, 32>(g, stream);
        if (g.r <= 64) return forward_tile<TX, TW, 4, 64>(g, stream);
        return forward_tile<TX, TW, 4, kMaxRank>(g, stream);
    }
    const int groups = (g.outer + kThreads - 1) / kThreads;
    const int slices = std::max(1, std::min(groups, kRowTarget / g.T)), cols = (groups + slices - 1) / slices * kThreads;
    return launch(k_adapters_row<TX, TW>, dim3(g.T, (g.outer + cols - 1) / cols), dim3(kThreads), stream, nullptr, nullptr,
                  g, cols);
}

template <typename TX, typename TW, int NT, int RM>
hipError_t back_tile(const BackBlocks &g, hipStream_t stream) {
    const int tiles = (g.T + kTileRows - 1) / kTileRows, groups = (g.ip + 63) / 64;
    const int slices = std::max(1, std::min(groups / kTileWaves, 512 / tiles));
    const int cols = (groups + slices - 1) / slices * 64, used = (g.ip + cols - 1) / cols;
    const int turns = std::min(g.n, std::max(2, std::min(16, 1024 / (tiles * slices))));
    return launch(k_back_tile<TX, TW, NT, RM>, dim3((tiles + 7) / 8 * 8 * (used + 1), turns), dim3(kTileThreads),
                  stream, nullptr, nullptr, g, cols, used, turns);
}

template <typename TX, typename TW>
hipError_t backward(int dtype, const AdapterBackArgs &g, void *workspace, hipStream_t stream) {
    const BackSpace s = back_space(g.T, g.inner, g.outer, g.n, g.r);
    char *ws = static_cast<char *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + s.offsets), *order = reinterpret_cast<int32_t *>(ws + s.order);
    float *v = reinterpret_cast<float *>(ws + s.v), *u = reinterpret_cast<float *>(ws + s.u);
    constexpr size_t z = sizeof(TX);
    const bool blocks =
        g.T > 0 && (int64_t)s.rp * std::max(s.ip, s.op) * (int64_t)sizeof(TW) < kBufferBytes &&
        (15 + 1) * (int64_t)std::max(s.ip, s.op) * (int64_t)z < kBufferBytes &&
        (s.padded || (piecewise(g.x, g.ld_x, g.inner, z) && piecewise(g.d_out, g.ld_d_out, g.outer, z) &&
                      piecewise(g.d_x, g.ld_d_x, g.inner, z) && reinterpret_cast<uintptr_t>(g.a) % 16 == 0 &&
                      (!g.dx_base || piecewise(g.dx_base, g.ld_dx_base, g.inner, z))));
    const bool small = blocks && g.T <= kSmallBack;
    hipError_t err = hipSuccess;
    if (!small) {
        DispatchArgs d{};
        d.ids = g.adapter;
        d.offsets = offsets;
        d.src = order;
        d.T = g.T;
        d.H = 1;
        d.k = 1;
        d.E = g.n;
        err = launch_dispatch(dtype, d, ws + s.sort, stream);
        if (err != hipSuccess) return err;
    }
    if (!blocks) {
        if (g.T > 0) err = launch(k_back_row<TX, TW>, dim3(g.T), dim3(kThreads), stream, nullptr, nullptr, g, v, u);
        if (err != hipSuccess) return err;
        const dim3 grid((g.inner + 63) / 64 + (g.outer + 63) / 64, (g.r + 15) / 16, g.n);
        return launch(k_back_weights<TX>, grid, dim3(kThreads), stream, nullptr, nullptr, g,
                      static_cast<const int32_t *>(offsets), static_cast<const int32_t *>(order),
                      static_cast<const float *>(v), static_cast<const float *>(u));
    }

    TW *at = reinterpret_cast<TW *>(ws + s.at), *bt = reinterpret_cast<TW *>(ws + s.bt);
    TW *ap = s.padded ? reinterpret_cast<TW *>(ws + s.ap) : nullptr;
    err = launch(k_back_layout<TW>, dim3((s.ip + 63) / 64 + (s.op + 63) / 64, (s.rp + 31) / 32, g.n), dim3(kThreads), stream,
                 nullptr, nullptr, static_cast<const TW *>(g.a), static_cast<const TW *>(g.b), at, bt, ap, g.inner, g.outer,
                 s.ip, s.op, g.r, s.rp);
    if (err != hipSuccess) return err;
    BackBlocks b{g.x, g.d_out, g.dx_base, g.d_x, g.ld_x, g.ld_d_out, g.ld_dx_base, g.ld_d_x, g.a, at, bt,
                 g.adapter, g.scale, v, u, g.T, s.ip, s.op, g.n, g.r, s.rp};
    const int copies = std::min((g.T + 3) / 4, 2048);
    if (s.padded) {
        Reshape m{{g.x, g.d_out, g.dx_base}, {ws + s.x, ws + s.d_out, ws + s.d_x}, {g.ld_x, g.ld_d_out, g.ld_dx_base},
                  {s.ip, s.op, s.ip}, {g.inner, g.outer, g.inner}, {s.ip, s.op, s.ip}};
        err = launch(k_back_reshape<TX>, dim3(copies, 3), dim3(kThreads), stream, nullptr, nullptr, m, g.T);
        if (err != hipSuccess) return err;
        b.x = ws + s.x;
        b.d_out = ws + s.d_out;
        b.dx_base = b.d_x = ws + s.d_x;
        b.ld_x = b.ld_dx_base = b.ld_d_x = s.ip;
        b.ld_d_out = s.op;
        b.a = ap;
    }
    err = g.r <= 16   ? back_tile<TX, TW, 1, 32>(b, stream)
          : g.r <= 32 ? back_tile<TX, TW, 2, 32>(b, stream)
          : g.r <= 64 ? back_tile<TX, TW, 4, 64>(b, stream)
                      : back_tile<TX, TW, 4, kMaxRank>(b, stream);
    if (err != hipSuccess) return err;
    if (s.padded) {
        Reshape m{{b.d_x}, {g.d_x}, {s.ip}, {g.ld_d_x}, {g.inner}, {g.inner}};
        err = launch(k_back_reshape<TX>, dim3(copies, 1), dim3(kThreads), stream, nullptr, nullptr, m, g.T);
        if (err != hipSuccess) return err;
    }
    const BackWeights w{g.adapter, b.x, b.d_out, b.ld_x, b.ld_d_out, offsets, order, v, u, reinterpret_cast<float *>(ws + s.partial),
                        g.d_a, g.d_b, g.T, g.inner, g.outer, s.ip, s.op, g.n, g.r, s.piece_rows};
    const int nt = g.r <= 16 ? 1 : g.r <= 32 ? 2 : 4;
    const dim3 grid((s.ip + kPieceCols - 1) / kPieceCols + (s.op + kPieceCols - 1) / kPieceCols, small ? g.n : s.max_pieces,
                    (g.r + 16 * nt - 1) / (16 * nt));
    auto pieces = [&](auto sm) {
        constexpr bool SMALL = decltype(sm)::value;
        return nt == 1   ? launch(k_back_pieces<TX, 1, SMALL>, grid, dim3(kThreads), stream, nullptr, nullptr, w)
               : nt == 2 ? launch(k_back_pieces<TX, 2, SMALL>, grid, dim3(kThreads), stream, nullptr, nullptr, w)
                         : launch(k_back_pieces<TX, 4, SMALL>, grid, dim3(kThreads), stream, nullptr, nullptr, w);
    };
    if (small) return pieces(std::true_type{});
    err = pieces(std::false_type{});
    if (err != hipSuccess) return err;
    return launch(k_back_join, dim3((g.inner + g.outer + kThreads - 1) / kThreads, g.r, g.n), dim3(kThreads), stream,
                  nullptr, nullptr, w);
}

}  // namespace

size_t adapters_workspace(int T, int inner, int outer, int n, int r) { return back_space(T, inner, outer, n, r).bytes; }

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
