// Low-rank adapters (include/moe_tokens.h): out = base + scale B (A x) with a row's own A and B, and
// the gradients.
#include <algorithm>
#include <type_traits>

#include "elements.hpp"
#include "order.hpp"

namespace moe {
namespace {

// A call takes a workgroup a row (k_adapters_row) up to this many rows and products, else blocks of rows.
// The row's cost grows with the work, the blocks' start at 7 to 11 us and grow with the adapters mixed in a
// block.  Rank 16 of 2048 x 2048: 256 rows 8.8 us a row against 11.1, 512 rows 13.3 against 11.3, but 16.5
// against 26.8 with 256 adapters mixed; 1024 rows 16.3 against 12.4.  Rank 64, 128 rows: 19.5 against 11.7,
// but 23 against 36 with 128 adapters mixed (how many are mixed is known on the device alone; n, which the rule
// does not ask, only bounds it).
// Rank 8 of 512 x 512: 1024 rows 5.5 against 7.8, 2048 rows 7.9 against 8.4, 4096 rows 12.2 against 9.3.
constexpr int kRowCalls = 1024;
constexpr int64_t kRowWork = 1 << 25;    // rows x rank x (inner + outer)
// Above, rows that have to be copied to aligned ones first are worth it from here on.  2048 x 2048, rank
// 16: 2048 rows 25 us a row against 29 with copies, 4096 rows 44 against 36; rank 32: 1024 rows 26 against
// 24, 4096 rows 87 against 41.
constexpr int kCopyCalls = 8192;
constexpr int64_t kCopyWork = 1 << 27;
// Workgroups of such a call, of 256 threads: two a CU.  Rank 16 of 2048 x 2048, 256 rows: 8.8 us, 11.0 with 256 and 9.1 with
// 1024; 128 rows: 6.7, 7.7 and 8.0.
constexpr int kRowTarget = 512;

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
template <int THREADS, typename TX, typename TW>
__device__ inline void shrink_row(const TX *x, const TW *a, int inner, int r, float *v) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int q0 = wave * 4; q0 < r; q0 += THREADS / 64 * 4) {
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
// of b and base is requested before v is made.  32 rows with an adapter each, rank 16 of 2048 x 2048, fp32
// with bf16 adapters: 5.4 us for 5 MB, mostly the latency of three loads that wait for each other.
template <typename TX, typename TW, int THREADS>
__global__ __launch_bounds__(THREADS) void k_adapters_row(AdapterArgs g, int slice_cols) {
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
        shrink_row<THREADS>(static_cast<const TX *>(g.x) + row * g.ld_x,
                            static_cast<const TW *>(g.a) + (size_t)e * g.r * g.inner, g.inner, g.r, v);
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
    for (int o = o0; o < o1; o += THREADS) {
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

constexpr int kMostRows = 32;   // rows of a block
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

// The first 8 bits of fp32 values as bf16, and what is left of them.
__device__ __forceinline__ bf16x8 cut(float (&f)[8]) {
    u32x4 top;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t a = __float_as_uint(f[2 * d]), b = __float_as_uint(f[2 * d + 1]);
        top[d] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        f[2 * d] -= __uint_as_float(a & 0xFFFF0000u);
        f[2 * d + 1] -= __uint_as_float(b & 0xFFFF0000u);
    }
    return __builtin_bit_cast(bf16x8, top);
}
// All 24 bits: f = hi + mid + lo (of an infinity the latter two are NaN).
__device__ __forceinline__ void three_parts(float (&f)[8], bf16x8 &hi, bf16x8 &mid, bf16x8 &lo) {
    hi = cut(f);
    mid = cut(f);
    lo = cut(f);
}
// The 11 bits of fp16 values: w = hi + lo.
__device__ __forceinline__ void two_parts(f16x8 w, bf16x8 &hi, bf16x8 &lo) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = widen(w[i]);
    hi = cut(f);
    lo = cut(f);
}

// The low parts' products of a sum whose high parts' products are added to it.  Beside an infinite operand they are a
// NaN (inf * 0) or an infinity of any sign, and the high parts alone give what the sum is; a finite number here, as
// every finite sum is left, keeps it so.  (Of a NaN the median is one of the bounds.)
__device__ __forceinline__ f32x4 bounded(f32x4 v) {
    constexpr float kMost = 3.402823466e38f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_fmed3f(v[i], -kMost, kMost);
    return v;
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

// Waves of a block (16: backward of 16384 rows of 2048 bf16 with rank 32 147 us against 138, rank 64 210 against 196).
constexpr int kShrinkWaves = 8;

// The first product of a block of 16 MT rows: v = m w^T.  The waves take runs of 128 bytes of the
// rows in turn, two chunks a lane, 64 bytes of a row in an instruction.  NT: tiles of 16 ranks at a time.
// More rows a block read w from L2 less often, which is what bounds this beside m.  TILED: w lies in the
// order in which it is loaded (tiled_at), 1 KB an instruction, which L2 gives faster than 64 bytes of 16
// rows (both products of a backward call of 16384 rows at rank 32: 44 us against 52).
template <typename TX, typename TW, int NT, int MT, bool TILED>
struct Shrink {
    typedef Mma<TX> M;
    static constexpr int C = M::kChunk, kRun = 8 * C;
    static constexpr int U = NT * MT == 1 ? 2 : NT * MT == 2 ? 2 : 1;   // runs in flight
    Buffer m, w;
    unsigned row, step;   // the lane's first row in m, and 16 rows, in bytes
    int cols;

    // part[wave][row][q] = the wave's share of sum_k m[row, k] w[q0 + q, k]
    __device__ __forceinline__ void run(const Lane &lane, int q0, int r, float *part) const {
        const Lane l = lane.again();
        f32x4 acc[NT][MT] = {};
        unsigned wr[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int q = q0 + 16 * i + l.l16;
            if constexpr (TILED)
                wr[i] = ((q0 / 16 + i) * 2 * 64 + (threadIdx.x & 63)) * C;
            else
                wr[i] = q < r ? (unsigned)q * cols : kNowhere / sizeof(TW);
        }
        const int runs = (cols + kRun - 1) / kRun;
        for (int d = l.wave; d < runs; d += U * kShrinkWaves) {
            Chunk<TX, TX> x[U][MT][2];
            Chunk<TX, TW> a[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = (d + u * kShrinkWaves) * kRun + 4 * s * C + l.quad * C;
                    const bool in = k < cols;
#pragma unroll
                    for (int j = 0; j < MT; ++j) x[u][j][s].load(m, in ? row + j * step + k * (unsigned)sizeof(TX) : kNowhere);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if constexpr (TILED)   // (beyond the last run: out of the buffer's range)
                            a[u][i][s].load(w, (wr[i] + ((d + u * kShrinkWaves) * ((r + 15) / 16) * 2 + s) * 64 * C) *
                                                   (unsigned)sizeof(TW));
                        else
                            a[u][i][s].load(w, in ? (wr[i] + k) * (unsigned)sizeof(TW) : kNowhere);
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < MT; ++j) acc[i][j] = M::mul(a[u][i][s].frag(), x[u][j][s].frag(), acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                *reinterpret_cast<f32x4 *>(part + ((l.wave * MT + j) * 16 + l.l16) * (16 * NT) + 16 * i + 4 * l.quad) =
                    acc[i][j];
    }
};

// Where element (q, c) of an adapter's [r x cols] matrix lies in that order, of chunks of C elements.
__host__ __device__ inline size_t tiled_at(int q, int c, int r, int C) {
    const int run = c / (8 * C), s = c / (4 * C) % 2, quad = c / C % 4;
    return ((((size_t)run * ((r + 15) / 16) + q / 16) * 2 + s) * 64 + quad * 16 + q % 16) * C + c % C;
}
__host__ __device__ inline size_t tiled_size(int r, int cols, int C) {
    return (size_t)((cols + 8 * C - 1) / (8 * C)) * (8 * C) * ((r + 15) / 16 * 16);
}

// The adapters of a lane's rows (e < 0: done or none): the smallest number left in the block, the same in
// every lane of every wave; -1 if there is none.
template <int MT>
__device__ __forceinline__ int next_adapter(const int (&e)[MT]) {
    unsigned now = ~0u;
#pragma unroll
    for (int j = 0; j < MT; ++j) now = min(now, (unsigned)e[j]);   // a negative number is a large one
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) now = min(now, (unsigned)__shfl_xor((int)now, d));
    return max(__builtin_amdgcn_readfirstlane((int)now), -1);
}
template <int MT>
__device__ __forceinline__ void adapters_of(const int32_t *adapter, int row, int T, int n, int (&e)[MT]) {
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int id = adapter[min(row + 16 * j, T - 1)];
        e[j] = row + 16 * j < T && (unsigned)id < (unsigned)n ? id : -1;
    }
}

// Rows row0 .. row0 + count - 1 of a matrix (as many as there are), as a buffer.
template <typename T>
__device__ __forceinline__ Buffer rows_of(const void *p, int64_t ld, int row0, int count, int rows, int cols) {
    return buffer(p ? static_cast<const T *>(p) + row0 * ld : nullptr,
                  ((size_t)(min(rows - row0, count) - 1) * ld + cols) * sizeof(T));
}

// v = scale (m w^T) for rows with their own adapters' w: the forward's x and A; the backward's x and A,
// and d_out and B transposed.
struct ShrinkJob {
    const void *m, *w;    // [T x cols]; [n][r x cols] (or tiled), w_step elements from one adapter to the next
    int64_t ld, w_step;
    float *v;             // [T x vr], zeros from rank r on
    int cols;
};
struct ShrinkArgs {
    ShrinkJob job[2];
    const int32_t *adapter;
    const float *scale;
    int T, n, r, vr;
};

// 16 MT rows a workgroup, for each adapter among them: the reduction split over the waves and joined in
// LDS.  A block's adapters are dealt to the workgroups of blockIdx.y (one without an adapter ends when it
// has seen the numbers), so that a block with several does not end a whole turn after the rest; with few
// blocks the ranks are dealt to them too.  8192 rows of 2048 bf16 with rank 16: 15 us for 34 MB of x and as
// much of A from L2, which is what it waits for; both products of a backward call of 16384 rows with rank
// 32: 37 to 45 us for 134 MB.
template <typename TX, typename TW, int NT, int MT, bool TILED>
__global__ __launch_bounds__(64 * kShrinkWaves) __attribute__((amdgpu_waves_per_eu(4))) void k_shrink(ShrinkArgs g, int rank_groups) {
    constexpr int kPart = 256 * NT * MT;
    __shared__ __align__(16) float part[kShrinkWaves * kPart];
    const ShrinkJob &job = g.job[blockIdx.z];
    const Lane l;
    Shrink<TX, TW, NT, MT, TILED> x;
    x.row = l.l16 * (unsigned)job.ld * sizeof(TX);
    x.step = 16 * (unsigned)job.ld * sizeof(TX);
    x.cols = job.cols;
    auto product = [&](int row0, int now, unsigned long long rows) __attribute__((always_inline)) {
        int r = g.r;
        asm volatile("" : "+s"(r));
        x.m = rows_of<TX>(job.m, job.ld, row0, 16 * MT, g.T, job.cols);
        x.w = buffer(static_cast<const TW *>(job.w) + now * job.w_step, (size_t)job.w_step * sizeof(TW));
        const float scale = g.scale[now];
        for (int q0 = blockIdx.y % rank_groups * 16 * NT; q0 < g.vr; q0 += rank_groups * 16 * NT) {
            x.run(l, q0, r, part);
            __syncthreads();
            for (int i = threadIdx.x; i < kPart; i += 64 * kShrinkWaves) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kShrinkWaves; ++w) s += part[w * kPart + i];
                const int k = i / (16 * NT), q = q0 + i % (16 * NT);
                if (q < g.vr && (rows >> k) & 1) job.v[(size_t)(row0 + k) * g.vr + q] = q < r ? s * scale : 0.f;
            }
            __syncthreads();
        }
    };
    const int turns = gridDim.y / rank_groups, turn = blockIdx.y / rank_groups, row0 = blockIdx.x * 16 * MT;
    int e[MT];
    adapters_of(g.adapter, row0 + l.l16, g.T, g.n, e);
    int seen = 0;
    for (int now = next_adapter(e); now >= 0; now = next_adapter(e)) {
        // its rows, taken out of e
        unsigned long long rows = 0;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            rows |= (__ballot(e[j] == now) & 0xFFFFull) << (16 * j);
            if (e[j] == now) e[j] = -1;
        }
        if (seen++ % turns == turn) product(row0, now, rows);
    }
}

// v's operand for the second product: fp32 as it is, beside 16-bit weights in three parts of bf16, which has the range
// that v may take (fp16 parts lost components 2^14 below a row's largest).  Two parts beside bf16 weights were no
// faster (8192 rows of 2048 columns, rank 16: the call 36.0 us against 36.3; rank 64: 57.2 against 56.6).
template <typename TX>
struct Left {
    static constexpr int C = Mma<TX>::kChunk;
    typedef typename std::conditional<sizeof(TX) == 4, f32x4, bf16x8>::type Part;
    float raw[C];
    Part hi, mid, lo;
    __device__ __forceinline__ void load(Buffer v, unsigned at) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const f32x4 f = __builtin_bit_cast(f32x4, load16(v, at + 4 * i));
#pragma unroll
            for (int k = 0; k < 4; ++k) raw[i + k] = f[k];
        }
    }
    __device__ __forceinline__ void part() {
        if constexpr (sizeof(TX) == 4) {
#pragma unroll
            for (int i = 0; i < C; ++i) hi[i] = raw[i];
        } else {
            three_parts(raw, hi, mid, lo);
        }
    }
};

// Adds w v to the sums of the high parts' products and of the others.  fp16 weights are cut into two bf16 parts (the
// kernel with 8192 rows of 2048 columns, rank 64: 29.0 us, with fp32 products 37.4; rank 16: 23.1 and 25.0).
template <typename TX, typename TW>
__device__ __forceinline__ void multiply(const Chunk<TX, TW> &w, const Left<TX> &f, f32x4 &high, f32x4 &low) {
    if constexpr (std::is_same_v<TX, f16>) {
        bf16x8 wh, wl;
        two_parts(w.frag(), wh, wl);
        low = Mma<bf16>::mul(wl, f.lo, low);
        low = Mma<bf16>::mul(wl, f.mid, low);
        low = Mma<bf16>::mul(wh, f.lo, low);
        low = Mma<bf16>::mul(wl, f.hi, low);
        low = Mma<bf16>::mul(wh, f.mid, low);
        high = Mma<bf16>::mul(wh, f.hi, high);
    } else {
        if constexpr (sizeof(TX) == 2) low = Mma<TX>::mul(w.frag(), f.mid, Mma<TX>::mul(w.frag(), f.lo, low));
        high = Mma<TX>::mul(w.frag(), f.hi, high);
    }
}

// out = base + v w^T, w a row's own adapter's: the forward's B, the backward's A transposed.
struct ExpandArgs {
    const void *base, *w;   // [T x cols] or null; [n x w_rows x wr], zeros from w_rows on to cols
    void *out;
    const float *v;         // [T x vr]
    const int32_t *adapter;
    int64_t ld_base, ld_out;
    int T, cols, n, w_rows, wr, vr, groups;   // groups: of 64 columns, that a wave takes
};

// 16 MT rows and a few groups of 64 columns a wave, without a barrier: bound by reading base and writing
// out, and by reading w from L2, the less often the more rows; v, split once a wave, is there too.  A lane
// gets 16 columns of its row in pieces of 16 bytes: the four lanes of a row have 64 bytes of it in each
// piece.  kTiles: products of 16x16 that make a piece.  For a block with several adapters each one's
// product is made in turn and the rows keep their own.  Workgroups go to the 8 XCDs in turn by index:
// those of a block have one index modulo 8, and follow each other there.  KB: blocks of ranks whose operand
// stays in registers.  8192 rows of 2048 bf16 with rank 16: 67 MB in 18.2 us, 3.7 TB/s; 16384 rows with
// rank 32: 134 MB in 32 us, 4.2 TB/s.  Waves a SIMD: what 512 registers allow without a spill; left to itself the
// compiler copied accumulators to and fro (rank 64, 2048 rows of fp16: the call 30.1 us against 26.0).
template <typename TX, typename TW, int KB, int MT>
__global__ __launch_bounds__(kThreads)
__attribute__((amdgpu_waves_per_eu(MT == 2 ? 2 : sizeof(TX) == 2 && KB == 1 ? 4 : 3))) void k_expand(ExpandArgs g, int col_wgs) {
    typedef Mma<TX> M;
    constexpr int C = M::kChunk, kBlock = 4 * C, V = kVec<TX>, kPieces = 16 / V, kTiles = V / 4;
    const Lane l;
    const int of = blockIdx.x >> 3, row0 = (of / col_wgs * 8 + (blockIdx.x & 7)) * 16 * MT;
    if (row0 >= g.T) return;
    int e[MT];
    adapters_of(g.adapter, row0 + l.l16, g.T, g.n, e);
    const Buffer base = rows_of<TX>(g.base, g.ld_base, row0, 16 * MT, g.T, g.cols);
    const Buffer out = rows_of<TX>(g.out, g.ld_out, row0, 16 * MT, g.T, g.cols);
    const Buffer v = rows_of<float>(g.v, g.vr, row0, 16 * MT, g.T, g.vr);
    unsigned base_row[MT], out_row[MT];   // a row behind the last: nowhere
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const bool in = row0 + 16 * j + l.l16 < g.T;
        base_row[j] = in ? (16 * j + l.l16) * (unsigned)g.ld_base * sizeof(TX) : kNowhere;
        out_row[j] = in ? (16 * j + l.l16) * (unsigned)g.ld_out * sizeof(TX) : kNowhere;
    }
    const int blocks = (g.vr + kBlock - 1) / kBlock;
    const int first = next_adapter(e);
    int todo[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) todo[j] = e[j] == first ? -1 : e[j];
    const bool several = next_adapter(todo) >= 0;

    auto left_at = [&](int b, int j) {
        const int q = b * kBlock + l.quad * C;
        return e[j] >= 0 && q < g.vr ? ((16 * j + l.l16) * g.vr + q) * 4u : kNowhere;   // 0 for a row without an adapter
    };
    Left<TX> left[KB][MT];
    if (first >= 0) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int j = 0; j < MT; ++j) left[b][j].load(v, left_at(b, j));
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int j = 0; j < MT; ++j) left[b][j].part();
    }
    auto weights = [&](int now) {
        return buffer(static_cast<const TW *>(g.w) + (size_t)now * g.w_rows * g.wr, (size_t)g.w_rows * g.wr * sizeof(TW));
    };
    auto load_weights = [&](Chunk<TX, TW> (&a)[4], Buffer w, int c0, int b) __attribute__((always_inline)) {
        const int q = b * kBlock + l.quad * C;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = c0 + t / kTiles * 4 * V + (l.l16 >> 2) * V + 4 * (t % kTiles) + (l.l16 & 3);
            a[t].load(w, c < g.cols && q < g.wr ? ((unsigned)c * g.wr + q) * (unsigned)sizeof(TW) : kNowhere);
        }
    };
    const int g0 = ((of % col_wgs) * (kThreads / 64) + l.wave) * g.groups, g1 = min(g0 + g.groups, (g.cols + 63) / 64);
    auto or_nowhere = [](unsigned row, unsigned c) { return (row | c) >= kNowhere ? kNowhere : row + c; };
    auto column = [&](int k, int p) {
        const int c = k * 64 + p * 4 * V + l.quad * V;
        return c < g.cols ? c * (unsigned)sizeof(TX) : kNowhere;
    };
    // the products of one adapter's w with every row
    auto product = [&](f32x4 (&acc)[MT][4], Buffer w, int k) __attribute__((always_inline)) {
        Chunk<TX, TW> a[KB][4];
#pragma unroll
        for (int b = 0; b < KB; ++b) load_weights(a[b], w, k * 64, b);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                f32x4 low = {};
#pragma unroll
                for (int b = 0; b < KB; ++b) multiply(a[b][t], left[b][j], acc[j][t], low);
                if constexpr (sizeof(TX) == 2) acc[j][t] += bounded(low);
            }
        for (int b = KB; b < blocks; ++b) {
            Chunk<TX, TW> o[4];
            load_weights(o, w, k * 64, b);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                Left<TX> f;
                f.load(v, left_at(b, j));
                f.part();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 low = {};
                    multiply(o[t], f, acc[j][t], low);
                    if constexpr (sizeof(TX) == 2) acc[j][t] += bounded(low);
                }
            }
        }
    };
    const Buffer w = weights(max(first, 0));
    for (int k = g0; k < g1; ++k) {
        u32x4 held[MT][kPieces];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int p = 0; p < kPieces; ++p) held[j][p] = load16(base, or_nowhere(base_row[j], column(k, p)));
        f32x4 res[MT][4] = {};
        if (first >= 0) {
            product(res, w, k);
            if (several) {
                int left_over[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j) left_over[j] = todo[j];
                for (int now = next_adapter(left_over); now >= 0; now = next_adapter(left_over)) {
                    f32x4 acc[MT][4] = {};
                    product(acc, weights(now), k);
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) res[j][t][i] = e[j] == now ? acc[j][t][i] : res[j][t][i];
                        if (left_over[j] == now) left_over[j] = -1;
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                float sum[V];
                unpack<TX>(__builtin_bit_cast(uint4, held[j][p]), sum);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float s = res[j][(p * V + i) / 4][i % 4];
                    sum[i] += e[j] >= 0 ? s : 0.f;
                }
                store16(out, or_nowhere(out_row[j], column(k, p)), __builtin_bit_cast(u32x4, pack<TX>(sum)));
            }
    }
}

// ------------------------------------------------------------------ gradients, a workgroup a row
//
// For rows that the block kernels cannot read where the workspace has no room for copies of them: right,
// and slow (16384 rows of 2048 bf16, rank 32: 3.4 ms against 0.11 aligned and 0.21 with copies).

// v and u of a row to memory, and its d_x.
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void k_back_row(AdapterBackArgs g, float *gv, float *gu) {
    __shared__ float v[kMaxRank], u[kMaxRank];
    const int row = blockIdx.x, e = g.adapter[row], lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool has = (unsigned)e < (unsigned)g.n;
    const TW *a = static_cast<const TW *>(g.a) + (has ? (size_t)e * g.r * g.inner : 0);
    const TX *dy = static_cast<const TX *>(g.d_out) + row * g.ld_d_out;
    if (has) {
        shrink_row<kThreads>(static_cast<const TX *>(g.x) + row * g.ld_x, a, g.inner, g.r, v);
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

// at[e][c][q] = a[e][q][c] with zeros in the padding, and a and b transposed in the order in which the first
// product loads them (tiled_at), zeros behind their last column.  32 ranks by 64 columns a workgroup.  The
// first `order_wgs` workgroups make the order of the rows by adapter meanwhile (16384 rows, 4 adapters of
// rank 32, 2048 x 2048: 11 us, against 9 and 11 as two launches).  C: a chunk's elements.
constexpr int kOrderedHere = 256;   // adapters that this has room for
template <typename TW, int C>
__global__ __launch_bounds__(kThreads) void k_back_layout(const TW *a, const TW *b, TW *at, TW *aw, TW *bw, int inner, int outer,
                                                          int ip, int r, int rp, DispatchArgs order, int order_wgs) {
    __shared__ union {
        TW tile[32][65];
        OrderSpace<kOrderedHere> order;
    } lds;
    auto &tile = lds.tile;
    const int tile_at = (int)blockIdx.x - order_wgs;
    if (tile_at < 0) {
        if (blockIdx.y == 0 && blockIdx.z == 0) order_picks<kOrderedHere>(order, blockIdx.x, kWgPicks, nullptr, 0, 1, lds.order);
        return;
    }
    const int tiles_a = (ip + 63) / 64, e = blockIdx.z, q0 = blockIdx.y * 32;
    const bool is_b = tile_at >= tiles_a;
    const int c0 = (is_b ? tile_at - tiles_a : tile_at) * 64;
    const int cols = is_b ? outer : inner;
    const size_t ea = (size_t)e * r * inner, eb = (size_t)e * r * outer;
    TW *to = (is_b ? bw : aw) + e * tiled_size(r, cols, C);
    const int whole = (cols + 8 * C - 1) / (8 * C) * (8 * C);   // columns of whole runs
#pragma unroll
    for (int k = 0; k < 32 * 64 / kThreads; ++k) {
        const int i = threadIdx.x + k * kThreads, q = is_b ? i % 32 : i / 64, c = is_b ? i / 32 : i % 64;
        TW v = narrow<TW>(0.f);
        if (q0 + q < r && c0 + c < cols)
            v = is_b ? b[eb + (size_t)(c0 + c) * r + q0 + q] : a[ea + (size_t)(q0 + q) * inner + c0 + c];
        tile[q][c] = v;
    }
    __syncthreads();
    // consecutive threads write consecutive elements: a chunk of a rank's, then the next rank's
#pragma unroll
    for (int k = 0; k < 32 * 64 / kThreads; ++k) {
        const int i = threadIdx.x + k * kThreads, c = i % C + i / (32 * C) * C, q = i / C % 32;
        if (q0 + q < (r + 15) / 16 * 16 && c0 + c < whole) to[tiled_at(q0 + q, c0 + c, r, C)] = tile[q][c];
    }
    if (is_b) return;
#pragma unroll
    for (int k = 0; k < 32 * 64 / kThreads; ++k) {
        const int i = threadIdx.x + k * kThreads, q = i % 32, c = i / 32;
        if (q0 + q < rp && c0 + c < ip) at[((size_t)e * ip + c0 + c) * rp + q0 + q] = tile[q][c];
    }
}

// Matrices copied row by row to another row distance and width: zeros behind the narrower source (and for
// a missing one).
struct Copy {
    const void *from;
    void *to;
    int64_t ld_from, ld_to;
    int cols_from, cols_to, rows;
    bool weights;   // of the weights' type
};
struct Reshape {
    Copy copy[4];
    int n;
    void add(Copy c) { copy[n++] = c; }
};
template <typename T>
__device__ __forceinline__ void copy_rows(const Copy &g) {
    for (int row = blockIdx.x * 4 + ((int)threadIdx.x >> 6); row < g.rows; row += gridDim.x * 4) {
        const T *from = static_cast<const T *>(g.from) + row * g.ld_from;
        T *to = static_cast<T *>(g.to) + row * g.ld_to;
        for (int c = (threadIdx.x & 63) * kVec<T>; c < g.cols_to; c += 64 * kVec<T>) {
            const uint4 v = g.from && c < g.cols_from ? load_piece(from + c, g.cols_from - c) : uint4{0, 0, 0, 0};
            store_piece(to + c, v, g.cols_to - c);
        }
    }
}
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void k_reshape(Reshape g) {
    const Copy &c = g.copy[blockIdx.y];
    if (c.weights)
        copy_rows<TW>(c);
    else
        copy_rows<TX>(c);
}
template <typename TX, typename TW>
hipError_t reshape(const Reshape &g, hipStream_t stream) {
    if (g.n == 0) return hipSuccess;
    int rows = 0;
    for (int i = 0; i < g.n; ++i) rows = std::max(rows, g.copy[i].rows);
    return launch(k_reshape<TX, TW>, dim3(std::min((rows + 3) / 4, 2048), g.n), dim3(kThreads), stream, nullptr, nullptr, g);
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
// and there is neither a sort nor a join.  512 rows, rank 16 of 2048 x 2048: 23.4 us against 24.8 (64
// adapters mixed: 65 against 72); 1024 rows 31.8 against 30.0.
constexpr int kSmallBack = 512;
// Rows whose order is made in the layout's launch, each ordering workgroup counting them all: 32768 rows of
// 2048 columns 210 us against 218 with a launch of its own, 131072 rows of 256 columns 188 against 168.
constexpr int kOrderRows = 32768;

struct BackWeights {
    const int32_t *adapter;
    const void *x, *d_out;
    int64_t ld_x, ld_d_out;
    const int32_t *offsets, *order;
    const float *v, *u;
    float *partial;      // [piece][r][ip + op]
    float *d_a, *d_b;
    int T, inner, outer, ip, op, n, r, vr, piece_rows;
};

__device__ __forceinline__ float *grad_at(const BackWeights &g, int e, bool is_b, int q, int c) {
    return is_b ? g.d_b + ((size_t)e * g.outer + c) * g.r + q : g.d_a + ((size_t)e * g.r + q) * g.inner + c;
}

// d_a and d_b of one piece: 128 columns and 16 NT ranks a workgroup, 32 rows a wave at a time.
// left[q][col] = sum over rows of (u or v)[row][q] (x or d_out)[row][col], the rows being the reduction:
// a lane loads 16 bytes of 8 rows, and for bf16 turns them into the eight columns' operands, pairs of
// rows a dword (v_perm), with u and v in three parts, which hold all of an fp32 value's 24 bits (two parts
// made the gradients' error 2.5 times that of fp32 products); other types multiply in fp32, whose operand is
// one element.  16384 rows of 2048 bf16, rank 32, both gradients: 134 MB in 28 us, 4.8 TB/s, when they come
// from the memory-side cache, 38 us when not; the join after it 5 us.
template <typename TX, int NT, bool SMALL>
__global__ __launch_bounds__(kThreads)
__attribute__((amdgpu_waves_per_eu(NT == 4 && sizeof(TX) == 4 ? 1 : 2))) void k_back_pieces(BackWeights g) {
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
    const int tiles_a = (g.ip + kPieceCols - 1) / kPieceCols;
    const bool is_b = (int)blockIdx.x >= tiles_a;
    const int c0 = (is_b ? blockIdx.x - tiles_a : blockIdx.x) * kPieceCols, cols = is_b ? g.op : g.ip;
    const int q0 = blockIdx.z * 16 * NT;
    const TX *m = static_cast<const TX *>(is_b ? g.d_out : g.x);
    const int64_t ld = is_b ? g.ld_d_out : g.ld_x;
    const float *left = is_b ? g.v : g.u;
    // Beside an infinite x or d_out the parts' products are infinities of any sign and NaN (0 * inf): if a result is not
    // finite, a second pass takes the first part three times, whose sums are NaN or an infinity where the result is.
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        bool bad = false;
        int id = threadIdx.x;
        asm volatile("" : "+v"(id));   // or addresses of all of a pass are computed ahead of the first, and spill
        const int lane = id & 63, l16 = lane & 15, quad = lane >> 4, wave = id >> 6;
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
                for (int k = 0; k < NT; ++k) f[k][j] = left[(size_t)row * g.vr + rank[k]];
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
                bf16x8 hi[NT], mid[NT], lo[NT];
#pragma unroll
                for (int k = 0; k < NT; ++k) three_parts(f[k], hi[k], mid[k], lo[k]);
                if (pass == 1)
#pragma unroll
                    for (int k = 0; k < NT; ++k) mid[k] = lo[k] = hi[k];
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
                        acc[k][t] = Mma<bf16>::mul(mid[k], right, acc[k][t]);
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
                    float *to = p.count == 1 ? grad_at(g, p.e, is_b, q, c)
                                             : g.partial + ((size_t)blockIdx.y * g.r + q) * width + (is_b ? g.ip : 0) + c;
                    if (pass == 0) {
                        *to = sum[i];
                        bad |= !__builtin_isfinite(sum[i]);
                    } else if (!__builtin_isfinite(sum[i]) && !__builtin_isfinite(*to)) {
                        *to = sum[i];
                    }
                }
            }
        }
        if constexpr (!kPairs) break;
        if (!__syncthreads_or(bad)) break;
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
#pragma unroll 4
    for (int p = 0; p < count; ++p) s += g.partial[((size_t)(first + p) * g.r + q) * width + at];
    *grad_at(g, e, is_b, q, c) = s;
}

// Sizes of a backward call and where its workspace holds what (element sizes as for fp32: the entry
// point does not ask for the types).
struct BackSpace {
    int ip, op, rp, piece_rows, max_pieces;
    bool padded;   // rows are copied to whole, aligned pieces of 8 elements: odd sizes, or if asked for
    size_t offsets, order, sort, v, u, at, aw, bw, partial, x, d_out, d_x, bytes;
};
BackSpace back_space(int T, int inner, int outer, int n, int r, bool copies) {
    BackSpace s;
    s.ip = (inner + 7) / 8 * 8;
    s.op = (outer + 7) / 8 * 8;
    s.rp = (r + 7) / 8 * 8;
    s.padded = copies || s.ip != inner || s.op != outer;
    // pieces such that their workgroups are about two and a half rounds of the chip's CUs (16384 rows, rank
    // 32, one adapter: 99 us, 106 with half as many, 102 with twice; 8 adapters: 136, 137 and 142)
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
    s.v = take(row * s.rp * 4);
    s.u = take(row * s.rp * 4);
    s.at = take(adapters * s.ip * s.rp * 4);
    // whole runs of columns, 64 elements for 16-bit activations
    s.aw = take(adapters * tiled_size(r, inner, 8) * 4);
    s.bw = take(adapters * tiled_size(r, outer, 8) * 4);
    s.partial = take(T <= kSmallBack ? 0 : (size_t)s.max_pieces * r * (s.ip + s.op) * 4);   // (few rows: no pieces to join)
    s.x = take(s.padded ? row * s.ip * 4 : 0);
    s.d_out = take(s.padded ? row * s.op * 4 : 0);
    s.d_x = take(s.padded ? row * s.ip * 4 : 0);
    s.bytes = at;
    return s;
}

// A forward call of blocks holds v; b with its rows padded where the rank is no multiple of 8, a where
// inner is none; and copies of x, and of base and out, as above.
struct ForwardSpace {
    int ip, op, rp;
    bool copy_x, copy_out;
    size_t v, b, a, x, out, bytes;
};
int64_t work_of(int64_t T, int inner, int outer, int r) { return T * r * (inner + outer); }
ForwardSpace forward_space(int T, int inner, int outer, int n, int r, bool copies) {
    ForwardSpace s{};
    if (T <= kRowCalls && work_of(T, inner, outer, r) <= kRowWork) return s;
    s.ip = (inner + 7) / 8 * 8;
    s.op = (outer + 7) / 8 * 8;
    s.rp = (r + 7) / 8 * 8;
    s.copy_x = copies || s.ip != inner;
    s.copy_out = copies || s.op != outer;
    auto take = [&](size_t bytes) {
        const size_t here = s.bytes;
        s.bytes += (bytes + 255) & ~(size_t)255;
        return here;
    };
    const size_t rows = T, adapters = n;
    s.v = take(rows * s.rp * 4);
    s.b = take(s.rp == r ? 0 : adapters * outer * s.rp * 4);
    s.a = take(s.ip == inner ? 0 : adapters * r * s.ip * 4);
    s.x = take(s.copy_x ? rows * s.ip * 4 : 0);
    s.out = take(s.copy_out ? rows * s.op * 4 : 0);
    return s;
}

// Whether a matrix can be read by the block kernels: rows of whole, aligned 16-byte pieces, a block of
// them within a buffer.
bool piecewise(const void *p, int64_t ld, int cols, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && cols * size % 16 == 0 &&
           ((kMostRows - 1) * ld + cols) * (int64_t)size < kBufferBytes;
}
// Whether an adapter's matrices, as they are laid out, fit a buffer.
bool fits_buffer(int64_t ip, int64_t op, int64_t rp, size_t size) { return rp * std::max(ip, op) * (int64_t)size < kBufferBytes; }

// Blocks up to which a workgroup takes 16 ranks only and the others go to more of them.  Rank 64 of 2048
// columns: 512 rows 15.0 us against 20.3; backward of 59 rows of 5056 columns 45 against 65; with blocks up
// to 256, backward of 2000 rows 63 against 59.
constexpr int kFewTiles = 64;
template <typename TX, typename TW, int MT, bool TILED>
hipError_t shrink(const ShrinkArgs &g, int jobs, hipStream_t stream) {
    const int tiles = (g.T + 16 * MT - 1) / (16 * MT);
    // turns: four workgroups a CU (8 adapters of rank 64, 2048 rows: 27 us, 35 with two turns; 64 mixed
    // adapters of rank 16: 51 and 55)
    const int turns = std::min(g.n, std::max(2, std::min(16, 1024 / tiles)));
    const dim3 grid(tiles, turns, jobs), block(64 * kShrinkWaves);
    if constexpr (MT == 1) {   // (taller blocks are for ranks from 17 on and many rows)
        if (g.r <= 16) return launch(k_shrink<TX, TW, 1, MT, TILED>, grid, block, stream, nullptr, nullptr, g, 1);
        if (tiles * jobs <= kFewTiles) {
            const int groups = (g.r + 15) / 16;
            return launch(k_shrink<TX, TW, 1, MT, TILED>, dim3(tiles, turns * groups, jobs), block, stream, nullptr, nullptr, g, groups);
        }
    }
    if (g.r <= 32) return launch(k_shrink<TX, TW, 2, MT, TILED>, grid, block, stream, nullptr, nullptr, g, 1);
    return launch(k_shrink<TX, TW, 4, MT, TILED>, grid, block, stream, nullptr, nullptr, g, 1);
}

template <typename TX, typename TW, int MT>
hipError_t expand(ExpandArgs g, hipStream_t stream) {
    const int tiles = (g.T + 16 * MT - 1) / (16 * MT), groups = (g.cols + 63) / 64;
    // a wave takes more groups (v is read and split once) as long as there are 16 waves a CU (8192 rows of
    // 2048 bf16: rank 16 35.5 us, 40 with 8 waves; rank 64 54, 56 with 32)
    g.groups = (int)std::max<int64_t>(1, std::min<int64_t>(8, (int64_t)tiles * groups / 4096));
    const int col_wgs = (groups + 4 * g.groups - 1) / (4 * g.groups);
    const dim3 grid((tiles + 7) / 8 * 8 * col_wgs), block(kThreads);
    constexpr int kBlock = 4 * Mma<TX>::kChunk;
    if constexpr (MT == 1 || kBlock > 16)
        if (g.wr <= kBlock) return launch(k_expand<TX, TW, 1, MT>, grid, block, stream, nullptr, nullptr, g, col_wgs);
    if constexpr (kBlock < 32)
        if (g.wr > 2 * kBlock) return launch(k_expand<TX, TW, 4, MT>, grid, block, stream, nullptr, nullptr, g, col_wgs);
    return launch(k_expand<TX, TW, 2, MT>, grid, block, stream, nullptr, nullptr, g, col_wgs);
}

// Both products of a call.  A block of 32 rows instead of 16 halves the reads of the adapters' matrices
// from L2, and the number of workgroups: worth it from rank 17 on and this many rows x ranks, four times as
// many where the first product's matrices are tiled.  2048 columns, rank 32: 4096 rows 22.9 us against 24.9,
// 1024 rows 17.7 against 14.9; rank 64: 4096 rows 31.6 against 38.3.  Backward: rank 32, 16384 rows 136
// against 141, 4096 rows 56.2 against 54.8. 
constexpr int64_t kTallWork = 1 << 17;
template <typename TX, typename TW, bool TILED>
hipError_t products(const ShrinkArgs &sa, int jobs, const ExpandArgs &ea, hipStream_t stream) {
    const bool tall = sa.r > 16 && (int64_t)sa.r * sa.T >= kTallWork * (TILED ? 4 : 1);
    const hipError_t err = tall ? shrink<TX, TW, 2, TILED>(sa, jobs, stream) : shrink<TX, TW, 1, TILED>(sa, jobs, stream);
    if (err != hipSuccess) return err;
    return tall ? expand<TX, TW, 2>(ea, stream) : expand<TX, TW, 1>(ea, stream);
}

template <typename TX, typename TW, int THREADS>
hipError_t row_calls(const AdapterArgs &g, hipStream_t stream) {
    const int groups = (g.outer + THREADS - 1) / THREADS;
    const int slices = std::max(1, std::min(groups, kRowTarget * kThreads / THREADS / g.T));
    const int cols = (groups + slices - 1) / slices * THREADS;
    return launch(k_adapters_row<TX, TW, THREADS>, dim3(g.T, (g.outer + cols - 1) / cols), dim3(THREADS), stream, nullptr, nullptr,
                  g, cols);
}

template <typename TX, typename TW>
hipError_t forward(const AdapterArgs &g, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    constexpr size_t z = sizeof(TX);
    char *ws = static_cast<char *>(workspace);
    auto fits = [&](const ForwardSpace &s) {
        return (s.copy_x ? piecewise(ws, s.ip, s.ip, z) : piecewise(g.x, g.ld_x, g.inner, z)) &&
               (s.copy_out ? piecewise(ws, s.op, s.op, z)
                           : piecewise(g.out, g.ld_out, g.outer, z) && (!g.base || piecewise(g.base, g.ld_base, g.outer, z)));
    };
    ForwardSpace s = forward_space(g.T, g.inner, g.outer, g.n, g.r, false);
    if (s.bytes && !fits(s)) {
        const ForwardSpace c = forward_space(g.T, g.inner, g.outer, g.n, g.r, true);
        if (c.bytes <= workspace_bytes) s = c;
    }
    const bool pad_a = s.ip != g.inner, pad_b = s.rp != g.r;
    const bool worth = !(s.copy_x || s.copy_out) || g.T > kCopyCalls || work_of(g.T, g.inner, g.outer, g.r) >= kCopyWork;
    if (s.bytes && worth && fits(s) && fits_buffer(s.ip, s.op, s.rp, sizeof(TW)) &&
        (pad_a || reinterpret_cast<uintptr_t>(g.a) % 16 == 0) && (pad_b || reinterpret_cast<uintptr_t>(g.b) % 16 == 0) &&
        (int64_t)g.n * std::max(g.outer, g.r) < (1 << 30)) {
        float *v = reinterpret_cast<float *>(ws + s.v);
        Reshape m{};
        if (s.copy_x) m.add({g.x, ws + s.x, g.ld_x, s.ip, g.inner, s.ip, g.T, false});
        if (s.copy_out) m.add({g.base, ws + s.out, g.ld_base, s.op, g.outer, s.op, g.T, false});
        if (pad_a) m.add({g.a, ws + s.a, g.inner, s.ip, g.inner, s.ip, g.n * g.r, true});
        if (pad_b) m.add({g.b, ws + s.b, g.r, s.rp, g.r, s.rp, g.n * g.outer, true});
        hipError_t err = reshape<TX, TW>(m, stream);
        if (err != hipSuccess) return err;
        const void *x = s.copy_x ? ws + s.x : g.x, *a = pad_a ? ws + s.a : g.a, *b = pad_b ? ws + s.b : g.b;
        void *out = s.copy_out ? ws + s.out : g.out;
        const void *base = s.copy_out ? out : g.base;
        const int64_t ld_x = s.copy_x ? s.ip : g.ld_x;
        const int64_t ld_out = s.copy_out ? s.op : g.ld_out, ld_base = s.copy_out ? s.op : g.ld_base;
        const ShrinkArgs sa{{{x, a, ld_x, (int64_t)g.r * s.ip, v, s.ip}}, g.adapter, g.scale, g.T, g.n, g.r, s.rp};
        const ExpandArgs ea{base, b, out, v, g.adapter, ld_base, ld_out, g.T, s.op, g.n, g.outer, s.rp, s.rp, 0};
        err = products<TX, TW, false>(sa, 1, ea, stream);
        if (err != hipSuccess || !s.copy_out) return err;
        Reshape back{};
        back.add({out, g.out, s.op, g.ld_out, g.outer, g.outer, g.T, false});
        return reshape<TX, TW>(back, stream);
    }
    // threads: four ranks a wave at once (one row of 2048 x 2048, rank 64: 9.9 us with 1024, 13.7 with 256; 64 rows
    // with rank 32: 6.7 us with 512, 9.4 with 256); fp32 adapters' registers allow 512
    // (a launch's threads stay under 2^32)
    if (g.r <= 16 || g.T >= 1 << 22) return row_calls<TX, TW, 256>(g, stream);
    if (g.r <= 32 || sizeof(TW) == 4) return row_calls<TX, TW, 512>(g, stream);
    if constexpr (sizeof(TW) == 2) return row_calls<TX, TW, 1024>(g, stream);
}

template <typename TX, typename TW>
hipError_t backward(int dtype, const AdapterBackArgs &g, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    constexpr size_t z = sizeof(TX);
    char *ws = static_cast<char *>(workspace);
    auto fits = [&](const BackSpace &s) {
        return s.padded ? piecewise(ws, s.ip, s.ip, z) && piecewise(ws, s.op, s.op, z)
                        : piecewise(g.x, g.ld_x, g.inner, z) && piecewise(g.d_out, g.ld_d_out, g.outer, z) &&
                              piecewise(g.d_x, g.ld_d_x, g.inner, z) &&
                              (!g.dx_base || piecewise(g.dx_base, g.ld_dx_base, g.inner, z));
    };
    BackSpace s = back_space(g.T, g.inner, g.outer, g.n, g.r, false);
    if (!fits(s)) {
        const BackSpace c = back_space(g.T, g.inner, g.outer, g.n, g.r, true);
        if (c.bytes <= workspace_bytes) s = c;
    }
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + s.offsets), *order = reinterpret_cast<int32_t *>(ws + s.order);
    float *v = reinterpret_cast<float *>(ws + s.v), *u = reinterpret_cast<float *>(ws + s.u);
    const bool blocks = g.T > 0 && fits(s) && fits_buffer(s.ip, s.op, (s.rp + 15) / 16 * 16, sizeof(TW));
    const bool small = blocks && g.T <= kSmallBack;
    DispatchArgs d{};
    d.ids = g.adapter;
    d.offsets = offsets;
    d.src = order;
    d.T = g.T;
    d.H = 1;
    d.k = 1;
    d.E = g.n;
    // a call of few rows needs no order, and most others make it in the launch of the layout
    const bool order_here = blocks && !small && g.T <= kOrderRows && g.n <= kOrderedHere;
    hipError_t err = hipSuccess;
    if (!small && !order_here) err = launch_dispatch(dtype, d, ws + s.sort, stream);
    if (err != hipSuccess) return err;
    if (!blocks) {
        if (g.T > 0) err = launch(k_back_row<TX, TW>, dim3(g.T), dim3(kThreads), stream, nullptr, nullptr, g, v, u);
        if (err != hipSuccess) return err;
        const dim3 grid((g.inner + 63) / 64 + (g.outer + 63) / 64, (g.r + 15) / 16, g.n);
        return launch(k_back_weights<TX>, grid, dim3(kThreads), stream, nullptr, nullptr, g,
                      static_cast<const int32_t *>(offsets), static_cast<const int32_t *>(order),
                      static_cast<const float *>(v), static_cast<const float *>(u));
    }

    constexpr int C = Mma<TX>::kChunk;
    TW *at = reinterpret_cast<TW *>(ws + s.at), *aw = reinterpret_cast<TW *>(ws + s.aw), *bw = reinterpret_cast<TW *>(ws + s.bw);
    const int order_wgs = order_here ? (g.T + kWgPicks - 1) / kWgPicks : 0;
    err = launch(k_back_layout<TW, C>, dim3(order_wgs + (s.ip + 63) / 64 + (g.outer + 63) / 64, (g.r + 31) / 32, g.n),
                 dim3(kThreads), stream, nullptr, nullptr, static_cast<const TW *>(g.a), static_cast<const TW *>(g.b), at, aw, bw,
                 g.inner, g.outer, s.ip, g.r, s.rp, d, order_wgs);
    if (err != hipSuccess) return err;
    // what the block kernels read and write: the caller's matrices, or padded copies
    const void *x = g.x, *d_out = g.d_out, *dx_base = g.dx_base;
    void *d_x = g.d_x;
    int64_t ld_x = g.ld_x, ld_d_out = g.ld_d_out, ld_dx_base = g.ld_dx_base, ld_d_x = g.ld_d_x;
    if (s.padded) {
        Reshape m{};
        m.add({g.x, ws + s.x, g.ld_x, s.ip, g.inner, s.ip, g.T, false});
        m.add({g.d_out, ws + s.d_out, g.ld_d_out, s.op, g.outer, s.op, g.T, false});
        m.add({g.dx_base, ws + s.d_x, g.ld_dx_base, s.ip, g.inner, s.ip, g.T, false});
        err = reshape<TX, TW>(m, stream);
        if (err != hipSuccess) return err;
        x = ws + s.x;
        d_out = ws + s.d_out;
        dx_base = d_x = ws + s.d_x;
        ld_x = ld_dx_base = ld_d_x = s.ip;
        ld_d_out = s.op;
    }
    const ShrinkArgs sa{{{x, aw, ld_x, (int64_t)tiled_size(g.r, g.inner, C), v, s.ip},
                         {d_out, bw, ld_d_out, (int64_t)tiled_size(g.r, g.outer, C), u, s.op}},
                        g.adapter, g.scale, g.T, g.n, g.r, s.rp};
    const ExpandArgs ea{dx_base, at, d_x, u, g.adapter, ld_dx_base, ld_d_x, g.T, s.ip, g.n, s.ip, s.rp, s.rp, 0};
    err = products<TX, TW, true>(sa, 2, ea, stream);
    if (err != hipSuccess) return err;
    if (s.padded) {
        Reshape m{};
        m.add({d_x, g.d_x, s.ip, g.ld_d_x, g.inner, g.inner, g.T, false});
        err = reshape<TX, TW>(m, stream);
        if (err != hipSuccess) return err;
    }
    const BackWeights w{g.adapter, x, d_out, ld_x, ld_d_out, offsets, order, v, u, reinterpret_cast<float *>(ws + s.partial),
                        g.d_a, g.d_b, g.T, g.inner, g.outer, s.ip, s.op, g.n, g.r, s.rp, s.piece_rows};
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

size_t adapters_forward_workspace(int T, int inner, int outer, int n, int r, bool copies) {
    return forward_space(T, inner, outer, n, r, copies).bytes;
}
size_t adapters_workspace(int T, int inner, int outer, int n, int r, bool copies) {
    return back_space(T, inner, outer, n, r, copies).bytes;
}

hipError_t launch_adapters(int dtype, int wtype, const AdapterArgs &g, void *workspace, size_t bytes, hipStream_t stream) {
    if (g.T == 0) return hipSuccess;
    if (dtype == T_F16) return forward<f16, f16>(g, workspace, bytes, stream);
    if (dtype == T_BF16) return forward<bf16, bf16>(g, workspace, bytes, stream);
    if (wtype == T_F16) return forward<float, f16>(g, workspace, bytes, stream);
    if (wtype == T_BF16) return forward<float, bf16>(g, workspace, bytes, stream);
    return forward<float, float>(g, workspace, bytes, stream);
}

hipError_t launch_adapters_back(int dtype, int wtype, const AdapterBackArgs &g, void *workspace, size_t bytes,
                                hipStream_t stream) {
    if (dtype == T_F16) return backward<f16, f16>(dtype, g, workspace, bytes, stream);
    if (dtype == T_BF16) return backward<bf16, bf16>(dtype, g, workspace, bytes, stream);
    if (wtype == T_F16) return backward<float, f16>(dtype, g, workspace, bytes, stream);
    if (wtype == T_BF16) return backward<float, bf16>(dtype, g, workspace, bytes, stream);
    return backward<float, float>(dtype, g, workspace, bytes, stream);
}

}  // namespace moe
