// Products over the rows of experts (include/moe_experts.h) on the matrix cores of gfx950.
//
// Every product is C[n][m] = sum over k of A[m][k] B[n][k] with m along the columns of the result:
//   hidden, product   m: rows of W (k along them), n: rows of x (k along them)
//   d_x, d_h          m: columns of W (k: its rows), n: rows of d_out (k along them)
//   d_w               m: columns of x (k: its rows), n: columns of d_out (k: its rows)
// so one kernel body serves all, with an operand either "along k" (KC) or "across k" (KR, read from LDS
// by the transposing 8-byte reads of gfx950).  The accumulators hold 4 columns next to each other a lane.
#include <algorithm>

#include "expert_kernels.hpp"
#include "pieces8.hpp"
#include "segments.hpp"

namespace moe {
namespace {

typedef float float16v __attribute__((ext_vector_type(16)));
typedef f16 half8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) short4v lds_short4;

enum Kind { KC, KR, KR_CODES };
enum Epi { E_HIDDEN, E_PLAIN, E_HIDDEN_BACK, E_GRAD };

constexpr int BM = 256, BN = 256;         // tile of a workgroup: columns and rows of the result
constexpr int kThreads = 512;             // 8 waves, 2 along m and 4 along n
constexpr int FM = 4, FN = 2;             // 32 x 32 pieces of a wave: 128 columns, 64 rows
constexpr int kPieces = 2048;             // 16-byte pieces of one operand's step (256 x 128 bytes)
constexpr int kLoads = kPieces / kThreads;
constexpr int kRsrcWord3 = 0x00020000;    // buffer resource flags of the gfx9 family (raw, untyped)
constexpr int kOut = (int)0x80000000;     // a buffer offset past every range: the load gives zeros
constexpr int64_t kReach = 0x7FFFFFF0;    // bytes that buffer offsets reach

template <typename T>
constexpr int KE = 8 * kVec<T>;           // reduction elements of a step

__device__ inline int swz(int line) { return (line & 7) ^ ((line >> 3) & 1); }

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(const void *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)kReach, kRsrcWord3);
}
// 16 bytes per lane straight into LDS: lane l's bytes land at lds + 16 l
__device__ inline void dma16(__amdgpu_buffer_rsrc_t r, uint4 *lds, int voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, voff, 0, 0, 0);
}
__device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename T>
__device__ inline float16v mma(float16v c, uint4 a, uint4 b) {
    if constexpr (std::is_same_v<T, f16>) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
    } else if constexpr (std::is_same_v<T, bf16>) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else {
        const float4 x = __builtin_bit_cast(float4, a), y = __builtin_bit_cast(float4, b);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(x.x, y.x, c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(x.y, y.y, c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(x.z, y.z, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x2f32(x.w, y.w, c, 0, 0, 0);
    }
}

// Where the lines (KC) or columns (KR) of an operand's 256 are.
struct Source {
    const void *p;        // element (line 0, k 0)
    int64_t ld;           // elements from one row in memory to the next
    int lines;            // that there are (of the first 128 and, of a split operand, of the second 128 too)
    int64_t split;        // > 0: lines 128 .. 255 are `split` elements on (hidden's up rows)
    int K;                // length of the reduction
    const uint8_t *s;     // KR_CODES
    int64_t ld_s;
};

// One operand's steps from memory to LDS: 256 lines x KE, 2048 pieces, piece `slot` by thread slot % 512.
// DIRECT: rows start at multiples of 16 bytes and are whole pieces, offsets fit 31 bits.
template <typename T, int KIND, bool DIRECT>
struct Loader {
    Source s;
    int voff[DIRECT ? kLoads : 1];
    uint4 r[DIRECT ? 1 : kLoads];

    static constexpr int PR = 256 / kVec<T>;   // pieces of a KR row
    __device__ static int line(int slot) { return KIND == KC ? slot >> 3 : slot / PR; }
    __device__ static int piece(int slot) {
        if constexpr (KIND == KC) return (slot & 7) ^ swz(slot >> 3);
        if constexpr (sizeof(T) == 4) return slot % PR;
        const int row = slot / PR, phys = slot % PR;
        return ((((phys >> 1) ^ (row & 7)) << 1) | (phys & 1));
    }
    __device__ bool there(int l) const { return (s.split > 0 ? l & 127 : l) < s.lines; }
    __device__ int64_t at(int l) const { return s.split > 0 && l >= 128 ? s.split + (int64_t)(l - 128) * s.ld : l * s.ld; }

    __device__ void begin(const Source &src) {
        s = src;
        if constexpr (DIRECT) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int slot = i * kThreads + threadIdx.x, l = line(slot), pc = piece(slot);
                if constexpr (KIND == KC)
                    voff[i] = there(l) ? (int)(at(l) * sizeof(T)) + pc * 16 : kOut;
                else
                    voff[i] = pc * kVec<T> < s.lines ? (int)(l * s.ld * sizeof(T)) + pc * 16 : kOut;
            }
        }
    }
    // starts the loads of a step; with DIRECT they go to buf
    __device__ void load(int step, uint4 *buf) {
        const int k0 = step * KE<T>;
        if constexpr (DIRECT) {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const T *base = static_cast<const T *>(s.p) + (KIND == KC ? (int64_t)k0 : k0 * s.ld);
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(base);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int slot = i * kThreads + threadIdx.x;
                const int k = k0 + (KIND == KC ? piece(slot) * kVec<T> : line(slot));
                dma16(rs, buf + i * kThreads + wave * 64, k < s.K ? voff[i] : kOut);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int slot = i * kThreads + threadIdx.x, l = line(slot), pc = piece(slot) * kVec<T>;
                if constexpr (KIND == KC) {
                    r[i] = load_piece(static_cast<const T *>(s.p) + at(l) + k0 + pc, there(l) ? s.K - k0 - pc : 0);
                } else if constexpr (KIND == KR) {
                    r[i] = load_piece(static_cast<const T *>(s.p) + (k0 + l) * s.ld + pc, k0 + l < s.K ? s.lines - pc : 0);
                } else {
                    const int n = k0 + l < s.K ? s.lines - pc : 0;
                    const int8_t *q = static_cast<const int8_t *>(s.p) + (k0 + l) * s.ld + pc;
                    uint2 c = {0, 0};
                    if (n >= kVec<T>) {
                        __builtin_memcpy(&c, q, kVec<T>);
                    } else {
                        int8_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < kVec<T>; ++j)
                            if (j < n) e[j] = q[j];
                        __builtin_memcpy(&c, e, 8);
                    }
                    r[i] = {c.x, c.y, n > 0 ? s.s[(k0 + l) * s.ld_s + pc / kBlock] : 0u, 0u};
                }
            }
        }
    }
    __device__ void store(uint4 *buf) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                uint4 v = r[i];
                if constexpr (KIND == KR_CODES) {
                    float f[8], g[kVec<T>];
                    decode8<T>({v.x, v.y}, v.z, f);
#pragma unroll
                    for (int j = 0; j < kVec<T>; ++j) g[j] = f[j];
                    v = pack<T>(g);
                }
                buf[i * kThreads + threadIdx.x] = v;
            }
        }
    }
};

// An operand of 32 lines (from `first`, a multiple of 32) and the kk-th eighth.. of a step's pieces:
// 8 (4 in fp32) reduction elements a lane, the upper half of the wave the next ones.
template <typename T, int KIND>
__device__ inline uint4 fragment(const uint4 *buf, int first, int kk) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    if constexpr (KIND == KC) {
        const int l = first + (lane & 31);
        return buf[l * 8 + ((2 * kk + half) ^ swz(lane & 31))];
    } else if constexpr (sizeof(T) == 4) {
        const float *f = reinterpret_cast<const float *>(buf) + (8 * kk + 4 * half) * 256 + first + (lane & 31);
        const float4 v = {f[0], f[256], f[512], f[768]};
        return __builtin_bit_cast(uint4, v);
    } else {
        const int col = first + 16 * ((lane >> 4) & 1) + 4 * (lane & 3), k = 16 * kk + 8 * half + ((lane & 15) >> 2);
        uint2 v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = k + 4 * t;
            const char *p = reinterpret_cast<const char *>(buf) + row * 512 + (((col >> 4) ^ (row & 7)) << 5) + (col & 15) * 2;
            v[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)p));
        }
        return {v[0].x, v[0].y, v[1].x, v[1].y};
    }
}

// The whole reduction of a tile.  One barrier a step: every wave has read the step's buffers, and the next
// step's loads, requested a step ahead, have landed.
template <typename T, int AK, int BK, bool DIRECT_A, bool DIRECT_B>
__device__ inline void reduce(const Source &sa, const Source &sb, const int (&fa)[FM], const int (&fb)[FN], int steps,
                              uint4 *A0, uint4 *A1, uint4 *B0, uint4 *B1, float16v (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    if (steps <= 0) return;
    Loader<T, AK, DIRECT_A> la;
    Loader<T, BK, DIRECT_B> lb;
    la.begin(sa);
    lb.begin(sb);
    la.load(0, A0);
    lb.load(0, B0);
    la.store(A0);
    lb.store(B0);
    wait_loads();
    __syncthreads();
    auto step = [&](int s, uint4 *a, uint4 *b, uint4 *an, uint4 *bn) {
        const bool more = s + 1 < steps;
        if (more) {
            la.load(s + 1, an);
            lb.load(s + 1, bn);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint4 x[FM], y[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) x[i] = fragment<T, AK>(a, fa[i], kk);
#pragma unroll
            for (int j = 0; j < FN; ++j) y[j] = fragment<T, BK>(b, fb[j], kk);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mma<T>(acc[i][j], x[i], y[j]);
        }
        if (more) {
            la.store(an);
            lb.store(bn);
        }
        wait_loads();
        __syncthreads();
    };
    int s = 0;
    for (; s + 2 <= steps; s += 2) {
        step(s, A0, B0, A1, B1);
        step(s + 1, A1, B1, A0, B0);
    }
    if (s < steps) step(s, A0, B0, A1, B1);
}

__device__ inline float sigmoid(float g) { return 1.f / (1.f + expf(-g)); }

// act(g) and its slope
__device__ inline void activation(float g, int act, float &a, float &slope) {
    if (act == MOE_ACT_SILU) {
        const float p = sigmoid(g);
        a = g * p;
        slope = p * (1.f + g * (1.f - p));
    } else {
        const float c = 0.7978845608028654f, t = tanhf(c * (g + 0.044715f * g * g * g));
        a = 0.5f * g * (1.f + t);
        slope = 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * c * (1.f + 0.134145f * g * g);
    }
}
__device__ inline float activate(float g, int act) {
    float a, s;
    activation(g, act, a, s);
    return a;
}

// 8 columns of a row of hidden, and what is kept of it.  Every lane of a block of 32 takes part.
template <typename T>
__device__ inline void put_hidden(const ExpertArgs &g, int row, int col, bool there, const float (&gv)[8],
                                  const float (&uv)[8]) {
    const int n = there ? g.M - col : 0;
    if (g.kept.q) {
        const int nb = (g.M + kBlock - 1) / kBlock;
        int sg, su;
        const uint2 cg = encode8(gv, n, sg), cu = encode8(uv, n, su);
        if (n > 0) {
            int8_t *q = g.kept.q + row * g.kept.ld + col;
            store_codes(q, cg, n);
            store_codes(q + g.M, cu, n);
            if (col % kBlock == 0) {
                uint8_t *s = g.kept.s + row * g.kept.ld_s + col / kBlock;
                s[0] = (uint8_t)sg;
                s[nb] = (uint8_t)su;
            }
        }
    }
    if (n <= 0) return;
    if (g.pre.p) {
        T *p = static_cast<T *>(g.pre.p) + row * g.pre.ld + col;
        store8(p, gv, n);
        store8(p + g.M, uv, n);
    }
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = activate(gv[i], g.act) * uv[i];
    store8(static_cast<T *>(g.out.p) + row * g.out.ld + col, h, n);
}

// 8 columns of a row through the activation's gradient.
template <typename T>
__device__ inline void put_hidden_back(const ExpertArgs &g, int row, int col, const float (&d)[8]) {
    const int n = g.M - col;
    float gv[8], uv[8], dg[8], du[8], h[8];
    if (g.kept_in.q) {
        const int nb = (g.M + kBlock - 1) / kBlock;
        const int8_t *q = g.kept_in.q + row * g.kept_in.ld + col;
        const uint8_t *s = g.kept_in.s + row * g.kept_in.ld_s + col / kBlock;
        decode8<float>(load_codes(q, n), s[0], gv);
        decode8<float>(load_codes(q + g.M, n), s[nb], uv);
    } else {
        const T *p = static_cast<const T *>(g.pre_in.p) + row * g.pre_in.ld + col;
        load8(p, gv, n);
        load8(p + g.M, uv, n);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, slope;
        activation(gv[i], g.act, a, slope);
        dg[i] = d[i] * uv[i] * slope;
        du[i] = d[i] * a;
        h[i] = a * uv[i];
    }
    T *p = static_cast<T *>(g.pre.p) + row * g.pre.ld + col;
    store8(p, dg, n);
    store8(p + g.M, du, n);
    if (g.out.p) store8(static_cast<T *>(g.out.p) + row * g.out.ld + col, h, n);
}

// LDS operations of one wave are done in order; this keeps the compiler from reordering them.
__device__ inline void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's 64 rows x 128 columns through its own 16 KB of LDS, 32 rows at a time: written 4 columns a lane,
// read back 8 next to each other, so that global stores are whole lines.  put(row, piece, f, PAIR's second):
// piece p holds columns 8p .. 8p+7; with PAIR p < 8 comes with piece p + 8.
template <bool PAIR, typename Put>
__device__ inline void spill(uint4 *stage, const float16v (&acc)[FM][FN], Put put) {
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        wave_fence();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                stage[r * 32 + ((i * 8 + q * 2 + half) ^ r)] = __builtin_bit_cast(uint4, v);
            }
        wave_fence();
        auto get = [&](int row, int p, float (&f)[8]) {
            const float4 a = __builtin_bit_cast(float4, stage[row * 32 + ((2 * p) ^ row)]);
            const float4 b = __builtin_bit_cast(float4, stage[row * 32 + ((2 * p + 1) ^ row)]);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        };
        constexpr int PP = PAIR ? 8 : 16;
#pragma unroll 1
        for (int it = 0; it < 32 * PP / 64; ++it) {
            const int x = it * 64 + lane, row = x / PP, p = x % PP;
            float f[8], g[8];
            get(row, p, f);
            if constexpr (PAIR) get(row, p + 8, g);
            put(j * 32 + row, p, f, g);
        }
    }
}

#define MOE_TILES                                                                                   \
    __shared__ __align__(16) uint4 A0[kPieces], A1[kPieces], B0[kPieces], B1[kPieces];              \
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1; \
    uint4 *const stage = (wave < 2 ? A0 : wave < 4 ? A1 : wave < 6 ? B0 : B1) + (wave & 1) * 1024;

// Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles next to each other, so that the rows
// and the weights that they share are in one L2.  Tile `b` of `total`, or -1.
__device__ inline int xcd_tile(int b, int total) {
    const int per = (total + 7) >> 3, i = b >> 3, t = (b & 7) * per + i;
    return i < per && t < total ? t : -1;
}

template <typename T, int AK, int EPI, bool DA, bool DB>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_rows(ExpertArgs g, int tiles_m) {
    MOE_TILES
    Tile t;
    int mt = 0;
    if (!find_tile(g.offsets, g.E, g.R, BN, [&](int total) {
            const int x = xcd_tile(blockIdx.x, total * tiles_m);
            mt = x % tiles_m;
            return x < 0 ? -1 : x / tiles_m;
        }, t))
        return;
    constexpr int COLS = EPI == E_HIDDEN ? BM / 2 : BM;
    const int m0 = mt * COLS;
    Source sa{}, sb{};
    const T *w = static_cast<const T *>(g.w);
    if constexpr (AK == KC) {
        const int64_t rows = EPI == E_HIDDEN ? 2 * (int64_t)g.M : g.M;
        sa.p = w + (t.e * rows + m0) * g.K;
        sa.ld = g.K;
        sa.split = EPI == E_HIDDEN ? (int64_t)g.M * g.K : 0;
    } else {
        sa.p = w + (int64_t)t.e * g.K * g.M + m0;
        sa.ld = g.M;
    }
    sa.lines = min(g.M - m0, COLS);
    sa.K = sb.K = g.K;
    sb.p = static_cast<const T *>(g.x.p) + t.row * g.x.ld;
    sb.ld = g.x.ld;
    sb.lines = min(t.end - t.row, BN);
    int fa[FM], fb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = EPI == E_HIDDEN ? (i >> 1) * 128 + wm * 64 + (i & 1) * 32 : wm * 128 + i * 32;
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = wn * 64 + j * 32;
    float16v acc[FM][FN];
    reduce<T, AK, KC, DA, DB>(sa, sb, fa, fb, (g.K + KE<T> - 1) / KE<T>, A0, A1, B0, B1, acc);
    const int row0 = t.row + wn * 64;
    if constexpr (EPI == E_HIDDEN) {
        spill<true>(stage, acc, [&](int r, int p, const float(&gv)[8], const float(&uv)[8]) {
            const int col = m0 + wm * 64 + 8 * p;
            put_hidden<T>(g, row0 + r, col, row0 + r < t.end, gv, uv);
        });
    } else {
        spill<false>(stage, acc, [&](int r, int p, const float(&f)[8], const float(&)[8]) {
            const int row = row0 + r, col = m0 + wm * 128 + 8 * p;
            if (row >= t.end || col >= g.M) return;
            if constexpr (EPI == E_PLAIN)
                store8(static_cast<T *>(g.out.p) + row * g.out.ld + col, f, g.M - col);
            else
                put_hidden_back<T>(g, row, col, f);
        });
    }
}

// d_w of one expert's tile and one of `splits` runs of its rows.
template <typename T, int AK, bool DA, bool DB>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_grad(ExpertGradArgs g, int tiles_m,
                                                                                        int tiles_n, int splits, float *parts) {
    MOE_TILES
    const int x = xcd_tile(blockIdx.x, g.E * tiles_m * tiles_n * splits);
    if (x < 0) return;
    const int mt = x % tiles_m, nt = x / tiles_m % tiles_n, sp = x / (tiles_m * tiles_n) % splits, e = x / (tiles_m * tiles_n * splits);
    int begin, end;
    rows_of(g.offsets, e, g.R, begin, end);
    if (splits > 1) {   // whole steps a run
        const int steps = (end - begin + KE<T> - 1) / KE<T>, per = (steps + splits - 1) / splits * KE<T>;
        begin = min(begin + sp * per, end);
        end = min(begin + per, end);
    }
    const int m0 = mt * BM, n0 = nt * BN;
    Source sa{}, sb{};
    if constexpr (AK == KR_CODES) {
        sa.p = g.codes.q + begin * g.codes.ld + m0;
        sa.ld = g.codes.ld;
        sa.s = g.codes.s + begin * g.codes.ld_s + m0 / kBlock;
        sa.ld_s = g.codes.ld_s;
    } else {
        sa.p = static_cast<const T *>(g.x.p) + begin * g.x.ld + m0;
        sa.ld = g.x.ld;
    }
    sa.lines = min(g.M - m0, BM);
    sb.p = static_cast<const T *>(g.d_out.p) + begin * g.d_out.ld + n0;
    sb.ld = g.d_out.ld;
    sb.lines = min(g.N - n0, BN);
    sa.K = sb.K = end - begin;
    int fa[FM], fb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = wm * 128 + i * 32;
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = wn * 64 + j * 32;
    float16v acc[FM][FN];
    reduce<T, AK, KR, DA, DB>(sa, sb, fa, fb, (end - begin + KE<T> - 1) / KE<T>, A0, A1, B0, B1, acc);
    float *out = (splits > 1 ? parts + (int64_t)sp * g.E * g.N * g.M : g.d_w) + (int64_t)e * g.N * g.M;
    spill<false>(stage, acc, [&](int r, int p, const float(&f)[8], const float(&)[8]) {
        const int row = n0 + wn * 64 + r, col = m0 + wm * 128 + 8 * p;
        if (row < g.N && col < g.M) store8(out + (int64_t)row * g.M + col, f, g.M - col);
    });
}

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

// ------------------------------------------------------------------------------------------- launches

bool aligned(const void *p, int64_t ld, size_t size) { return !(((uintptr_t)p | (uintptr_t)(ld * size)) & 15); }

// Whether 256 rows of `ld` elements go straight into LDS.
bool direct(const void *p, int64_t ld, int64_t along, size_t size) {
    return aligned(p, ld, size) && along * (int64_t)size % 16 == 0 && 256 * ld * (int64_t)size < kReach;
}

int row_tiles(int R, int E) { return R / BN + std::min(E, R); }

template <typename T, int AK, int EPI>
hipError_t rows_launch(const ExpertArgs &a, hipStream_t stream) {
    if (a.R == 0) return hipSuccess;
    const int cols = EPI == E_HIDDEN ? BM / 2 : BM, tiles_m = (a.M + cols - 1) / cols;
    const int64_t n = (int64_t)row_tiles(a.R, a.E) * tiles_m;
    const dim3 grid((unsigned)((n + 7) / 8 * 8)), block(kThreads);
    const int64_t ld = AK == KC ? a.K : a.M;
    bool da = direct(a.w, ld, ld, sizeof(T)), db = direct(a.x.p, a.x.ld, a.K, sizeof(T));
    if (EPI == E_HIDDEN) da = da && ((int64_t)a.M + 256) * a.K * (int64_t)sizeof(T) < kReach;
    if (da && db) return launch(k_rows<T, AK, EPI, true, true>, grid, block, stream, nullptr, nullptr, a, tiles_m);
    return launch(k_rows<T, AK, EPI, false, false>, grid, block, stream, nullptr, nullptr, a, tiles_m);
}

template <int AK, int EPI>
hipError_t rows_any(int dtype, const ExpertArgs &a, hipStream_t stream) {
    if (dtype == T_F32) return rows_launch<float, AK, EPI>(a, stream);
    if (dtype == T_F16) return rows_launch<f16, AK, EPI>(a, stream);
    return rows_launch<bf16, AK, EPI>(a, stream);
}

int grad_splits(int R, int M, int N, int E) {
    const int64_t tiles = (int64_t)((M + BM - 1) / BM) * ((N + BN - 1) / BN) * E;
    return (int)std::max<int64_t>(1, std::min<int64_t>({512 / std::max<int64_t>(tiles, 1), R / 512, 16}));
}

template <typename T>
hipError_t grad_launch(const ExpertGradArgs &a, void *workspace, hipStream_t stream) {
    const int tiles_m = (a.M + BM - 1) / BM, tiles_n = (a.N + BN - 1) / BN, splits = grad_splits(a.R, a.M, a.N, a.E);
    const int64_t n = (int64_t)tiles_m * tiles_n * a.E * splits, size = (int64_t)a.E * a.M * a.N;
    const dim3 grid((unsigned)((n + 7) / 8 * 8)), block(kThreads);
    float *parts = static_cast<float *>(workspace);
    const bool db = direct(a.d_out.p, a.d_out.ld, a.N, sizeof(T));
    hipError_t e;
    if (!a.x.p) {
        e = db ? launch(k_grad<T, KR_CODES, false, true>, grid, block, stream, nullptr, nullptr, a, tiles_m, tiles_n, splits, parts)
               : launch(k_grad<T, KR_CODES, false, false>, grid, block, stream, nullptr, nullptr, a, tiles_m, tiles_n, splits, parts);
    } else if (db && direct(a.x.p, a.x.ld, a.M, sizeof(T))) {
        e = launch(k_grad<T, KR, true, true>, grid, block, stream, nullptr, nullptr, a, tiles_m, tiles_n, splits, parts);
    } else {
        e = launch(k_grad<T, KR, false, false>, grid, block, stream, nullptr, nullptr, a, tiles_m, tiles_n, splits, parts);
    }
    if (e != hipSuccess || splits == 1) return e;
    return launch(k_grad_join, dim3((unsigned)((size + 1023) / 1024)), dim3(256), stream, nullptr, nullptr,
                  static_cast<const float *>(parts), a.d_w, size, splits);
}

}  // namespace

hipError_t launch_hidden(int dtype, const ExpertArgs &a, hipStream_t stream) { return rows_any<KC, E_HIDDEN>(dtype, a, stream); }
hipError_t launch_product(int dtype, const ExpertArgs &a, hipStream_t stream) { return rows_any<KC, E_PLAIN>(dtype, a, stream); }
hipError_t launch_hidden_back(int dtype, const ExpertArgs &a, hipStream_t stream) {
    return rows_any<KR, E_HIDDEN_BACK>(dtype, a, stream);
}
hipError_t launch_product_back(int dtype, const ExpertArgs &a, hipStream_t stream) { return rows_any<KR, E_PLAIN>(dtype, a, stream); }

size_t expert_grad_workspace(int R, int M, int N, int E) {
    const int s = grad_splits(R, M, N, E);
    return s == 1 ? 0 : (size_t)s * E * M * N * sizeof(float);
}

hipError_t launch_expert_grad(int dtype, const ExpertGradArgs &a, void *workspace, hipStream_t stream) {
    if (dtype == T_F32) return grad_launch<float>(a, workspace, stream);
    if (dtype == T_F16) return grad_launch<f16>(a, workspace, stream);
    return grad_launch<bf16>(a, workspace, stream);
}

}  // namespace moe
