// Products over the rows of experts (include/moe_experts.h) on the matrix cores of gfx950.
//
// Every product is C[n][m] = sum over k of A[m][k] B[n][k] with m along the columns of the result:
//   hidden, product   m: rows of W (k along them), n: rows of x (k along them)
//   d_x, d_h          m: columns of W (k: its rows), n: rows of d_out (k along them)
//   d_w               m: columns of x (k: its rows), n: columns of d_out (k: its rows)
// so one kernel body serves all, with an operand either "along k" (KC) or "across k" (KR, read from LDS
// by the transposing 8-byte reads of gfx950).  The accumulators hold 4 columns next to each other a lane.
#pragma once

#include <algorithm>
#include <utility>

#include "expert_kernels.hpp"
#include "expert_shapes.hpp"
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
// How an operand comes from memory.  DIRECT: rows start at multiples of 16 bytes and are whole pieces, offsets fit 31
// bits; the loads write LDS (codes: registers, by as many instructions whatever is asked for).  Otherwise through
// registers, STAGES steps of them: PIECES, 16 bytes at any element; ELEMENTS, where a row is shorter than a piece.
enum Way { DIRECT, PIECES, ELEMENTS };
enum Epi { E_HIDDEN, E_PLAIN, E_HIDDEN_BACK };

constexpr int kRsrcWord3 = 0x00020000;    // buffer resource flags of the gfx9 family (raw, untyped)
constexpr int kOut = (int)0x80000000;     // a buffer offset past every range: the load gives zeros
constexpr int64_t kReach = 0x7FFFFFF0;    // bytes that buffer offsets reach

template <typename T>
constexpr int KE = 4 * kVec<T>;           // reduction elements of a step

// Swizzle of a line's 4 pieces: 16 lines read at one piece meet each 16-byte bank group once.
__device__ inline int swz(int line) { return (line >> 2) & 3; }

typedef int int4v __attribute__((ext_vector_type(4)));

__device__ inline int4v make_rsrc(const void *base) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return {__builtin_amdgcn_readfirstlane((int)p), __builtin_amdgcn_readfirstlane((int)(p >> 32) & 0xFFFF), (int)kReach,
            kRsrcWord3};
}
// 16 bytes per lane straight into LDS: lane l's bytes land at lds + 16 l (lds uniform).  In assembly, since the
// compiler waits for all of its own loads into LDS before it reads any of LDS (it tells 8 of them apart, a tile has
// 32), so that none could be a step ahead; wait_and_meet waits for these.  No register is written.  The s_nop:
// a vector instruction may just have written a scalar register that the load reads (5 wait states), and M0 wants one.
__device__ inline void dma16(int4v r, uint4 *lds, int voff) {
    const int at = __builtin_amdgcn_readfirstlane((int)reinterpret_cast<uintptr_t>((lds_void *)lds));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(voff), "s"(r)
                 : "memory", "m0");
}
// All but the last N of this wave's loads and stores have landed (N = 63: nothing is asked of them), and its LDS
// operations are done; then every wave's are.
template <int N>
__device__ inline void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

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

// One operand's steps from memory to LDS: DIM lines x KE; the piece at `slot` by thread slot % THREADS.
template <typename T, int KIND, int DIM, typename C, int WAY>
struct Loader {
    static constexpr int LOADS = DIM * 4 / C::THREADS, GROUPS = DIM / 16;   // GROUPS: of 16 columns (KR)
    static constexpr bool TO_LDS = WAY == DIRECT && KIND != KR_CODES;
    Source s;
    int voff[WAY == DIRECT ? LOADS : 1], soff[KIND == KR_CODES && WAY == DIRECT ? LOADS : 1];
    uint4 r[TO_LDS ? 1 : C::STAGES][TO_LDS ? 1 : LOADS];

    // The line (KC) or row (KR) and the piece along it that LDS holds at `slot`.  KC: a line's 4 pieces, swizzled.  KR,
    // 16 bits: 4 rows x 16 columns next to each other, as the transposing reads take them; 32 bits: row by row.
    __device__ static int line(int slot) {
        return KIND == KC ? slot >> 2 : sizeof(T) == 4 ? slot / (DIM / 4) : slot / (8 * GROUPS) * 4 + ((slot >> 1) & 3);
    }
    __device__ static int piece(int slot) {
        return KIND == KC ? (slot & 3) ^ swz(slot >> 2) : sizeof(T) == 4 ? slot % (DIM / 4) : (slot >> 3) % GROUPS * 2 + (slot & 1);
    }
    __device__ bool there(int l) const { return (s.split > 0 ? l % (DIM / 2) : l) < s.lines; }
    __device__ int64_t at(int l) const {
        return s.split > 0 && l >= DIM / 2 ? s.split + (int64_t)(l - DIM / 2) * s.ld : l * s.ld;
    }

    __device__ void begin(const Source &src) {
        s = src;
        if constexpr (WAY == DIRECT) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int slot = i * C::THREADS + threadIdx.x, l = line(slot), pc = piece(slot);
                if constexpr (KIND == KC) {
                    voff[i] = there(l) ? (int)(at(l) * sizeof(T)) + pc * 16 : kOut;
                } else if constexpr (KIND == KR) {
                    voff[i] = pc * kVec<T> < s.lines ? (int)(l * s.ld * sizeof(T)) + pc * 16 : kOut;
                } else {
                    const bool in = pc * kVec<T> < s.lines;
                    voff[i] = in ? (int)(l * s.ld) + pc * kVec<T> : kOut;
                    soff[i] = in ? (int)(l * s.ld_s) + pc * kVec<T> / kBlock : kOut;
                }
            }
        }
    }
    // the i-th load of a step straight to LDS
    __device__ void direct(int step, uint4 *buf, int i) {
        if constexpr (TO_LDS) {
            const int k0 = step * KE<T>, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const T *base = static_cast<const T *>(s.p) + (KIND == KC ? (int64_t)k0 : k0 * s.ld);
            const int slot = i * C::THREADS + threadIdx.x;
            const int k = k0 + (KIND == KC ? piece(slot) * kVec<T> : line(slot));
            dma16(make_rsrc(base), buf + i * C::THREADS + wave * 64, k < s.K ? voff[i] : kOut);
        }
    }
    // all of a step's loads to registers
    __device__ void load(int step, int stage) {
        if constexpr (TO_LDS) return;
        const int k0 = step * KE<T>;
        if constexpr (WAY == DIRECT && KIND == KR_CODES) {
            const __amdgpu_buffer_rsrc_t q = codes_rsrc(static_cast<const int8_t *>(s.p) + k0 * s.ld), c = codes_rsrc(s.s + k0 * s.ld_s);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const bool in = k0 + line(i * C::THREADS + threadIdx.x) < s.K;
                uint2 v = {0, 0};
                if constexpr (sizeof(T) == 4) v.x = __builtin_amdgcn_raw_buffer_load_b32(q, in ? voff[i] : kOut, 0, 0);
                else v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(q, in ? voff[i] : kOut, 0, 0));
                r[stage][i] = {v.x, v.y, (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(c, in ? soff[i] : kOut, 0, 0), 0u};
            }
        } else {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int slot = i * C::THREADS + threadIdx.x, l = line(slot), pc = piece(slot) * kVec<T>, n = left(k0, l, pc);
                const int64_t to = KIND == KC ? at(l) + k0 + pc : (k0 + l) * s.ld + pc;
                if constexpr (WAY == PIECES) {
                    // no branches, so that loads of several steps are on their way: a piece past the end of its row is read
                    // as the row's last one, and shifted in store; where there is nothing, the first one of all
                    const int64_t from = n > 0 ? to - max(kVec<T> - n, 0) : KIND == KC ? 0 : min(s.lines - kVec<T>, 0);
                    if constexpr (KIND == KR_CODES) {
                        uint2 q = {0, 0};
                        __builtin_memcpy(&q, static_cast<const int8_t *>(s.p) + from, kVec<T>);
                        r[stage][i] = {q.x, q.y, s.s[n > 0 ? (k0 + l) * s.ld_s + pc / kBlock : 0], 0u};
                    } else {
                        __builtin_memcpy(&r[stage][i], static_cast<const T *>(s.p) + from, 16);
                    }
                } else if constexpr (KIND == KR_CODES) {
                    const uint2 c = load_codes(static_cast<const int8_t *>(s.p) + to, min(n, kVec<T>));
                    r[stage][i] = {c.x, c.y, n > 0 ? s.s[(k0 + l) * s.ld_s + pc / kBlock] : 0u, 0u};
                } else {
                    r[stage][i] = load_piece(static_cast<const T *>(s.p) + to, n);
                }
            }
        }
    }
    // elements from a piece on that there are
    __device__ int left(int k0, int l, int pc) const {
        if constexpr (KIND == KC) return there(l) ? s.K - k0 - pc : 0;
        return k0 + l < s.K ? s.lines - pc : 0;
    }
    // v without its lowest bits
    __device__ static uint4 shifted(uint4 v, int bits) {
        uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
        if (bits >= 64) lo = hi, hi = 0, bits -= 64;
        if (bits) lo = lo >> bits | hi << (64 - bits), hi >>= bits;
        return {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    __device__ static __amdgpu_buffer_rsrc_t codes_rsrc(const void *p) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)kReach, kRsrcWord3);
    }
    // Takes every register as read, so that no load is left out where a tile ends: the waits count them.
    __device__ void use() const {
        if constexpr (WAY == DIRECT && KIND == KR_CODES) {
#pragma unroll
            for (int k = 0; k < C::STAGES; ++k)
#pragma unroll
                for (int i = 0; i < LOADS; ++i) asm volatile("" ::"v"(r[k][i].x), "v"(r[k][i].y), "v"(r[k][i].z));
        }
    }
    // and from there to LDS
    __device__ void store(int step, int stage, uint4 *buf) {
        if constexpr (TO_LDS) return;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            uint4 v = r[stage][i];
            if constexpr (WAY == PIECES) {
                const int slot = i * C::THREADS + threadIdx.x, n = left(step * KE<T>, line(slot), piece(slot) * kVec<T>);
                if (n < kVec<T>) {
                    const uint32_t scale = v.z;
                    if (KIND == KR_CODES) v.z = 0;
                    v = n > 0 ? shifted(v, (kVec<T> - n) * (KIND == KR_CODES ? 8 : 8 * (int)sizeof(T))) : uint4{0, 0, 0, 0};
                    if (KIND == KR_CODES) v.z = n > 0 ? scale : 0;
                }
            }
            if constexpr (KIND == KR_CODES) {
                float f[8], g[kVec<T>];
                decode8<T>({v.x, v.y}, v.z, f);
#pragma unroll
                for (int j = 0; j < kVec<T>; ++j) g[j] = f[j];
                v = pack<T>(g);
            }
            buf[i * C::THREADS + threadIdx.x] = v;
        }
    }
};

// Where a lane reads an operand's pieces of 32 lines, in bytes: the kk-th pair of a step's 4 pieces, the upper
// half of the wave the pair's second.
template <typename T, int KIND, int DIM>
struct Reader {
    int at[KIND == KC ? 2 : 1];
    __device__ explicit Reader(int first) {   // first: the wave's first line, a multiple of 32
        const int lane = threadIdx.x & 63, half = lane >> 5;
        if constexpr (KIND == KC) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) at[kk] = ((first + (lane & 31)) * 4 + ((2 * kk + half) ^ swz(lane & 31))) * 16;
        } else if constexpr (sizeof(T) == 4) {
            at[0] = (4 * half * DIM + first + (lane & 31)) * 4;
        } else {
            at[0] = 2 * half * (DIM * 8) + (first >> 4) * 128 + ((lane >> 4) & 1) * 128 + (lane & 15) * 8;
        }
    }
    // lines `more` (a multiple of 32) on
    __device__ uint4 get(const uint4 *buf, int kk, int more) const {
        const char *p = reinterpret_cast<const char *>(buf);
        if constexpr (KIND == KC) {
            return *reinterpret_cast<const uint4 *>(p + at[kk] + more * 64);
        } else if constexpr (sizeof(T) == 4) {
            const float *f = reinterpret_cast<const float *>(p + at[0]) + 8 * kk * DIM + more;
            const float4 v = {f[0], f[DIM], f[2 * DIM], f[3 * DIM]};
            return __builtin_bit_cast(uint4, v);
        } else {
            const char *q = p + at[0] + kk * DIM * 32 + (more >> 4) * 128;   // 4 rows take DIM * 8 bytes
            const uint2 u = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)q));
            const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(q + DIM * 8)));
            return {u.x, u.y, v.x, v.y};
        }
    }
};

// LDS of a workgroup: the steps' two operands.
template <typename C>
struct Stages {
    uint4 *all;
    __device__ uint4 *a(int stage) const { return all + stage * (C::BM * 4); }
    __device__ uint4 *b(int stage) const { return all + C::STAGES * (C::BM * 4) + stage * (C::BN * 4); }
};

template <typename F, int... I>
__device__ inline void each(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

// The whole reduction of a tile.  fa, fb: lines of the wave's first 32 x 32 piece; da: lines between its pieces.
// One barrier a step: every wave has read the step's buffers, and the next step's loads, requested S - 1 steps
// before, have landed.  A piece of the reduction is read from LDS while the one before is multiplied,
// across steps too.  Loads are spread between the products: a wave that issues them at once waits for the
// address unit that all waves share, and its products with it.  A wave without work (`active` false) only loads.
template <typename T, int AK, int BK, typename C, int WAY, typename Da>
__device__ inline void reduce(const Source &sa, const Source &sb, int fa, Da da, int fb, bool active, int steps,
                              const Stages<C> &l, float16v (&acc)[C::FM][C::FN]) {
    constexpr int FM = C::FM, FN = C::FN, S = C::STAGES;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    if (steps <= 0) return;
    using LA = Loader<T, AK, C::BM, C, WAY>;
    using LB = Loader<T, BK, C::BN, C, WAY>;
    LA la;
    LB lb;
    la.begin(sa);
    lb.begin(sb);
    // A step's products are 2 FM groups of FN; its loads to LDS go between them: the first ones, by their order, in the last
    // FM / 2 groups of the step S before, behind its barrier, and the others in the first groups of the next step.
    constexpr int NA = LA::TO_LDS ? LA::LOADS : 0, ALL = NA + (LB::TO_LDS ? LB::LOADS : 0), GROUPS = 2 * FM, BEHIND = FM / 2;
    auto issue = [&](int step, int stage, int order) {
#pragma unroll
        for (int q = 0; q < ALL; ++q)
            if (q * GROUPS / ALL == order) {
                if (q < NA) la.direct(step, l.a(stage), q);
                else lb.direct(step, l.b(stage), q - NA);
            }
    };
    constexpr int FIRST = (BEHIND * ALL + GROUPS - 1) / GROUPS;   // loads of order < BEHIND
    // Loads that may still be on their way when the next step's have to be there: those of the S - 2 steps behind
    // it.  Codes are two loads each, in every step, past the last one too (Loader::use).  Loads to registers alone: the
    // compiler waits for them.
    constexpr int CODES = WAY == DIRECT && AK == KR_CODES ? 2 * LA::LOADS : 0;
    constexpr int LEFT = ALL ? (S - 2) * (ALL + CODES) : 63;
    const Reader<T, AK == KR_CODES ? KR : AK, C::BM> ra(fa);
    const Reader<T, BK, C::BN> rb(fb);
    uint4 x[2][FM], y[2][FN];
    auto read = [&](int stage, int kk) {
#pragma unroll
        for (int j = 0; j < FN; ++j) y[kk][j] = rb.get(l.b(stage), kk, j * 32);
#pragma unroll
        for (int i = 0; i < FM; ++i) x[kk][i] = ra.get(l.a(stage), kk, da(i));
    };
#pragma unroll
    for (int k = 0; k < S; ++k) {
        la.load(k, k);
        lb.load(k, k);
#pragma unroll
        for (int order = 0; order < (k + 1 < S ? GROUPS : BEHIND); ++order) issue(k, k, order);
    }
    la.store(0, 0, l.a(0));
    lb.store(0, 0, l.b(0));
    wait_and_meet<ALL ? (S - 2) * ALL + FIRST : 63>();
    auto run = [&](auto works) {   // a loop for each kind of wave: branches inside would join the waits for LDS
        constexpr bool W = decltype(works)::value;
        if (W) read(0, 0);
        auto products = [&](int group) {
            const int kk = group / FM, i = group % FM;
            if constexpr (W)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mma<T>(acc[i][j], x[kk][i], y[kk][j]);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto step = [&](auto stage, int s) {
            constexpr int c = decltype(stage)::value, n = (c + 1) % S, last = (c + S - 1) % S;
            if (W) read(c, 1);
#pragma unroll
            for (int i = 0; i < GROUPS - BEHIND; ++i) {
                products(i);
                issue(s + S - 1, last, i + BEHIND);
            }
            la.store(s + 1, n, l.a(n));
            lb.store(s + 1, n, l.b(n));
            wait_and_meet<LEFT>();
            // past the last step the loads give zeros, and what is read is not used
            if (W) read(n, 0);
            la.load(s + S, c);
            lb.load(s + S, c);
#pragma unroll
            for (int i = GROUPS - BEHIND; i < GROUPS; ++i) {
                issue(s + S, c, i - (GROUPS - BEHIND));
                products(i);
            }
        };
        int s = 0;
        constexpr auto stages = std::make_integer_sequence<int, S>{};
        for (; s + S <= steps; s += S) each([&](auto i) { step(i, s + decltype(i)::value); }, stages);
        each([&](auto i) {
            if (s + decltype(i)::value < steps) step(i, s + decltype(i)::value);
        }, stages);
    };
    if (active) run(std::true_type{});
    else run(std::false_type{});
    la.use();
    wait_and_meet<0>();   // the LDS is free for the results
}

// 1 / (1 + exp(-g)); the 16-bit types take the hardware's exponential and reciprocal (half the time of a tile's
// activations).  Off by (|g| + 5) 2^-23 of itself at most: two roundings of the exponential's argument, 1 unit in the last
// place each of the two instructions, and 0 from about g = -87 down, where it is no normal number.  An activation that is
// a normal number of its type has g > -13 in f16 and, above that cut, g > -88 in bf16: under a hundredth of its rounding.
template <typename T>
__device__ inline float sigmoid(float g) {
    if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-g));
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
}

// act(g) = g p and its slope p + g p', p = sigmoid(z): z = g (silu), or z = sqrt(8/pi) (g + 0.044715 g^3), as
// (1 + tanh(z/2)) / 2 = sigmoid(z) (gelu).
template <typename T>
__device__ inline void activation(float g, int act, float &a, float &slope) {
    const float c = 1.5957691216057308f, q = fminf(0.044715f * g * g, 1e10f);
    const bool silu = act == MOE_ACT_SILU;
    const float p = sigmoid<T>(silu ? g : c * (g + q * g));
    a = g * p;
    slope = p + a * (1.f - p) * (silu ? 1.f : c * (1.f + 3.f * q));   // p is 0 or 1 long before q is cut
}

// 8 values of a row; in fp32 through the caches, since a lane's 32 bytes take two stores that each leave half lines.
template <typename T>
__device__ inline void put8(T *p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) store8(p, f, n);
    else stream8(p, f, n);
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
        put8(p, gv, n);
        put8(p + g.M, uv, n);
    }
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float slope;
        activation<T>(gv[i], g.act, h[i], slope);
        h[i] *= uv[i];
    }
    put8(static_cast<T *>(g.out.p) + row * g.out.ld + col, h, n);
}

// What the activation's gradient needs of 8 columns of a row, as it lies in memory.
template <typename T>
struct Kept {
    uint4 g[sizeof(T) / 2], u[sizeof(T) / 2];   // codes: .xy and the scale in .z
};

template <typename T>
__device__ inline Kept<T> get_kept(const ExpertArgs &g, int row, int col, bool there) {
    const int n = there ? g.M - col : 0;
    Kept<T> k;
    if (g.kept_in.q) {
        const int nb = (g.M + kBlock - 1) / kBlock;
        const int8_t *q = g.kept_in.q + row * g.kept_in.ld + col;
        const uint8_t *s = g.kept_in.s + row * g.kept_in.ld_s + col / kBlock;
        const uint2 a = load_codes(q, n), b = load_codes(q + g.M, n);
        k.g[0] = {a.x, a.y, n > 0 ? s[0] : 0u, 0u};
        k.u[0] = {b.x, b.y, n > 0 ? s[nb] : 0u, 0u};
    } else {
        const T *p = static_cast<const T *>(g.pre_in.p) + row * g.pre_in.ld + col;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            k.g[i] = load_piece(p + i * kVec<T>, n - i * kVec<T>);
            k.u[i] = load_piece(p + g.M + i * kVec<T>, n - i * kVec<T>);
        }
    }
    return k;
}

template <typename T>
__device__ inline void values(const uint4 (&k)[sizeof(T) / 2], bool codes, float (&f)[8]) {
    if (codes) {
        decode8<float>({k[0].x, k[0].y}, k[0].z, f);
    } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            float v[kVec<T>];
            unpack<T>(k[i], v);
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) f[i * kVec<T> + j] = v[j];
        }
    }
}

// 8 columns of a row through the activation's gradient.
template <typename T>
__device__ inline void put_hidden_back(const ExpertArgs &g, int row, int col, const float (&d)[8], const Kept<T> &k) {
    const int n = g.M - col;
    float gv[8], uv[8], dg[8], du[8], h[8];
    values<T>(k.g, g.kept_in.q, gv);
    values<T>(k.u, g.kept_in.q, uv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, slope;
        activation<T>(gv[i], g.act, a, slope);
        dg[i] = d[i] * uv[i] * slope;
        du[i] = d[i] * a;
        h[i] = a * uv[i];
    }
    T *p = static_cast<T *>(g.pre.p) + row * g.pre.ld + col;
    put8(p, dg, n);
    put8(p + g.M, du, n);
    if (g.out.p) put8(static_cast<T *>(g.out.p) + row * g.out.ld + col, h, n);
}

// LDS operations of one wave are done in order; this keeps the compiler from reordering them.
__device__ inline void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's rows and columns through LDS of its own, 32 rows at a time: written 4 columns a lane, read back 8 next
// to each other, so that global stores are whole lines.  Piece p holds columns 8p .. 8p+7; with PAIR the first half of
// the pieces come with the second half.  fetch(row, p) gives what put(row, p, f, g, fetched) needs from memory; it is
// called BATCH pieces ahead.
template <typename C, bool PAIR, bool APART, int BATCH, typename Fetch, typename Put>
__device__ inline void spill(uint4 *stage, const float16v (&acc)[C::FM][C::FN], Fetch fetch, Put put) {
    constexpr int UNITS = C::FM * 8, PP = UNITS / (PAIR ? 4 : 2), ITS = 32 * PP / 64, ALL = C::FN * ITS;
    static_assert(ITS % BATCH == 0, "batches within 32 rows");
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31, p = lane % PP, row0 = lane / PP;
    decltype(fetch(0, 0)) ahead[2][BATCH];
    auto get = [&](int row, int piece, float (&f)[8]) {
        const int u = APART ? piece : 2 * piece, w = APART ? piece + UNITS / 2 : 2 * piece + 1;
        const float4 a = __builtin_bit_cast(float4, stage[row * UNITS + (u ^ (row % UNITS))]);
        const float4 b = __builtin_bit_cast(float4, stage[row * UNITS + (w ^ (row % UNITS))]);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    };
    auto row_of = [&](int it) { return it / ITS * 32 + it % ITS * (64 / PP) + row0; };
#pragma unroll
    for (int i = 0; i < BATCH; ++i) ahead[0][i] = fetch(row_of(i), p);
#pragma unroll
    for (int b = 0; b < ALL / BATCH; ++b) {
        if (b + 1 < ALL / BATCH)
#pragma unroll
            for (int i = 0; i < BATCH; ++i) ahead[(b + 1) & 1][i] = fetch(row_of((b + 1) * BATCH + i), p);
        if (b * BATCH % ITS == 0) {
            const int j = b * BATCH / ITS;
            wave_fence();
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    stage[r * UNITS + ((i * 8 + q * 2 + half) ^ (r % UNITS))] = __builtin_bit_cast(uint4, v);
                }
            wave_fence();
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int row = row_of(b * BATCH + i);
            float f[8], g[8];
            get(row & 31, p, f);
            if constexpr (PAIR) get(row & 31, p + PP, g);
            put(row, p, f, g, ahead[b & 1][i]);
        }
    }
}
struct Nothing {};

// Piece p of a row of M columns, from column col0 on, as spill gives it.
template <typename C, typename T>
__device__ inline void put_plain(T *row, int col0, int p, int M, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        const int a = col0 + 4 * p, b = a + C::FM * 16;
        stream4(row + a, f[0], f[1], f[2], f[3], M - a);
        stream4(row + b, f[4], f[5], f[6], f[7], M - b);
    } else {
        const int col = col0 + 8 * p;
        if (col < M) stream8(row + col, f, M - col);
    }
}

#define MOE_TILES                                                                                                  \
    __shared__ __align__(16) uint4 steps[C::STAGES * (C::BM + C::BN) * 4];                                           \
    static_assert(C::WAVES * C::FM * 256 <= C::STAGES * (C::BM + C::BN) * 4, "room for the results of every wave");  \
    const Stages<C> l = {steps};                                                                                     \
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave % C::MW, wn = wave / C::MW;         \
    uint4 *const stage = steps + wave * (C::FM * 256);

// Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles next to each other, so that the rows
// and the weights that they share are in one L2.  Tile `b` of `total`, or -1.
__device__ inline int xcd_tile(int b, int total) {
    const int per = (total + 7) >> 3, i = b >> 3, t = (b & 7) * per + i;
    return i < per && t < total ? t : -1;
}

template <typename T, int AK, int EPI, typename C, int WAY>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_rows(ExpertArgs g, int tiles_m) {
    MOE_TILES
    Tile t;
    int mt = 0;
    if (!find_tile(g.offsets, g.E, g.R, C::BN, [&](int total) {
            const int x = xcd_tile(blockIdx.x, total * tiles_m);
            mt = x % tiles_m;
            return x < 0 ? -1 : x / tiles_m;
        }, t))
        return;
    constexpr int COLS = EPI == E_HIDDEN ? C::BM / 2 : C::BM, MINE = COLS / C::MW;   // columns of a tile, and of a wave
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
    sb.lines = min(t.end - t.row, C::BN);
    float16v acc[C::FM][C::FN];
    const bool active = wm * MINE < sa.lines && wn * C::WN < sb.lines;
    // hidden: the second half of a wave's pieces are up's, of the same columns
    reduce<T, AK, KC, C, WAY>(
        sa, sb, wm * MINE, [](int i) { return EPI == E_HIDDEN ? i / (C::FM / 2) * (C::BM / 2) + i % (C::FM / 2) * 32 : i * 32; },
        wn * C::WN, active, (g.K + KE<T> - 1) / KE<T>, l, acc);
    if (!active) return;
    const int row0 = t.row + wn * C::WN, col0 = m0 + wm * MINE;
    const auto nothing = [](int, int) { return Nothing{}; };
    if constexpr (EPI == E_HIDDEN) {
        spill<C, true, false, 2>(stage, acc, nothing, [&](int r, int p, const float(&gv)[8], const float(&uv)[8], Nothing) {
            put_hidden<T>(g, row0 + r, col0 + 8 * p, row0 + r < t.end, gv, uv);
        });
    } else if constexpr (EPI == E_HIDDEN_BACK) {
        const auto fetch = [&](int r, int p) { return get_kept<T>(g, row0 + r, col0 + 8 * p, row0 + r < t.end); };
        spill<C, false, false, sizeof(T) == 4 ? 2 : 4>(stage, acc, fetch, [&](int r, int p, const float(&f)[8], const float(&)[8], const Kept<T> &k) {
            const int row = row0 + r, col = col0 + 8 * p;
            if (row < t.end && col < g.M) put_hidden_back<T>(g, row, col, f, k);
        });
    } else {
        spill<C, false, sizeof(T) == 4, 2>(stage, acc, nothing, [&](int r, int p, const float(&f)[8], const float(&)[8], Nothing) {
            if (row0 + r < t.end) put_plain<C>(static_cast<T *>(g.out.p) + (row0 + r) * g.out.ld, col0, p, g.M, f);
        });
    }
}

// d_w of one expert's tile and one of `splits` runs of its rows.
template <typename T, int AK, typename C, int WAY>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_grad(ExpertGradArgs g, int tiles_m,
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
    const int m0 = mt * C::BM, n0 = nt * C::BN;
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
    sa.lines = min(g.M - m0, C::BM);
    sb.p = static_cast<const T *>(g.d_out.p) + begin * g.d_out.ld + n0;
    sb.ld = g.d_out.ld;
    sb.lines = min(g.N - n0, C::BN);
    sa.K = sb.K = end - begin;
    float16v acc[C::FM][C::FN];
    const bool active = wm * C::WM < sa.lines && wn * C::WN < sb.lines;
    reduce<T, AK, KR, C, WAY>(sa, sb, wm * C::WM, [](int i) { return i * 32; }, wn * C::WN, active,
                                 (end - begin + KE<T> - 1) / KE<T>, l, acc);
    if (!active) return;
    float *out = (splits > 1 ? parts + (int64_t)sp * g.E * g.N * g.M : g.d_w) + (int64_t)e * g.N * g.M;
    spill<C, false, true, 2>(stage, acc, [](int, int) { return Nothing{}; }, [&](int r, int p, const float(&f)[8], const float(&)[8], Nothing) {
        const int row = n0 + wn * C::WN + r;
        if (row < g.N) put_plain<C>(out + (int64_t)row * g.M, m0 + wm * C::WM, p, g.M, f);
    });
}

// ------------------------------------------------------------------------------------------- launches

bool aligned(const void *p, int64_t ld, size_t size) { return !(((uintptr_t)p | (uintptr_t)(ld * size)) & 15); }

// Whether 256 rows of `ld` elements, `along` of them read, go straight into LDS.
bool direct(const void *p, int64_t ld, int64_t along, size_t size) {
    return aligned(p, ld, size) && along * (int64_t)size % 16 == 0 && 256 * ld * (int64_t)size < kReach;
}

template <typename T, int AK, int EPI, typename C, int WAY>
hipError_t rows_shape(const ExpertArgs &a, hipStream_t stream) {
    const int tiles_m = tiles(a.M, EPI == E_HIDDEN ? C::BM / 2 : C::BM);
    const int64_t n = ((int64_t)a.R / C::BN + std::min(a.E, a.R)) * tiles_m;
    return launch(k_rows<T, AK, EPI, C, WAY>, dim3((unsigned)((n + 7) / 8 * 8)), dim3(C::THREADS), stream, nullptr, nullptr, a, tiles_m);
}

template <typename T, int AK, int EPI>
hipError_t rows_launch(const ExpertArgs &a, hipStream_t stream) {
    if (a.R == 0) return hipSuccess;
    const int64_t ld = AK == KC ? a.K : a.M;
    bool d = direct(a.w, ld, ld, sizeof(T)) && direct(a.x.p, a.x.ld, a.K, sizeof(T));
    if (EPI == E_HIDDEN) d = d && ((int64_t)a.M + 256) * a.K * (int64_t)sizeof(T) < kReach;   // from a gate row to its up row
    if (!d && std::min(ld, (int64_t)a.K) < kVec<T>) return rows_shape<T, AK, EPI, Small, ELEMENTS>(a, stream);
    // Small where the middle one has fewer tiles than there are CUs (8 rows of 8 experts, hidden 2048 to 768: 13.0 us against 16.0;
    // 999 odd rows of 16 experts 28 / 36).  The larger one from 160 rows an expert and 192 tiles on (128 experts, 768 to 2048: 128 rows each
    // 108 us against the middle one's 110, 192 rows 123 / 159, 512 rows 257 / 339; 16 experts, 2048 to 2048: 64 rows 35 / 24, 256 rows
    // and 128 tiles 46 / 46, 512 rows 61 / 85; hidden of 8192 rows of one expert, 192 tiles, 54 / 65).
    const auto columns = [&](int bm) { return (int64_t)tiles(a.M, EPI == E_HIDDEN ? bm / 2 : bm); };
    const bool small = std::max(tiles(a.R, Mid::BN), std::min(a.E, a.R)) * columns(Mid::BM) < 256;
    if (!d) return small ? rows_shape<T, AK, EPI, Small, PIECES>(a, stream) : rows_shape<T, AK, EPI, Mid, PIECES>(a, stream);
    if (small) return rows_shape<T, AK, EPI, Small, DIRECT>(a, stream);
    if (a.R / a.E < 160 || tiles(a.R, Wide::BN) * columns(Wide::BM) < 192) return rows_shape<T, AK, EPI, Mid, DIRECT>(a, stream);
    return rows_shape<T, AK, EPI, Wide, DIRECT>(a, stream);
}

template <typename T, int AK, typename C, int WAY>
hipError_t grad_shape(const ExpertGradArgs &a, int splits, float *parts, hipStream_t stream) {
    const int tiles_m = tiles(a.M, C::BM), tiles_n = tiles(a.N, C::BN);
    const int64_t n = (int64_t)tiles_m * tiles_n * a.E * splits;
    return launch(k_grad<T, AK, C, WAY>, dim3((unsigned)((n + 7) / 8 * 8)), dim3(C::THREADS), stream, nullptr, nullptr, a, tiles_m,
                  tiles_n, splits, parts);
}

template <typename T>
hipError_t grad_launch(const ExpertGradArgs &a, const GradPlan &plan, float *parts, hipStream_t stream) {
    bool d = direct(a.d_out.p, a.d_out.ld, a.N, sizeof(T));
    const bool tiny = std::min(a.M, a.N) < kVec<T>;
    hipError_t e;
    if (a.x.p) {
        d = d && direct(a.x.p, a.x.ld, a.M, sizeof(T));
        e = d && plan.wide ? grad_shape<T, KR, Wide, DIRECT>(a, plan.splits, parts, stream)
            : d            ? grad_shape<T, KR, Mid, DIRECT>(a, plan.splits, parts, stream)
            : tiny         ? grad_shape<T, KR, Mid, ELEMENTS>(a, plan.splits, parts, stream)
                           : grad_shape<T, KR, Mid, PIECES>(a, plan.splits, parts, stream);
    } else {
        // pieces of 8 codes (4 beside fp32) are whole and aligned
        d = d && !(((uintptr_t)a.codes.q | (uintptr_t)a.codes.ld | (uintptr_t)a.M) & 7) && 256 * std::max(a.codes.ld, a.codes.ld_s) < kReach;
        e = d && plan.wide ? grad_shape<T, KR_CODES, Wide, DIRECT>(a, plan.splits, parts, stream)
            : d            ? grad_shape<T, KR_CODES, Mid, DIRECT>(a, plan.splits, parts, stream)
            : tiny         ? grad_shape<T, KR_CODES, Mid, ELEMENTS>(a, plan.splits, parts, stream)
                           : grad_shape<T, KR_CODES, Mid, PIECES>(a, plan.splits, parts, stream);
    }
    return e;
}

}  // namespace

// The launches of one type (a file each, since they take half a minute to compile).
#define MOE_EXPERTS_OF(T, NAME)                                                                                      \
    hipError_t hidden_##NAME(const ExpertArgs &a, hipStream_t s) { return rows_launch<T, KC, E_HIDDEN>(a, s); }       \
    hipError_t product_##NAME(const ExpertArgs &a, hipStream_t s) { return rows_launch<T, KC, E_PLAIN>(a, s); }       \
    hipError_t hidden_back_##NAME(const ExpertArgs &a, hipStream_t s) { return rows_launch<T, KR, E_HIDDEN_BACK>(a, s); } \
    hipError_t product_back_##NAME(const ExpertArgs &a, hipStream_t s) { return rows_launch<T, KR, E_PLAIN>(a, s); }  \
    hipError_t grad_##NAME(const ExpertGradArgs &a, const GradPlan &p, float *parts, hipStream_t s) {                 \
        return grad_launch<T>(a, p, parts, s);                                                                        \
    }

}  // namespace moe
