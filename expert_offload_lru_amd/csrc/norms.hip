// Norms around a block with its gate and residual scale, and rows kept in 8 bits (include/moe_experts.h).
//
// Both are bound by memory: a row is read once, held in registers while its sums are made, and its results
// are written from there.
#include <algorithm>

#include "expert_kernels.hpp"
#include "pieces8.hpp"

namespace moe {
namespace {

// ------------------------------------------------------------------------------------- rows in 8 bits

constexpr int kRowsPer = 4;   // rows a thread has in flight

// A thread holds 8 columns of kRowsPer rows; `lanes` threads (a power of two, whole blocks) go along a row.
template <typename T>
__global__ __launch_bounds__(256) void k_encode(Rows x, CodesOut c, int R, int C, int lanes) {
    const int per = 256 / lanes, groups = (C + kBlock - 1) / kBlock * 4;
    const int64_t row0 = (int64_t)blockIdx.x * per * kRowsPer + threadIdx.x / lanes;
    for (int at = threadIdx.x & (lanes - 1); at < groups; at += lanes) {
        float f[kRowsPer][8];
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const int64_t row = row0 + i * per;
            load8(static_cast<const T *>(x.p) + row * x.ld + at * 8, f[i], row < R ? C - at * 8 : 0);
        }
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const int64_t row = row0 + i * per;
            int scale;
            const uint2 q = encode8(f[i], C - at * 8, scale);
            if (row < R) {
                store_codes(c.q + row * c.ld + at * 8, q, C - at * 8);
                if ((at & 3) == 0) c.s[row * c.ld_s + at / 4] = (uint8_t)scale;
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_decode(Codes c, RowsOut x, int R, int C, int lanes) {
    const int per = 256 / lanes, groups = (C + 7) / 8;
    const int64_t row0 = (int64_t)blockIdx.x * per * kRowsPer + threadIdx.x / lanes;
    for (int at = threadIdx.x & (lanes - 1); at < groups; at += lanes) {
        uint2 q[kRowsPer];
        int s[kRowsPer];
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const int64_t row = row0 + i * per;
            q[i] = load_codes(c.q + row * c.ld + at * 8, row < R ? C - at * 8 : 0);
            s[i] = row < R ? c.s[row * c.ld_s + at / 4] : 0;
        }
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const int64_t row = row0 + i * per;
            float f[8];
            decode8<T>(q[i], s[i], f);
            if (row < R) store8(static_cast<T *>(x.p) + row * x.ld + at * 8, f, C - at * 8);
        }
    }
}

int lanes_of(int groups) {
    int l = 4;
    while (l < groups && l < 256) l *= 2;
    return l;
}
unsigned row_blocks(int R, int lanes) {
    const int64_t per = (int64_t)256 / lanes * kRowsPer;
    return (unsigned)((R + per - 1) / per);
}

// --------------------------------------------------------------------------------------------- norms

// v plus the value that a lane gets by `CTRL` (0 in rows of 16 lanes outside MASK).
template <int CTRL, int MASK>
__device__ inline float plus_from(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, MASK, 0xf, false));
}
// The wave's sum: by moves between lanes within the vector unit (through LDS: 2048 rows of 8192 forward 28.5 us, so 26.1).
__device__ inline float wave_sum(float v) {
    v = plus_from<0x111, 0xf>(v);   // row_shr:1 .. 8: lane 15 of each 16 has their sum
    v = plus_from<0x112, 0xf>(v);
    v = plus_from<0x114, 0xf>(v);
    v = plus_from<0x118, 0xf>(v);
    v = plus_from<0x142, 0xa>(v);   // row_bcast:15
    v = plus_from<0x143, 0xc>(v);   // row_bcast:31: lane 63 has all
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sums over the waves of a row; the buffer `s` has a place for each wave and is not written again before
// the next barrier but one.
template <int WAVES, int N>
__device__ inline void row_sum(float (&v)[N], float *s, int wave_in_row, int first_wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[(first_wave + wave_in_row) * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v[i] += s[(first_wave + w) * N + i];
        }
    }
}

// 1 / sqrt(mean square + eps) of a row; sum: a lane's part of the sum of squares, squares(k): the same of k times the
// values.  A sum of squares leaves fp32's range where a row's root mean square is 2^64 / sqrt(columns) and more, and loses
// squares below 2^-126 where eps does not outweigh them; such a row is summed once more, from its values times 2^-80 or
// 2^80 (exact, and enough for every row whose inverse root is an fp32 number).  Other rows pay a comparison (65536 rows of
// 64 columns 37.8 -> 39.6 us; nothing to 2 % from 512 columns on).  s, again: a place for each of the ALL waves, as row_sum
// wants them.
template <int WAVES, int ALL, typename Squares>
__device__ inline float inverse_root(float sum, Squares squares, float inv, float eps, float *s, float *again,
                                     int wave_in_row, int first_wave) {
    constexpr float kFar = 1.2089258196146292e24f;   // 2^80
    constexpr uint32_t kLeast = (127 - 100) << 23, kInf = 0x7F800000u;   // 2^-100; a mean below it, infinite or NaN is far
    const auto far = [](float m) { return __float_as_uint(m) - kLeast >= kInf - kLeast; };
    float v[1] = {sum};
    row_sum<WAVES, 1>(v, s, wave_in_row, first_wave);
    const float mean = v[0] * inv + eps;
    bool any = false;   // the same in all waves that meet at the sums' barrier: of all their rows, from the same numbers
    if constexpr (WAVES > 1 && ALL > WAVES) {
#pragma unroll
        for (int g = 0; g < ALL; g += WAVES) {
            float m = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) m += s[g + w];
            any |= far(m * inv + eps);
        }
    } else {
        any = far(mean);
    }
    if (__builtin_expect(any, 0)) {
        const float k = mean < 1.f ? kFar : 1.f / kFar;
        v[0] = squares(k);
        row_sum<WAVES, 1>(v, again, wave_in_row, first_wave);
        if (far(mean)) return k / sqrtf(v[0] * inv + eps * k * k);
    }
    return 1.f / sqrtf(mean);
}

// A lane's 8 columns of a row: next to each other in the 16-bit types; in fp32 4 and, 256 columns on, 4 more, so that each
// load and store of 16 bytes a lane is whole lines (8192 rows: 3.3 TB/s otherwise).  Column of element i, behind the first:
template <typename T>
__device__ constexpr int column(int i) { return sizeof(T) == 4 ? (i & 3) + (i >> 2) * 256 : i; }
// The first column of piece v of V, of wave w of W a row.
template <typename T>
__device__ inline int first_column(int v, int W, int w) {
    return (v * W + w) * 512 + (threadIdx.x & 63) * (sizeof(T) == 4 ? 4 : 8);
}
// n: columns from the first on that there are.
template <typename T, typename U>
__device__ inline void load_columns(const U *p, float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        float a[4], b[4];
        unpack<float>(load_piece(p, n), a);
        unpack<float>(load_piece(p + 256, n - 256), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
        load8(p, f, n);
    }
}
// A row's results, past the caches (8192 rows of 2048, bf16: 32 -> 28 us).
template <typename T>
__device__ inline void put_columns(T *p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        stream4(p, f[0], f[1], f[2], f[3], n);
        stream4(p + 256, f[4], f[5], f[6], f[7], n - 256);
    } else {
        stream8(p, f, n);
    }
}
// Sums in fp32, beside rows of T.
template <typename T>
__device__ inline void put_sums(float *p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 4) {
        store_piece(p, pack<float>({f[0], f[1], f[2], f[3]}), n);
        store_piece(p + 256, pack<float>({f[4], f[5], f[6], f[7]}), n - 256);
    } else {
        store8(p, f, n);
    }
}

// A parameter's columns; `other` where it is not there.
template <typename T>
__device__ inline void load_vector(const float *p, int col, int n, float (&f)[8], float other) {
    if (p) {
        load_columns<T>(p + col, f, n);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = other;
    }
}

// 8 columns x V of a row, as they lie in memory.
template <typename T, int V>
struct Raw {
    uint4 v[V][sizeof(T) / 2];
    __device__ void load(const Rows &m, int64_t row, const int (&col)[V], const int (&n)[V], bool there) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j)
                v[i][j] = load_piece(static_cast<const T *>(m.p) + row * m.ld + col[i] + column<T>(j * kVec<T>),
                                     there && m.p ? n[i] - column<T>(j * kVec<T>) : 0);
    }
    __device__ void get(int i, float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
            float e[kVec<T>];
            unpack<T>(v[i][j], e);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) f[j * kVec<T> + k] = e[k];
        }
    }
};

// WAVES waves next to each other a row, 8 columns x V a lane; GROUPS rows a workgroup at a time.  A workgroup takes rows
// gridDim.x * GROUPS apart, so that the parameters stay in registers (read for every row they were twice its bytes), and
// requests the next row while it works on one.
template <typename T, int WAVES, int V>
__global__ __launch_bounds__(WAVES < 4 ? 256 : WAVES * 64) void k_norm(NormArgs g) {
    constexpr int GROUPS = WAVES < 4 ? 4 / WAVES : 1, ALL = GROUPS * WAVES;
    __shared__ float s_y[2][ALL], s_o[2][ALL], again[ALL];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = wave / WAVES, w = wave % WAVES;
    int col[V], n[V];
    float post[V][8], pre[V][8], alpha[V][8], gate[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = first_column<T>(v, WAVES, w);
        n[v] = g.H - col[v];
        load_vector<T>(g.w_post, col[v], n[v], post[v], 1.f);
        load_vector<T>(g.w_pre, col[v], n[v], pre[v], 1.f);
        load_vector<T>(g.alpha, col[v], n[v], alpha[v], 1.f);
        load_vector<T>(nullptr, col[v], n[v], gate[v], 1.f);
    }
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    const int steps = (int)((g.T + step - 1) / step);
    int64_t row = (int64_t)blockIdx.x * GROUPS + group, gate_row = -1;
    Raw<T, V> rx[2], ry[2];
    rx[0].load(g.x, row, col, n, row < g.T);
    ry[0].load(g.y, row, col, n, row < g.T);
    const float inv = 1.f / (float)g.H;
    auto one = [&](const Raw<T, V> &nx, const Raw<T, V> &ny, Raw<T, V> &fx, Raw<T, V> &fy, int it) {
        const bool there = row < g.T;
        fx.load(g.x, row + step, col, n, row + step < g.T);
        fy.load(g.y, row + step, col, n, row + step < g.T);
        if (g.gate && there && row / g.per_gate != gate_row) {
            gate_row = row / g.per_gate;
#pragma unroll
            for (int v = 0; v < V; ++v) load_vector<T>(g.gate + gate_row * g.H, col[v], n[v], gate[v], 1.f);
        }
        float x[V][8], y[V][8], r_y = 0.f, r_o = 0.f;
        if (g.y.p) {
            float s = 0.f, r = 1.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ny.get(v, y[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(y[v][i], y[v][i], s);
            }
            if (g.w_post) {
                const auto squares = [&](float k) {
                    float s = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int i = 0; i < 8; ++i) s += (k * y[v][i]) * (k * y[v][i]);
                    return s;
                };
                r = r_y = inverse_root<WAVES, ALL>(s, squares, inv, g.eps, s_y[it & 1], again, w, group * WAVES);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                nx.get(v, x[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] = alpha[v][i] * x[v][i] + gate[v][i] * (post[v][i] * (y[v][i] * r));
                if (g.out.p && there && n[v] > 0) put_columns(static_cast<T *>(g.out.p) + row * g.out.ld + col[v], x[v], n[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) nx.get(v, x[v]);
        }
        if (g.w_pre) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += n[v] > column<T>(i) ? x[v][i] * x[v][i] : 0.f;
            const auto squares = [&](float k) {
                float s = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s += n[v] > column<T>(i) ? (k * x[v][i]) * (k * x[v][i]) : 0.f;
                return s;
            };
            r_o = inverse_root<WAVES, ALL>(s, squares, inv, g.eps, s_o[it & 1], again, w, group * WAVES);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = pre[v][i] * (x[v][i] * r_o);
                if (there && n[v] > 0) put_columns(static_cast<T *>(g.normed.p) + row * g.normed.ld + col[v], p, n[v]);
            }
        }
        if (g.stats && lane == 0 && w == 0 && there) {
            g.stats[2 * row] = r_y;
            g.stats[2 * row + 1] = r_o;
        }
        row += step;
    };
    for (int it = 0; it < steps; it += 2) {
        one(rx[0], ry[0], rx[1], ry[1], it);
        if (it + 1 < steps) one(rx[1], ry[1], rx[0], ry[0], it + 1);
    }
}

// How the rows of a backward call are dealt: `chunks` workgroups; rows of a chunk share a row of gate
// (rows_each of them, or what is left), or, where a gate's rows are fewer than a chunk's, a chunk has `units`
// whole gates of `unit` rows.
struct Deal {
    int chunks, rows_each, per_gate_chunks, unit;   // unit 0: rows of one gate
};

constexpr int kBackWaves = 4;   // waves of a workgroup, at least

// Waves along a row; a lane has 8 columns, 16 above 4096 (bf16: 16384 rows of 500 columns, 1 wave 45 us, 2 72; of 1000, 2 waves 76,
// 4 121, one with 16 columns a lane 66; 8192 of 2048, 4 waves 56, 8 82, 2 with 16 55; 6000 of 2560, 8 waves 74, 6 105, 4 with 16 79;
// 4096 of 4096, 8 waves 64, 16 275, 4 with 16 62; 2048 of 8192, 8 with 16 71, 16 waves 218).
inline int back_waves(int H) { return H <= 512 ? 1 : H <= 1024 ? 2 : H <= 2048 ? 4 : H <= 8192 ? 8 : 16; }
inline int back_groups(int H) { return std::max(1, kBackWaves / back_waves(H)); }
// One round of workgroups: two waves a SIMD, as the registers allow (16384 rows of 2048: 97 us; two rows
// ahead 105, three waves 130).
inline int back_chunks(int H) { return std::max(256, 2048 / std::max(kBackWaves, back_waves(H))); }

Deal deal(int T, int H, int per_gate, bool gate) {
    const int groups = back_groups(H), n = std::max(1, gate ? std::min(per_gate, T) : T);
    const int most = back_chunks(H), gates = std::max(1, (T + n - 1) / n);
    int each = std::max(groups, (T + most - 1) / most);
    if (!gate || n >= each) {   // as many whole parts a gate as still make one round
        each = std::max(groups, (n + std::max(1, most / gates) - 1) / std::max(1, most / gates));
        const int parts = (n + each - 1) / each;
        return {T > 0 ? parts * gates : 0, each, parts, 0};
    }
    each = (each + n - 1) / n * n;   // whole gates
    each = std::max(each, n * groups);
    return {(T + each - 1) / each, each, 0, n};
}

template <typename T, int WAVES, int V>
__global__ __launch_bounds__(WAVES > kBackWaves ? WAVES * 64 : kBackWaves * 64) void k_norm_back(NormBackArgs g, Deal d,
                                                                                              float *parts) {
    constexpr int GROUPS = WAVES > kBackWaves ? 1 : kBackWaves / WAVES, ALL = GROUPS * WAVES;
    constexpr bool ROOM = V == 1;   // registers for a row ahead
    __shared__ float sums[2][ALL * 3];
    __shared__ float join[GROUPS > 1 ? GROUPS * WAVES * 64 * 8 * V : 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = wave / WAVES, w = wave % WAVES;
    int64_t begin, end;
    if (d.unit == 0) {
        const int n = g.gate ? min(g.per_gate, g.T) : g.T;
        const int64_t gate = blockIdx.x / d.per_gate_chunks;
        begin = gate * n + (int64_t)(blockIdx.x % d.per_gate_chunks) * d.rows_each;
        end = min(min(begin + d.rows_each, (gate + 1) * n), (int64_t)g.T);
    } else {
        begin = (int64_t)blockIdx.x * d.rows_each;
        end = min(begin + d.rows_each, (int64_t)g.T);
    }
    const int steps = d.unit == 0 ? (d.rows_each + GROUPS - 1) / GROUPS
                                  : (d.rows_each / d.unit + GROUPS - 1) / GROUPS * d.unit;
    float post[V][8], pre[V][8], alpha[V][8], gate[V][8];
    float a_post[V][8] = {}, a_pre[V][8] = {}, a_alpha[V][8] = {}, a_gate[V][8] = {};
    int col[V], n[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = first_column<T>(v, WAVES, w);
        n[v] = g.H - col[v];
        load_vector<T>(g.w_post, col[v], n[v], post[v], 1.f);
        load_vector<T>(g.w_pre, col[v], n[v], pre[v], 0.f);
        load_vector<T>(g.alpha, col[v], n[v], alpha[v], 1.f);
        load_vector<T>(g.gate && begin < end && d.unit == 0 ? g.gate + begin / g.per_gate * g.H : nullptr, col[v], n[v], gate[v], 1.f);
    }
    const float inv = 1.f / (float)g.H;
    // a row of step `it`; last: of its gate
    auto row_of = [&](int it, bool &first, bool &last) {
        if (d.unit == 0) {
            first = last = false;
            return begin + (int64_t)it * GROUPS + group;
        }
        const int u = it / d.unit, i = it - u * d.unit;
        first = i == 0;
        last = i == d.unit - 1;
        return begin + (int64_t)(u * GROUPS + group) * d.unit + i;
    };
    struct Four {
        Raw<T, V> x, y, d, n;
        float r_y, r_o;
    };
    auto fetch = [&](Four &f, int it) {
        bool a, b;
        const int64_t row = row_of(it, a, b);
        const bool there = it < steps && row < end;
        f.x.load(g.x, row, col, n, there);
        f.y.load(g.y, row, col, n, there);
        f.d.load(g.d_out, row, col, n, there);
        f.n.load(g.d_normed, row, col, n, there);
        f.r_y = there && g.w_post ? g.stats[2 * row] : 1.f;
        f.r_o = there && g.w_pre ? g.stats[2 * row + 1] : 0.f;
    };
    auto one = [&](Four &at, int it) {
        bool first, last;
        const int64_t row = row_of(it, first, last);
        if (first)
#pragma unroll
            for (int v = 0; v < V; ++v)
                load_vector<T>(row < end ? g.gate + row / g.per_gate * g.H : nullptr, col[v], n[v], gate[v], 1.f);
        const bool there = row < end;
        // Sums are of y r_y and out r_out, numbers of size 1, so that no row's size leaves fp32's range in them:
        //   D = d_out + r_out (t - o mean(t o)), o = out r_out;   d_y = r_y (c - z mean(c z)), z = y r_y,
        // and mean(c z) from sums that need no D, made together with mean(t o): one exchange between the waves a row.
        float x[V][8], z[V][8], dd[V][8], t[V][8], o[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            at.x.get(v, x[v]);
            at.y.get(v, z[v]);
            at.d.get(v, dd[v]);
            at.n.get(v, t[v]);
        }
        const float r_y = at.r_y, r_o = at.r_o;
        if (ROOM) fetch(at, it + 1);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (n[v] > column<T>(i) && there) {
                    z[v][i] *= r_y;
                    o[v][i] = (alpha[v][i] * x[v][i] + (g.y.p ? gate[v][i] * (post[v][i] * z[v][i]) : 0.f)) * r_o;
                    if (g.d_normed.p) {
                        a_pre[v][i] += t[v][i] * o[v][i];
                        t[v][i] *= pre[v][i];
                        s[0] += t[v][i] * o[v][i];
                        dd[v][i] += r_o * t[v][i];
                    }
                    const float kz = gate[v][i] * post[v][i] * z[v][i];
                    s[1] += kz * dd[v][i];
                    s[2] += kz * o[v][i];
                }
            }
        row_sum<WAVES, 3>(s, sums[it & 1], w, group * WAVES);
        const float c1 = g.d_normed.p ? r_o * (s[0] * inv) : 0.f;
        // What is not part of a formula stays out of it, not times 0: out and y may be infinite.  The selection in the loop
        // costs 1024 rows of 16384 columns 306 -> 320 us and up to 2 % elsewhere; the loop twice, with and without w_post, takes 30
        // registers more.
        const float c2 = (g.d_normed.p ? s[1] - c1 * s[2] : s[1]) * inv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!there || n[v] <= 0) continue;
            float dx[8], dy[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float D = g.d_normed.p ? dd[v][i] - c1 * o[v][i] : dd[v][i];
                dx[i] = alpha[v][i] * D;
                dy[i] = r_y * (gate[v][i] * post[v][i] * D - (g.w_post ? c2 * z[v][i] : 0.f));
                a_alpha[v][i] += D * x[v][i];
                a_post[v][i] += gate[v][i] * D * z[v][i];
                a_gate[v][i] += post[v][i] * D * z[v][i];
            }
            if (g.d_x.p) put_columns(static_cast<T *>(g.d_x.p) + row * g.d_x.ld + col[v], dx, n[v]);
            if (g.d_y.p) put_columns(static_cast<T *>(g.d_y.p) + row * g.d_y.ld + col[v], dy, n[v]);
        }
        if (last && g.d_gate) {   // this gate's rows are all this group's
            const int64_t q = (begin + (int64_t)((it / d.unit) * GROUPS + group) * d.unit) / g.per_gate;
            if (q * g.per_gate < end)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (n[v] > 0) put_sums<T>(g.d_gate + q * g.H + col[v], a_gate[v], n[v]);
        }
        if (last)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) a_gate[v][i] = 0.f;
    };
    Four row;
    fetch(row, 0);
    for (int it = 0; it < steps; ++it) {
        one(row, it);
        if (!ROOM) fetch(row, it + 1);
    }
    if (!parts) return;
    // the groups' sums, in order, then the chunk's row of each parameter's partial sums
    auto put = [&](float(&a)[V][8], int which) {
        if constexpr (GROUPS > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) join[(v * 8 + i) * (ALL * 64) + threadIdx.x] = a[v][i];
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int k = 1; k < GROUPS; ++k) a[v][i] += join[(v * 8 + i) * (ALL * 64) + k * WAVES * 64 + threadIdx.x];
            }
        }
        if (group == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (n[v] > 0) put_sums<T>(parts + ((int64_t)which * d.chunks + blockIdx.x) * g.H + col[v], a[v], n[v]);
    };
    if (g.d_w_post) put(a_post, 0);
    if (g.d_alpha) put(a_alpha, 1);
    if (g.d_w_pre) put(a_pre, 2);
    if (g.d_gate && d.unit == 0) put(a_gate, 3);
}

// Sums of the chunks' rows, in order, 64 columns a workgroup.  y: parameter (0 .. 2), from 3 on a row of gate.
__global__ __launch_bounds__(1024) void k_norm_join(NormBackArgs g, Deal d, const float *parts) {
    __shared__ float s[16][64];
    const int c = threadIdx.x & 63, k = threadIdx.x >> 6, col = blockIdx.x * 64 + c, which = blockIdx.y;
    float *out = which == 0 ? g.d_w_post : which == 1 ? g.d_alpha : which == 2 ? g.d_w_pre : g.d_gate;
    if (!out) return;
    int64_t first = 0, rows = d.chunks;
    if (which >= 3) {
        first = (int64_t)(which - 3) * d.per_gate_chunks;
        rows = d.per_gate_chunks;
        out += (int64_t)(which - 3) * g.H;
    }
    const float *p = parts + ((int64_t)min(which, 3) * d.chunks + first) * g.H + col;
    const int64_t per = (rows + 15) / 16, b = k * per, e = min(b + per, rows);
    float v = 0.f;
    if (col < g.H)
#pragma unroll 8
        for (int64_t i = b; i < e; ++i) v += p[i * g.H];
    s[k][c] = v;
    __syncthreads();
    if (k == 0 && col < g.H) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += s[i][c];
        out[col] = v;
    }
}

template <typename T>
hipError_t norm_launch(const NormArgs &a, hipStream_t stream) {
    // Waves a row: 8 columns a lane, 16 above 8192 columns (bf16: 16384 rows of 500 columns, 1 wave 18 us, 2 30; of 1000, 2 waves 27,
    // 4 40, one with 16 columns a lane 28; 8192 of 2048, 4 waves 25, 8 37, 2 with 16 28; 6000 of 2560, 6 waves 29, 8 30, 4 with 16 34;
    // 4096 of 4096, 8 waves 25, 16 40, 4 with 16 26; 2048 of 8192, 16 waves 26, 8 with 16 28).
    // Workgroups: as many as run at a time, since more rows each keep the parameters longer (the same cases with 256, 512, 1024 and
    // 2048: 40 26 18 19 us; 65 38 27 27; 48 30 25 25; 43 29 30 35; 32 25 26 28; 26 29 33 39; 1024 of 16384 columns 54 68 89 89).
    const auto grid = [&](int rows, int most) { return dim3((unsigned)std::min((a.T + rows - 1) / rows, most)); };
    if (a.H <= 512) return launch(k_norm<T, 1, 1>, grid(4, 2048), dim3(256), stream, nullptr, nullptr, a);
    if (a.H <= 1024) return launch(k_norm<T, 2, 1>, grid(2, 1024), dim3(256), stream, nullptr, nullptr, a);
    if (a.H <= 2048) return launch(k_norm<T, 4, 1>, grid(1, 1024), dim3(256), stream, nullptr, nullptr, a);
    if (a.H <= 6 * 512) return launch(k_norm<T, 6, 1>, grid(1, 512), dim3(384), stream, nullptr, nullptr, a);
    if (a.H <= 4096) return launch(k_norm<T, 8, 1>, grid(1, 512), dim3(512), stream, nullptr, nullptr, a);
    if (a.H <= 8192) return launch(k_norm<T, 16, 1>, grid(1, 256), dim3(1024), stream, nullptr, nullptr, a);
    return launch(k_norm<T, 16, 2>, grid(1, 256), dim3(1024), stream, nullptr, nullptr, a);
}

template <typename T>
hipError_t norm_back_launch(const NormBackArgs &a, float *parts, hipStream_t stream) {
    const Deal d = deal(a.T, a.H, a.per_gate, a.gate != nullptr);
    const dim3 grid((unsigned)d.chunks);
    hipError_t e = hipSuccess;
    if (a.T > 0) {
        const int w = back_waves(a.H);
        const dim3 block((unsigned)(back_groups(a.H) * w * 64));
        if (w == 1) e = launch(k_norm_back<T, 1, 1>, grid, block, stream, nullptr, nullptr, a, d, parts);
        else if (w == 2) e = launch(k_norm_back<T, 2, 1>, grid, block, stream, nullptr, nullptr, a, d, parts);
        else if (w == 4) e = launch(k_norm_back<T, 4, 1>, grid, block, stream, nullptr, nullptr, a, d, parts);
        else if (a.H <= 4096) e = launch(k_norm_back<T, 8, 1>, grid, block, stream, nullptr, nullptr, a, d, parts);
        else if (w == 8) e = launch(k_norm_back<T, 8, 2>, grid, block, stream, nullptr, nullptr, a, d, parts);
        else e = launch(k_norm_back<T, 16, 2>, grid, block, stream, nullptr, nullptr, a, d, parts);
    }
    if (e != hipSuccess || !(a.d_w_post || a.d_alpha || a.d_w_pre || a.d_gate)) return e;
    const bool gates = a.d_gate && d.unit == 0;
    const int y = gates ? 3 + (a.T + std::max(1, std::min(a.per_gate, a.T)) - 1) / std::max(1, std::min(a.per_gate, a.T)) : 3;
    return launch(k_norm_join, dim3((unsigned)((a.H + 63) / 64), (unsigned)y), dim3(1024), stream, nullptr, nullptr, a, d,
                  static_cast<const float *>(parts));
}

}  // namespace

hipError_t launch_encode(int dtype, Rows x, CodesOut c, int R, int C, hipStream_t stream) {
    const int lanes = lanes_of((C + kBlock - 1) / kBlock * 4);
    const dim3 grid(row_blocks(R, lanes)), block(256);
    if (dtype == T_F32) return launch(k_encode<float>, grid, block, stream, nullptr, nullptr, x, c, R, C, lanes);
    if (dtype == T_F16) return launch(k_encode<f16>, grid, block, stream, nullptr, nullptr, x, c, R, C, lanes);
    return launch(k_encode<bf16>, grid, block, stream, nullptr, nullptr, x, c, R, C, lanes);
}

hipError_t launch_decode(int dtype, Codes c, RowsOut x, int R, int C, hipStream_t stream) {
    const int lanes = lanes_of((C + 7) / 8);
    const dim3 grid(row_blocks(R, lanes)), block(256);
    if (dtype == T_F32) return launch(k_decode<float>, grid, block, stream, nullptr, nullptr, c, x, R, C, lanes);
    if (dtype == T_F16) return launch(k_decode<f16>, grid, block, stream, nullptr, nullptr, c, x, R, C, lanes);
    return launch(k_decode<bf16>, grid, block, stream, nullptr, nullptr, c, x, R, C, lanes);
}

hipError_t launch_norm(int dtype, const NormArgs &a, hipStream_t stream) {
    if (dtype == T_F32) return norm_launch<float>(a, stream);
    if (dtype == T_F16) return norm_launch<f16>(a, stream);
    return norm_launch<bf16>(a, stream);
}

size_t norm_workspace(int T, int H, int per_gate) {
    const int with = deal(T, H, per_gate, true).chunks, without = deal(T, H, per_gate, false).chunks;
    return (size_t)std::max(with, without) * 4 * H * sizeof(float);
}

hipError_t launch_norm_back(int dtype, const NormBackArgs &a, void *workspace, hipStream_t stream) {
    float *parts = a.d_w_post || a.d_alpha || a.d_w_pre || a.d_gate ? static_cast<float *>(workspace) : nullptr;
    if (dtype == T_F32) return norm_back_launch<float>(a, parts, stream);
    if (dtype == T_F16) return norm_back_launch<f16>(a, parts, stream);
    return norm_back_launch<bf16>(a, parts, stream);
}

}  // namespace moe
