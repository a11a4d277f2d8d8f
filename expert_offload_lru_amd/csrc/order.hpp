// The order of picks by expert: a stable counting sort whose workgroups need nothing of each other
// (device code, shared by the token dispatch and the adapters' gradients).
#pragma once

#include "token_kernels.hpp"

namespace moe {

constexpr int kThreads = 256;
constexpr int kWgPicks = 512;   // picks a workgroup ranks at most
constexpr int kCopies = 8;      // copies of a histogram, by lane: picks of one expert in a wave
                                // would otherwise add to one LDS word in turn

// Adds picks p0 .. p1 to the histogram copies, eight picks a thread in flight.
__device__ inline void count(const int32_t *ids, int p0, int p1, int E, int *hist) {
    const int copy = threadIdx.x & (kCopies - 1);
    auto add = [&](int e) {
        if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e * kCopies + copy], 1);
    };
    int p = p0 + 4 * (int)threadIdx.x;
    for (; p + 4 * kThreads + 4 <= p1; p += 8 * kThreads) {
        int e[8];
        __builtin_memcpy(e, ids + p, 16);
        __builtin_memcpy(e + 4, ids + p + 4 * kThreads, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) add(e[i]);
    }
    for (; p < p1; p += 4 * kThreads) {
        int e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = p + i < p1 ? ids[p + i] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) add(e[i]);
    }
}

__device__ inline int total_of(const int *hist, int e) {
    int s = 0;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) s += hist[e * kCopies + c];
    return s;
}

// LDS of order_picks, for up to EM experts.
template <int EM>
struct OrderSpace {
    int hist[EM * kCopies];
    int next[EM];            // picks before the workgroup's, then the next row, of each expert
    int all[EM];             // picks of each expert
    int row_of[kWgPicks];    // out: rows of the workgroup's picks (written by the first wave)
    int wave_sum[kThreads / 64];
};

// Workgroup wg takes `tokens` consecutive tokens.  The row of pick p with expert e is
//   offsets[e] + (valid picks of e before p),
// so it counts, per expert, all picks and the picks before its own -- from the ids themselves, or for
// many picks from the counts of slices of `per` picks -- and then ranks its own picks in order, 64 at a
// time by one wave: the lanes with the same expert are found by one ballot per bit of the id.
template <int EM>
__device__ __forceinline__ void order_picks(const DispatchArgs &a, int wg, int tokens, const int32_t *counts, int slices, int per,
                                            OrderSpace<EM> &o) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E, N = a.T * a.k;
    const int p0 = wg * tokens * a.k, p1 = min(a.T, (wg + 1) * tokens) * a.k;
    for (int i = tid; i < E * kCopies; i += kThreads) o.hist[i] = 0;
    __syncthreads();
    const int slice = counts ? p0 / per : 0;
    count(a.ids, counts ? slice * per : 0, p0, E, o.hist);
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        int before = total_of(o.hist, e), sum = 0;
        if (counts) {
#pragma unroll 8
            for (int s = 0; s < slices; ++s) {
                const int n = counts[(size_t)s * E + e];
                sum += n;
                before += s < slice ? n : 0;
            }
        }
        o.next[e] = before;
        o.all[e] = sum;
    }
    if (!counts) {
        __syncthreads();
        count(a.ids, p0, N, E, o.hist);
        __syncthreads();
        for (int e = tid; e < E; e += kThreads) o.all[e] = total_of(o.hist, e);
    }
    __syncthreads();
    // the experts' first rows: consecutive experts a thread
    constexpr int EP = EM / kThreads;
    int total[EP], mine = 0;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        total[i] = EP * tid + i < E ? o.all[EP * tid + i] : 0;
        mine += total[i];
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) o.wave_sum[wave] = upto;
    __syncthreads();
    int start = upto - mine;
    for (int w = 0; w < wave; ++w) start += o.wave_sum[w];
    const int n_rows = o.wave_sum[0] + o.wave_sum[1] + o.wave_sum[2] + o.wave_sum[3];
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int e = EP * tid + i;
        if (e < E) {
            o.next[e] += start;
            if (wg == 0) a.offsets[e] = start;
        }
        start += total[i];
    }
    if (wg == 0 && tid == 0) a.offsets[E] = n_rows;
    __syncthreads();

    if (wave == 0) {
        volatile int *nx = o.next;
        for (int p = p0; p < p1; p += 64) {
            const int q = p + lane;
            const int e = q < p1 ? a.ids[q] : -1;
            const bool valid = (unsigned)e < (unsigned)E;
            unsigned long long same = __ballot(valid);
            for (int bit = 0; (1 << bit) < E; ++bit) {
                const bool set = (e >> bit) & 1;
                const unsigned long long m = __ballot(set);
                same &= set ? m : ~m;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            int row = -1;
            if (valid) {
                const int at = nx[e];
                row = at + rank;
                if (rank == 0) nx[e] = at + __popcll(same);
            }
            if (q < p1) {
                o.row_of[q - p0] = row;
                if (a.pos) a.pos[q] = row;
                if (valid) {
                    a.src[row] = q;
                    if (a.expert) a.expert[row] = e;
                }
            }
        }
    }
    // rows behind the last
    for (int p = p0 + tid; p < p1; p += kThreads)
        if (p >= n_rows) {
            a.src[p] = -1;
            if (a.expert) a.expert[p] = -1;
        }
}

}  // namespace moe
