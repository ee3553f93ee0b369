// q8_kv4_shares.h -- how the attention's steps are cut into shares, one for a
// workgroup: plain arithmetic, which the kernel does on the GPU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

// Least share: two steps a wave.  With 4 or 16 steps, 7 sessions with a window of
// 1000 take 12.8 or 13.3 us against 12.1, the larger cases the same.
constexpr int kMinSteps = 8;

// The room cut into shares.  Even layout: kMinSteps each.  End to end: one for
// each resident workgroup.  Where several share a CU, those dispatched first
// get ahead of the others in its issue slots, and the last ones would run on
// alone: shares are weighted by rank, 23 : 20 : 17 for three (16 sessions up to
// 8192 tokens 31.5 -> 28.6 us, near 32768 tokens 103.8 -> 99.0, against equal
// shares; at 26 : 20 : 14, 29.0 and 100.8) and 5 : 4 for two (4 drafted tokens of
// 16 sessions 35.9 us; equal shares 38.2, 4 : 3 39.5).  Those are full grids.  One
// that the context or kMostParts keeps smaller, with fewer workgroups to a CU or
// one, is cut by the same weights, and its longest share is 15% (11%) above the mean.
struct Shares {
    int64_t room;
    double unit;   // room of a share of weight 1
    int n, rank;   // shares in all, and of one rank
    int w[3];      // weight of a share by its rank
    bool even;

    __host__ __device__ Shares(int64_t room_, int n_, bool even_, int on_cu)
        : room(room_), n(n_), rank(n_ / on_cu), even(even_) {
        w[0] = on_cu == 3 ? 23 : on_cu == 2 ? 5 : 1;
        w[1] = on_cu == 3 ? 20 : on_cu == 2 ? 4 : 1;
        w[2] = on_cu == 3 ? 17 : w[1];
        unit = (double)room / weight(n);
    }
    __host__ __device__ int weight(int i) const {  // of the first i shares
        const int second = i - rank < rank ? i - rank : rank, third = i - 2 * rank;
        return w[0] * (i < rank ? i : rank) + w[1] * (second > 0 ? second : 0) +
               w[2] * (third > 0 ? third : 0);
    }
    __host__ __device__ int64_t start(int i) const {
        if (even) return (int64_t)kMinSteps * i < room ? (int64_t)kMinSteps * i : room;
        return i >= n ? room : (int64_t)(unit * weight(i));
    }
    // The share that holds pos, for any pos >= 0 one of the n.
    __host__ __device__ int at(int64_t pos) const {
        if (even) return pos < room ? (int)(pos / kMinSteps) : n - 1;
        const double x = (double)pos / unit;
        const int v = x < 1e9 ? (int)x : 1000000000;  // past the room it may be anything
        const int v0 = w[0] * rank, v1 = v0 + w[1] * rank;
        int i = v < v0 ? v / w[0] : v < v1 ? rank + (v - v0) / w[1] : 2 * rank + (v - v1) / w[2];
        if (i > n - 1) i = n - 1;
        while (start(i) > pos) --i;
        while (i + 1 < n && start(i + 1) <= pos) ++i;
        return i;
    }
};

}  // namespace q8
