// Device helpers shared by the streaming-attention kernels.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rvq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <typename T>
__device__ inline float to_float(T x) { return static_cast<float>(x); }

// One clip of a packed batch: its queries and keys, ends clamped into the arrays.
struct Clip {
    int q0, nq;      // first query row, number of queries
    int k0, nk;
};

__device__ inline void clip_range(const int32_t *cu, int b, int64_t tokens, int &first, int &count)
{
    const int top = static_cast<int>(tokens);
    const int lo = min(max(cu[b], 0), top), hi = min(max(cu[b + 1], 0), top);
    first = lo;
    count = max(hi - lo, 0);
}

// The last b in [0, n) with cu[b] / per + b <= slot (0 if there is none). With per = tile rows this names the
// clip of a tile: clip b owns the slots cu[b] / per + b .. cu[b + 1] / per + b, enough for its rows.
__device__ inline int clip_of_slot(const int32_t *cu, int n, int slot, int per)
{
    int lo = 0, hi = n;      // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] / per + mid <= slot) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The last b in [0, n) with cu[b] <= row: the clip of a row (empty clips are passed over).
__device__ inline int clip_of_row(const int32_t *cu, int n, int row)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ inline float wave_sum(float x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

}  // namespace rvq
