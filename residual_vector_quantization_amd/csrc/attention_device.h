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

template <typename T> inline constexpr bool kNarrow = false;      // few exponent bits
template <> inline constexpr bool kNarrow<f16_t> = true;

// A number known to the compiler, as an argument.
template <int kN> struct Constant { static constexpr int value = kN; };

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

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));
typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Matrix-core operand: 8 values along the contracted dimension. A 16-wide product contracts 32 of them (lane / 16
// names the group of 8), a 32-wide one 16 (lane / 32 names it); float32 takes one instruction per value of the 8,
// each contracting one value of every group, so that operands are laid out alike for all types.
template <typename T> struct Vec8;
template <> struct Vec8<float> { typedef f32x8 type; };
template <> struct Vec8<f16_t> { typedef f16x8 type; };
template <> struct Vec8<bf16_t> { typedef bf16x8 type; };
template <typename T> using vec8 = typename Vec8<T>::type;

__device__ inline f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mma16(f32x8 a, f32x8 b, f32x4 c)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// Eight float32 values as three bfloat16 parts each, x = high + middle + low to 2^-24 of x: high is x cut off after 8
// bits, what is left is exact in float32, middle its rounding to 8 bits and low that of the exact rest.
struct Split8 {
    bf16x8 high, middle, low;

    __device__ Split8() {}
    __device__ explicit Split8(f32x8 x)
    {
        union Pairs { uint32_t pair[4]; bf16x8 whole; } h, m, l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            const uint32_t ah = __float_as_uint(a) & 0xffff0000u, bh = __float_as_uint(b) & 0xffff0000u;
            h.pair[i] = __builtin_amdgcn_perm(bh, ah, 0x07060302u);     // both high halves
            const float ar = a - __uint_as_float(ah), br = b - __uint_as_float(bh);
            m.pair[i] = round_pair(ar, br);
            l.pair[i] = round_pair(ar - __uint_as_float(m.pair[i] << 16), br - __uint_as_float(m.pair[i] & 0xffff0000u));
        }
        high = h.whole;
        middle = m.whole;
        low = l.whole;
    }
    __device__ static uint32_t round_pair(float a, float b)
    {
        typedef float two __attribute__((ext_vector_type(2)));
        typedef bf16_t half_two __attribute__((ext_vector_type(2)));
        union { half_two x; uint32_t bits; } u;
        u.x = __builtin_convertvector(two{a, b}, half_two);
        return u.bits;
    }
};

// What a 32-wide product takes for 8 values of type T. Float32 values are split: six bfloat16 products of 32 cycles
// give what eight float32 products of 64 do, but for the parts' products left out. A middle part is up to 2^-7 of its
// value (high is cut off, not rounded: rounded up it would leave float32's range), a low one up to 2^-16, so middle times
// low, twice, is up to 2^-22 of the product of two values; in the mean square of normal ones 2^-25.4, where a float32
// rounding is 2^-24 at most. Infinities split into NaN.
template <typename T> struct OperandOf { typedef vec8<T> type; };
template <> struct OperandOf<float> { typedef Split8 type; };
template <typename T> using Operand = typename OperandOf<T>::type;

__device__ inline f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x16 mma32(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ inline f32x16 mma32(f32x8 a, f32x8 b, f32x16 c)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
}
__device__ inline f32x16 mma32(const Split8 &a, const Split8 &b, f32x16 c)
{
    c = mma32(a.low, b.high, c);       // small terms first
    c = mma32(a.high, b.low, c);
    c = mma32(a.middle, b.middle, c);
    c = mma32(a.middle, b.high, c);
    c = mma32(a.high, b.middle, c);
    return mma32(a.high, b.high, c);
}
__device__ inline float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ inline float wave_sum(float x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

}  // namespace rvq
