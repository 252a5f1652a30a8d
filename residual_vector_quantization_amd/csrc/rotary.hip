// Rotary positions of packed query and key heads, alone or on the way into the
// paged cache.
//
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),  t = position * frequency of the pair
//
// and, as the gradient, the same with -t (a rotation's transpose). Bound by
// HBM: every value is read once and written once. Measured: 65,536 tokens of 16
// and 4 heads of 128 in bfloat16, out of a fused projection, 0.67 GB in 127 to
// 131 us, 5.1 to 5.3 TB/s, what a large copy reaches; 27,224 new frames of 32, 8 and 8 heads of 128
// turned and written into pages of 16, 0.67 GB in 134 us; the next frames of 96
// streams 5 us, the launch and three reads one after another.
// A thread keeps to one token and to the same pairs of every head it goes
// through, so that a pair's sine and cosine are made once for several heads;
// neighbouring threads have neighbouring heads (of the first case, 4 side by side:
// 153 us with one after another, 131 so). It takes 32 bytes of a head at a time, as two loads of 16:
// in the half layout these are the two partners of its pairs, 16 bytes of each
// half; in the interleaved one they are neighbours. What does not turn is
// copied by the other threads of the row.
// Angles: positions go up to 2^31, and a turn has to be known to 2^-26 or so, 2^-55 of
// what position * frequency can be in turns. So the frequency is taken in turns as
// the sum of two float64, and the product less its whole turns comes out of one
// fma, with 2^-53 of a turn left; quarters leave exactly, and the rest (an
// eighth of a turn at most) goes through
// the Taylor series of sine and cosine in float32; they are cut off where the
// next term is below 2^-28. Values turn in float32 and are rounded once.
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"

namespace rvq {
namespace {

constexpr int kThreads = 256;
constexpr int kStagedClips = 1023;     // clips up to which a workgroup brings the offsets into the LDS to search them
constexpr int kWantedGroups = 6144;    // workgroups up to which a token's heads are shared out among threads

struct Params {
    RotaryArgs a;
    int units, unit_shift;     // threads a head: one takes 32 bytes
    int apart, apart_shift;    // threads that share a token's heads; one takes every apart-th
    int tokens;                // tokens a workgroup
};

// cos and sin of 2 pi position f.
__device__ inline void turn(double position, double f, float &c, float &s)
{
    // f / 2 pi in two parts; the product with the position keeps what rounding would cut off
    const double high = f * 0x1.45f306dc9c883p-3;
    const double low = __builtin_fma(f, 0x1.45f306dc9c883p-3, -high) + f * -0x1.6b01ec5417056p-57;
    double t = __builtin_fma(position, high, -__builtin_rint(position * high)) + position * low;
    const double quarters = __builtin_rint(4.0 * t);
    const float x = static_cast<float>(__builtin_fma(quarters, -0.25, t)) * 6.283185307179586f;
    const float y = x * x;
    float sine = __builtin_fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
    sine = __builtin_fmaf(y, sine, 1.0f / 120.0f);
    sine = __builtin_fmaf(y, sine, -1.0f / 6.0f);
    sine = __builtin_fmaf(x * y, sine, x);
    float cosine = __builtin_fmaf(y, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    cosine = __builtin_fmaf(y, cosine, -1.0f / 720.0f);
    cosine = __builtin_fmaf(y, cosine, 1.0f / 24.0f);
    cosine = __builtin_fmaf(y, cosine, -0.5f);
    cosine = __builtin_fmaf(y, cosine, 1.0f);
    const int q = static_cast<int>(quarters);
    s = q & 1 ? cosine : sine;
    c = q & 1 ? sine : cosine;
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

// 16 bytes of a row.
template <typename T> struct Piece {
    static constexpr int kValues = 16 / sizeof(T);
    union {
        u32x4 whole;
        T x[kValues];
    };
    __device__ inline void load(const T *p) { whole = *reinterpret_cast<const u32x4 *>(p); }
    __device__ inline void store(T *p) const { *reinterpret_cast<u32x4 *>(p) = whole; }
};

// kAppend: keys and values go into the cache's pages. kPieces: pairs fill whole pieces (rot_dim is a multiple of 32
// bytes); otherwise values are taken one by one.
template <typename T, bool kAppend, bool kPieces, bool kNeighbours>
__global__ __launch_bounds__(kThreads)
void turn_heads(Params p)
{
    constexpr int kValues = Piece<T>::kValues;
    const RotaryArgs &a = p.a;
    __shared__ int32_t s_cu[kStagedClips + 1];
    const int unit = threadIdx.x & (p.units - 1), at = threadIdx.x >> p.unit_shift;
    const int first_head = at & (p.apart - 1);
    const int64_t token = static_cast<int64_t>(blockIdx.x) * p.tokens + (at >> p.apart_shift);
    const bool staged = a.cu && a.n_clips <= kStagedClips;
    if (staged) {
        for (int i = threadIdx.x; i <= a.n_clips; i += kThreads) s_cu[i] = a.cu[i];
        __syncthreads();
    }
    if (token >= a.n_tokens) return;
    const int pairs = a.rot_dim / 2;
    double f[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) f[i] = unit * kValues + i < pairs ? a.frequencies[unit * kValues + i] : 0.0;

    int64_t position, row = -1;      // row: the frame's place in the pools at head 0
    if (a.positions) {
        position = a.positions[token];
    } else {
        int clip = static_cast<int>(token), nth = 0;
        if (a.cu) {
            clip = clip_of_row(staged ? s_cu : a.cu, a.n_clips, static_cast<int>(token));
            nth = static_cast<int>(token) - (staged ? s_cu : a.cu)[clip];
            if (nth < 0 || token >= (staged ? s_cu : a.cu)[clip + 1]) return;      // outside every clip
        }
        position = (a.first ? static_cast<int64_t>(a.first[clip]) : 0) + nth;
        if (kAppend && position >= 0 && position < static_cast<int64_t>(a.table_ld) * a.page_size) {
            const int e = static_cast<int>(position) / a.page_size, slot = static_cast<int>(position) - e * a.page_size;
            const int page = a.table[static_cast<int64_t>(clip) * a.table_ld + e];
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
                row = static_cast<int64_t>(page) * a.kv_heads * a.page_size + slot;
        }
    }
    float c[kValues], s[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
        turn(static_cast<double>(position), f[i], c[i], s[i]);
        c[i] *= a.amplitude;
        s[i] *= a.inverse ? -a.amplitude : a.amplitude;
    }

    const T *q = static_cast<const T *>(a.q.data) + token * a.q.token;
    const T *k = static_cast<const T *>(a.k.data) + token * a.k.token;
    T *q_out = static_cast<T *>(a.q_out.data) + token * a.q_out.token;
    const int heads = a.q_heads + (kAppend ? (row < 0 ? 0 : 2 * a.kv_heads) : a.kv_heads);
    const bool turns = unit * kValues < pairs;      // with kPieces: this thread's values turn, or none of them
    // of the two pieces
    const int one = !turns || kNeighbours ? 2 * kValues * unit : kValues * unit;
    const int two = !turns || kNeighbours ? one + kValues : pairs + kValues * unit;
    // a row that stays in its place needs no copy of what does not turn
    const bool copies = turns || !(a.q_out.data == a.q.data);
    const bool k_copies = turns || kAppend || !(a.k_out.data == a.k.data);
    // where head h is and goes; false: it stays as it is
    auto place = [&](int h, const T *&from, T *&to, bool &still) {
        still = false;
        if (h < a.q_heads) {
            from = q + h * a.q.head;
            to = q_out + h * a.q_out.head;
            return !kPieces || copies;
        }
        if (!kAppend) {
            from = k + (h - a.q_heads) * a.k.head;
            to = static_cast<T *>(a.k_out.data) + token * a.k_out.token + (h - a.q_heads) * a.k_out.head;
            return !kPieces || k_copies;
        }
        still = h >= a.q_heads + a.kv_heads;        // a value row
        const int kv = h - a.q_heads - (still ? a.kv_heads : 0);
        from = still ? static_cast<const T *>(a.v.data) + token * a.v.token + kv * a.v.head : k + kv * a.k.head;
        to = static_cast<T *>(still ? a.v_pool : a.k_pool) + (row + static_cast<int64_t>(kv) * a.page_size) * a.dim;
        return true;
    };
    if constexpr (kPieces) {
        for (int h = first_head; h < heads; h += p.apart) {
            const T *from;
            T *to;
            bool still;
            if (!place(h, from, to, still)) continue;
            Piece<T> x, y;
            x.load(from + one);
            y.load(from + two);
            if (turns && !still) {
                float v[2 * kValues];
#pragma unroll
                for (int i = 0; i < kValues; ++i) {
                    const Piece<T> &z = kNeighbours && i >= kValues / 2 ? y : x;
                    const float u = to_float(z.x[kNeighbours ? 2 * i % kValues : i]);
                    const float w = to_float(kNeighbours ? z.x[2 * i % kValues + 1] : y.x[i]);
                    v[kNeighbours ? 2 * i : i] = __builtin_fmaf(u, c[i], -(w * s[i]));
                    v[kNeighbours ? 2 * i + 1 : kValues + i] = __builtin_fmaf(w, c[i], u * s[i]);
                }
#pragma unroll
                for (int i = 0; i < kValues; ++i) {
                    x.x[i] = static_cast<T>(v[i]);
                    y.x[i] = static_cast<T>(v[kValues + i]);
                }
            }
            x.store(to + one);
            y.store(to + two);
        }
    } else {
        for (int h = first_head; h < heads; h += p.apart) {
            const T *from;
            T *to;
            bool still;
            place(h, from, to, still);
            const int n = still ? 0 : pairs;       // pairs of this row; the values behind them are copied
#pragma unroll
            for (int i = 0; i < kValues; ++i) {
                const int pair = unit * kValues + i;
                if (pair >= n) break;
                const int d0 = kNeighbours ? 2 * pair : pair, d1 = kNeighbours ? d0 + 1 : pairs + pair;
                const float u = to_float(from[d0]), w = to_float(from[d1]);
                to[d0] = static_cast<T>(__builtin_fmaf(u, c[i], -(w * s[i])));
                to[d1] = static_cast<T>(__builtin_fmaf(w, c[i], u * s[i]));
            }
            for (int d = 2 * n + unit; d < a.dim; d += p.units) to[d] = from[d];
        }
    }
}

template <typename T, bool kAppend>
hipError_t run(Params p, hipStream_t stream)
{
    const RotaryArgs &a = p.a;
    constexpr int kValues = Piece<T>::kValues;
    p.units = a.dim / (2 * kValues);
    while ((1 << p.unit_shift) < p.units) ++p.unit_shift;
    // Every thread makes the sines of its pairs, as much work as several heads' rotations: a token's heads are shared
    // out among no more threads than it takes to fill the chip several times over.
    const int heads = a.q_heads + (kAppend ? 2 : 1) * a.kv_heads, most = kThreads / p.units;
    p.apart = 1;
    while (p.apart < heads && p.apart < most && a.n_tokens * p.units * p.apart < static_cast<int64_t>(kWantedGroups) * kThreads) {
        p.apart *= 2;
        ++p.apart_shift;
    }
    p.tokens = kThreads / (p.units * p.apart);
    const int64_t groups = (a.n_tokens + p.tokens - 1) / p.tokens;
    if (!fits(groups, kThreads)) return hipErrorNotSupported;
    const bool pieces = a.rot_dim % (2 * kValues) == 0;
    const unsigned n = static_cast<unsigned>(groups);
    if (pieces && a.interleaved) turn_heads<T, kAppend, true, true><<<n, kThreads, 0, stream>>>(p);
    else if (pieces) turn_heads<T, kAppend, true, false><<<n, kThreads, 0, stream>>>(p);
    else if (a.interleaved) turn_heads<T, kAppend, false, true><<<n, kThreads, 0, stream>>>(p);
    else turn_heads<T, kAppend, false, false><<<n, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool kAppend>
hipError_t launch(const RotaryArgs &a, hipStream_t stream)
{
    Params p = {};
    p.a = a;
    if (a.dtype == RVQ_F32) return run<float, kAppend>(p, stream);
    if (a.dtype == RVQ_F16) return run<f16_t, kAppend>(p, stream);
    return run<bf16_t, kAppend>(p, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream) { return launch<false>(a, stream); }

hipError_t launch_rotary_append(const RotaryArgs &a, hipStream_t stream) { return launch<true>(a, stream); }

}  // namespace rvq
