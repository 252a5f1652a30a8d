// Windowed attention with sinks, forward pass.
//
//   x_ij = scale q_i . k_j over the keys j that query i sees,
//   w = softmax(x), out_i = sum_j w_ij v_j, lse_i = log sum_j exp(x_ij)
//
// Bound by the matrix cores, the LDS reads that feed them and the exponentials,
// all of about the same weight: 4 dim flops, 1 exponential a pair.
// Measured: 16384 queries, window 4096, 4 sinks, 16 heads of 128 over 4, bfloat16:
// 524 us, 997 TFLOP/s, where a large library product reaches 1250 (both at a
// clock that the power limit brings to about 1.9 GHz); matrix cores busy in 50%
// of the cycles, no LDS bank conflicts.
// A workgroup takes 128 queries of one head and clip, 32 a wavefront, and goes
// once over the keys they see: the sinks' tiles, then the window's, 64 keys a
// tile. With transposed products a lane keeps to one query:
//   S^T [key][query] = K Q^T, 32-wide products; Q stays in registers
//   O^T [dim][query] += V^T P^T
// so maxima and sums run inside a lane (and once with the lane 32 further), and
// the scores that a lane holds are, in order, the P^T operand of the second
// product: the keys of a V^T operand are numbered as the scores come out.
// While one tile is worked on, the next is on its way from global memory.
// Weights enter the second product in the inputs' type, rounded once: half a step
// of theirs beside the half step of the result (mean error in bfloat16 0.0017 to
// 0.0024 where the result's rounding alone gives 0.0015 to 0.0017; two parts a
// weight would double the second product). Their sum is of the unrounded ones. In
// float16 they are taken times 2^kShift, so that the many small ones beside a
// large one do not sink below its exponents: half a step is 2^-32 of the largest.
// Steps, on that case: one wavefront a row 95.5 ms; matrix products with V
// transposed in registers 0.81; V read across its rows in the LDS, rows copied
// there directly 0.68; copies from a scalar base address 0.60; a whole tile
// between branches 0.55; the queries' loads waited for before the loop 0.53.
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"
#include "attention_tiles.h"

namespace rvq {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;     // queries a workgroup
constexpr float kSlack = 8.0f;         // how far (powers of two) a score may exceed the running maximum

template <typename T, int kD>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
void forward_tiles(AttentionArgs a, float factor, int slots)
{
    typedef Feed<T, kD, kWaves> Keys;
    typedef typename Keys::Rows Rows;
    __shared__ __attribute__((aligned(16))) char s_mem[Keys::kBytes];
    constexpr float kShift = kNarrow<T> ? 15.0f - kSlack : 0.0f;      // weights are below 2^(kSlack + kShift)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, half = lane >> 5;
    // heads change fastest: with 8 of them or more, one chiplet sees the same heads' keys again and again; the
    // last queries of a clip, which see most, start first
    const int slot = slots - 1 - static_cast<int>(blockIdx.x / a.q_heads), head = blockIdx.x % a.q_heads;
    const int kv = head / (a.q_heads / a.kv_heads);
    const int clip = clip_of_slot(a.cu_q, a.n_clips, slot, kRows);
    int q0, nq, k0, nk;
    clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int i0 = (slot - (a.cu_q[clip] / kRows + clip)) * kRows;
    if (i0 < 0 || i0 >= nq) return;

    const int back = nk - nq;                               // position of query 0
    const int row = i0 + 32 * wave + c;                     // this lane's query
    const bool real = row < nq;
    const int p = row + back;
    const KeyRange range = keys_seen(i0 + back, min(i0 + kRows, nq) - 1 + back, a.window, a.sinks);
    // this wavefront's first and last position
    const int w_first = i0 + 32 * wave + back, w_last = min(i0 + 32 * wave + 31, nq - 1) + back;
    // positions above these are in the window of this query, of the wavefront's first and of its last
    const int p_low = below_window(p, a.window), w_low = below_window(w_first, a.window);
    const int w_high = below_window(w_last, a.window);

    const T *own = static_cast<const T *>(a.q.data) + static_cast<int64_t>(q0 + min(row, nq - 1)) * a.q.token + head * a.q.head;
    Operand<T> q[kD / 16];
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) q[t] = Operand<T>(load8(own + 16 * t + 8 * half));
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) arrive(q[t]);
    Keys feed(s_mem, a.k.token, a.v.token);
    const T *keys = static_cast<const T *>(a.k.data) + static_cast<int64_t>(k0) * a.k.token + kv * a.k.head;
    const T *values = static_cast<const T *>(a.v.data) + static_cast<int64_t>(k0) * a.v.token + kv * a.v.head;

    f32x16 o[kD / 32];
    float m, l;

    // One tile of keys. The buffer's number is a constant, so that LDS addresses are; markers and clean (the values
    // of a tile are rewritten) make the later passes.
    auto tile = [&](int t, auto buffer, auto markers, auto clean) {
        char *s_k = feed.tile_one(buffer), *s_v = feed.tile_two(buffer);
        feed.turn(buffer, t + 1 < range.tiles, keys, values, range.start(t + 1), nk);
        if (clean.value) {
            only_finite<Rows, kD, kThreads>(s_v, markers.value);
            __syncthreads();
        }
        const int j0 = range.start(t);
        // nothing of these keys is seen by this wavefront
        if (j0 > w_last || (j0 + kTileRows - 1 <= w_low && j0 >= a.sinks)) return;
        f32x16 x[2] = {};
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < kD / 16; ++n) x[b] = mma32(Rows::along(s_k, 32 * b + c, 2 * n + half), q[n], x[b]);
        if constexpr (clean.value && sizeof(T) == 4) {
            // scores that the split made NaN, again by float32 products: they may be infinite
            bool odd = false;
#pragma unroll
            for (int r = 0; r < 32; ++r) odd = odd || x[r >> 4][r & 15] != x[r >> 4][r & 15];
            if (__any(odd)) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    f32x16 y = {};
                    const T *key = keys + min(j0 + 32 * b + c, nk - 1) * a.k.token + 8 * half;
                    for (int n = 0; n < kD / 16; ++n) y = mma32(load8(key + 16 * n), load8(own + 16 * n + 8 * half), y);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[b][r] = x[b][r] != x[b][r] ? y[r] : x[b][r];
                }
            }
        }
        if (!(j0 + kTileRows - 1 <= w_first && (j0 > w_high || j0 + kTileRows - 1 < a.sinks))) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = j0 + 32 * b + 8 * (r >> 2) + 4 * half + (r & 3);
                    x[b][r] = j <= p && (j > p_low || j < a.sinks) ? x[b][r] : -INFINITY;
                }
        }
        float top = x[0][0];
#pragma unroll
        for (int r = 1; r < 32; ++r) top = fmaxf(top, x[r >> 4][r & 15]);
        top *= factor;
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            if (top > m + kSlack) {
                const float keep = fast_exp2(m - top);
                m = top;
                l *= keep;
                if (!markers.value) {
#pragma unroll
                    for (int n = 0; n < kD / 32; ++n) o[n] *= keep;
                }
            }
        }
        const float safe = m == -INFINITY ? 0.0f : m - kShift;
        float sum[4] = {};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            vec8<T> w[2];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float e = fast_exp2(__builtin_fmaf(x[b][r], factor, -safe));
                sum[r & 3] += e;
                if (markers.value) e = x[b][r] == -INFINITY ? 0.0f : 1.0f;
                w[r >> 3][r & 7] = static_cast<T>(e);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Operand<T> weights(w[s]);
#pragma unroll
                for (int n = 0; n < kD / 32; ++n) o[n] = mma32(Rows::across(s_v, n, 2 * b + s), weights, o[n]);
            }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (markers.value) {
            // counts of a tile and the one before stay below 1 / kMinus: whole and broken part apart
#pragma unroll
            for (int n = 0; n < kD / 32; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[n][r] = (o[n][r] >= 1.0f ? 1.0f : 0.0f) + (o[n][r] > floorf(o[n][r]) ? kMinus : 0.0f);
        }
    };
    auto pass = [&](auto markers, auto clean) {
        if (range.tiles > 0) feed.start(keys, values, range.start(0), nk);
#pragma unroll
        for (int n = 0; n < kD / 32; ++n) o[n] = f32x16{};
        m = -INFINITY;
        l = 0.0f;
        for (int t = 0; t < range.tiles; t += 2) {
            tile(t, Constant<0>{}, markers, clean);
            if (t + 1 < range.tiles) tile(t + 1, Constant<1>{}, markers, clean);
        }
    };

    pass(Constant<0>{}, Constant<0>{});
    bool odd = false;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) odd = odd || !(fabsf(o[n][r]) <= FLT_MAX);
    // Weights of unseen keys are 0, but 0 times a value that is not finite is not 0. So when a result is not finite, a
    // second pass finds, for every result, whether keys that are seen have an infinity of either sign there (a NaN is
    // both), and a third computes the results with these values taken as 0: results with one sign are that infinity,
    // with both NaN, the others are what they would be without the values that are not seen.
    if (__syncthreads_or(odd)) {
        pass(Constant<1>{}, Constant<1>{});
        uint32_t up[kD / 64] = {}, down[kD / 64] = {};
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                up[n >> 1] |= static_cast<uint32_t>(o[n][r] >= 1.0f) << (16 * (n & 1) + r);
                down[n >> 1] |= static_cast<uint32_t>(o[n][r] > floorf(o[n][r])) << (16 * (n & 1) + r);
            }
        __syncthreads();     // the tiles are no longer read
        pass(Constant<0>{}, Constant<1>{});
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const bool plus = up[n >> 1] >> (16 * (n & 1) + r) & 1, minus = down[n >> 1] >> (16 * (n & 1) + r) & 1;
                if (plus || minus) o[n][r] = plus && minus ? __builtin_nanf("") : plus ? INFINITY : -INFINITY;
            }
    }
    if (!real) return;
    l += __shfl_xor(l, 32);
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    T *out = static_cast<T *>(a.out.data) + static_cast<int64_t>(q0 + row) * a.out.token + head * a.out.head;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            T y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = static_cast<T>(o[n][4 * r + i] * inverse);
            store4(out + 32 * n + 8 * r + 4 * half, y);
        }
    if (a.lse && half == 0)
        a.lse[static_cast<int64_t>(head) * a.q_tokens + q0 + row] = l == 0.0f ? -INFINITY : (m - kShift + log2f(l)) * kLn2;
}

template <typename T, int kD>
hipError_t forward(const AttentionArgs &a, hipStream_t stream)
{
    const int64_t slots = a.q_tokens / kRows + a.n_clips + 1;
    if (!fits(slots * a.q_heads, kThreads)) return hipErrorNotSupported;
    // scale 0 (equal weights) becomes the smallest factor: 0 times the -inf of an unseen key does not arise
    const float factor = fmaxf(a.scale * kLog2e, FLT_MIN);
    forward_tiles<T, kD><<<static_cast<unsigned>(slots * a.q_heads), kThreads, 0, stream>>>(a, factor, static_cast<int>(slots));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_window_attention(const AttentionArgs &a, hipStream_t stream)
{
    if (a.dtype == RVQ_F32) return a.dim == 64 ? forward<float, 64>(a, stream) : forward<float, 128>(a, stream);
    if (a.dtype == RVQ_F16) return a.dim == 64 ? forward<f16_t, 64>(a, stream) : forward<f16_t, 128>(a, stream);
    return a.dim == 64 ? forward<bf16_t, 64>(a, stream) : forward<bf16_t, 128>(a, stream);
}

}  // namespace rvq
