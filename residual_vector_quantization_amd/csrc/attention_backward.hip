// Gradient of the windowed attention with sinks.
//
//   x_ij = scale q_i . k_j,  w_ij = exp(x_ij - lse_i),  delta_i = dout_i . out_i
//   dw_ij = dout_i . v_j,  dx_ij = w_ij (dw_ij - delta_i)
//   dq_i = scale sum_j dx_ij k_j,  dk_j = scale sum_i dx_ij q_i,  dv_j = sum_i w_ij dout_i
//
// Two main launches and no atomics, so the sums' order is fixed: dq and the rows'
// delta (queries in registers, keys go by), dk and dv (keys in registers, queries
// go by, all query heads of a key head one after another); a small one before them
// in float16, and one behind them where dk and dv come in parts (both below). Scores
// and dw are made twice, 14 dim flops a pair with the forward pass' 4 make 18 where
// 14 would do; in exchange no partial dq goes through memory.
// Bound by the matrix cores and the LDS reads that feed them, as in the
// forward pass, with the same operand layouts: a lane keeps to one query (dq)
// or one key (dk, dv), and what a product leaves in it is the next one's operand.
// Measured: two clips of up to 8192 frames, window 750, 4 sinks, 16 heads of 128
// over 4, bfloat16: dq 204 us (matrix cores busy 32% of the cycles), dk and dv
// 286 us (27%; accumulators and operands take 400 registers, so 1 wavefront a
// SIMD, and exponentials are not hidden behind another's products), sinks 6 us.
// 8 clips of 2000 frames, all seen, 16 heads of 64 over 8, float16: 145 and 211 us.
//
// Weights and dx enter the products in the inputs' type. bfloat16 has float32's
// range, but float16 has 5 bits of exponent, so there weights are taken times
// 2^14 and dx times 2^14 over a power of two that bounds |dw - delta|: no value
// can overflow, and those down to 2^-28 of the bound keep all their bits.
//   dq: |dw_ij - delta_i| <= 2 |dout_i| |v|, the largest |v| of the keys gone over
//     (a launch before the two finds it for every 128 keys, 16 MB of values in 5 us;
//     a small call of 36 us takes 3 us longer by it);
//   dk: |dw_ij - delta_i| <= |dout| |v_j| + |delta|, the largest |dout| and |delta| of
//     the rows gone over (from dq_tiles). A lane keeps to one key, so it may have
//     its own factor.
// The factors leave again in float32 at the end; powers of two change no rounding.
//
// delta comes from the rounded out. Its error enters dx as (1 / number of keys
// that matter) of the size of dx's own rounding squared, so it shows only where
// few keys do. Where queries see few (kFewKeys) dq_tiles first goes over the keys
// for sum_j w_ij (dw_ij - delta_i), which is what delta lacks, and corrects it,
// for the keys' gradients as well. Small windows in float16, error of dq and dk
// over that of a correct result rounded once: 1.52 without, 1.41 with (two
// roundings); over windows of 2 to 600 frames 1.39 to 1.47. Queries that see many
// keys and give their weight to few keep delta's error (the additional pass would
// cost two thirds of dq's time): 600 frames, all seen, scores of N(0, 1) times 1,
// 2.4, 4, 8 and 16: 1.41, 1.65, 2.2, 3.1 and 3.8.
//
// Where keys and key heads make few workgroups, the query heads of a key head
// are shared out among several (parts_of), and a further launch adds their float32
// sums in order.
//
// The first sinks of a clip are seen by all of its later queries, hundreds of
// tiles where other keys have a window's. When that matters (see split_sinks)
// the queries beyond the window go in pieces of kFarRows to workgroups of their
// own, and a further launch adds the float32 parts in order.
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
constexpr int kRows = 32 * kWaves;      // queries (dq) or keys (dk, dv) a workgroup
constexpr int kFewKeys = 128;           // keys up to which delta is corrected
constexpr int kFarRows = 256;           // queries of a piece beyond the window
constexpr int kLongClip = 2048;         // average clip from which the sinks are split off
constexpr int kMaxSplitSinks = 64;

// Workspace: lse in powers of two (less kWeightShift in float16; +inf for rows that see nothing, so that their weights
// are 0) and -delta a query and head, then the float32 parts of the sinks' gradients, { dk, dv } [sinks][dim] each.
struct Work {
    float *lse2, *minus_delta;     // [q_heads][q_tokens]
    float *largest;          // float16: [q_heads][q_slots] the largest |dout| and |delta| of the rows of dq_tiles' workgroups
    float *values;           // float16: [kv_heads][k_slots] the largest |v| of 128 keys
    int q_slots, k_slots;
    float *near;             // [n_clips][kv_heads]
    float *far;              // [far slots][kv_heads][2]
    bool split;
    float *part;                   // [parts][k_tokens][kv_heads] where parts > 1, laid out as near
    int parts;
};

int64_t rounded(int64_t floats) { return (floats + 3) / 4 * 4; }

int64_t far_slots(int64_t q_tokens, int n_clips) { return q_tokens / kFarRows + n_clips + 1; }

// Sinks are split off where clips are long on average: short ones have too few queries for their sinks to last
// longer than the rest.
bool split_sinks(int64_t q_tokens, int n_clips, int sinks)
{
    return sinks > 0 && sinks <= kMaxSplitSinks && q_tokens >= static_cast<int64_t>(n_clips) * kLongClip;
}

int64_t k_slots(int64_t k_tokens, int n_clips) { return k_tokens / kRows + n_clips + 1; }

// Among how many workgroups the query heads of a key head are shared out: as many as fill the chip's 256 CUs twice, if
// each has some 32 tiles of queries to go over (a float32 tile counts as 3); otherwise the additional launch (4 us, and
// as much for the sums) is not made up for. Forward and gradient, us: 8 query heads over 1 of 64, 1500 frames, 295 ->
// 99; 4 clips of up to 600, 8 heads over 1 of 128, 207 -> 85; 8 clips of up to 300, 8 over 4 of 64, 43 against 55 if
// shared. Not where the sinks are split off.
int parts_of(const AttentionArgs &a)
{
    if (split_sinks(a.q_tokens, a.n_clips, a.sinks) || a.n_clips == 0) return 1;
    const int group = a.q_heads / a.kv_heads;
    const int64_t length = a.k_tokens / a.n_clips, seen = static_cast<int64_t>(a.window) + kRows;
    const int64_t tiles = ((length < seen ? length : seen) / kTileRows + 1) * group;
    if (tiles * (a.dtype == RVQ_F32 ? 3 : 1) < 32) return 1;
    const int64_t n = 512 / (k_slots(a.k_tokens, a.n_clips) * a.kv_heads);
    return n < 2 ? 1 : n < group ? static_cast<int>(n) : group;
}

int64_t q_slots(int64_t q_tokens, int n_clips) { return q_tokens / kRows + n_clips + 1; }

int64_t work_floats(const AttentionArgs &a)
{
    int64_t n = 2 * rounded(a.q_tokens * a.q_heads);
    if (a.dtype == RVQ_F16)
        n += rounded(2 * q_slots(a.q_tokens, a.n_clips) * a.q_heads) + rounded(k_slots(a.k_tokens, a.n_clips) * a.kv_heads);
    if (split_sinks(a.q_tokens, a.n_clips, a.sinks))
        n += (a.n_clips + 2 * far_slots(a.q_tokens, a.n_clips)) * a.kv_heads * a.sinks * a.dim * 2;
    const int parts = parts_of(a);
    if (parts > 1) n += parts * a.k_tokens * a.kv_heads * a.dim * 2;
    return n;
}

Work work_of(const AttentionArgs &a)
{
    Work w;
    w.lse2 = static_cast<float *>(a.workspace);
    w.minus_delta = w.lse2 + rounded(a.q_tokens * a.q_heads);
    w.largest = w.minus_delta + rounded(a.q_tokens * a.q_heads);
    w.q_slots = static_cast<int>(q_slots(a.q_tokens, a.n_clips));
    w.k_slots = static_cast<int>(k_slots(a.k_tokens, a.n_clips));
    const bool narrow = a.dtype == RVQ_F16;
    w.values = w.largest + (narrow ? rounded(static_cast<int64_t>(2) * w.q_slots * a.q_heads) : 0);
    w.near = w.values + (narrow ? rounded(static_cast<int64_t>(w.k_slots) * a.kv_heads) : 0);
    w.far = w.near + static_cast<int64_t>(a.n_clips) * a.kv_heads * a.sinks * a.dim * 2;
    w.split = a.window != INT_MAX && split_sinks(a.q_tokens, a.n_clips, a.sinks);
    w.part = w.near;               // never both
    w.parts = parts_of(a);
    return w;
}

constexpr float kWeightShift = 14.0f;                      // float16 weights are taken times 2^this

__device__ inline bool not_finite(float x) { return !(fabsf(x) <= FLT_MAX); }

// e with 2^(e - 1) <= x < 2^e, 0 for x = 0 and values that are not finite.
__device__ inline int exponent_of(float x) { return x == 0.0f || not_finite(x) ? 0 : __builtin_amdgcn_frexp_expf(x); }

__device__ inline float finite_or_0(float x) { return not_finite(x) ? 0.0f : x; }

__device__ inline float wave_max(float x)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}

template <typename V>
__device__ inline float square_sum(V x)
{
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += to_float(x[i]) * to_float(x[i]);
    return sum;
}

// float16: the largest finite |v| (as a vector's length) of every 128 keys of a clip and key head.
template <typename T, int kD>
__global__ __launch_bounds__(kThreads)
void value_sizes(AttentionArgs a, Work work)
{
    constexpr int kLanes = kD / 8, kStep = kThreads / kLanes;      // lanes a row, rows at a time
    __shared__ float s_top[kWaves];
    const int slot = blockIdx.x / a.kv_heads, kv = blockIdx.x % a.kv_heads;
    const int clip = clip_of_slot(a.cu_k, a.n_clips, slot, kRows);
    int k0, nk;
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int first = (slot - (a.cu_k[clip] / kRows + clip)) * kRows;
    if (first < 0 || first >= nk) return;
    const T *rows = static_cast<const T *>(a.v.data) + static_cast<int64_t>(k0 + first) * a.v.token + kv * a.v.head;
    const int at = threadIdx.x / kLanes, end = min(kRows, nk - first);
    float top = 0.0f;
#pragma unroll
    for (int n = 0; n < kRows / kStep; ++n) {
        const int row = n * kStep + at;
        float sum = square_sum(load8(rows + min(row, end - 1) * a.v.token + threadIdx.x % kLanes * 8));
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) sum += __shfl_xor(sum, m);
        top = fmaxf(top, finite_or_0(sum));
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0)
        work.values[static_cast<int64_t>(kv) * work.k_slots + slot] = sqrtf(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])));
}

// dq, and lse2 and delta of the rows. As in the forward pass a workgroup takes 128 queries and goes over the tiles of
// keys they see. If a result is not finite, a second pass takes rows of K that are not finite as zeros and the weights of
// the queries that do see them as NaN, so that only those get it.
template <typename T, int kD>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? (kD == 64 ? 3 : 2) : 1)
void dq_tiles(AttentionArgs a, Work work, float factor)
{
    typedef Feed<T, kD, kWaves> Keys;
    typedef typename Keys::Rows Rows;
    __shared__ __attribute__((aligned(16))) char s_mem[Keys::kBytes];
    __shared__ int s_bad[kTileRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int slot = work.q_slots - 1 - static_cast<int>(blockIdx.x / a.q_heads), head = blockIdx.x % a.q_heads;
    const int kv = head / (a.q_heads / a.kv_heads);
    const int clip = clip_of_slot(a.cu_q, a.n_clips, slot, kRows);
    int q0, nq, k0, nk;
    clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int i0 = (slot - (a.cu_q[clip] / kRows + clip)) * kRows;
    if (i0 < 0 || i0 >= nq) return;

    const int back = nk - nq;
    const int row = i0 + 32 * wave + c;
    const int p = row + back;
    const KeyRange range = keys_seen(i0 + back, min(i0 + kRows, nq) - 1 + back, a.window, a.sinks);
    const int w_first = i0 + 32 * wave + back, w_last = min(i0 + 32 * wave + 31, nq - 1) + back;
    const int p_low = below_window(p, a.window), w_low = below_window(w_first, a.window);
    const int w_high = below_window(w_last, a.window);
    const int64_t at = q0 + min(row, nq - 1);

    const T *own_q = static_cast<const T *>(a.q.data) + at * a.q.token + head * a.q.head + 8 * half;
    const T *own_g = static_cast<const T *>(a.dout.data) + at * a.dout.token + head * a.dout.head + 8 * half;
    const T *own_o = static_cast<const T *>(a.out.data) + at * a.out.token + head * a.out.head + 8 * half;
    Operand<T> q[kD / 16], g[kD / 16];
    float lse2 = a.lse[head * a.q_tokens + at], minus_delta = 0.0f, unshift = 1.0f;
    lse2 = lse2 == -INFINITY ? INFINITY : lse2 * kLog2e - (kNarrow<T> ? kWeightShift : 0.0f);
    float size = 0.0f;      // |dout| of the row, squared at first
    vec8<T> rows[3][kD / 16];
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
        rows[0][t] = load8(own_q + 16 * t);
        rows[1][t] = load8(own_g + 16 * t);
        rows[2][t] = load8(own_o + 16 * t);
    }
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
        q[t] = Operand<T>(rows[0][t]);
        g[t] = Operand<T>(rows[1][t]);
        arrive(q[t]);
        arrive(g[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) minus_delta -= to_float(rows[1][t][i]) * to_float(rows[2][t][i]);
        if constexpr (kNarrow<T>) size += square_sum(rows[1][t]);
    }
    minus_delta += __shfl_xor(minus_delta, 32);
    if (half == 0 && row < nq) work.lse2[head * a.q_tokens + at] = lse2;
    if constexpr (kNarrow<T>) {
        __shared__ float s_top[2][kWaves];
        float value = 0.0f;
        const float *values = work.values + static_cast<int64_t>(kv) * work.k_slots + k0 / kRows + clip;
#pragma unroll 4
        for (int t = lane; t < range.tiles; t += 64) value = fmaxf(value, values[range.start(t) / kRows]);
        value = wave_max(value);
        size = sqrtf(size + __shfl_xor(size, 32));
        const float e = static_cast<float>(exponent_of(2.0f * size * value));
        lse2 += e;
        unshift = fast_exp2(e - kWeightShift);
        s_top[0][wave] = wave_max(finite_or_0(size));
        s_top[1][wave] = wave_max(finite_or_0(fabsf(minus_delta)));
        __syncthreads();
        if (threadIdx.x < 2) {
            const float *top = s_top[threadIdx.x];
            work.largest[2 * (static_cast<int64_t>(head) * work.q_slots + slot) + threadIdx.x] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        }
    }
    Keys feed(s_mem, a.k.token, a.v.token);
    const T *keys = static_cast<const T *>(a.k.data) + static_cast<int64_t>(k0) * a.k.token + kv * a.k.head;
    const T *values = static_cast<const T *>(a.v.data) + static_cast<int64_t>(k0) * a.v.token + kv * a.v.head;

    f32x16 dq[kD / 32];
    float lack = 0.0f;
    // One tile of keys; buffer and pass are constants: 0 the usual one, 1 the one after a result that is not finite,
    // 2 the one that finds what delta lacks.
    auto tile = [&](int t, auto buffer, auto which) {
        constexpr bool second = which.value == 1;
        char *s_k = feed.tile_one(buffer), *s_v = feed.tile_two(buffer);
        feed.turn(buffer, t + 1 < range.tiles, keys, values, range.start(t + 1), nk);
        if (second) {
            if (threadIdx.x < kTileRows) s_bad[threadIdx.x] = 0;
            __syncthreads();
            clear_bad_rows<Rows, kD, kThreads>(s_k, s_bad);
            __syncthreads();
        }
        const int j0 = range.start(t);
        if (j0 > w_last || (j0 + kTileRows - 1 <= w_low && j0 >= a.sinks)) return;
        const bool whole = j0 + kTileRows - 1 <= w_first && (j0 > w_high || j0 + kTileRows - 1 < a.sinks);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x16 x = {}, y = {};
#pragma unroll
            for (int n = 0; n < kD / 16; ++n) {
                x = mma32(Rows::along(s_k, 32 * b + c, 2 * n + half), q[n], x);
                y = mma32(Rows::along(s_v, 32 * b + c, 2 * n + half), g[n], y);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                y[r] = fast_exp2(__builtin_fmaf(x[r], factor, -lse2)) * (y[r] + minus_delta);
                if (second && s_bad[32 * b + 8 * (r >> 2) + 4 * half + (r & 3)]) y[r] = __builtin_nanf("");
            }
            if (!whole) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = j0 + 32 * b + 8 * (r >> 2) + 4 * half + (r & 3);
                    y[r] = j <= p && (j > p_low || j < a.sinks) ? y[r] : 0.0f;
                }
            }
            if constexpr (which.value == 2) {
#pragma unroll
                for (int r = 0; r < 16; ++r) lack += y[r];
                continue;
            }
            vec8<T> w[2];
#pragma unroll
            for (int r = 0; r < 16; ++r) w[r >> 3][r & 7] = static_cast<T>(y[r]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Operand<T> weights(w[s]);
#pragma unroll
                for (int n = 0; n < kD / 32; ++n) dq[n] = mma32(Rows::across(s_k, n, 2 * b + s), weights, dq[n]);
            }
        }
    };
    auto pass = [&](auto which) {
        if (range.tiles > 0) feed.start(keys, values, range.start(0), nk);
#pragma unroll
        for (int n = 0; n < kD / 32; ++n) dq[n] = f32x16{};
        for (int t = 0; t < range.tiles; t += 2) {
            tile(t, Constant<0>{}, which);
            if (t + 1 < range.tiles) tile(t + 1, Constant<1>{}, which);
        }
    };
    if (sizeof(T) == 2 && min(static_cast<int64_t>(a.window) + a.sinks, static_cast<int64_t>(min(i0 + kRows, nq) + back)) <= kFewKeys) {
        pass(Constant<2>{});
        lack += __shfl_xor(lack, 32);
        minus_delta -= lack * unshift;
        __syncthreads();     // the tiles are no longer read
    }
    if (half == 0 && row < nq) work.minus_delta[head * a.q_tokens + at] = minus_delta;
    pass(Constant<0>{});
    bool odd = false;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) odd = odd || not_finite(dq[n][r]);
    if (__syncthreads_or(odd)) pass(Constant<1>{});
    if (row >= nq) return;
    T *out = static_cast<T *>(a.dq.data) + at * a.dq.token + head * a.dq.head;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            T e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = static_cast<T>(dq[n][4 * r + i] * (a.scale * unshift));
            store4(out + 32 * n + 8 * r + 4 * half, e);
        }
}

// dk and dv. A workgroup takes 128 keys of a key head, 32 a wavefront, and goes over the queries that see them, one
// query head after another. kFar: the sinks with the queries beyond the first keys' window, kFarRows of them; the
// wavefronts share the sinks (32 each) and take half of a tile's queries each.
template <typename T, int kD, bool kFar>
__device__ inline void dkv_group(const AttentionArgs &a, const Work &work, float factor, int block, char *s_mem,
                                 float (&s_stats)[2][2][kTileRows], int *s_bad)
{
    typedef Feed<T, kD, kWaves> Queries;
    typedef typename Queries::Rows Rows;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, half = lane >> 5;
    const int parts = kFar ? 1 : work.parts, part = block % parts;
    const int slot = block / parts / a.kv_heads, kv = block / parts % a.kv_heads, group = a.q_heads / a.kv_heads;
    const int first_head = kv * group + group * part / parts, heads = kv * group + group * (part + 1) / parts - first_head;
    const int32_t *cu = kFar ? a.cu_q : a.cu_k;
    constexpr int kPer = kFar ? kFarRows : kRows;
    const int clip = clip_of_slot(cu, a.n_clips, slot, kPer);
    int q0, nq, k0, nk;
    clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int64_t first = (slot - (cu[clip] / kPer + clip)) * static_cast<int64_t>(kPer);
    if (first < 0 || first >= (kFar ? nq : nk) || nk == 0) return;

    const int back = nk - nq;
    const int j_tile = kFar ? 0 : static_cast<int>(first);       // the workgroup's first key
    const int key = j_tile + (kFar ? 32 * (wave >> 1) : 32 * wave) + c;
    // positions that see the workgroup's keys: below near_end through the window, all later ones see the sinks
    const int near_end = static_cast<int>(min(static_cast<int64_t>(nk), static_cast<int64_t>(j_tile) + kRows - 1 + a.window));
    int i_first, i_end, hi = 0;       // queries gone over; position below which this lane's key is seen
    if (kFar) {
        i_first = max(static_cast<int>(first), near_end - back);
        i_end = static_cast<int>(min(static_cast<int64_t>(nq), first + kFarRows));
        if (key < min(a.sinks, nk)) hi = nk;
    } else {
        const bool all = !work.split && j_tile < a.sinks;
        i_first = max(0, j_tile - back);
        i_end = (all ? nk : near_end) - back;
        if (key < nk) hi = static_cast<int>(min(static_cast<int64_t>(all && key < a.sinks ? INT_MAX : static_cast<int64_t>(key) + a.window), static_cast<int64_t>(nk)));
        // with the sinks split off, their queries up to near_end still belong here
        if (work.split && key < min(a.sinks, nk)) hi = near_end;
    }
    const int i_start = i_first / kTileRows * kTileRows;
    const int per_head = i_end > i_first ? (i_end - i_start + kTileRows - 1) / kTileRows : 0;
    const int tiles = per_head * heads;
    const int key_first = __builtin_amdgcn_readfirstlane(key - c), key_last = key_first + 31;
    // below this position all of the wavefront's keys are seen, from the other on none
    int hi_all = hi, hi_any = hi;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        hi_all = min(hi_all, __shfl_xor(hi_all, m));
        hi_any = max(hi_any, __shfl_xor(hi_any, m));
    }
    hi_all = __builtin_amdgcn_readfirstlane(hi_all);     // the same in both halves of the wavefront
    hi_any = __builtin_amdgcn_readfirstlane(hi_any);

    const int64_t own = k0 + min(key, nk - 1);
    const T *own_k = static_cast<const T *>(a.k.data) + own * a.k.token + kv * a.k.head + 8 * half;
    const T *own_v = static_cast<const T *>(a.v.data) + own * a.v.token + kv * a.v.head + 8 * half;
    Queries feed(s_mem, a.q.token, a.dout.token);
    const T *queries = static_cast<const T *>(a.q.data) + static_cast<int64_t>(q0) * a.q.token;
    const T *slopes_of = static_cast<const T *>(a.dout.data) + static_cast<int64_t>(q0) * a.dout.token;
    auto load_stats = [&](int buffer, int head, int i) {
        if (wave < 2)
            copy4((wave ? work.minus_delta : work.lse2) + head * a.q_tokens + q0 + i, 4 * min(lane, nq - 1 - i), s_stats[buffer][wave]);
    };

    // The keys' and values' operands stay in registers, but for float32 values of dim 128: with as many registers of
    // accumulators beside them they come from the caches in every tile (the compiler would put some of them into
    // scratch memory and fetch them from there).
    constexpr bool kKeep = sizeof(T) == 2 || kD == 64;
    // 16-bit operands are read from the LDS well ahead of their products: those along the rows all at once, those across
    // them before the exponentials (dim 128 with 1 wavefront a SIMD 302 -> 282 us, dim 64 with 2 237 -> 221 us). Split
    // float32 operands would take three times the registers.
    constexpr bool kAhead = sizeof(T) == 2;
    Operand<T> k[kD / 16], v[kKeep ? kD / 16 : 1];
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
        k[t] = Operand<T>(load8(own_k + 16 * t));
        if constexpr (kKeep) v[t] = Operand<T>(load8(own_v + 16 * t));
    }
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
        arrive(k[t]);
        if constexpr (kKeep) arrive(v[t]);
    }
    // float16: dw - delta times `small`, weights times 2^kWeightShift
    float small = 1.0f, unit_v = 1.0f;
    if constexpr (kNarrow<T>) {
        // the rows gone over, in the slots that dq_tiles took them by
        const int slot0 = q0 / kRows + clip + i_first / kRows, slots = per_head > 0 ? (i_end - 1) / kRows - i_first / kRows + 1 : 0;
        float size = 0.0f, delta = 0.0f, value = 0.0f;
#pragma unroll 4
        for (int n = lane; n < slots * heads; n += 64) {
            const int h = n / slots;
            const float *top = work.largest + 2 * (static_cast<int64_t>(first_head + h) * work.q_slots + slot0 + n - h * slots);
            size = fmaxf(size, top[0]);
            delta = fmaxf(delta, top[1]);
        }
#pragma unroll
        for (int t = 0; t < kD / 16; ++t) value += square_sum(v[t]);
        value = finite_or_0(sqrtf(value + __shfl_xor(value, 32)));
        small = fast_exp2(static_cast<float>(-exponent_of(wave_max(size) * value + wave_max(delta))));
        unit_v = fast_exp2(-kWeightShift);
    }
    f32x16 dk[kD / 32], dv[kD / 32];
    int head, i;     // of the next tile to load
    // One tile of queries; buffer and pass are constants.
    auto tile = [&](int t, int i_tile, auto buffer, auto second) {
        typedef Operand<T> Op;
        char *s_q = feed.tile_one(buffer), *s_g = feed.tile_two(buffer);
        feed.turn(buffer, t + 1 < tiles, queries + head * a.q.head, slopes_of + head * a.dout.head, i, nq);
        if (t + 1 < tiles) load_stats(1 - buffer.value, head, i);
        if (second.value) {
            if (threadIdx.x < kTileRows) s_bad[threadIdx.x] = 0;
            __syncthreads();
            clear_bad_rows<Rows, kD, kThreads>(s_q, s_bad);
            clear_bad_rows<Rows, kD, kThreads>(s_g, s_bad);
            __syncthreads();
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int p0 = i_tile + 32 * b + back;       // position of the first of these 32 queries
            if (p0 + 31 < key_first || p0 >= hi_any) continue;
            if (kFar && (b != (wave & 1) || p0 + 31 < i_first + back)) continue;
            f32x16 x = {}, y;
            f32x4 lse2[4];
            Op tg[2][kAhead ? kD / 32 : 1], tq[2][kAhead ? kD / 32 : 1];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int in = 32 * b + 8 * f + 4 * half;
                lse2[f] = *reinterpret_cast<const f32x4 *>(&s_stats[buffer.value][0][in]);
                const f32x4 minus_delta = *reinterpret_cast<const f32x4 *>(&s_stats[buffer.value][1][in]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 * f + e] = minus_delta[e];     // dw - delta comes out of the product
            }
            if constexpr (kAhead) {
                Op aq[kD / 16], ag[kD / 16];
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) {
                    aq[n] = Rows::along(s_q, 32 * b + c, 2 * n + half);
                    ag[n] = Rows::along(s_g, 32 * b + c, 2 * n + half);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) {
                    x = mma32(aq[n], k[n], x);
                    y = mma32(ag[n], v[n], y);
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int n = 0; n < kD / 32; ++n) {
                        tg[s][n] = Rows::across(s_g, n, 2 * b + s);
                        tq[s][n] = Rows::across(s_q, n, 2 * b + s);
                    }
                __builtin_amdgcn_sched_barrier(0);
            } else {
#pragma unroll
                for (int n = 0; n < kD / 16; ++n) {
                    x = mma32(Rows::along(s_q, 32 * b + c, 2 * n + half), k[n], x);
                    if constexpr (kKeep) y = mma32(Rows::along(s_g, 32 * b + c, 2 * n + half), v[n], y);
                    else y = mma32(Rows::along(s_g, 32 * b + c, 2 * n + half), Op(load8(own_v + 16 * n)), y);
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                x[r] = fast_exp2(__builtin_fmaf(x[r], factor, -lse2[r >> 2][r & 3]));
                y[r] = x[r] * (kNarrow<T> ? y[r] * small : y[r]);
                if (second.value && s_bad[32 * b + 8 * (r >> 2) + 4 * half + (r & 3)]) x[r] = y[r] = __builtin_nanf("");
            }
            if (kFar || !(p0 >= key_last && p0 + 31 < hi_all)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int p = p0 + 8 * (r >> 2) + 4 * half + (r & 3);
                    bool sees = p >= key && p < hi;
                    if (kFar) sees = sees && p - back >= i_first && p - back < i_end;
                    x[r] = sees ? x[r] : 0.0f;
                    y[r] = sees ? y[r] : 0.0f;
                }
            }
            vec8<T> w[2], d[2];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                w[r >> 3][r & 7] = static_cast<T>(x[r]);
                d[r >> 3][r & 7] = static_cast<T>(y[r]);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Op weights(w[s]), slopes(d[s]);
#pragma unroll
                for (int n = 0; n < kD / 32; ++n) {
                    if constexpr (kAhead) {
                        dv[n] = mma32(tg[s][n], weights, dv[n]);
                        dk[n] = mma32(tq[s][n], slopes, dk[n]);
                    } else {
                        dv[n] = mma32(Rows::across(s_g, n, 2 * b + s), weights, dv[n]);
                        dk[n] = mma32(Rows::across(s_q, n, 2 * b + s), slopes, dk[n]);
                    }
                }
            }
        }
    };
    auto pass = [&](auto second) {
        head = first_head;
        i = i_start;
        if (tiles > 0) {
            feed.start(queries + head * a.q.head, slopes_of + head * a.dout.head, i, nq);
            load_stats(0, head, i);
        }
#pragma unroll
        for (int n = 0; n < kD / 32; ++n) dk[n] = dv[n] = f32x16{};
        auto step = [&](int t, auto buffer) {
            const int now = i;
            i += kTileRows;
            if (i >= i_end) {
                i = i_start;
                ++head;
            }
            tile(t, now, buffer, second);
        };
        for (int t = 0; t < tiles; t += 2) {
            step(t, Constant<0>{});
            if (t + 1 < tiles) step(t + 1, Constant<1>{});
        }
    };
    pass(Constant<0>{});
    bool odd = false;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) odd = odd || not_finite(dk[n][r]) || not_finite(dv[n][r]);
    if (__syncthreads_or(odd)) pass(Constant<1>{});
    if (key >= nk) return;
    const float unit_k = unit_v / small;
    if (kFar || parts > 1 || (work.split && key < a.sinks)) {
        if (kFar && key >= a.sinks) return;
        const int64_t which = kFar ? (static_cast<int64_t>(slot) * a.kv_heads + kv) * 2 + (wave & 1)
                                   : static_cast<int64_t>(clip) * a.kv_heads + kv;
        float *to = parts > 1 ? work.part + ((part * a.k_tokens + k0 + key) * a.kv_heads + kv) * 2 * kD
                              : (kFar ? work.far : work.near) + (which * a.sinks + key) * 2 * kD;
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d0 = 32 * n + 8 * r + 4 * half;
                *reinterpret_cast<f32x4 *>(to + d0) = f32x4{dk[n][4 * r], dk[n][4 * r + 1], dk[n][4 * r + 2], dk[n][4 * r + 3]} * unit_k;
                *reinterpret_cast<f32x4 *>(to + kD + d0) = f32x4{dv[n][4 * r], dv[n][4 * r + 1], dv[n][4 * r + 2], dv[n][4 * r + 3]} * unit_v;
            }
        return;
    }
    T *out_k = static_cast<T *>(a.dk.data) + (k0 + static_cast<int64_t>(key)) * a.dk.token + kv * a.dk.head;
    T *out_v = static_cast<T *>(a.dv.data) + (k0 + static_cast<int64_t>(key)) * a.dv.token + kv * a.dv.head;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            T e[4], f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                e[x] = static_cast<T>(dk[n][4 * r + x] * (a.scale * unit_k));
                f[x] = static_cast<T>(dv[n][4 * r + x] * unit_v);
            }
            store4(out_k + 32 * n + 8 * r + 4 * half, e);
            store4(out_v + 32 * n + 8 * r + 4 * half, f);
        }
}

// The pieces of queries beyond the window come last: they are shorter than the others and fill up their last round.
template <typename T, int kD>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && kD == 64 ? 2 : 1)
void dkv_tiles(AttentionArgs a, Work work, float factor, int near_groups)
{
    __shared__ __attribute__((aligned(16))) char s_mem[Feed<T, kD, kWaves>::kBytes];
    __shared__ __attribute__((aligned(16))) float s_stats[2][2][kTileRows];     // [buffer][lse2, -delta][query]
    __shared__ int s_bad[kTileRows];
    const int block = blockIdx.x;
    if (block < near_groups) dkv_group<T, kD, false>(a, work, factor, block, s_mem, s_stats, s_bad);
    else dkv_group<T, kD, true>(a, work, factor, block - near_groups, s_mem, s_stats, s_bad);
}

// The parts' sums: a workgroup takes kJoinRows of the 128 keys that those of dkv_group took, a thread 4 values at a time.
constexpr int kJoinRows = 16;

template <typename T, int kD>
__global__ __launch_bounds__(kThreads)
void join_parts(AttentionArgs a, Work work)
{
    const int slot = blockIdx.x / a.kv_heads, kv = blockIdx.x % a.kv_heads;
    const int clip = clip_of_slot(a.cu_k, a.n_clips, slot, kRows);
    int k0, nk;
    clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
    const int tile = (slot - (a.cu_k[clip] / kRows + clip)) * kRows, first = tile + blockIdx.y * kJoinRows;
    if (tile < 0 || first >= nk) return;
    constexpr int kFours = 2 * kD / 4;
    for (int at = threadIdx.x; at < min(kJoinRows, nk - first) * kFours; at += kThreads) {
        const int64_t row = k0 + first + at / kFours;
        const int d = at % kFours * 4;      // below kD: dk, others dv
        f32x4 sum = {};
#pragma unroll 4
        for (int part = 0; part < work.parts; ++part)
            sum += *reinterpret_cast<const f32x4 *>(work.part + ((part * a.k_tokens + row) * a.kv_heads + kv) * 2 * kD + d);
        if (d < kD) sum *= a.scale;
        T y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = static_cast<T>(sum[i]);
        if (d < kD) store4(static_cast<T *>(a.dk.data) + row * a.dk.token + kv * a.dk.head + d, y);
        else store4(static_cast<T *>(a.dv.data) + row * a.dv.token + kv * a.dv.head + d - kD, y);
    }
}

// The sinks' gradients: the part within the first keys' window, then the pieces beyond it in order.
template <typename T, int kD>
__global__ __launch_bounds__(2 * kD)
void join_sinks(AttentionArgs a, Work work)
{
    const int key = blockIdx.x, kv = blockIdx.y, d = threadIdx.x;      // d < kD: dk, others dv
    for (int clip = blockIdx.z; clip < a.n_clips; clip += gridDim.z) {
        int q0, nq, k0, nk;
        clip_range(a.cu_q, clip, a.q_tokens, q0, nq);
        clip_range(a.cu_k, clip, a.k_tokens, k0, nk);
        if (key >= nk) continue;
        float sum = work.near[((static_cast<int64_t>(clip) * a.kv_heads + kv) * a.sinks + key) * 2 * kD + d];
        const int64_t base = q0 / kFarRows + clip;
#pragma unroll 8
        for (int piece = 0; piece < (nq + kFarRows - 1) / kFarRows; ++piece)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                sum += work.far[((((base + piece) * a.kv_heads + kv) * 2 + h) * a.sinks + key) * 2 * kD + d];
        const int64_t row = k0 + key;
        if (d < kD)
            (static_cast<T *>(a.dk.data) + row * a.dk.token + kv * a.dk.head)[d] = static_cast<T>(sum * a.scale);
        else
            (static_cast<T *>(a.dv.data) + row * a.dv.token + kv * a.dv.head)[d - kD] = static_cast<T>(sum);
    }
}

template <typename T, int kD>
hipError_t backward(const AttentionArgs &a, hipStream_t stream)
{
    const Work work = work_of(a);
    const float factor = fmaxf(a.scale * kLog2e, FLT_MIN);     // as in the forward pass
    const int64_t q_groups = q_slots(a.q_tokens, a.n_clips) * a.q_heads;
    const int64_t far_groups = work.split ? far_slots(a.q_tokens, a.n_clips) * a.kv_heads : 0;
    const int64_t key_groups = k_slots(a.k_tokens, a.n_clips) * a.kv_heads, near_groups = key_groups * work.parts;
    if (!fits(q_groups, kThreads) || !fits(near_groups + far_groups, kThreads)) return hipErrorNotSupported;
    if constexpr (kNarrow<T>)
        if (a.q_tokens > 0 && a.k_tokens > 0)
            value_sizes<T, kD><<<static_cast<unsigned>(key_groups), kThreads, 0, stream>>>(a, work);
    if (a.q_tokens > 0)
        dq_tiles<T, kD><<<static_cast<unsigned>(q_groups), kThreads, 0, stream>>>(a, work, factor);
    if (a.k_tokens > 0) {
        dkv_tiles<T, kD><<<static_cast<unsigned>(near_groups + far_groups), kThreads, 0, stream>>>(
            a, work, factor, static_cast<int>(near_groups));
        if (work.parts > 1) join_parts<T, kD><<<dim3(static_cast<unsigned>(key_groups), kRows / kJoinRows), kThreads, 0, stream>>>(a, work);
        if (work.split)
            join_sinks<T, kD><<<dim3(a.sinks, a.kv_heads, a.n_clips < 1024 ? a.n_clips : 1024), 2 * kD, 0, stream>>>(a, work);
    }
    return hipGetLastError();
}

}  // namespace

int64_t window_attention_backward_bytes(const AttentionArgs &a) { return work_floats(a) * 4; }

hipError_t launch_window_attention_backward(const AttentionArgs &a, hipStream_t stream)
{
    if (a.dtype == RVQ_F32) return a.dim == 64 ? backward<float, 64>(a, stream) : backward<float, 128>(a, stream);
    if (a.dtype == RVQ_F16) return a.dim == 64 ? backward<f16_t, 64>(a, stream) : backward<f16_t, 128>(a, stream);
    return a.dim == 64 ? backward<bf16_t, 64>(a, stream) : backward<bf16_t, 128>(a, stream);
}

}  // namespace rvq
