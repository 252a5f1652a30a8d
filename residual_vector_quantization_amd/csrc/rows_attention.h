// Attention of each clip's packed queries over keys that lie elsewhere: in the
// pages of a cache (a chunk of new frames) or packed (an encoder's states).
//
//   x_ij = scale q_i . k_j over the keys j that query i sees,
//   w = softmax(x), out_i = sum_j w_ij v_j, lse_i = log sum_j exp(x_ij)
//
// The query heads that share a key head are rows of the same matrix products:
// row r of a block is query r / heads and head r % heads, so that a key is read
// once for all of them. Two kinds of workgroups share one launch, as the
// lengths of the clips' queries are known on the device alone:
// - few_rows takes a whole clip of up to 16 kSets rows (where there are few rows in
//   all, also one with more, in turns) and is bound by HBM. Its wavefronts take 32
//   keys in turn, which go from memory into registers and from there into 16-wide
//   products with the rows as columns:
//     S^T [key][row] = K Q^T,  O^T [dim][row] = V^T P^T.
//   Only keys that some row sees are gone over (sinks, then the window), and
//   the keys of S^T's rows are numbered so that a lane's scores belong to the 8
//   keys of its V^T operand.
// - tile_rows takes 128 rows, 32 a wavefront, of a clip with more, goes over
//   tiles of 64 keys in the LDS and is bound by the matrix cores, with 32-wide
//   products of the same form; while a tile is worked on, the next is on its way.
// Where clips and heads make few workgroups, the keys of a row are split over
// several; each leaves its maximum, sum and accumulator in the workspace and a
// second launch (join_rows) joins them in order.
//
// Measured, bfloat16: 2048 new frames over 45,000 in pages of 64, 32 heads of 128
// over 8: 1.56 to 1.65 ms, 935 to 990 TFLOP/s, where a large library product
// reaches 1130 to 1170 (matrix cores busy in 44% of the cycles, no LDS bank
// conflicts). The next frame of 12 clips of up to 45,000: 248 us, 5.3 TB/s. 64
// single queries over up to 1500 packed states, 16 heads of 64: 38 us and 4 for the
// join, 4.3 TB/s (a plain read of as much reaches 6.2 where all workgroups move
// through memory side by side and 4.5 to 5.4 where each has a stretch of its own, as
// here). 8 clips of up to 4 frames over up to 1500, 16 heads of 128 over 8: 13.5 us and 4,
// of which 6 to 8 are the chain of reads before the first product (offsets, count, page
// number, row) and the launch. float16, 12 clips of up to 2000 queries over up to 750
// states, 16 heads of 128 over 4: 113 us, 600 TFLOP/s, and 4 for a join launch that finds
// nothing to join, for a workgroup has 12 tiles at most: 16,384 queries over 64 n keys take 41 + 7.7 n us, 27 of the 41 for 134 MB of
// queries and results.
//
// Running maxima move only when a score exceeds them by more than 2^kSlack.
// Weights are rounded to the inputs' type where they enter the second product:
// in tile_rows once (half a step of theirs beside the result's own, 1.41 of its
// error in the mean; a second part would double the product); in few_rows, which
// does not wait for the matrix cores, as two parts, so that the result's own
// rounding is all (64 single queries 46 -> 48 us). In float16 they are taken times
// 2^kShift, so that many small ones beside a large one do not sink below its
// exponents. Their sum is of the unrounded ones, in float32, as are maxima and
// accumulators.
//
// Values that a row does not see: its weights there are 0, but 0 times a value
// that is not finite is not 0. And of a value that is seen, an infinity times a
// weight of 0 (a second part, or one below float32's numbers) would be NaN. So
// where a result is not finite, few_rows goes over its part of the keys again for
// each such row alone, with what it sees only (one_row), and tile_rows repeats its
// pass to find, for every result, whether keys that are seen have an infinity of
// either sign there (a NaN is both), and once more with these values taken as 0.
// The joins leave sums that are not finite unscaled, for a factor may be 0 too.
#pragma once

#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"
#include "attention_tiles.h"
#include "cache_index.h"

namespace rvq {
namespace rows {

#define RVQ_INLINE __device__ inline __attribute__((always_inline))

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kTileQueries = 32 * kWaves;   // rows of tile_rows
constexpr int kKeys = kSharedTile;          // keys a wavefront of few_rows takes at a time
constexpr float kSlack = 8.0f;              // how far (powers of two) a score may exceed the running maximum
constexpr int kMaxSplits = 256;

struct Plan {
    int group, chunks;          // query heads a key head; blocks of them that rows are made of
    int few_limit;              // queries that few_rows takes at a time
    bool any_few, all_few;      // whether few_rows takes the clips with at most so many, and whether all others too
    int tile_queries;           // queries of a workgroup of tile_rows
    int few_splits, tile_splits;
    int tile_slots;             // blocks of queries of tile_rows, all clips
    int mark;                   // how they are found, see below
    bool join_clips;            // join_rows goes by clips and their first few_limit queries, not by rows
    bool by_chiplet;            // how few_rows' workgroups are numbered, see there
    float factor;               // scale in powers of two
    Divisor page;
    float *few, *tile;          // partial results
    int64_t few_rows, tile_rows;
};

// Partial results of `rows` rows in `splits` splits: { max, sum } of each, then the accumulators.
__host__ __device__ inline int64_t stats_floats(int64_t slots) { return (2 * slots + 3) / 4 * 4; }

__device__ inline int heads_first(const Plan &p, int chunk) { return p.group * chunk / p.chunks; }

// The last b in [0, n) that is before, which those up to some b are (0 if there is none), searched by a whole wavefront,
// 64 at a time: one read of the offsets for up to 64 clips, two for 4096.
template <typename Before>
RVQ_INLINE int last_before(int n, Before before)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, size = n;
    while (size > 1) {
        const int step = (size + 63) / 64, b = lo + lane * step;
        const int count = __popcll(__ballot(b < lo + size && before(b)));
        if (count == 0) break;
        size = min(step, size - (count - 1) * step);
        lo += (count - 1) * step;
    }
    return lo;
}

// As clip_of_slot and clip_of_row.
RVQ_INLINE int clip_of_slot_wide(const int32_t *cu, int n, int slot, int per)
{
    return last_before(n, [=](int b) { return cu[b] / per + b <= slot; });
}
RVQ_INLINE int clip_of_row_wide(const int32_t *cu, int n, int row)
{
    return last_before(n, [=](int b) { return cu[b] <= row; });
}

// Clips and their blocks of tile_queries queries are numbered without reading their lengths. mark 0: clip b owns the
// numbers cu[b] / tile_queries + b .., enough for its queries, q_tokens / tile_queries + n_clips + 1 in all. Where clips
// are many and short, few have more than few_limit queries: every such clip has a row that is a multiple of mark =
// few_limit + 1, at least as many of them as blocks (mark is at most half of tile_queries), and those rows' numbers are
// its blocks'; others find that they are not needed.

// A clip's queries and how many keys it has.
struct ClipRows {
    int q0, nq, nk;
    bool beyond;       // more keys than the table can hold: nothing is read and results are NaN
};

// ---------------------------------------------------------------- where keys lie

// Pages of a cache. A query at position p sees the frames j <= p of its window and the sinks.
template <typename T, int kD>
struct Paged {
    static constexpr bool kAll = false;
    const T *keys, *values;
    const int32_t *row;
    Divisor page;
    int table_ld, n_pages, kv_heads, kv;

    RVQ_INLINE static ClipRows clip(const RowsArgs &a, int b)
    {
        ClipRows r;
        if (a.cu_q) clip_range(a.cu_q, b, a.q_tokens, r.q0, r.nq);
        else r.q0 = b, r.nq = 1;
        r.nk = max(a.lens[b], 0);
        r.beyond = r.nk > static_cast<int64_t>(a.table_ld) * a.page_size;
        return r;
    }
    RVQ_INLINE Paged(const RowsArgs &a, const Plan &p, int b, int kv_head)
        : keys(static_cast<const T *>(a.k_pool)), values(static_cast<const T *>(a.v_pool)),
          row(a.table + static_cast<int64_t>(b) * a.table_ld), page(p.page), table_ld(a.table_ld), n_pages(a.n_pages),
          kv_heads(a.kv_heads), kv(kv_head) {}
    RVQ_INLINE uint32_t find(int position) const { return cache_row(row, position, page, table_ld, n_pages, kv_heads, kv); }
    RVQ_INLINE const T *key(uint32_t at) const { return keys + static_cast<uint64_t>(at) * kD; }
    RVQ_INLINE const T *value(uint32_t at) const { return values + static_cast<uint64_t>(at) * kD; }
};

// Packed rows. Every query sees all of its clip's keys.
template <typename T, int kD>
struct Packed {
    static constexpr bool kAll = true;
    const T *keys, *values;
    int64_t key_stride, value_stride;

    RVQ_INLINE static ClipRows clip(const RowsArgs &a, int b)
    {
        ClipRows r;
        int k0;
        if (a.cu_q) clip_range(a.cu_q, b, a.q_tokens, r.q0, r.nq);
        else r.q0 = b, r.nq = 1;
        clip_range(a.cu_k, b, a.k_tokens, k0, r.nk);
        r.beyond = false;
        return r;
    }
    RVQ_INLINE Packed(const RowsArgs &a, const Plan &, int b, int kv_head) : key_stride(a.k.token), value_stride(a.v.token)
    {
        int k0, nk;
        clip_range(a.cu_k, b, a.k_tokens, k0, nk);
        keys = static_cast<const T *>(a.k.data) + k0 * key_stride + kv_head * a.k.head;
        values = static_cast<const T *>(a.v.data) + k0 * value_stride + kv_head * a.v.head;
    }
    RVQ_INLINE uint32_t find(int position) const { return static_cast<uint32_t>(position); }
    RVQ_INLINE const T *key(uint32_t at) const { return keys + static_cast<int64_t>(at) * key_stride; }
    RVQ_INLINE const T *value(uint32_t at) const { return values + static_cast<int64_t>(at) * value_stride; }
};

template <typename Keys>
RVQ_INLINE int position_of(const ClipRows &r, int i) { return Keys::kAll ? r.nk - 1 : r.nk - r.nq + i; }

// ---------------------------------------------------------------- few rows

// kN values of 8 keys, as the kN operands of 8 keys at one dim.
template <typename T, int kN>
struct Block8 {
    T x[8][kN];

    __device__ inline void load(int i, const T *p)
    {
#pragma unroll
        for (int w = 0; w < static_cast<int>(kN * sizeof(T) / 8); ++w)
            reinterpret_cast<u32x2 *>(x[i])[w] = reinterpret_cast<const u32x2 *>(p)[w];
    }
    __device__ inline void clear(int i)
    {
#pragma unroll
        for (int n = 0; n < kN; ++n) x[i][n] = static_cast<T>(0.0f);
    }
    __device__ inline vec8<T> at(int n) const
    {
        vec8<T> r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = x[i][n];
        return r;
    }
};

// Maximum and sum over the four lane groups that hold one row.
__device__ inline float groups_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ inline float groups_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

template <int kD> constexpr int kJoinBytes = kWaves * 16 * (kD + 4 + 2) * 4;
// Where two sets of rows would not leave registers enough their queries stay in the LDS (48 clips of 4 frames over up to
// 4000, 32 heads of 128 over 4: 85.6 -> 74.3 us, spilled registers 17 -> none; 8 such clips 26.4 -> 25.3).
template <typename T, int kD, int kSets> constexpr bool kStaged = kSets == 2 && kD == 128 && sizeof(T) == 2;
template <typename T, int kD, int kSets> constexpr int kStagedBytes = kJoinBytes<kD> + (kStaged<T, kD, kSets> ? kSets * kD / 32 * 1024 : 0);
template <typename T, int kD, int kSets> constexpr int kFewBytes = kStagedBytes<T, kD, kSets> + 16;

// A partial sum times a factor. An infinite one stays so if the factor is 0.
__device__ inline float scaled(float x, float factor) { return fabsf(x) <= FLT_MAX ? x * factor : x; }

// A row's place among the partial results of few_rows' splits.
RVQ_INLINE int64_t few_slot(const RowsArgs &a, const Plan &p, const ClipRows &r, int clip, int split, int i, int h)
{
    const int64_t row = p.all_few ? r.q0 + i : static_cast<int64_t>(clip) * p.few_limit + i;
    return (row * a.q_heads + h) * p.few_splits + split;
}

// One row of few_rows again, query i and head h over the workgroup's own part of the keys, after a result that is not
// finite though the sum of its weights is no NaN: only what the query sees counts, and infinities and NaN are noted apart
// from the sums. Maximum and sum, and so lse, stay as they are. Rare and simple: a thread a key for the scores of
// kThreads keys, then a thread a dim for their values; where all dims of the row are NaN it stops. If every value of the cache is NaN the next frame of 12 clips of up to 45,000
// takes 1.4 ms for 0.25, drafts of 48 clips over up to 4000 0.87 for 0.07, 64 single queries over up to 1500 states 0.37 for
// 0.05; a few such values cost a few of these rows.
template <typename T, int kD, typename Keys>
RVQ_INLINE void one_row(const RowsArgs &a, const Plan &p, const ClipRows &r, const Keys &keys, const Shared &shared, int clip,
                        int split, int i, int h, char *s_mem)
{
    constexpr int kSlices = kThreads / kD;
    float *s_weight = reinterpret_cast<float *>(s_mem);                       // of each key; -1: not seen
    uint32_t *s_place = reinterpret_cast<uint32_t *>(s_weight + kThreads);
    float *s_value = reinterpret_cast<float *>(s_place + kThreads);           // one a thread
    float *s_wave = s_value + kThreads;
    const int wave = threadIdx.x >> 6, d = threadIdx.x % kD, slice = threadIdx.x / kD;
    const T *q = static_cast<const T *>(a.q.data) + static_cast<int64_t>(r.q0 + i) * a.q.token + h * a.q.head;
    const int position = position_of<Keys>(r, i);
    const int last = min(min(shared.tiles, (split + 1) * shared.per) * kKeys, shared.seen.count);
    float top = -INFINITY, sum = 0.0f, y = 0.0f;
    bool plus = false, minus = false;
    for (int nth0 = split * shared.per * kKeys; nth0 < last; nth0 += kThreads) {
        const int nth = nth0 + static_cast<int>(threadIdx.x);
        const int j = nth < last ? shared_frame(shared, nth, !Keys::kAll, position, a.window, a.sinks) : -1;
        uint32_t place = j < 0 ? kPastEnd : keys.find(j);
        float x = -INFINITY;
        if (place < kPastEnd) {
            x = 0.0f;
            const T *key = keys.key(place);
#pragma unroll 4
            for (int n = 0; n < kD; n += 8) {
                const vec8<T> u = load8(q + n), w = load8(key + n);
#pragma unroll
                for (int e = 0; e < 8; ++e) x = __builtin_fmaf(to_float(u[e]), to_float(w[e]), x);
            }
            x *= p.factor;
        }
        float most = x;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor(most, m));
        __syncthreads();      // what was left in the LDS has been read
        const bool odd = __all(plus && minus);
        if ((threadIdx.x & 63) == 0) {
            s_wave[wave] = most;
            s_wave[kWaves + wave] = odd ? 1.0f : 0.0f;
        }
        __syncthreads();
        float all = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) all += s_wave[kWaves + w];
        if (all == kWaves) break;      // the row's results are all NaN already
        const float before = top;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_wave[w]);
        const float keep = before == -INFINITY ? 0.0f : fast_exp2(before - top);
        const bool sees = x != -INFINITY;
        const float weight = sees ? fast_exp2(x - top) : -1.0f;
        sum = sum * keep + (sees ? weight : 0.0f);
        s_weight[threadIdx.x] = weight;
        s_place[threadIdx.x] = place;
        __syncthreads();
        y *= keep;
#pragma unroll 4
        for (int n = slice; n < min(kThreads, last - nth0) && !(plus && minus); n += kSlices) {
            const float w = s_weight[n];
            const bool seen = w != -1.0f;
            const float v = to_float(keys.value(seen ? s_place[n] : 0)[d]);
            const bool up = seen && !(v <= FLT_MAX), down = seen && !(v >= -FLT_MAX);
            plus = plus || up;
            minus = minus || down;
            y += up || down || !seen ? 0.0f : w * v;
        }
    }
    if (plus || minus) y = plus && minus ? __builtin_nanf("") : plus ? INFINITY : -INFINITY;
    sum = wave_sum(sum);
    __syncthreads();
    s_value[threadIdx.x] = y;
    if ((threadIdx.x & 63) == 0) s_wave[wave] = sum;
    __syncthreads();
    if (slice == 0) {
        float total = 0.0f;
        y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) total += s_wave[w];
#pragma unroll
        for (int n = 0; n < kSlices; ++n) y += s_value[n * kD + d];
        if (p.few_splits == 1) {
            T *out = static_cast<T *>(a.out.data) + static_cast<int64_t>(r.q0 + i) * a.out.token + h * a.out.head;
            out[d] = static_cast<T>(total == 0.0f ? 0.0f : y / total);
        } else {
            const int64_t slot = few_slot(a, p, r, clip, split, i, h);
            // this workgroup's own, written before the fence
            const float most = __hip_atomic_load(p.few + 2 * slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float factor = top == -INFINITY || most == -INFINITY ? 0.0f : fast_exp2(top - most);
            p.few[stats_floats(p.few_rows * p.few_splits) + slot * kD + d] = scaled(y, factor);
        }
    }
    __syncthreads();
}

template <typename T, int kD, typename Keys, int kSets>
RVQ_INLINE void few_rows(const RowsArgs &a, const Plan &p, int block, char *s_mem)
{
    constexpr int kSteps = kD / 32;      // products along the head dim
    constexpr int kN = kD / 16;          // dims a lane holds of a value row
    constexpr float kShift = kNarrow<T> ? 15.0f - kSlack : 0.0f;      // weights are below 2^(kSlack + kShift)
    float (*s_out)[16][kD + 4] = reinterpret_cast<float (*)[16][kD + 4]>(s_mem);
    float (*s_max)[16] = reinterpret_cast<float (*)[16]>(s_mem + kWaves * 16 * (kD + 4) * 4);
    float (*s_sum)[16] = s_max + kWaves;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // Heads change fastest, then splits, then clips. Workgroups go to the 8 chiplets in turn; where a key's heads lie
    // side by side, all heads of a clip's split go to one of them, so that its cache sees whole keys, not every
    // eighth head's part of them, which would use few of its channels (64 single queries 52.7 -> 50.2 us).
    const int columns = a.kv_heads * p.chunks;
    const int rest = p.by_chiplet ? block / (8 * columns) * 8 + block % 8 : block / columns;
    const int column = p.by_chiplet ? block / 8 % columns : block - rest * columns;
    const int kv = column / p.chunks, chunk = column - kv * p.chunks;
    const int clip = rest / p.few_splits, split = rest - clip * p.few_splits;
    if (clip >= a.n_clips) return;
    const ClipRows r = Keys::clip(a, clip);
    if (r.nq == 0 || (!p.all_few && r.nq > p.few_limit)) return;
    const int heads = heads_first(p, chunk + 1) - heads_first(p, chunk), head0 = kv * p.group + heads_first(p, chunk);
    const Keys keys(a, p, clip, kv);

    for (int base = 0; base < r.nq; base += p.few_limit) {
        const int count = min(p.few_limit, r.nq - base);     // queries of this turn
        // this lane's row of every set
        int query[kSets], head[kSets];
        constexpr bool kLds = kStaged<T, kD, kSets>;
        vec8<T> *s_q = reinterpret_cast<vec8<T> *>(s_mem + kJoinBytes<kD>) + lane;      // [set][step][lane]
        vec8<T> q[kLds ? 1 : kSets][kLds ? 1 : kSteps];
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int at = min(16 * s + c, count * heads - 1);
            query[s] = base + at / heads;
            head[s] = head0 + at - (query[s] - base) * heads;
            const T *from = static_cast<const T *>(a.q.data) + static_cast<int64_t>(r.q0 + query[s]) * a.q.token + head[s] * a.q.head;
#pragma unroll
            for (int t = 0; t < kSteps; ++t) {
                if constexpr (!kLds) q[s][t] = load8(from + 32 * t + 8 * g);
                else if (t == wave) s_q[(s * kSteps + t) * 64] = load8(from + 32 * t + 8 * g);
            }
        }
        if constexpr (kLds) __syncthreads();
        const int sets = (count * heads + 15) / 16;       // the others hold no row

        f32x4 o[kSets][kN];
        float m[kSets], l[kSets];
        const int p_first = position_of<Keys>(r, base), p_last = position_of<Keys>(r, base + count - 1);
        const Shared shared = share(r.beyond ? -1 : p_first, r.beyond ? -1 : p_last, a.window, a.sinks, p.few_splits);
        const Seen &seen = shared.seen;
        {
            // positions up to `through` are seen by all of the queries if they are above `from` (or sinks)
            const int through = p_first, from = below_window(p_last, a.window);
#pragma unroll
            for (int s = 0; s < kSets; ++s) {
                m[s] = -INFINITY;
                l[s] = r.beyond ? __builtin_nanf("") : 0.0f;
#pragma unroll
                for (int n = 0; n < kN; ++n) o[s][n] = f32x4{};
            }
            const int end = min(shared.tiles, (split + 1) * shared.per);
            // lane n holds the place of the tile's key n % 32
            auto find = [&](int tile) -> uint32_t {
                if (tile >= end) return kPastEnd;
                const int j = shared_frame(shared, tile * kKeys + (lane & 31), false, 0, a.window, a.sinks);
                return j < 0 ? kPastEnd : keys.find(j);
            };
            struct Part {
                int tile;
                uint32_t mine;         // of the keys' places, this lane's
                vec8<T> k[2][kSteps];
                Block8<T, kN> v;
            };
            // sets out for a tile's keys and values; row 0 in the place of keys that are not there, so that nothing branches
            auto load = [&](Part &d, int tile, uint32_t mine) __attribute__((always_inline)) {
                d.tile = tile;
                d.mine = mine;
                const uint32_t at = mine < kPastEnd ? mine : 0;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const T *key = keys.key(__shfl(at, 8 * (c >> 2) + 4 * b + (c & 3))) + 8 * g;
#pragma unroll
                    for (int t = 0; t < kSteps; ++t) d.k[b][t] = load8(key + 32 * t);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) d.v.load(i, keys.value(__shfl(at, 8 * g + i)) + kN * c);
            };
            auto use = [&](Part &d) __attribute__((always_inline)) {
                const bool there = __all(d.mine < kPastEnd), lost = __any(d.mine == kNoPage);
                if (!there) {
                    // keys that are not there are zeros: their weights are 0
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (__shfl(d.mine, 8 * (c >> 2) + 4 * b + (c & 3)) >= kPastEnd)
#pragma unroll
                            for (int t = 0; t < kSteps; ++t) d.k[b][t] = vec8<T>{};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (__shfl(d.mine, 8 * g + i) >= kPastEnd) d.v.clear(i);
                }
                // all keys of the tile are there and seen by every row
                const int j_first = seen_position(seen, d.tile * kKeys);
                const int j_last = seen_position(seen, min(d.tile * kKeys + kKeys, seen.count) - 1);
                const bool whole = there && (Keys::kAll || (j_last <= through && (j_first > from || j_last < a.sinks)));
#pragma unroll
                for (int s = 0; s < kSets; ++s) {
                    if (kSets > 1 && s >= sets) break;
                    if (kSets > 1) __builtin_amdgcn_sched_barrier(0);
                    // scores in powers of two: key 8 g + 4 b + i of the tile, row c
                    f32x4 x[2] = {};
#pragma unroll
                    for (int t = 0; t < kSteps; ++t)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            if constexpr (kLds) x[b] = mma16(d.k[b][t], s_q[(s * kSteps + t) * 64], x[b]);
                            else x[b] = mma16(d.k[b][t], q[s][t], x[b]);
                        }
                    float top = -INFINITY;
                    if (!whole) {
                        const int position = position_of<Keys>(r, query[s]), low = below_window(position, a.window);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int nth = d.tile * kKeys + 8 * g + 4 * b + i, j = seen_position(seen, nth);
                                const bool sees = nth < seen.count && (Keys::kAll || (j <= position && (j > low || j < a.sinks)));
                                x[b][i] = sees ? x[b][i] : -INFINITY;
                            }
                    }
                    if (!Keys::kAll && lost) {     // rare; their scores are 0 where they are seen
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (__shfl(d.mine, 8 * g + 4 * b + i) == kNoPage) {
                                    if (x[b][i] != -INFINITY) l[s] = __builtin_nanf("");
                                    x[b][i] = -INFINITY;
                                }
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = fmaxf(top, x[b][i]);
                    top *= p.factor;
                    if (__any(top > m[s] + kSlack)) {
                        top = groups_max(top);
                        if (top > m[s] + kSlack) {
                            const float keep = fast_exp2(m[s] - top);
                            m[s] = top;
                            l[s] *= keep;
#pragma unroll
                            for (int n = 0; n < kN; ++n) o[s][n] *= keep;
                        }
                    }
                    const float safe = m[s] == -INFINITY ? 0.0f : m[s] - kShift;
                    // weights in two parts where they are rounded: the second product is not what the time goes to
                    vec8<T> w, rest;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = fast_exp2(__builtin_fmaf(x[b][i], p.factor, -safe));
                            l[s] += e;
                            w[4 * b + i] = static_cast<T>(e);
                            if constexpr (sizeof(T) == 2) rest[4 * b + i] = static_cast<T>(e - to_float(w[4 * b + i]));
                        }
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        const vec8<T> v = d.v.at(n);
                        if constexpr (sizeof(T) == 2) o[s][n] = mma16(v, rest, o[s][n]);
                        o[s][n] = mma16(v, w, o[s][n]);
                    }
                }
            };
            Part part;
            int tile = split * shared.per + wave;
            uint32_t next = find(tile);
            for (; tile < end; tile += kWaves) {
                load(part, tile, next);
                next = find(tile + kWaves);
                use(part);
            }
        }
        // joins the wavefronts and writes the rows
        uint32_t *s_odd = reinterpret_cast<uint32_t *>(s_mem + kStagedBytes<T, kD, kSets>);   // rows with something not finite, a bit each
        if (threadIdx.x == 0) *s_odd = 0;
        {
#pragma unroll
            for (int s = 0; s < kSets; ++s) {
                if (s >= sets) break;
                if (s > 0) __syncthreads();
                const float sum = groups_sum(l[s]);
                if (g == 0) {
                    s_max[wave][c] = m[s];
                    s_sum[wave][c] = sum;
                }
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_out[wave][c][kN * (4 * g + i) + n] = o[s][n][i];
                __syncthreads();
                const int rows = min(16, count * heads - 16 * s);
                for (int at = threadIdx.x; at < rows * kD; at += kThreads) {
                    const int row = at / kD, d = at - row * kD, nth = (16 * s + row) / heads;
                    const int i = base + nth, h = head0 + (16 * s + row) - nth * heads;
                    float top = -INFINITY, total = 0.0f, y = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_max[w][row]);
                    const float safe = top == -INFINITY ? 0.0f : top;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) {
                        const float f = fast_exp2(s_max[w][row] - safe);
                        total += s_sum[w][row] * f;
                        y += s_out[w][row][d] * f;
                    }
                    if (!(fabsf(y) <= FLT_MAX) && total == total) atomicOr(s_odd, 1u << (16 * s + row));
                    if (p.few_splits == 1) {
                        T *out = static_cast<T *>(a.out.data) + static_cast<int64_t>(r.q0 + i) * a.out.token + h * a.out.head;
                        out[d] = static_cast<T>(total == 0.0f ? 0.0f : y / total);
                        if (a.lse && d == 0)
                            a.lse[static_cast<int64_t>(h) * a.q_tokens + r.q0 + i] =
                                total == 0.0f ? -INFINITY : (top - kShift + log2f(total)) * kLn2;
                    } else {
                        const int64_t slot = few_slot(a, p, r, clip, split, i, h);
                        p.few[stats_floats(p.few_rows * p.few_splits) + slot * kD + d] = y;
                        if (d == 0) {
                            p.few[2 * slot] = top - kShift;
                            p.few[2 * slot + 1] = total;
                        }
                    }
                }
            }
        }
        __syncthreads();
        uint32_t rows = *s_odd;
        if (rows != 0) {
            __threadfence();      // what these rows are now is written before what they become
            __syncthreads();
            while (rows != 0) {
                const int row = __builtin_ctz(rows), nth = row / heads;
                rows &= rows - 1;
                one_row<T, kD, Keys>(a, p, r, keys, shared, clip, split, base + nth, head0 + row - nth * heads, s_mem);
            }
        }
        if (base + count < r.nq) __syncthreads();
    }
}

// ---------------------------------------------------------------- tiles of many rows

// As copy16, from an address of 64 bits in each lane.
__device__ inline void copy16_from(const void *src, void *dst)
{
    const unsigned m0 = static_cast<unsigned>(reinterpret_cast<size_t>((lds_void *)dst));
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(m0) : "memory");
}

// Tiles of keys and values that go by, as Feed, from where they lie. start sets out for a tile, turn waits for it and
// sets out for the next. gone: a bit for each of the current tile's keys that is not there (what lies in its place is
// some other row).
template <typename T, int kD, typename Keys> struct Tiles;

template <typename T, int kD>
struct Tiles<T, kD, Packed<T, kD>> {
    typedef Feed<T, kD, kWaves> Memory;
    typedef typename Memory::Rows Rows;
    static constexpr int kBytes = Memory::kBytes;
    Memory feed;
    const Packed<T, kD> keys;
    const KeyRange range;
    int last;

    RVQ_INLINE Tiles(char *s, const Packed<T, kD> &from, const KeyRange &r, int last_position)
        : feed(s, from.key_stride, from.value_stride), keys(from), range(r), last(last_position) {}
    RVQ_INLINE void start(int t, int) { feed.start(keys.keys, keys.values, range.start(t), last + 1); }
    template <int kBuffer>
    RVQ_INLINE uint64_t turn(Constant<kBuffer> buffer, int t, int end)
    {
        feed.turn(buffer, t + 1 < end, keys.keys, keys.values, range.start(t + 1), last + 1);
        return 0;
    }
    template <int kBuffer> __device__ char *tile_keys(Constant<kBuffer> b) const { return feed.tile_one(b); }
    template <int kBuffer> __device__ char *tile_values(Constant<kBuffer> b) const { return feed.tile_two(b); }
};

// From pages: lane n holds the place of the next tile's key n, looked up one tile ahead of the copies that need it.
template <typename T, int kD>
struct PagedPlaces {
    const Paged<T, kD> keys;
    const KeyRange range;
    int last;
    uint32_t next;
    uint64_t gone;

    RVQ_INLINE PagedPlaces(const Paged<T, kD> &from, const KeyRange &r, int last_position)
        : keys(from), range(r), last(last_position), next(0), gone(0) {}
    // keys behind the last one that is seen: that one again
    RVQ_INLINE void look(int t, int end)
    {
        if (t < end) next = keys.find(min(range.start(t) + static_cast<int>(threadIdx.x & 63), last));
    }
    // row 0 of the pools in the place of keys that are not there
    RVQ_INLINE void take()
    {
        gone = __ballot(next == kNoPage);
        if (next == kNoPage) next = 0;
    }
};

template <typename T, int kD>
struct Tiles<T, kD, Paged<T, kD>> {
    typedef Tile<T, kD, kWaves> Rows;
    static constexpr int kBytes = 4 * Rows::kBytes;
    PagedPlaces<T, kD> places;
    char *s;

    RVQ_INLINE Tiles(char *memory, const Paged<T, kD> &from, const KeyRange &r, int last_position)
        : places(from, r, last_position), s(memory) {}
    RVQ_INLINE void load(int buffer)
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        places.take();
        char *to = s + buffer * 2 * Rows::kBytes;
#pragma unroll
        for (int n = 0; n < Rows::kCopies; ++n) {
            const int at = (n * kWaves + wave) * 64 + lane, row = at / Rows::kRowPieces;
            const uint64_t place = __shfl(places.next, row);
            const uint64_t offset = place * Rows::kRowBytes + Rows::place(row, at % Rows::kRowPieces) * 16;
            copy16_from(reinterpret_cast<const char *>(places.keys.keys) + offset, to + (n * kWaves + wave) * 1024);
            copy16_from(reinterpret_cast<const char *>(places.keys.values) + offset, to + Rows::kBytes + (n * kWaves + wave) * 1024);
        }
    }
    RVQ_INLINE void start(int t, int end)
    {
        places.look(t, end);
        load(0);
        places.look(t + 1, end);
    }
    template <int kBuffer>
    RVQ_INLINE uint64_t turn(Constant<kBuffer>, int t, int end)
    {
        const uint64_t gone = places.gone;
        wait_copies();
        __syncthreads();
        if (t + 1 < end) {
            load(1 - kBuffer);
            places.look(t + 2, end);
        }
        return gone;
    }
    template <int kBuffer> __device__ char *tile_keys(Constant<kBuffer>) const { return s + kBuffer * 2 * Rows::kBytes; }
    template <int kBuffer> __device__ char *tile_values(Constant<kBuffer>) const { return s + (kBuffer * 2 + 1) * Rows::kBytes; }
};

template <int kD>
struct Tiles<float, kD, Paged<float, kD>> {
    typedef SplitTile<kD, kWaves> Rows;
    static constexpr int kBytes = 2 * Rows::kBytes;
    PagedPlaces<float, kD> places;
    typename Rows::Loader one, two;
    char *s;

    RVQ_INLINE Tiles(char *memory, const Paged<float, kD> &from, const KeyRange &r, int last_position)
        : places(from, r, last_position), one(0), two(0), s(memory) {}
    RVQ_INLINE void load()
    {
        places.take();
#pragma unroll
        for (int n = 0; n < Rows::kUnits; ++n) {
            const int at = n * kThreads + threadIdx.x, row = at / (kD / 8), piece = at % (kD / 8);
            const uint32_t place = __shfl(places.next, row);
            one.x[n] = load8(places.keys.key(place) + 8 * piece);
            two.x[n] = load8(places.keys.value(place) + 8 * piece);
        }
    }
    RVQ_INLINE void start(int t, int end)
    {
        places.look(t, end);
        load();
        places.look(t + 1, end);
    }
    template <int kBuffer>
    RVQ_INLINE uint64_t turn(Constant<kBuffer>, int t, int end)
    {
        const uint64_t gone = places.gone;
        __syncthreads();
        one.store(s);
        two.store(s + Rows::kBytes);
        __syncthreads();
        if (t + 1 < end) {
            load();
            places.look(t + 2, end);
        }
        return gone;
    }
    template <int kBuffer> __device__ char *tile_keys(Constant<kBuffer>) const { return s; }
    template <int kBuffer> __device__ char *tile_values(Constant<kBuffer>) const { return s + Rows::kBytes; }
};

template <typename T, int kD, typename Keys>
RVQ_INLINE void tile_rows(const RowsArgs &a, const Plan &p, int block, char *s_mem)
{
    typedef Tiles<T, kD, Keys> Source;
    typedef typename Source::Rows Rows;
    constexpr float kShift = kNarrow<T> ? 15.0f - kSlack : 0.0f;      // weights are below 2^(kSlack + kShift)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, half = lane >> 5;
    // heads change fastest, then splits; the last queries of a clip, which see most, start first
    const int columns = a.kv_heads * p.chunks;
    const int rest = block / columns, column = block - rest * columns;
    const int kv = column / p.chunks, chunk = column - kv * p.chunks;
    const int slot = p.tile_slots - 1 - rest / p.tile_splits, split = rest % p.tile_splits;
    const int clip = p.mark ? clip_of_row_wide(a.cu_q, a.n_clips, slot * p.mark)
                            : clip_of_slot_wide(a.cu_q, a.n_clips, slot, p.tile_queries);
    const ClipRows r = Keys::clip(a, clip);
    const int64_t nth = p.mark ? slot - (r.q0 + p.mark - 1) / p.mark : slot - (a.cu_q[clip] / p.tile_queries + clip);
    if (nth < 0 || nth * p.tile_queries >= r.nq || r.nq <= p.few_limit) return;
    const int i0 = static_cast<int>(nth) * p.tile_queries;
    const int heads = heads_first(p, chunk + 1) - heads_first(p, chunk), head0 = kv * p.group + heads_first(p, chunk);
    const Keys keys(a, p, clip, kv);

    const int used = min(p.tile_queries, r.nq - i0) * heads;      // rows
    const int row = min(32 * wave + c, used - 1);
    const bool real = 32 * wave + c < used;
    const int query = i0 + row / heads, head = head0 + row % heads;
    const int position = position_of<Keys>(r, query);
    const int p_last = r.beyond ? -1 : position_of<Keys>(r, i0 + (used - 1) / heads);
    const KeyRange range = keys_seen(r.beyond ? -1 : position_of<Keys>(r, i0), p_last, a.window, a.sinks);
    const int per = (range.tiles + p.tile_splits - 1) / p.tile_splits;
    const int begin = min(split * per, range.tiles), end = min(begin + per, range.tiles);
    // this wavefront's first and last position; one without a row of its own sees no tile
    const int w_first = position_of<Keys>(r, i0 + min(32 * wave, used - 1) / heads);
    const int w_last = 32 * wave < used ? position_of<Keys>(r, i0 + min(32 * wave + 31, used - 1) / heads) : -1;
    // positions above these are in the window of this query, of the wavefront's first and of its last
    const int p_low = below_window(position, a.window), w_low = below_window(w_first, a.window);
    const int w_high = below_window(w_last, a.window);

    const T *own = static_cast<const T *>(a.q.data) + static_cast<int64_t>(r.q0 + query) * a.q.token + head * a.q.head;
    Operand<T> q[kD / 16];
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) q[t] = Operand<T>(load8(own + 16 * t + 8 * half));
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) arrive(q[t]);
    Source source(s_mem, keys, range, p_last);

    f32x16 o[kD / 32];
    float m, l;
    bool bad = r.beyond;

    // One tile of keys. The buffer's number is a constant, so that LDS addresses are; markers and clean (the values
    // of a tile are rewritten) make the later passes.
    auto tile = [&](int t, auto buffer, auto markers, auto clean) __attribute__((always_inline)) {
        const uint64_t gone = source.turn(buffer, t, end);
        char *s_k = source.tile_keys(buffer), *s_v = source.tile_values(buffer);
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
            for (int i = 0; i < 32; ++i) odd = odd || x[i >> 4][i & 15] != x[i >> 4][i & 15];
            if (__any(odd)) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    f32x16 y = {};
                    uint32_t at = keys.find(min(j0 + 32 * b + c, p_last));
                    if (at == kNoPage) at = 0;
                    const T *key = keys.key(at) + 8 * half;
                    for (int n = 0; n < kD / 16; ++n) y = mma32(load8(key + 16 * n), load8(own + 16 * n + 8 * half), y);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[b][i] = x[b][i] != x[b][i] ? y[i] : x[b][i];
                }
            }
        }
        if (!(j0 + kTileRows - 1 <= w_first && (j0 > w_high || j0 + kTileRows - 1 < a.sinks))) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = j0 + 32 * b + 8 * (i >> 2) + 4 * half + (i & 3);
                    x[b][i] = j <= position && (j > p_low || j < a.sinks) ? x[b][i] : -INFINITY;
                }
        }
        if (gone != 0) {      // rare
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t some = static_cast<uint32_t>(gone >> 32 * b) >> 4 * half;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = j0 + 32 * b + 8 * (i >> 2) + 4 * half + (i & 3);
                    const bool lost = some >> (8 * (i >> 2) + (i & 3)) & 1;
                    bad = bad || (lost && j <= position && (j > p_low || j < a.sinks));
                    x[b][i] = lost ? -INFINITY : x[b][i];
                }
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i >> 4][i & 15]);
        top *= p.factor;
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
            for (int i = 0; i < 16; ++i) {
                float e = fast_exp2(__builtin_fmaf(x[b][i], p.factor, -safe));
                sum[i & 3] += e;
                if (markers.value) e = x[b][i] == -INFINITY ? 0.0f : 1.0f;
                w[i >> 3][i & 7] = static_cast<T>(e);
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
                for (int i = 0; i < 16; ++i) o[n][i] = (o[n][i] >= 1.0f ? 1.0f : 0.0f) + (o[n][i] > floorf(o[n][i]) ? kMinus : 0.0f);
        }
    };
    auto pass = [&](auto markers, auto clean) __attribute__((always_inline)) {
        if (begin < end) source.start(begin, end);
#pragma unroll
        for (int n = 0; n < kD / 32; ++n) o[n] = f32x16{};
        m = -INFINITY;
        l = 0.0f;
        for (int t = begin; t < end; t += 2) {
            tile(t, Constant<0>{}, markers, clean);
            if (t + 1 < end) tile(t + 1, Constant<1>{}, markers, clean);
        }
    };

    pass(Constant<0>{}, Constant<0>{});
    bool odd = false;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) odd = odd || !(fabsf(o[n][i]) <= FLT_MAX);
    if (__syncthreads_or(odd)) {
        pass(Constant<1>{}, Constant<1>{});
        uint32_t up[kD / 64] = {}, down[kD / 64] = {};
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                up[n >> 1] |= static_cast<uint32_t>(o[n][i] >= 1.0f) << (16 * (n & 1) + i);
                down[n >> 1] |= static_cast<uint32_t>(o[n][i] > floorf(o[n][i])) << (16 * (n & 1) + i);
            }
        __syncthreads();     // the tiles are no longer read
        pass(Constant<0>{}, Constant<1>{});
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool plus = up[n >> 1] >> (16 * (n & 1) + i) & 1, minus = down[n >> 1] >> (16 * (n & 1) + i) & 1;
                if (plus || minus) o[n][i] = plus && minus ? __builtin_nanf("") : plus ? INFINITY : -INFINITY;
            }
    }
    l += __shfl_xor(l, 32);
    bad = __shfl_xor(static_cast<int>(bad), 32) || bad;      // in this order: all lanes take part
    if (!real) return;
    if (bad) l = __builtin_nanf("");
    if (p.tile_splits > 1) {
        const int64_t at = (static_cast<int64_t>(r.q0 + query) * a.q_heads + head) * p.tile_splits + split;
        float *out = p.tile + stats_floats(p.tile_rows * p.tile_splits) + at * kD;
#pragma unroll
        for (int n = 0; n < kD / 32; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4 *>(out + 32 * n + 8 * i + 4 * half) =
                    f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
        if (half == 0) {
            p.tile[2 * at] = m - kShift;
            p.tile[2 * at + 1] = l;
        }
        return;
    }
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    T *out = static_cast<T *>(a.out.data) + static_cast<int64_t>(r.q0 + query) * a.out.token + head * a.out.head;
#pragma unroll
    for (int n = 0; n < kD / 32; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(o[n][4 * i + e] * inverse);
            store4(out + 32 * n + 8 * i + 4 * half, y);
        }
    if (a.lse && half == 0)
        a.lse[static_cast<int64_t>(head) * a.q_tokens + r.q0 + query] = l == 0.0f ? -INFINITY : (m - kShift + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- launches

// The tiles' workgroups come first: they last longer. Registers spilled, here and in only_few_rows: over pages 9 of 168 in
// 16 bits at dim 64 with two sets of rows, 68 in float32 at dim 128; none elsewhere.
template <typename T, int kD, typename Keys, int kSets>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? (kD == 64 ? 3 : 2) : 1)
void all_rows(RowsArgs a, Plan p, int tile_groups)
{
    constexpr int kTileBytes = Tiles<T, kD, Keys>::kBytes;
    constexpr int kRest = kFewBytes<T, kD, kSets>;
    __shared__ __attribute__((aligned(16))) char s_mem[kTileBytes > kRest ? kTileBytes : kRest];
    const int block = blockIdx.x;
    if (block < tile_groups) tile_rows<T, kD, Keys>(a, p, block, s_mem);
    else few_rows<T, kD, Keys, kSets>(a, p, block - tile_groups, s_mem);
}

template <typename T, int kD, typename Keys, int kSets>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
void only_few_rows(RowsArgs a, Plan p)
{
    __shared__ __attribute__((aligned(16))) char s_mem[kFewBytes<T, kD, kSets>];
    few_rows<T, kD, Keys, kSets>(a, p, blockIdx.x, s_mem);
}

// One wavefront a query and kJoined of its heads, kD / 4 lanes each: they find the largest maximum and the scaled sums
// over the splits, then add up the accumulators in order, 4 dims a lane.
template <int kD> constexpr int kJoined = 256 / kD;

template <typename T, int kD, typename Keys>
__global__ __launch_bounds__(64)
void join_rows(RowsArgs a, Plan p)
{
    constexpr int kLanes = kD / 4;
    const int lane = threadIdx.x & (kLanes - 1), nth = threadIdx.x / kLanes;
    int clip = blockIdx.x;
    if (p.join_clips) clip = blockIdx.x / p.few_limit;
    else if (a.cu_q) clip = clip_of_row_wide(a.cu_q, a.n_clips, blockIdx.x);
    const ClipRows r = Keys::clip(a, clip);
    const int i = p.join_clips ? blockIdx.x - clip * p.few_limit : blockIdx.x - r.q0, token = r.q0 + i;
    if (i < 0 || i >= r.nq) return;
    const bool few = p.all_few || r.nq <= p.few_limit;
    const int splits = few ? p.few_splits : p.tile_splits;
    if (splits == 1) return;
    const int own = blockIdx.y * kJoined<kD> + nth, head = min(own, a.q_heads - 1);
    const float *part = few ? p.few : p.tile;
    const int64_t row = (few && !p.all_few ? static_cast<int64_t>(clip) * p.few_limit + i : token) * a.q_heads + head;
    const float *stats = part + 2 * row * splits;
    const float *sums = part + stats_floats((few ? p.few_rows : p.tile_rows) * splits) + row * splits * kD + 4 * lane;
    __shared__ float s_factor[kJoined<kD>][kMaxSplits];
    float top = -INFINITY;
    for (int s = lane; s < splits; s += kLanes) top = fmaxf(top, stats[2 * s]);
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float safe = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int s = lane; s < splits; s += kLanes) {
        const float f = fast_exp2(stats[2 * s] - safe);
        s_factor[nth][s] = f;
        sum += stats[2 * s + 1] * f;
    }
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
    __syncthreads();
    f32x4 y = {};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) y += *reinterpret_cast<const f32x4 *>(sums + s * kD) * s_factor[nth][s];
    bool odd = false;
#pragma unroll
    for (int n = 0; n < 4; ++n) odd = odd || !(fabsf(y[n]) <= FLT_MAX);
    if (odd) {
        y = f32x4{};
        for (int s = 0; s < splits; ++s)
            for (int n = 0; n < 4; ++n) y[n] += scaled(sums[s * kD + n], s_factor[nth][s]);
    }
    if (own >= a.q_heads) return;
    T *out = static_cast<T *>(a.out.data) + static_cast<int64_t>(token) * a.out.token + head * a.out.head;
    T z[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) z[n] = static_cast<T>(sum == 0.0f ? 0.0f : y[n] / sum);
    store4(out + 4 * lane, z);
    if (a.lse && lane == 0)
        a.lse[static_cast<int64_t>(head) * a.q_tokens + token] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// How the rows are shared out. It depends on shapes alone, so that the workspace's size is known beforehand. keys: the
// most that a clip can have.
inline Plan plan(const RowsArgs &a, int64_t keys, int64_t &floats)
{
    // few_rows: up to kWanted workgroups, each with kTurns tiles a wavefront or more, as every split of a row writes its
    // accumulator (8 clips of 4 frames over up to 4000, 8 query heads a key head of 128: kTurns 1, 2, 3, 4 take 31, 26, 25,
    // 30 us; 12 clips of up to 45000 frames: 1024, 2048, 4096, 8192 workgroups take 262, 256, 248, 264 us); with 32
    // rows, which take more registers and write twice as much, up to 768 (the same drafts of 48 clips: 512, 768, 1024, 2048,
    // 4096 take 80, 74, 76, 83, 83 us; 24 single frames beside 8 chunks 75, 74, 78, 78, 78).
    // tile_rows: as many workgroups as the chip holds at once, 2 a CU in 16 bits (256 frames over 8000: 256, 384, 512, 768
    // workgroups take 84, 72, 62, 74 us), with least_tiles tiles each. In dim 64 it holds 3, which pays where keys are many
    // (2 clips of 1024 frames over 8000, 16 heads over 4: 256, 512, 768 workgroups take 202, 125, 111 us; 27 tiles a row in
    // one workgroup and in two: 84 and 93 us). Float32 takes six products for one, so that its
    // workgroups' starts and ends weigh less (16 clips of 400 over 4000, dim 128: 512, 768, 1024 take 445, 407, 410 us; 6
    // clips of 50 frames over 250 seen: splits of 8, 3, 2, 1 tiles take 26.6, 22.3, 20.6, 22.7 us).
    constexpr int64_t kWanted = 4096, kTurns = 3;
    const int64_t wanted_tiles = a.dtype == RVQ_F32 ? 768 : 512, least_tiles = a.dtype == RVQ_F32 ? 2 : 4;
    Plan p = {};
    p.group = a.q_heads / a.kv_heads;
    p.chunks = (p.group + 31) / 32;
    const int heads = (p.group + p.chunks - 1) / p.chunks;
    const int64_t columns = static_cast<int64_t>(a.kv_heads) * p.chunks;
    const int64_t average = a.n_clips ? (a.q_tokens + a.n_clips - 1) / a.n_clips : 0;
    // 16 rows of few_rows where they do for most clips, 32 otherwise
    const int rows = heads <= 16 && average * heads <= 16 ? 16 : 32;
    p.few_limit = rows / heads;
    // One clip alone has either many or few. few_rows takes all where there are so few that tile_rows' workgroups do not
    // pay: up to 4 turns, or 8 where that is no more than 64 queries. 4 and 8 turns: 8 clips of 4 frames, 8 query heads a
    // key head of 128, bfloat16 32.0 and 31.0 us, float32 91.0 and 87.6; 4 heads of 64 16.3 and 16.0, 22.7 and 20.9; 16
    // clips of 4, 2 heads of 128 27.5 and 26.7, 62.6 and 59.8. With one query head a key head 8 turns are 128 queries: 8
    // clips of 12 take 16.5 and 16.0, 22.9 and 20.8, but 6 float32 clips of up to 50, which go through all of the turns one
    // after another, 19.7 and 25.0.
    const int64_t turns = 8 * p.few_limit <= 64 ? 8 : 4;
    p.all_few = !a.cu_q || a.q_tokens <= (a.n_clips == 1 ? 1 : turns) * p.few_limit;
    p.any_few = p.all_few || a.n_clips != 1;
    if (!p.any_few) p.few_limit = 0;
    p.few_splits = p.tile_splits = 1;
    p.tile_queries = kTileQueries / heads;
    if (p.any_few) {
        const int64_t tiles = (keys + kKeys - 1) / kKeys, base = a.n_clips * columns;
        int64_t n = base > 0 ? (rows == 16 ? kWanted : 768) / base : 1;
        const int64_t most = tiles <= 4 * kWaves ? 1 : tiles / (kWaves * kTurns);
        n = n < most ? n : most;
        p.few_splits = static_cast<int>(n < 1 ? 1 : n < kMaxSplits ? n : kMaxSplits);
    }
    if (!p.all_few) {
        const int64_t slots = a.q_tokens / p.tile_queries + a.n_clips + 1, marked = a.q_tokens / (p.few_limit + 1) + 1;
        if (p.any_few && marked < slots) p.mark = p.few_limit + 1;
        p.tile_slots = static_cast<int>(p.mark ? marked : slots);
        const int64_t tiles = (keys + kTileRows - 1) / kTileRows;
        const int64_t full = a.q_tokens / p.tile_queries;      // blocks of queries, those at clips' ends not counted
        const int64_t groups = (full > 0 ? full : 1) * columns;
        int64_t n = wanted_tiles / groups;
        n = n < tiles / least_tiles ? n : tiles / least_tiles;
        if (a.dtype != RVQ_F32 && a.dim == 64) {
            const int64_t third = 768 / groups < tiles / 32 ? 768 / groups : tiles / 32;
            n = n > third ? n : third;
        }
        p.tile_splits = static_cast<int>(n < 1 ? 1 : n < kMaxSplits ? n : kMaxSplits);
    }
    p.join_clips = !p.all_few && p.tile_splits == 1 && static_cast<int64_t>(a.n_clips) * p.few_limit < a.q_tokens;
    p.few_rows = p.few_splits > 1 ? (p.all_few ? a.q_tokens : static_cast<int64_t>(a.n_clips) * p.few_limit) * a.q_heads : 0;
    p.tile_rows = p.tile_splits > 1 ? a.q_tokens * a.q_heads : 0;
    p.factor = fmaxf(a.scale * kLog2e, FLT_MIN);   // scale 0: equal weights, and 0 times -inf does not arise
    const int64_t few = stats_floats(p.few_rows * p.few_splits) + p.few_rows * p.few_splits * a.dim;
    const int64_t tile = stats_floats(p.tile_rows * p.tile_splits) + p.tile_rows * p.tile_splits * a.dim;
    p.few = static_cast<float *>(a.workspace);
    p.tile = p.few + few;
    floats = few + tile;
    return p;
}

template <typename T, int kD, typename Keys>
hipError_t run(const RowsArgs &a, Plan p, hipStream_t stream)
{
    const int64_t columns = static_cast<int64_t>(a.kv_heads) * p.chunks;
    // whole rounds of the chiplets
    const int64_t blocks = static_cast<int64_t>(a.n_clips) * p.few_splits;
    const int64_t few = !p.any_few ? 0 : (p.by_chiplet ? (blocks + 7) / 8 * 8 : blocks) * columns;
    const int64_t tile = p.tile_slots * static_cast<int64_t>(p.tile_splits) * columns;
    const bool join = p.few_splits > 1 || p.tile_splits > 1;
    const int64_t join_rows_x = p.join_clips ? static_cast<int64_t>(a.n_clips) * p.few_limit : a.q_tokens;
    const int join_heads = (a.q_heads + kJoined<kD> - 1) / kJoined<kD>;
    if (!fits(few + tile, kThreads) || (join && !fits(join_rows_x * join_heads, 64))) return hipErrorNotSupported;
    const bool one = p.few_limit * ((p.group + p.chunks - 1) / p.chunks) <= 16;
    const unsigned n = static_cast<unsigned>(few + tile);
    if (p.all_few && one) only_few_rows<T, kD, Keys, 1><<<n, kThreads, 0, stream>>>(a, p);
    else if (p.all_few) only_few_rows<T, kD, Keys, 2><<<n, kThreads, 0, stream>>>(a, p);
    else if (one) all_rows<T, kD, Keys, 1><<<n, kThreads, 0, stream>>>(a, p, static_cast<int>(tile));
    else all_rows<T, kD, Keys, 2><<<n, kThreads, 0, stream>>>(a, p, static_cast<int>(tile));
    if (join) join_rows<T, kD, Keys><<<dim3(static_cast<unsigned>(join_rows_x), join_heads), 64, 0, stream>>>(a, p);
    return hipGetLastError();
}

template <template <typename, int> class Keys>
hipError_t launch(const RowsArgs &a, const Plan &p, hipStream_t stream)
{
    if (a.dtype == RVQ_F32)
        return a.dim == 64 ? run<float, 64, Keys<float, 64>>(a, p, stream) : run<float, 128, Keys<float, 128>>(a, p, stream);
    if (a.dtype == RVQ_F16)
        return a.dim == 64 ? run<f16_t, 64, Keys<f16_t, 64>>(a, p, stream) : run<f16_t, 128, Keys<f16_t, 128>>(a, p, stream);
    return a.dim == 64 ? run<bf16_t, 64, Keys<bf16_t, 64>>(a, p, stream) : run<bf16_t, 128, Keys<bf16_t, 128>>(a, p, stream);
}

}  // namespace rows
}  // namespace rvq
