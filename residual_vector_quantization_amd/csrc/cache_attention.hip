// Attention of every clip's newest frame over its paged key-value cache.
//
//   x_j = scale q . k_j over the frames j that are seen, out = sum_j exp(x_j) v_j / sum_j exp(x_j)
//
// Bound by HBM: every seen key and value is read once, 4 G dim flops for its
// 4 dim (16-bit) bytes with G query heads a key head. Measured: 12 clips of up to
// 45000 frames, 32 heads of 128 over 8, pages of 64, bfloat16: 1.35 GB in 244 us,
// 5.5 TB/s; 96 clips, window 1500, 16 heads of 64, float16: 0.59 GB in 102 us, 5.8
// TB/s (a large copy reaches 4.95 TB/s); one clip of 1500 frames: 5.4 us and 3.5
// us for the join. The G query heads of a
// key head (16 at most at a time) are the columns of 16-wide matrix products:
//   S^T [frame][query] = K Q^T: a K operand is 8 neighbouring dims of a frame,
//     which a lane loads from the cache as they are;
//   O^T [dim][query] = V^T P^T: a V^T operand is 8 frames at one dim. A lane
//     loads 8 dims of 8 frames (16 lanes a row, so each load of the wavefront
//     covers whole rows) and transposes the 8 x 8 values in its registers.
// The frames of S^T's rows are numbered so that the scores a lane holds belong
// to the 8 frames of its V^T operand: weights go from one product into the
// next without leaving the lane, and keys and values never enter the LDS.
// Weights enter the second product in the cache's type, rounded once (half a step
// of theirs beside the result's own, as in the windowed attention); their sum is
// of the unrounded ones. float16 weights are taken times 2^kShift: half a step is
// then 2^-32 of the largest, so that a long cache's many small ones are not lost
// beside a large one.
//
// A wavefront takes tiles of 32 seen frames; its running maximum moves only
// when a score exceeds it by more than 2^8, so most tiles need neither an
// exchange between lanes nor a rescale (weights stay below 2^8, sums are
// float32). When clips and heads alone do not fill the chip, a clip's frames go
// to 8 wavefronts of a workgroup instead of 4, and where that leaves each more
// than kManyTiles tiles they are split over workgroups: each split leaves its
// maximum, sum and accumulator in the workspace and a second launch joins them
// in order.
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "attention_device.h"
#include "attention_internal.h"
#include "attention_tiles.h"
#include "cache_index.h"

namespace rvq {
namespace {

constexpr int kWaves = 4;            // wavefronts of a workgroup; kWideWaves in a few workgroups with few frames
constexpr int kWideWaves = 8;
constexpr int kManyTiles = 2;
constexpr int kTile = 32;            // frames a wavefront takes at a time
constexpr int kQueries = 16;         // columns of the products
constexpr float kSlack = 8.0f;       // how far (powers of two) a score may exceed the running maximum
constexpr int kWantedGroups = 2048;  // workgroups that fill the chip evenly (8 a CU)
constexpr int kMaxSplits = 256;
constexpr int kCus = 256;

struct Params {
    CacheAttentionArgs a;
    Divisor page;
    int group, chunks, splits;       // query heads a key head, 16-wide chunks of them, splits of a clip's frames
    bool wide;                       // kWideWaves wavefronts a workgroup
    float factor;                    // scale in powers of two
};

// Partial results of a split: [clip][query head][split] of { max, sum } and [dim].
struct Partials {
    float *stats, *out;
};

// kN values of 8 frames, as the kN operands of 8 frames at one dim.
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

// Maximum over the four lane groups that hold one query.
__device__ inline float over_groups_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

__device__ inline float over_groups_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

template <typename T, int kD, int kWaves>
__global__ __launch_bounds__(64 * kWaves)
void newest_frame(Params p, Partials part)
{
    constexpr int kSteps = kD / 32;      // products along the head dim
    constexpr int kN = kD / 16;          // dims a lane holds of a value row
    constexpr float kShift = kNarrow<T> ? 15.0f - kSlack : 0.0f;      // weights are below 2^(kSlack + kShift)
    __shared__ float s_out[kWaves][kQueries][kD + 4];
    __shared__ float s_max[kWaves][kQueries], s_sum[kWaves][kQueries];
    const CacheAttentionArgs &a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    // heads change fastest, then splits, then clips
    const int columns = a.kv_heads * p.chunks;
    const int rest = blockIdx.x / columns, column = blockIdx.x - rest * columns;
    const int kv = column / p.chunks, chunk = column - kv * p.chunks;
    const int clip = rest / p.splits, split = rest - clip * p.splits;
    const int head0 = kv * p.group + chunk * kQueries, heads = min(kQueries, p.group - chunk * kQueries);
    // a count beyond the table: nothing is read and the result is NaN
    const int len = a.lens[clip];
    const bool beyond = len > static_cast<int64_t>(a.table_ld) * a.page_size;
    const Seen seen = seen_frames(beyond ? 0 : len, a.window, a.sinks);
    const int32_t *row = a.table + static_cast<int64_t>(clip) * a.table_ld;
    const T *keys = static_cast<const T *>(a.k_pool), *values = static_cast<const T *>(a.v_pool);

    vec8<T> q[kSteps];
    {
        const T *at = static_cast<const T *>(a.q.data) + clip * a.q.token + (head0 + min(c, heads - 1)) * a.q.head;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) q[t] = load8(at + 32 * t + 8 * g);
    }
    f32x4 o[kN] = {};
    float m = -INFINITY, l = 0.0f;
    bool bad = beyond;

    const int tiles = (seen.count + kTile - 1) / kTile;
    const int per = (tiles + p.splits - 1) / p.splits;
    const int last = min(tiles, (split + 1) * per);
    // lane n holds the pool row of the tile's frame n % 32
    auto find = [&](int tile) -> uint32_t {
        const int nth = tile * kTile + (lane & 31);
        if (tile >= last || nth >= seen.count) return kPastEnd;
        return cache_row(row, seen_position(seen, nth), p.page, a.table_ld, a.n_pages, a.kv_heads, kv);
    };
    int tile = split * per + wave;
    uint32_t mine = find(tile);
    for (; tile < last; tile += kWaves) {
        const bool whole = __all(mine < kPastEnd);
        bad = bad || mine == kNoPage;
        vec8<T> k[2][kSteps];
        Block8<T, kN> v;
        uint32_t kr[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) kr[b] = __shfl(mine, 8 * (c >> 2) + 4 * b + (c & 3));
        if (whole) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < kSteps; ++t) k[b][t] = load8(keys + static_cast<uint64_t>(kr[b]) * kD + 32 * t + 8 * g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v.load(i, values + static_cast<uint64_t>(__shfl(mine, 8 * g + i)) * kD + kN * c);
        } else {
            // rows that are not there are zeros: their weights are 0, and nothing is read for them
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < kSteps; ++t) {
                    k[b][t] = vec8<T>{};
                    if (kr[b] < kPastEnd) k[b][t] = load8(keys + static_cast<uint64_t>(kr[b]) * kD + 32 * t + 8 * g);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = __shfl(mine, 8 * g + i);
                v.clear(i);
                if (r < kPastEnd) v.load(i, values + static_cast<uint64_t>(r) * kD + kN * c);
            }
        }
        const uint32_t next = find(tile + kWaves);

        // scores in powers of two: frame 8 g + 4 b + i of the tile, query c
        f32x4 x[2] = {};
#pragma unroll
        for (int t = 0; t < kSteps; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b) x[b] = mma16(k[b][t], q[t], x[b]);
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[b][i] *= p.factor;
                if (!whole) x[b][i] = __shfl(mine, 8 * g + 4 * b + i) < kPastEnd ? x[b][i] : -INFINITY;
                top = fmaxf(top, x[b][i]);
            }
        if (__any(top > m + kSlack)) {
            top = over_groups_max(top);
            if (top > m + kSlack) {
                const float keep = fast_exp2(m - top);
                m = top;
                l *= keep;
#pragma unroll
                for (int n = 0; n < kN; ++n) o[n] *= keep;
            }
        }
        const float safe = m == -INFINITY ? 0.0f : m - kShift;
        vec8<T> w;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = fast_exp2(x[b][i] - safe);
                l += e;
                w[4 * b + i] = static_cast<T>(e);
            }
#pragma unroll
        for (int n = 0; n < kN; ++n) o[n] = mma16(v.at(n), w, o[n]);
        mine = next;
    }

    // join the workgroup's wavefronts
    l = over_groups_sum(l);
    if (__any(bad)) l = __builtin_nanf("");
    if (g == 0) {
        s_max[wave][c] = m;
        s_sum[wave][c] = l;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_out[wave][c][kN * (4 * g + i) + n] = o[n][i];
    __syncthreads();
    const int64_t heads_before = static_cast<int64_t>(clip) * a.q_heads + head0;
    for (int at = threadIdx.x; at < heads * kD; at += 64 * kWaves) {
        const int h = at / kD, d = at - h * kD;
        float top = -INFINITY, sum = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_max[w][h]);
        const float safe = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = fast_exp2(s_max[w][h] - safe);
            sum += s_sum[w][h] * f;
            y += s_out[w][h][d] * f;
        }
        if (p.splits == 1) {
            T *out = static_cast<T *>(a.out.data) + clip * a.out.token + (head0 + h) * a.out.head;
            out[d] = static_cast<T>(sum == 0.0f ? 0.0f : y / sum);
        } else {
            const int64_t slot = (heads_before + h) * p.splits + split;
            part.out[slot * kD + d] = y;
            if (d == 0) {
                part.stats[2 * slot] = top;
                part.stats[2 * slot + 1] = sum;
            }
        }
    }
}

// One wavefront a clip and query head: lanes find the largest maximum and the scaled sums over the splits, then
// add up the accumulators, a lane kD / 64 dims.
template <typename T, int kD>
__global__ __launch_bounds__(64)
void join_splits(Params p, Partials part)
{
    const CacheAttentionArgs &a = p.a;
    const int clip = blockIdx.x, head = blockIdx.y, lane = threadIdx.x;
    const int64_t slot = (static_cast<int64_t>(clip) * a.q_heads + head) * p.splits;
    __shared__ float s_factor[kMaxSplits];
    float top = -INFINITY;
    for (int s = lane; s < p.splits; s += 64) top = fmaxf(top, part.stats[2 * (slot + s)]);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float safe = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int s = lane; s < p.splits; s += 64) {
        const float f = fast_exp2(part.stats[2 * (slot + s)] - safe);
        s_factor[s] = f;
        sum += part.stats[2 * (slot + s) + 1] * f;
    }
    sum = wave_sum(sum);
    __syncthreads();
    float y[kD / 64] = {};
    for (int s = 0; s < p.splits; ++s)
#pragma unroll
        for (int i = 0; i < kD / 64; ++i) y[i] += part.out[(slot + s) * kD + 64 * i + lane] * s_factor[s];
    T *out = static_cast<T *>(a.out.data) + clip * a.out.token + head * a.out.head;
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) out[64 * i + lane] = static_cast<T>(sum == 0.0f ? 0.0f : y[i] / sum);
}

// How many splits of a clip's frames: enough workgroups to fill the chip, none with less than a tile a wavefront.
// It depends on shapes alone, so that the workspace's size is known beforehand.
int splits_for(int n_clips, int kv_heads, int group, int64_t capacity)
{
    const int64_t base = static_cast<int64_t>(n_clips) * kv_heads * ((group + kQueries - 1) / kQueries);
    const int64_t tiles = (capacity + kTile - 1) / kTile;
    int64_t n = base > 0 ? kWantedGroups / base : 1;
    // the second launch costs about 3 us, as much as a tile of a wavefront that nothing hides
    const int64_t most = tiles <= kWideWaves * kManyTiles ? 1 : tiles / kWaves;
    if (n > most) n = most;
    if (n > kMaxSplits) n = kMaxSplits;
    return n < 1 ? 1 : static_cast<int>(n);
}

int64_t stats_floats(int64_t slots) { return (2 * slots + 3) / 4 * 4; }

template <typename T, int kD>
hipError_t run(const Params &p, hipStream_t stream)
{
    const CacheAttentionArgs &a = p.a;
    Partials part = {};
    if (p.splits > 1) {
        part.stats = static_cast<float *>(a.workspace);
        part.out = part.stats + stats_floats(static_cast<int64_t>(a.n_clips) * a.q_heads * p.splits);
    }
    const int64_t groups = static_cast<int64_t>(a.n_clips) * p.splits * a.kv_heads * p.chunks;
    if (!fits(groups, 64 * (p.wide ? kWideWaves : kWaves))) return hipErrorNotSupported;
    if (p.wide) newest_frame<T, kD, kWideWaves><<<static_cast<unsigned>(groups), 64 * kWideWaves, 0, stream>>>(p, part);
    else newest_frame<T, kD, kWaves><<<static_cast<unsigned>(groups), 64 * kWaves, 0, stream>>>(p, part);
    if (p.splits > 1) join_splits<T, kD><<<dim3(a.n_clips, a.q_heads), 64, 0, stream>>>(p, part);
    return hipGetLastError();
}

}  // namespace

int64_t cache_attention_bytes(int n_clips, int q_heads, int kv_heads, int dim, int64_t capacity)
{
    const int splits = splits_for(n_clips, kv_heads, q_heads / kv_heads, capacity);
    if (splits == 1) return 0;
    const int64_t slots = static_cast<int64_t>(n_clips) * q_heads * splits;
    return (stats_floats(slots) + slots * dim) * 4;
}

hipError_t launch_cache_attention(const CacheAttentionArgs &a, hipStream_t stream)
{
    Params p = {};
    p.a = a;
    p.page = divisor(a.page_size);
    p.group = a.q_heads / a.kv_heads;
    p.chunks = (p.group + kQueries - 1) / kQueries;
    // no more frames than the window and the sinks hold; the workspace is sized for the table's capacity
    const int64_t capacity = static_cast<int64_t>(a.table_ld) * a.page_size;
    const int64_t seen = static_cast<int64_t>(a.window) + a.sinks;
    const int64_t frames = seen < capacity ? seen : capacity;
    p.splits = splits_for(a.n_clips, a.kv_heads, p.group, frames);
    p.wide = p.splits == 1 && frames > kWaves * kTile && static_cast<int64_t>(a.n_clips) * a.kv_heads * p.chunks <= kCus;
    p.factor = fmaxf(a.scale * kLog2e, FLT_MIN);   // scale 0: equal weights, and 0 times -inf does not arise
    if (a.dtype == RVQ_F32) return a.dim == 64 ? run<float, 64>(p, stream) : run<float, 128>(p, stream);
    if (a.dtype == RVQ_F16) return a.dim == 64 ? run<f16_t, 64>(p, stream) : run<f16_t, 128>(p, stream);
    return a.dim == 64 ? run<bf16_t, 64>(p, stream) : run<bf16_t, 128>(p, stream);
}

}  // namespace rvq
