// Tiles of head rows in the LDS, and the matrix operands read from them along
// the rows or across them.
//
// A tile of 16-bit values lies row after row, 16 bytes a piece; the pieces of a
// row are exchanged (place) so that reads along the rows (16 neighbouring rows,
// the same piece) and across them (4 neighbouring rows, 64 bytes each) spread
// over all banks. Rows come straight from global memory into the LDS, each lane
// picking the piece that belongs to its place. A tile of float32 values is
// three such tiles, of their bfloat16 parts: a workgroup splits each value
// once, on the way from registers into the LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention_device.h"

namespace rvq {

constexpr int kTileRows = 64;

__device__ inline f32x8 load8(const float *p)
{
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ inline f16x8 load8(const f16_t *p) { return *reinterpret_cast<const f16x8 *>(p); }
__device__ inline bf16x8 load8(const bf16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Four neighbouring values in one store.
template <typename T>
__device__ inline void store4(T *p, const T (&x)[4])
{
    typedef T four __attribute__((ext_vector_type(4)));
    *reinterpret_cast<four *>(p) = four{x[0], x[1], x[2], x[3]};
}

typedef __attribute__((address_space(3))) void lds_void;

// One wavefront-wide copy from global memory into the LDS: lane i's 16 (4) bytes at src + offset (offset in the lane,
// src the same for all) go to dst + 16 i (4 i), dst the same for all lanes. Issued as inline assembly so that the
// compiler does not order every LDS read behind it; the caller waits with wait_copies and a barrier. The instruction
// needs 1 wait state after a scalar write of m0 and 5 after a vector instruction's write of a scalar register that it
// reads (src brought back from a spill), which the compiler does not see to inside inline assembly.
__device__ inline void copy16(const void *src, uint32_t offset, void *dst)
{
    const unsigned m0 = static_cast<unsigned>(reinterpret_cast<size_t>((lds_void *)dst));
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(src), "{m0}"(m0) : "memory");
}
__device__ inline void copy4(const void *src, uint32_t offset, void *dst)
{
    const unsigned m0 = static_cast<unsigned>(reinterpret_cast<size_t>((lds_void *)dst));
    asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(offset), "s"(src), "{m0}"(m0) : "memory");
}
// Makes the compiler wait for a loaded operand here. Otherwise it waits where a loop first uses it, in every turn, and
// its count of outstanding loads, which knows nothing of the copies above, then waits for those as well.
template <typename V>
__device__ inline void arrive(V &x)
{
    asm volatile("" : "+v"(x));
}
__device__ inline void arrive(Split8 &x)
{
    arrive(x.high);
    arrive(x.middle);
    arrive(x.low);
}
__device__ inline void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The 64-key tiles that the queries at positions p_first .. p_last see some of: the sinks', then the window's.
struct KeyRange {
    int tiles, sink_tiles, skip;
    __device__ int start(int t) const { return kTileRows * (t < sink_tiles ? t : t + skip); }
};

__device__ inline KeyRange keys_seen(int p_first, int p_last, int window, int sinks)
{
    KeyRange r = {0, 0, 0};
    if (p_last < 0) return r;
    const int64_t low64 = static_cast<int64_t>(p_first) - window + 1;
    const int low = low64 > 0 ? static_cast<int>(low64) : 0;
    const int sunk = min(min(sinks, low), p_last + 1);
    r.sink_tiles = (sunk + kTileRows - 1) / kTileRows;
    const int first = max(r.sink_tiles, low / kTileRows), end = low <= p_last ? p_last / kTileRows + 1 : first;
    r.skip = first - r.sink_tiles;
    r.tiles = r.sink_tiles + max(0, end - first);
    return r;
}

// The position below which a query at p sees only sinks, less 1 (-1 at least).
__device__ inline int below_window(int p, int window)
{
    return static_cast<int>(max(static_cast<int64_t>(p) - window, static_cast<int64_t>(-1)));
}

// 64 rows of 16-bit values.
template <typename T, int kD, int kWaves>
struct Tile {
    static constexpr int kRowBytes = 2 * kD;
    static constexpr int kBytes = kTileRows * kRowBytes;
    static constexpr int kRowPieces = kRowBytes / 16;
    static constexpr int kCopies = kTileRows * kRowPieces / (64 * kWaves);
    static_assert(sizeof(T) == 2 && kCopies >= 1, "tile smaller than the workgroup");

    __device__ static int place(int row, int piece)
    {
        return piece ^ (kRowPieces >= 16 ? (row & 3) << 2 | ((row >> 2) & 3) : ((row >> 1) & 1) << 2 | ((row >> 2) & 3));
    }

    // What a lane needs to bring tiles of rows `stride` values apart into the LDS: the offset of each of its pieces
    // from the tile's first row. 64 rows span less than 2^31 bytes.
    struct Loader {
        uint32_t offset[kCopies];
        uint32_t step;      // bytes from row to row

        __device__ explicit Loader(int64_t stride)
        {
            const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
            step = static_cast<uint32_t>(stride) * static_cast<uint32_t>(sizeof(T));
#pragma unroll
            for (int n = 0; n < kCopies; ++n) {
                const int at = (n * kWaves + wave) * 64 + lane, row = at / kRowPieces;
                offset[n] = row * step + place(row, at % kRowPieces) * 16;
            }
        }
        // Rows first .. first + 63 of `rows` into the tile s, the last one (end - 1) again for rows past the end.
        __device__ void load(char *s, const T *rows, int first, int end) const
        {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const char *from = reinterpret_cast<const char *>(rows) + static_cast<int64_t>(first) * step;
            if (first + kTileRows <= end) {
#pragma unroll
                for (int n = 0; n < kCopies; ++n) copy16(from, offset[n], s + (n * kWaves + wave) * 1024);
            } else {
                const int last = end - 1 - first;
#pragma unroll
                for (int n = 0; n < kCopies; ++n) {
                    const int row = ((n * kWaves + static_cast<int>(threadIdx.x >> 6)) * 64 + static_cast<int>(threadIdx.x & 63)) / kRowPieces;
                    copy16(from, offset[n] - (row > last ? row - last : 0) * step, s + (n * kWaves + wave) * 1024);
                }
            }
        }
    };

    // Operand along the rows: values 8 k8 .. 8 k8 + 7 of a row.
    __device__ static vec8<T> along(const char *s, int row, int k8)
    {
        return *reinterpret_cast<const vec8<T> *>(s + row * kRowBytes + place(row, k8) * 16);
    }

    // Operand across the rows: lane l gets dim 32 n + l % 32 of rows 16 step + 4 half .. + 3 and 16 step + 8 + 4 half
    // .. + 3 (half = l / 32), the order in which a 32-wide product leaves its results. The values are transposed by
    // the LDS read: of each 16 lanes, lanes 4 r .. 4 r + 3 point at 16 neighbouring values of row r, and lane i gets
    // the four rows' value i.
    __device__ static vec8<T> across(const char *s, int n, int step)
    {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int lane = threadIdx.x & 63, half = lane >> 5;
        union { s16x4 part[2]; vec8<T> whole; } u;
        const int i = lane & 15, group = (lane >> 4) & 1;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = 16 * step + 8 * b + 4 * half + (i >> 2);
            const int piece = 4 * n + 2 * group + ((i >> 1) & 1);
            const char *at = s + row * kRowBytes + place(row, piece) * 16 + (i & 1) * 8;
            u.part[b] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at);
        }
        return u.whole;
    }

    // Value i of the tile, in no order of interest, and its rewriting.
    __device__ static float value(const char *s, int i) { return to_float(reinterpret_cast<const T *>(s)[i]); }
    __device__ static void set(char *s, int i, float x) { reinterpret_cast<T *>(s)[i] = static_cast<T>(x); }
};

// 64 rows of float32 values, in three parts.
template <int kD, int kWaves>
struct SplitTile {
    typedef Tile<bf16_t, kD, kWaves> Part;
    static constexpr int kBytes = 3 * Part::kBytes;
    static constexpr int kUnits = kTileRows * kD / 8 / (64 * kWaves);      // 8 values each a thread

    // Rows on their way: fetch sets out, store puts their parts into the tile.
    struct Loader {
        f32x8 x[kUnits];
        int64_t stride;

        __device__ explicit Loader(int64_t row_stride) : stride(row_stride) {}
        __device__ void fetch(const float *rows, int first, int end)
        {
#pragma unroll
            for (int n = 0; n < kUnits; ++n) {
                const int at = n * 64 * kWaves + threadIdx.x, row = at / (kD / 8), piece = at % (kD / 8);
                x[n] = load8(rows + min(first + row, end - 1) * stride + 8 * piece);
            }
        }
        __device__ void store(char *s) const
        {
#pragma unroll
            for (int n = 0; n < kUnits; ++n) {
                const int at = n * 64 * kWaves + threadIdx.x, row = at / (kD / 8), piece = at % (kD / 8);
                const Split8 y(x[n]);
                char *to = s + row * Part::kRowBytes + Part::place(row, piece) * 16;
                *reinterpret_cast<bf16x8 *>(to) = y.high;
                *reinterpret_cast<bf16x8 *>(to + Part::kBytes) = y.middle;
                *reinterpret_cast<bf16x8 *>(to + 2 * Part::kBytes) = y.low;
            }
        }
    };

    __device__ static Split8 along(const char *s, int row, int k8)
    {
        Split8 x;
        x.high = Part::along(s, row, k8);
        x.middle = Part::along(s + Part::kBytes, row, k8);
        x.low = Part::along(s + 2 * Part::kBytes, row, k8);
        return x;
    }
    __device__ static Split8 across(const char *s, int n, int step)
    {
        Split8 x;
        x.high = Part::across(s, n, step);
        x.middle = Part::across(s + Part::kBytes, n, step);
        x.low = Part::across(s + 2 * Part::kBytes, n, step);
        return x;
    }
    // The first part: of a value that is not finite, that value.
    __device__ static float value(const char *s, int i) { return Part::value(s, i); }
    __device__ static void set(char *s, int i, float x)     // a value of 8 bits
    {
        Part::set(s, i, x);
        Part::set(s + Part::kBytes, i, 0.0f);
        Part::set(s + 2 * Part::kBytes, i, 0.0f);
    }
};

template <typename T, int kD, int kWaves> struct RowsOf { typedef Tile<T, kD, kWaves> type; };
template <int kD, int kWaves> struct RowsOf<float, kD, kWaves> { typedef SplitTile<kD, kWaves> type; };

__device__ inline bool fine(float x) { return x - x == 0.0f; }

// Values of a tile that are not finite become 0; or, as markers, +inf becomes 1, -inf kMinus, NaN their sum and all others
// 0. Every thread of the workgroup takes part, barriers are the caller's.
constexpr float kMinus = 0.0078125f;

template <typename Rows, int kD, int kThreads>
__device__ inline void only_finite(char *s, bool markers)
{
    for (int i = threadIdx.x; i < kTileRows * kD; i += kThreads) {
        const float x = Rows::value(s, i);
        if (markers) Rows::set(s, i, fine(x) ? 0.0f : x > 0.0f ? 1.0f : x < 0.0f ? kMinus : 1.0f + kMinus);
        else if (!fine(x)) Rows::set(s, i, 0.0f);
    }
}

// Rows of a tile with a value that is not finite: their flag is set and they become zeros. Barriers are the caller's.
template <typename Rows, int kD, int kThreads>
__device__ inline void clear_bad_rows(char *s, int *flags)
{
    constexpr int kLanes = kThreads / kTileRows;
    const int row = threadIdx.x / kLanes;
    bool bad = false;
    for (int i = threadIdx.x % kLanes; i < kD; i += kLanes) bad = bad || !fine(Rows::value(s, row * kD + i));
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) bad = __shfl_xor(static_cast<int>(bad), m) || bad;
    if (bad) {
        flags[row] = 1;
        for (int i = threadIdx.x % kLanes; i < kD; i += kLanes) Rows::set(s, row * kD + i, 0.0f);
    }
}

// Two arrays of rows (keys and values, or queries and gradients) that go by tile after tile. 16-bit: two tiles of each
// in the LDS, one worked on, one on its way. Float32: one tile of each in the LDS, the next in registers.
template <typename T, int kD, int kWaves>
struct Feed {
    typedef Tile<T, kD, kWaves> Rows;
    static constexpr int kBytes = 4 * Rows::kBytes;
    typename Rows::Loader one, two;
    char *s;

    __device__ Feed(char *memory, int64_t stride_one, int64_t stride_two) : one(stride_one), two(stride_two), s(memory) {}
    __device__ void start(const T *rows_one, const T *rows_two, int first, int end) { load(0, rows_one, rows_two, first, end); }
    // Waits for the tile in `buffer`; then `go` sets out for the next one. Nothing of the tile before is read any more.
    template <int kBuffer>
    __device__ void turn(Constant<kBuffer>, bool go, const T *rows_one, const T *rows_two, int first, int end)
    {
        wait_copies();
        __syncthreads();
        if (go) load(1 - kBuffer, rows_one, rows_two, first, end);
    }
    template <int kBuffer> __device__ char *tile_one(Constant<kBuffer>) const { return s + kBuffer * 2 * Rows::kBytes; }
    template <int kBuffer> __device__ char *tile_two(Constant<kBuffer>) const { return s + (kBuffer * 2 + 1) * Rows::kBytes; }

private:
    __device__ void load(int buffer, const T *rows_one, const T *rows_two, int first, int end)
    {
        one.load(s + buffer * 2 * Rows::kBytes, rows_one, first, end);
        two.load(s + (buffer * 2 + 1) * Rows::kBytes, rows_two, first, end);
    }
};

template <int kD, int kWaves>
struct Feed<float, kD, kWaves> {
    typedef SplitTile<kD, kWaves> Rows;
    static constexpr int kBytes = 2 * Rows::kBytes;
    typename Rows::Loader one, two;
    char *s;

    __device__ Feed(char *memory, int64_t stride_one, int64_t stride_two) : one(stride_one), two(stride_two), s(memory) {}
    __device__ void start(const float *rows_one, const float *rows_two, int first, int end)
    {
        one.fetch(rows_one, first, end);
        two.fetch(rows_two, first, end);
    }
    template <int kBuffer>
    __device__ void turn(Constant<kBuffer>, bool go, const float *rows_one, const float *rows_two, int first, int end)
    {
        wait_copies();
        __syncthreads();
        one.store(s);
        two.store(s + Rows::kBytes);
        __syncthreads();
        if (go) start(rows_one, rows_two, first, end);
    }
    template <int kBuffer> __device__ char *tile_one(Constant<kBuffer>) const { return s; }
    template <int kBuffer> __device__ char *tile_two(Constant<kBuffer>) const { return s + Rows::kBytes; }
};

}  // namespace rvq
