// Tiles of head rows in the LDS, and the matrix operands read from them along
// the rows or across them.
//
// A tile lies row after row, 16 bytes a piece; the pieces of a row are
// exchanged (place) so that reads along the rows (16 neighbouring rows, the
// same piece) and across them (4 neighbouring rows, 64 bytes each) spread over
// all banks. Rows come straight from global memory into the LDS, each lane
// picking the piece that belongs to its place.
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

template <typename T, int kD, int kWaves>
struct Tile {
    static constexpr int kRowBytes = kD * static_cast<int>(sizeof(T));
    static constexpr int kBytes = kTileRows * kRowBytes;
    static constexpr int kPiece = 16 / static_cast<int>(sizeof(T));   // values in 16 bytes
    static constexpr int kRowPieces = kRowBytes / 16;
    static constexpr int kCopies = kTileRows * kRowPieces / (64 * kWaves);
    static_assert(kCopies >= 1, "tile smaller than the workgroup");

    __device__ static int place(int row, int piece)
    {
        return piece ^ (kRowPieces >= 16 ? (row & 3) << 2 | ((row >> 2) & 3) : ((row >> 1) & 1) << 2 | ((row >> 2) & 3));
    }

    // What a lane needs to bring tiles of rows `stride` values apart into the LDS: the offset of each of its pieces
    // from the tile's first row. 64 rows span less than 2^31 bytes.
    struct Loader {
        uint32_t offset[kCopies];
        uint32_t step;      // bytes from row to row

        __device__ Loader(int64_t stride)
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
        const char *r = s + row * kRowBytes;
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const vec8<T> *>(r + place(row, k8) * 16);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(r + place(row, 2 * k8) * 16);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(r + place(row, 2 * k8 + 1) * 16);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Operand across the rows: lane l gets dim 32 n + l % 32 of rows 16 step + 4 half .. + 3 and 16 step + 8 + 4 half
    // .. + 3 (half = l / 32), the order in which a 32-wide product leaves its results. 16-bit values are transposed by
    // the LDS read: of each 16 lanes, lanes 4 r .. 4 r + 3 point at 16 neighbouring values of row r, and lane i gets
    // the four rows' value i.
    __device__ static vec8<T> across(const char *s, int n, int step)
    {
        const int lane = threadIdx.x & 63, half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
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
        } else {
            vec8<T> x;
            const int dim = 32 * n + (lane & 31);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 16 * step + 8 * (e >> 2) + 4 * half + (e & 3);
                x[e] = *reinterpret_cast<const float *>(s + row * kRowBytes + place(row, dim >> 2) * 16 + (dim & 3) * 4);
            }
            return x;
        }
    }

    // Values of the tile that are not finite become 0; or, as markers, they become 1 and all others 0. Every thread
    // of the workgroup takes part, barriers are the caller's.
    __device__ static void only_finite(char *s, bool markers)
    {
        T *x = reinterpret_cast<T *>(s);
        for (int i = threadIdx.x; i < kTileRows * kD; i += 64 * kWaves) {
            const float y = to_float(x[i]);
            const bool fine = y - y == 0.0f;
            x[i] = static_cast<T>(markers ? (fine ? 0.0f : 1.0f) : (fine ? y : 0.0f));
        }
    }
};

}  // namespace rvq
