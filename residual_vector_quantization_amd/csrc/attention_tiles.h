// Tiles of 64 rows of head values on their way from global memory through
// registers into the LDS, as they are or transposed, and the matrix operands
// read back from there.
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
__device__ inline void store4(float *p, const float (&x)[4]) { *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]}; }
template <typename T>
__device__ inline void store4(T *p, const T (&x)[4])
{
    typedef T four __attribute__((ext_vector_type(4)));
    *reinterpret_cast<four *>(p) = four{x[0], x[1], x[2], x[3]};
}

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

template <typename T, int kD, int kThreads>
struct Tiles {
    static constexpr int kBytes = kTileRows * kD * static_cast<int>(sizeof(T));
    static constexpr int kPiece = 16 / static_cast<int>(sizeof(T));   // values in 16 bytes
    static constexpr int kRowPieces = kD / kPiece;
    static constexpr int kCount = kTileRows * kRowPieces / kThreads;  // 16-byte pieces a thread
    // transposed tiles come in as units of 4 rows and kWide columns, so that every thread has one or more
    static constexpr int kWide = sizeof(T) == 2 && kD == 128 ? 8 : 4;
    static constexpr int kUnitCols = kD / kWide;
    static constexpr int kUnits = kTileRows / 4 * kUnitCols / kThreads;
    static_assert(kCount >= 1 && kUnits >= 1, "tile smaller than the workgroup");

    struct Piece { u32x4 x[kCount]; };
    typedef T Part __attribute__((ext_vector_type(kWide)));
    struct Group { Part x[kUnits][4]; };

    // Exchange of the 16-byte pieces of a row: 16 neighbouring rows (of 8 pieces: pairs of rows) put the same piece
    // in different banks.
    __device__ static int row_place(int row, int piece)
    {
        return piece ^ (kRowPieces >= 16 ? row & 15 : (row >> 1) & 7);
    }
    // The same for a transposed row (64 values of one dim: 8 or 16 pieces), where the writes of one instruction are
    // kWide dims apart.
    __device__ static int dim_place(int dim, int piece)
    {
        return piece ^ (sizeof(T) == 2 ? ((dim >> 1) ^ (dim >> 3)) & 7 : (dim ^ (dim >> 3)) & 15);
    }

    // Rows first .. first + 63 of `rows`, zeros from row `end` on.
    __device__ static void fetch_rows(Piece &p, const T *rows, int64_t stride, int first, int end)
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            const int at = n * kThreads + threadIdx.x, row = first + at / kRowPieces, col = at % kRowPieces;
            p.x[n] = u32x4{0, 0, 0, 0};
            if (row < end) p.x[n] = *reinterpret_cast<const u32x4 *>(rows + row * stride + col * kPiece);
        }
    }
    __device__ static void store_rows(char *s, const Piece &p)
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            const int at = n * kThreads + threadIdx.x, row = at / kRowPieces, col = at % kRowPieces;
            *reinterpret_cast<u32x4 *>(s + (row * kRowPieces + row_place(row, col)) * 16) = p.x[n];
        }
    }
    // 8 values of row `row` from 8 * k8 on.
    __device__ static vec8<T> row_operand(const char *s, int row, int k8)
    {
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const vec8<T> *>(s + (row * kRowPieces + row_place(row, k8)) * 16);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(s + (row * kRowPieces + row_place(row, 2 * k8)) * 16);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(s + (row * kRowPieces + row_place(row, 2 * k8 + 1)) * 16);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    __device__ static void fetch_groups(Group &g, const T *rows, int64_t stride, int first, int end)
    {
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int at = n * kThreads + threadIdx.x, four = at / kUnitCols, col = at % kUnitCols;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = first + 4 * four + i;
                g.x[n][i] = Part{};
                if (row < end) g.x[n][i] = *reinterpret_cast<const Part *>(rows + row * stride + col * kWide);
            }
        }
    }
    // Row d of the transposed tile holds the 64 rows' values at dim d. 16-bit: 16-byte piece 2 s + half holds rows
    // 16 s + 4 half .. + 3 and 16 s + 8 + 4 half .. + 3, the order in which a 32-wide product leaves its results.
    __device__ static void store_transposed(char *s, const Group &g)
    {
        typedef T Four __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int at = n * kThreads + threadIdx.x, four = at / kUnitCols, col = at % kUnitCols;
#pragma unroll
            for (int j = 0; j < kWide; ++j) {
                const int dim = col * kWide + j;
                const Four y = {g.x[n][0][j], g.x[n][1][j], g.x[n][2][j], g.x[n][3][j]};
                char *row = s + dim * kTileRows * static_cast<int>(sizeof(T));
                if constexpr (sizeof(T) == 2) {
                    const int piece = 2 * (four >> 2) + (four & 1), part = (four >> 1) & 1;
                    *reinterpret_cast<Four *>(row + dim_place(dim, piece) * 16 + part * 8) = y;
                } else {
                    *reinterpret_cast<Four *>(row + dim_place(dim, four) * 16) = y;
                }
            }
        }
    }
    // Rows 16 s + 4 half .. + 3 and 16 s + 8 + 4 half .. + 3 at dim `dim`.
    __device__ static vec8<T> transposed_operand(const char *s, int dim, int step, int half)
    {
        const char *row = s + dim * kTileRows * static_cast<int>(sizeof(T));
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const vec8<T> *>(row + dim_place(dim, 2 * step + half) * 16);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(row + dim_place(dim, 4 * step + half) * 16);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(row + dim_place(dim, 4 * step + 2 + half) * 16);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Values that are not finite become 0; or, as markers, they become 1 and all others 0.
    __device__ static void only_finite(Group &g, bool markers)
    {
#pragma unroll
        for (int n = 0; n < kUnits; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < kWide; ++j) {
                    const float x = to_float(g.x[n][i][j]);
                    const bool fine = x - x == 0.0f;
                    g.x[n][i][j] = static_cast<T>(markers ? (fine ? 0.0f : 1.0f) : (fine ? x : 0.0f));
                }
    }
};

}  // namespace rvq
