// ar_matmul_fp8.cuh -- what the kernels of ar_matmul_fp8 share: the call as they see it, and which rows and
// weights a tile of it takes.
#pragma once

#include <cuda.h>

#include "ar_ffn.h"
#include "ar_kv4.cuh"

namespace tda {

constexpr int kBlock = 128;      // channels, and features of a weight, that share a scale

struct Product {
    ar_matmul_fp8_args a;
    int groups;                  // groups of 128 channels
};

// A tile's rows: first .. first + count - 1 of the call, of one expert.  count 0: the tile is not there.
struct Rows {
    int expert, first, count;
};

__device__ __forceinline__ int clamp_row(int v, int64_t rows) { return v < 0 ? 0 : v > rows ? (int)rows : v; }

// Which rows tile number `tile` of up to `size` rows takes; the whole warp calls it.  Experts' tiles are
// numbered in the experts' order, none for an expert without rows.
__device__ __forceinline__ Rows rows_of_tile(const ar_matmul_fp8_args &a, int64_t tile, int size) {
    if (!a.offsets) {
        const int64_t first = tile * size;
        return first < a.rows ? Rows{0, (int)first, (int)min((int64_t)size, a.rows - first)} : Rows{0, 0, 0};
    }
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        int begin = 0, n = 0;
        if (e < a.experts) {
            begin = clamp_row(a.offsets[e], a.rows);
            n = max(clamp_row(a.offsets[e + 1], a.rows) - begin, 0);
        }
        const int own = (n + size - 1) / size;
        int run = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(~0u, run, d);
            if (lane >= d) run += x;
        }
        const bool mine = tile >= before + run - own && tile < before + run;
        const unsigned who = __ballot_sync(~0u, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            const int at = (int)(tile - before - (run - own)) * size;
            return Rows{e0 + src, __shfl_sync(~0u, begin + at, src), __shfl_sync(~0u, min(size, n - at), src)};
        }
        before += __shfl_sync(~0u, run, 31);
    }
    return Rows{0, 0, 0};
}

// How many tiles of `size` rows there are; the whole warp calls it.
__device__ __forceinline__ int64_t tiles_of_rows(const ar_matmul_fp8_args &a, int size) {
    if (!a.offsets) return (a.rows + size - 1) / size;
    int64_t n = 0;
    for (int e = threadIdx.x & 31; e < a.experts; e += 32)
        n += (max(clamp_row(a.offsets[e + 1], a.rows) - clamp_row(a.offsets[e], a.rows), 0) + size - 1) / size;
#pragma unroll
    for (int d = 16; d; d /= 2) n += __shfl_xor_sync(~0u, n, d);
    return n;
}

// The most tiles of `size` rows that a call can have, whatever its offsets.
inline int64_t most_tiles(const ar_matmul_fp8_args &a, int size) {
    const int64_t whole = (a.rows + size - 1) / size;
    return a.offsets ? a.rows / size + (a.rows < a.experts ? a.rows : a.experts) : whole;
}

// The row of x that a row of the call belongs to; -1: none.
__device__ __forceinline__ int64_t source_row(const ar_matmul_fp8_args &a, int64_t row) {
    if (!a.row_of) return row;
    const int r = a.row_of[row];
    return r >= 0 && r < a.x_rows ? r : -1;
}

// How the copy engine sees the weight, a box of `box` features of a group; and the rows of x, a box of `box` rows,
// or one where they are picked by number.  False: it cannot (the addresses and strides are checked before).
bool map_weight(CUtensorMap *m, const ar_matmul_fp8_args &a, int box);
bool map_rows(CUtensorMap *m, const ar_matmul_fp8_args &a, int box);

// The kernels for rows on 16 bytes, and the first error that each has recorded (and forgets).
cudaError_t start_few(const Product &p, cudaStream_t s, int multiprocessors);
int take_few_status(int *code);
cudaError_t start_many(const Product &p, cudaStream_t s, int multiprocessors);
int take_many_status(int *code);

}  // namespace tda
