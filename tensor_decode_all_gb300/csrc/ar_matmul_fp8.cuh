// ar_matmul_fp8.cuh -- what the kernels of ar_matmul_fp8 share: the call as they see it, and which rows and
// weights a tile of it takes.
#pragma once

#include <cuda.h>

#include "ar_ffn.h"
#include "ar_kv4.cuh"
#include "ar_tensor.cuh"

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

// Rows of x that are picked by number, N of them, copied a group of channels at a time by one warp: 16 bytes to a lane, eight lanes to a row, in the
// order that the copy engine gives a tile's rows.  Where there is no row, another or none is copied: what comes of it is not used.
// (Two or three instructions to a copy: a warp has no time for more.)
template <int N> struct Picked {
    uint32_t at[N / 4];          // of row 4 i + which, in 16 bytes from x on
    int here;                    // rows that are there
    __device__ __forceinline__ void look_up(const ar_matmul_fp8_args &a, int first, int count) {
        const int64_t stride = a.x_rows > 1 ? a.x_stride / 16 : 0;
        here = count;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const int j = 4 * i + (threadIdx.x >> 3 & 3);
            at[i] = (uint32_t)(j < count ? max(source_row(a, first + j), (int64_t)0) * stride : 0);
        }
    }
    __device__ __forceinline__ void copy(const ar_matmul_fp8_args &a, uint32_t to, int group) const {
        const int piece = threadIdx.x & 7, which = threadIdx.x >> 3 & 3, channel = group * kBlock + piece * 16, bytes = max(0, min(a.dim - channel, 16));
        const uint8_t *from = static_cast<const uint8_t *>(a.x) + (bytes ? channel : 0);
        const uint32_t even = to + which * kBlock + ((piece ^ which) << 4), odd = to + which * kBlock + ((piece ^ (which + 4)) << 4);
        // Few rows: none is copied that is not there.  Many: eight copies at a time, so that their addresses are there before the first.
        constexpr int M = N <= 32 ? 1 : 8;
#pragma unroll
        for (int i0 = 0; i0 < N / 4; i0 += M) {
            if (4 * i0 >= here) break;
            const uint8_t *p[M];
#pragma unroll
            for (int i = 0; i < M; ++i) p[i] = from + (uint64_t)at[i0 + i] * 16;
#pragma unroll
            for (int i = 0; i < M; ++i) copy_piece(((i0 + i) & 1 ? odd : even) + (i0 + i) * 4 * kBlock, p[i], bytes);
        }
    }
};

// How the copy engine sees the weight, a box of `box` features of a group; and the rows of x, a box of `box` rows.  False: it cannot (the addresses and strides are checked before).
bool map_weight(CUtensorMap *m, const ar_matmul_fp8_args &a, int box);
bool map_rows(CUtensorMap *m, const ar_matmul_fp8_args &a, int box);

// Bytes from a picked row to the next in the workspace.
inline int64_t pitch_of(const ar_matmul_fp8_args &a) { return ((int64_t)a.dim + 15) / 16 * 16; }

// The kernels for rows on 16 bytes, and the first error that each has recorded (and forgets).
cudaError_t start_few(const Product &p, cudaStream_t s, int multiprocessors);
int take_few_status(int *code);
cudaError_t start_many(const Product &p, cudaStream_t s, int multiprocessors);
int take_many_status(int *code);

}  // namespace tda
