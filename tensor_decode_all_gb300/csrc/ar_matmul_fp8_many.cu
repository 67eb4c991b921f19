// ar_matmul_fp8_many.cu -- products of many rows with an e4m3 weight: the matrix instructions' rate is what counts.
//
// Two blocks of a cluster, on two multiprocessors, share a tile of 256 rows and 256 features: each keeps its 128 rows (the
// lanes) and half of the features' operand, so that a group of 128 channels costs a block 32 KB of copies and as much reading of
// shared memory as writing, which is what 512 cycles of matrix instructions leave time for (a block alone with 128 x 256 would
// copy 48 KB).  Block 0 issues for both.  The instructions sum one group of channels; then eight warps, a row
// and 128 features to a thread, multiply by the two scales and add up in registers, while the next group's sums go to the
// other half of tensor memory.
//
// Blocks stay and go from tile to tile; copies for the next tile are under way while one is stored.  Results leave by way of
// shared memory, 64 bytes of a row at a time.
#include "ar_matmul_fp8.cuh"
#include "ar_tensor.cuh"

namespace tda {
namespace {

__device__ int g_many_status;

constexpr int kManyThreads = 384;             // a warpgroup for copies and instructions (two of its warps idle), two that add up
// Registers a thread: 168 at the start, 384 * 168 = 128 * 72 + 256 * 216.
constexpr int kRegistersMoving = 72, kRegistersAdding = 216;
constexpr int kTileRows = 256, kTileFeatures = 256;
constexpr int kManyStages = 6, kOperandBytes = kBlock * kBlock, kManyScaleBytes = (kBlock + 4) * 4;
constexpr int kManyStageBytes = 2 * kOperandBytes + kManyScaleBytes, kOutBytes = 32 * 64;
constexpr int kManySmem = kManyStages * kManyStageBytes + 8 * kOutBytes + (3 * kManyStages + 4) * 8 + 16 + 1024;
constexpr int kRowTilesTogether = 8;

__device__ __forceinline__ unsigned long long pair_of_floats(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 floats_of(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__global__ void __launch_bounds__(kManyThreads, 1) many_kernel(const __grid_constant__ Product p, const __grid_constant__ CUtensorMap weight,
                                                               const __grid_constant__ CUtensorMap x, int row_tiles) {
    constexpr int S = kManyStages;
    extern __shared__ uint8_t raw[];
    const ar_matmul_fp8_args &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = (shared_address(raw) + 1023) & ~1023u;
    const uint32_t rows_at = base, weights = rows_at + S * kOperandBytes, out_at = weights + S * kOperandBytes, scales = out_at + 8 * kOutBytes;
    // full: block 0's, both blocks' operands; scaled: the scales; empty: a stage's; sums_full, sums_empty (block 0's): the halves of tensor memory
    const uint32_t full = scales + S * kManyScaleBytes, scaled = full + S * 8, empty = scaled + S * 8, sums_full = empty + S * 8, sums_empty = sums_full + 16;
    const uint32_t tmem_at = sums_empty + 16;
    uint8_t *const shared = raw + (base - shared_address(raw));
    const int rank = (int)cluster_rank();
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                bar_init(full + 8 * i, 1);
                bar_init(scaled + 8 * i, 32);
                bar_init(empty + 8 * i, 8);
            }
            for (int i = 0; i < 2; ++i) {
                bar_init(sums_full + 8 * i, 1);
                bar_init(sums_empty + 8 * i, 16);
            }
            bar_init_done();
            tensor_prefetch(&weight);
            tensor_prefetch(&x);
        }
    } else if (warp == 1) {
        pair_tmem_alloc(tmem_at, 512);
    }
    tmem_before_sync();
    __syncthreads();
    cluster_sync_all();           // (nobody signals a barrier that is not there yet)
    tmem_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(shared + (tmem_at - base));
    after_the_stream();

    const int wide = (a.out_dim + kTileFeatures - 1) / kTileFeatures, blocks = (a.out_dim + kBlock - 1) / kBlock;
    const int64_t step = gridDim.x / 2;
    // With one weight, 8 tiles of rows by all features, then the next 8: what the GPU works on at a time is a
    // patch with few different rows and features, which L2 holds.  Rows and feature are the pair's.
    auto tile_of = [&](int64_t u, int &feature) {
        int64_t t;
        if (row_tiles) {
            const int64_t band = u / ((int64_t)kRowTilesTogether * wide), in = u - band * kRowTilesTogether * wide;
            const int high = min(kRowTilesTogether, (int)max(row_tiles - band * kRowTilesTogether, (int64_t)1));
            t = band * kRowTilesTogether + in % high;
            feature = (int)(in / high) * kTileFeatures;
        } else {
            t = u / wide;
            feature = (int)(u - t * wide) * kTileFeatures;
        }
        return feature < a.out_dim ? rows_of_tile(a, t, kTileRows) : Rows{0, 0, 0};
    };
    bool fine = true;
    int feature = 0;

    if (warp < 4) {
    registers_down<kRegistersMoving>();
    if (warp == 0) {
        const uint32_t full_of_0 = cluster_address(full, 0);
        int issued = 0;
        for (int64_t u = blockIdx.x / 2; fine; u += step) {
            const Rows rows = tile_of(u, feature);
            if (rows.count == 0) break;
            const int first = rows.first + rank * kBlock, count = rows.count - rank * kBlock;
            int picked[4] = {0, 0, 0, 0};
            if (a.row_of) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * lane + i;
                    picked[i] = j < count ? (int)max(source_row(a, first + j), (int64_t)0) : 0;
                }
            }
            const float *scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = lane + 32 * i;
                const int64_t r = j < count ? source_row(a, first + j) : -1;
                scale[i] = r >= 0 ? a.x_scales + r * a.x_scales_stride : nullptr;
            }
            // the weight's scales of both halves, by two lanes
            const int half = feature / kBlock + lane;
            const float *weight_scale = lane < 2 && half < blocks ? a.weight_scales + ((int64_t)rows.expert * blocks + half) * p.groups : nullptr;
            for (int k = 0; k < p.groups; ++k, ++issued) {
                const int s = issued % S;
                if (!(fine = bar_wait_warp(empty + 8 * s, (issued / S & 1) ^ 1))) break;
                const uint32_t bar = full_of_0 + 8 * s, to = rows_at + s * kOperandBytes, words = scales + s * kManyScaleBytes;
                if (lane == 0) {
                    if (rank == 0) bar_expect(full + 8 * s, 4 * kOperandBytes);
                    pair_tensor_load(weights + s * kOperandBytes, &weight, bar, k * kBlock, feature + rank * kBlock, rows.expert);
                    if (!a.row_of) pair_tensor_load(to, &x, bar, k * kBlock, first);
                }
                if (a.row_of) pair_tensor_gather(to + lane * 4 * kBlock, &x, bar, k * kBlock, picked);
#pragma unroll
                for (int i = 0; i < 4; ++i) copy_word(words + 4 * (lane + 32 * i), scale[i] ? scale[i] + (a.x_row_scales ? 0 : k) : a.x_scales, scale[i] != nullptr);
                if (lane < 2) copy_word(words + 4 * (kBlock + lane), weight_scale ? weight_scale + k : a.weight_scales, weight_scale != nullptr);
                bar_arrive_copies(scaled + 8 * s);
                __syncwarp();
            }
        }
        if (!fine) {                                   // what is under way has to land before the blocks may end
            for (int i = max(issued - S, 0); i < issued; ++i) (void)bar_wait_warp(scaled + 8 * (i % S), i / S & 1);
            if (rank == 0)
                for (int i = max(issued - S, 0); i < issued; ++i) (void)bar_wait_warp(full + 8 * (i % S), i / S & 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int n = 0;
            for (int64_t u = blockIdx.x / 2; fine; u += step) {
                if (tile_of(u, feature).count == 0) break;
                for (int k = 0; k < p.groups; ++k, ++n) {
                    const int s = n % S, b = n & 1;
                    if (!(fine = bar_wait_warp(sums_empty + 8 * b, (n >> 1 & 1) ^ 1) && bar_wait_warp(full + 8 * s, n / S & 1))) break;
                    tmem_after_sync();
                    if (lane == 0) {
                        const uint64_t r = operand_of(rows_at + s * kOperandBytes), w = operand_of(weights + s * kOperandBytes);
#pragma unroll
                        for (int i = 0; i < 4; ++i) pair_mma_e4m3(tmem + b * kTileFeatures, r + 2 * i, w + 2 * i, product_shape(kTileRows, kTileFeatures), i > 0);
                        pair_mma_commit(sums_full + 8 * b);
                    }
                    __syncwarp();
                }
            }
            if (!fine)
                for (int i = max(n - 2, 0); i < n; ++i) (void)bar_wait_warp(sums_full + 8 * (i & 1), i >> 1 & 1);
        }
    }
    } else {
        registers_up<kRegistersAdding>();
        const int quarter = warp & 3, half = (warp - 4) >> 2, mine = quarter * 32 + lane;
        const uint32_t empty_of_0 = cluster_address(sums_empty, 0), from = tmem + ((uint32_t)(quarter * 32) << 16) + half * kBlock;
        const uint32_t out_words = out_at + (warp - 4) * kOutBytes;
        const bool vectors = !(reinterpret_cast<uintptr_t>(a.out) & 15) && a.out_stride % 8 == 0;
        int n = 0;
        for (int64_t u = blockIdx.x / 2; fine; u += step) {
            const Rows rows = tile_of(u, feature);
            if (rows.count == 0) break;
            const int first = rows.first + rank * kBlock, count = rows.count - rank * kBlock;
            unsigned long long sum[kBlock / 2];
#pragma unroll
            for (int j = 0; j < kBlock / 2; ++j) sum[j] = 0;
            for (int k = 0; k < p.groups; ++k, ++n) {
                const int s = n % S, b = n & 1;
                if (!(fine = bar_wait_warp(scaled + 8 * s, n / S & 1) && bar_wait_warp(sums_full + 8 * b, n >> 1 & 1))) break;
                tmem_after_sync();
                const float *words = reinterpret_cast<const float *>(shared + (scales - base) + s * kManyScaleBytes);
                const float f = words[mine] * words[kBlock + half];
                __syncwarp();
                if (lane == 0) bar_arrive(empty + 8 * s);      // (the sums are there: nothing reads the stage any more)
                const unsigned long long ff = pair_of_floats(f, f);
                // (16 columns are on their way while the 16 before are added)
                float v[2][16];
                tmem_load(from + b * kTileFeatures, v[0]);
                tmem_wait_loads(v[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j < 7) tmem_load(from + b * kTileFeatures + (j + 1) * 16, v[(j + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum[j * 8 + i / 2]) : "l"(pair_of_floats(v[j & 1][i], v[j & 1][i + 1])), "l"(ff));
                    if (j < 7) tmem_wait_loads(v[(j + 1) & 1]);
                }
                tmem_before_sync();
                __syncwarp();
                if (lane == 0) cluster_bar_arrive(empty_of_0 + 8 * b);
            }
            if (!fine) break;
            const bool real = mine < count && source_row(a, first + mine) >= 0;
#pragma unroll
            for (int j = 0; j < kBlock; j += 32) {
                // a row's 32 features (64 bytes) from a thread, in 16-byte pieces that two rows' order keeps apart
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 v = floats_of(sum[j / 2 + c * 4 + e]);
                        if (!real) v = make_float2(0, 0);
                        w[e] = a.dtype == AR_F16 ? to_pair<__half>(v) : to_pair<__nv_bfloat16>(v);
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out_words + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
                }
                __syncwarp();
                const int at = feature + half * kBlock + j + (lane & 3) * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 2), row = quarter * 32 + r;
                    union { uint4 v; uint16_t h[8]; } w;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.v.x), "=r"(w.v.y), "=r"(w.v.z), "=r"(w.v.w) : "r"(out_words + r * 64 + (((lane & 3) ^ (r >> 1 & 3)) << 4)) : "memory");
                    if (row < count && at < a.out_dim) {
                        uint16_t *to = static_cast<uint16_t *>(a.out) + (int64_t)(first + row) * a.out_stride + at;
                        if (vectors && at + 8 <= a.out_dim) {
                            *reinterpret_cast<uint4 *>(to) = w.v;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (at + e < a.out_dim) to[e] = w.h[e];
                        }
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!fine && lane == 0) atomicCAS(&g_many_status, 0, AR_ETIMEOUT);
    tmem_before_sync();
    __syncthreads();
    cluster_sync_all();
    tmem_after_sync();
    if (warp == 1) pair_tmem_free(tmem, 512);
}

}  // namespace

cudaError_t start_many(const Product &p, cudaStream_t s, int multiprocessors) {
    const ar_matmul_fp8_args &a = p.a;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kManySmem);
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    CUtensorMap weight, x;
    if (!map_weight(&weight, a, kBlock) || !map_rows(&x, a, kBlock)) return cudaErrorInvalidValue;
    const int64_t tiles = most_tiles(a, kTileRows), units = tiles * ((a.out_dim + kTileFeatures - 1) / kTileFeatures), pairs = multiprocessors / 2;
    return launch_next(many_kernel, dim3((unsigned)(2 * (units < pairs ? units : pairs))), kManyThreads, kManySmem, s, 2, p, weight, x, a.offsets ? 0 : (int)tiles);
}

int take_many_status(int *code) {
    const int none = AR_OK;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_many_status, sizeof(int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_many_status, &none, sizeof(int));
    return launch_status(e);
}

}  // namespace tda
