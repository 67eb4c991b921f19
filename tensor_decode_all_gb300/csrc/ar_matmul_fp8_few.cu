// ar_matmul_fp8_few.cu -- products of few rows with an e4m3 weight: the weight's bytes are what counts.
//
// 128 features of the weight are the matrix instruction's lanes, up to TOK rows its columns, so that few rows leave
// little of it empty: per group of 128 channels four tcgen05.mma sum the group's products in tensor memory,
// and four warps, a feature to a thread, multiply what came out by the two scales and add it up in registers.
//
// A warp copies, another issues the instructions; weight tiles (16 KB) and rows come by bulk tensor copies, the
// scales by word copies beside them, all to one barrier a stage.  Rows that are picked by number come four at a time.
//
// Where there are fewer tiles than the GPU has room for, a cluster of blocks shares a tile's channels: each block
// sums its part, deals its sums out to the cluster's shared memory by columns, and adds up its own columns in
// the blocks' order.
#include "ar_matmul_fp8.cuh"
#include "ar_tensor.cuh"

namespace tda {
namespace {

__device__ int g_few_status;

constexpr int kFewThreads = 192;              // copies, instructions, four warps that add up

template <int TOK> struct Few {
    static constexpr int WeightBytes = kBlock * kBlock, RowBytes = TOK * kBlock, ScaleBytes = (TOK + 4) * 4;
    static constexpr int Buffers = TOK <= 64 ? 4 : 2;                 // of sums in tensor memory
    static constexpr int Columns = TOK * Buffers;
    static constexpr int StageBytes = WeightBytes + RowBytes + ScaleBytes;
    static constexpr int Stages = 112 * 1024 / StageBytes;            // two blocks to a multiprocessor
    static constexpr int Smem = Stages * StageBytes + (2 * Stages + 2 * Buffers) * 8 + 16 + 1024;
};

template <int TOK>
__global__ void __launch_bounds__(kFewThreads, 2) few_kernel(const __grid_constant__ Product p, const __grid_constant__ CUtensorMap weight,
                                                             const __grid_constant__ CUtensorMap x, int cluster, int row_tiles) {
    using F = Few<TOK>;
    constexpr int S = F::Stages, B = F::Buffers;
    extern __shared__ uint8_t raw[];
    const ar_matmul_fp8_args &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = (shared_address(raw) + 1023) & ~1023u;
    const uint32_t weights = base, rows_at = weights + S * F::WeightBytes, scales = rows_at + S * F::RowBytes;
    const uint32_t full = scales + S * F::ScaleBytes, empty = full + S * 8, sums_full = empty + S * 8, sums_empty = sums_full + B * 8;
    const uint32_t tmem_at = sums_empty + B * 8;
    uint8_t *const shared = raw + (base - shared_address(raw));
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                bar_init(full + 8 * i, 33);            // the bulk copies' thread, and each lane's word copies
                bar_init(empty + 8 * i, 4);
            }
            for (int i = 0; i < B; ++i) {
                bar_init(sums_full + 8 * i, 1);
                bar_init(sums_empty + 8 * i, 4);
            }
            bar_init_done();
            tensor_prefetch(&weight);
            tensor_prefetch(&x);
        }
    } else if (warp == 1) {
        tmem_alloc(tmem_at, F::Columns);
    }
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(shared + (tmem_at - base));
    after_the_stream();

    const int features = (a.out_dim + kBlock - 1) / kBlock;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int k0 = p.groups * rank / cluster, k1 = p.groups * (rank + 1) / cluster;
    const int64_t step = gridDim.x / cluster;
    // Tiles of rows fastest where one weight is all there is: it is read once, and then comes from L2.
    auto tile_of = [&](int64_t u, int &feature) {
        const int64_t t = row_tiles ? u % row_tiles : u / features;
        feature = (int)(row_tiles ? u / row_tiles : u % features) * kBlock;
        return feature < a.out_dim ? rows_of_tile(a, t, TOK) : Rows{0, 0, 0};
    };
    bool fine = true, any = false, joined = false;     // no wait ran out; there was a tile; the cluster's blocks have met
    int feature = 0;
    Rows rows = {0, 0, 0};

    if (warp == 0) {
        int issued = 0;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            int picked[4] = {0, 0, 0, 0};
            if (a.row_of && lane < TOK / 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * lane + i;
                    picked[i] = j < rows.count ? (int)max(source_row(a, rows.first + j), (int64_t)0) : 0;
                }
            }
            const float *scale[(TOK + 31) / 32];
#pragma unroll
            for (int i = 0; i < (TOK + 31) / 32; ++i) {
                const int j = lane + 32 * i;
                const int64_t r = j < rows.count ? source_row(a, rows.first + j) : -1;
                scale[i] = r >= 0 ? a.x_scales + r * a.x_scales_stride : nullptr;
            }
            const float *weight_scale = a.weight_scales + ((int64_t)rows.expert * features + feature / kBlock) * p.groups;
            for (int k = k0; k < k1; ++k, ++issued) {
                const int s = issued % S;
                if (!(fine = bar_wait_warp(empty + 8 * s, (issued / S & 1) ^ 1))) break;
                const uint32_t bar = full + 8 * s, to = rows_at + s * F::RowBytes, words = scales + s * F::ScaleBytes;
                if (lane == 0) {
                    bar_expect(bar, F::WeightBytes + F::RowBytes);
                    tensor_load(weights + s * F::WeightBytes, &weight, bar, k * kBlock, feature, rows.expert);
                    if (!a.row_of) tensor_load(to, &x, bar, k * kBlock, rows.first);
                    copy_word(words + 4 * TOK, weight_scale + k, true);
                }
                if (a.row_of && lane < TOK / 4) tensor_gather(to + lane * 4 * kBlock, &x, bar, k * kBlock, picked);
#pragma unroll
                for (int i = 0; i < (TOK + 31) / 32; ++i)
                    if (TOK >= 32 || lane < TOK)
                        copy_word(words + 4 * (lane + 32 * i), scale[i] ? scale[i] + (a.x_row_scales ? 0 : k) : a.x_scales, scale[i] != nullptr);
                bar_arrive_copies(bar);
                __syncwarp();
            }
        }
        if (!fine)                                     // what is under way has to land before the block may end
            for (int i = max(issued - S, 0); i < issued; ++i) (void)bar_wait_warp(full + 8 * (i % S), i / S & 1);
    } else if (warp == 1) {
        int n = 0;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            for (int k = k0; k < k1; ++k, ++n) {
                const int s = n % S, b = n % B;
                if (!(fine = bar_wait_warp(sums_empty + 8 * b, (n / B & 1) ^ 1) && bar_wait_warp(full + 8 * s, n / S & 1))) break;
                tmem_after_sync();
                if (lane == 0) {
                    const uint64_t w = operand_of(weights + s * F::WeightBytes), r = operand_of(rows_at + s * F::RowBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_e4m3(tmem + b * TOK, w + 2 * i, r + 2 * i, product_shape(kBlock, TOK), i > 0);
                    mma_commit(sums_full + 8 * b);
                }
                __syncwarp();
            }
        }
        if (!fine)
            for (int i = max(n - B, 0); i < n; ++i) (void)bar_wait_warp(sums_full + 8 * (i % B), i / B & 1);
    } else {
        const int quarter = warp & 3, mine = quarter * 32 + lane;
        int n = 0;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            float sum[TOK];
#pragma unroll
            for (int j = 0; j < TOK; ++j) sum[j] = 0;
            for (int k = k0; k < k1; ++k, ++n) {
                const int s = n % S, b = n % B;
                // (the stage's own barrier too: the scales are ordinary copies)
                if (!(fine = bar_wait_warp(sums_full + 8 * b, n / B & 1) && bar_wait_warp(full + 8 * s, n / S & 1))) break;
                tmem_after_sync();
                const float *words = reinterpret_cast<const float *>(shared + (scales - base) + s * F::ScaleBytes);
                const float sw = words[TOK];
                constexpr int W = TOK < 32 ? TOK : 32;
#pragma unroll
                for (int j = 0; j < TOK; j += W) {
                    float v[W];
                    tmem_load(tmem + ((uint32_t)(quarter * 32) << 16) + b * TOK + j, v);
                    tmem_wait_loads(v);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 sx = *reinterpret_cast<const float4 *>(words + j + i);
                        sum[j + i] = fmaf(v[i], sx.x * sw, sum[j + i]);
                        sum[j + i + 1] = fmaf(v[i + 1], sx.y * sw, sum[j + i + 1]);
                        sum[j + i + 2] = fmaf(v[i + 2], sx.z * sw, sum[j + i + 2]);
                        sum[j + i + 3] = fmaf(v[i + 3], sx.w * sw, sum[j + i + 3]);
                    }
                }
                tmem_before_sync();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(sums_empty + 8 * b);
                    bar_arrive(empty + 8 * s);
                }
            }
            if (!fine) break;
            if (cluster > 1) {
                // (one tile to a cluster: nothing follows in the stages' memory)
                __syncwarp();
                cluster_sync_all();
                const int each = TOK / cluster;
#pragma unroll
                for (int j = 0; j < TOK; ++j)
                    cluster_store(cluster_address(base + ((rank * each + j % each) * kBlock + mine) * 4, j / each), sum[j]);
                __syncwarp();
                cluster_sync_all();
                const float *parts = reinterpret_cast<const float *>(shared);
#pragma unroll 1
                for (int j = 0; j < each; ++j) {
                    float v = parts[j * kBlock + mine];
                    for (int r = 1; r < cluster; ++r) v += parts[(r * each + j) * kBlock + mine];
                    const int row = rank * each + j;
                    if (row < rows.count && feature + mine < a.out_dim) {
                        if (a.row_of && source_row(a, rows.first + row) < 0) v = 0;
                        const int64_t at = (rows.first + row) * a.out_stride + feature + mine;
                        if (a.dtype == AR_F16) static_cast<__half *>(a.out)[at] = __float2half_rn(v);
                        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
                    }
                }
                joined = true;
                break;
            }
#pragma unroll
            for (int j0 = 0; j0 < TOK; j0 += 32) {
                unsigned there = ~0u;
                if (a.row_of) there = __ballot_sync(~0u, j0 + lane < rows.count && source_row(a, rows.first + j0 + lane) >= 0);
#pragma unroll
                for (int j = j0; j < j0 + 32 && j < TOK; ++j)
                    if (j < rows.count && feature + mine < a.out_dim) {
                        const float v = there >> (j - j0) & 1 ? sum[j] : 0.0f;
                        const int64_t at = (rows.first + j) * a.out_stride + feature + mine;
                        if (a.dtype == AR_F16) static_cast<__half *>(a.out)[at] = __float2half_rn(v);
                        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
                    }
            }
        }
    }
    if (!fine && lane == 0) atomicCAS(&g_few_status, 0, AR_ETIMEOUT);
    if (cluster > 1 && any && !joined) {
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    if (warp == 1) tmem_free(tmem, F::Columns);
}

template <int TOK>
cudaError_t start_few_of(const Product &p, cudaStream_t s, int cluster, int64_t units, int row_tiles, int multiprocessors) {
    using F = Few<TOK>;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(few_kernel<TOK>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::Smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_kernel<TOK>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    CUtensorMap weight, x;
    if (!map_weight(&weight, p.a, kBlock) || !map_rows(&x, p.a, TOK)) return cudaErrorInvalidValue;
    const int64_t blocks = cluster > 1 ? units * cluster : units < 2 * multiprocessors ? units : 2 * multiprocessors;
    return launch_next(few_kernel<TOK>, dim3((unsigned)blocks), kFewThreads, F::Smem, s, cluster > 1 ? cluster : 0, p, weight, x, cluster, row_tiles);
}

}  // namespace

cudaError_t start_few(const Product &p, cudaStream_t s, int multiprocessors) {
    const ar_matmul_fp8_args &a = p.a;
    // Columns for the rows that a tile is likely to have: all of them, or twice an expert's share.
    const int64_t likely = a.offsets ? 2 * a.rows / a.experts : a.rows;
    const int tok = likely <= 16 ? 16 : likely <= 32 ? 32 : likely <= 64 ? 64 : 128;
    const int features = (a.out_dim + kBlock - 1) / kBlock;
    const int64_t tiles = most_tiles(a, tok), units = tiles * features;
    int cluster = 1;
    while (cluster < 16 && units * cluster * 2 <= 2 * multiprocessors && p.groups >= cluster * 4) cluster *= 2;
    const int row_tiles = a.offsets ? 0 : (int)tiles;
    return tok == 16   ? start_few_of<16>(p, s, cluster, units, row_tiles, multiprocessors)
           : tok == 32 ? start_few_of<32>(p, s, cluster, units, row_tiles, multiprocessors)
           : tok == 64 ? start_few_of<64>(p, s, cluster, units, row_tiles, multiprocessors)
                       : start_few_of<128>(p, s, cluster, units, row_tiles, multiprocessors);
}

int take_few_status(int *code) {
    const int none = AR_OK;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_few_status, sizeof(int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_few_status, &none, sizeof(int));
    return launch_status(e);
}

}  // namespace tda
