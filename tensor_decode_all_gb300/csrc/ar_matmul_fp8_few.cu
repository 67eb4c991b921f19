// ar_matmul_fp8_few.cu -- products of few rows with an e4m3 weight: the weight's bytes are what counts.
//
// 128 features of the weight are the matrix instruction's lanes, up to TOK rows its columns, so that few rows leave
// little of it empty: per group of 128 channels four tcgen05.mma sum the group's products in tensor memory,
// and four warps (eight), a feature to a thread, multiply what came out by the two scales and add it up in registers.
//
// A warp copies, another issues the instructions; weight tiles (16 KB) and rows come by bulk tensor copies, the
// scales by word copies beside them.  Rows that are picked by number come 16 bytes to a lane.
//
// Where there are fewer tiles than the GPU has room for, a cluster of blocks shares a tile's channels: each block
// sums its part and sends its sums to the blocks' shared memory, each row's to one of them, which adds them up in the blocks' order as soon
// as a barrier has counted their bytes: no meeting of the cluster at the end.
//
// GB300 graph replays: 256 tokens with 8 of 128 experts, 4096 -> 2048 features, 156 us, 6.5 TB/s or 97% of what a plain copy
// reaches; 5 tokens with 4 of 32 25.5 us (84%); 8 x 8192 -> 1280 4.6 us (1.3 to the first sums, 1.0 for four groups, 0.3 to send, 0.4 until all
// is there, 0.3 to add and store, the launch); 61 x 3584 -> 8192 9.2 us.
#include <algorithm>

#include "ar_matmul_fp8.cuh"
#include "ar_tensor.cuh"

namespace tda {
namespace {

__device__ int g_few_status;

template <int TOK> struct Few {
    static constexpr int WeightBytes = kBlock * kBlock, RowBytes = TOK * kBlock, ScaleBytes = (TOK + 4) * 4;
    static constexpr int Buffers = TOK <= 64 ? 4 : 2;                 // of sums in tensor memory
    static constexpr int Columns = TOK * Buffers;
    static constexpr int StageBytes = WeightBytes + RowBytes;
    // Two blocks to a multiprocessor; with 128 rows one, whose sums are eight warps' (with four they would not fit their registers; with
    // eight 44 to 48 bytes of a thread still do not).
    static constexpr int Blocks = TOK <= 64 ? 2 : 1, Halves = TOK <= 64 ? 1 : 2, Own = TOK / Halves;
    static constexpr int Threads = 64 + 128 * Halves;               // copies, instructions, warps that add up
    static constexpr int Stages = (224 * 1024 / Blocks - 4 * ScaleBytes) / (StageBytes + ScaleBytes);
    // The sums that a block of a cluster is sent take the place of a stage (two).
    static constexpr int PartBytes = TOK * kBlock * 4, Given = TOK <= 64 ? 1 : 2;
    static constexpr int Room = std::max(Stages * StageBytes, (Stages - Given) * StageBytes + PartBytes);
    // A stage is free when the matrix instructions have read it, its scales when they have been multiplied by: up to
    // `Buffers` groups later.
    static constexpr int Scales = Stages + Buffers;
    static constexpr int Smem = Room + Scales * ScaleBytes + (2 * Stages + Scales + 2 * Buffers + 1) * 8 + 16 + 1024;
};

// kPicked: row_of is given.
template <int TOK, bool kPicked>
__global__ void __launch_bounds__(Few<TOK>::Threads, Few<TOK>::Blocks) few_kernel(const __grid_constant__ Product p,
                                                                                       const __grid_constant__ CUtensorMap weight,
                                                                                       const __grid_constant__ CUtensorMap x, int cluster, int row_tiles) {
    using F = Few<TOK>;
    constexpr int S = F::Stages, B = F::Buffers, Q = F::Scales;
    extern __shared__ uint8_t raw[];
    const ar_matmul_fp8_args &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = (shared_address(raw) + 1023) & ~1023u;
    // a stage: the weight's tile, and the rows after it
    const uint32_t scales = base + F::Room;
    const uint32_t full = scales + Q * F::ScaleBytes, empty = full + S * 8, scaled = empty + S * 8, sums_full = scaled + Q * 8, sums_empty = sums_full + B * 8;
    const uint32_t sent = sums_empty + B * 8, tmem_at = sent + 8;
    const uint32_t stages = cluster > 1 ? S - F::Given : S, parts = base + (S - F::Given) * F::StageBytes;
    uint8_t *const shared = raw + (base - shared_address(raw));
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                bar_init(full + 8 * i, kPicked ? 33 : 1);      // the bulk copies' thread, and each lane's copies of picked rows
                bar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < Q; ++i) bar_init(scaled + 8 * i, 32);      // each lane's copies
            for (int i = 0; i < B; ++i) {
                bar_init(sums_full + 8 * i, 1);
                bar_init(sums_empty + 8 * i, 4 * F::Halves);
            }
            bar_init(sent, 1);
            bar_init_done();
            if (cluster > 1) bar_expect(sent, F::PartBytes);
            tensor_prefetch(&weight);
            tensor_prefetch(&x);
        }
    } else if (warp == 1) {
        tmem_alloc(tmem_at, F::Columns);
    }
    tmem_before_sync();
    __syncthreads();
    if (cluster > 1) cluster_sync_all();           // (nobody sends to a barrier that is not there yet)
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
    bool fine = true, any = false;     // no wait ran out; there was a tile
    int feature = 0;
    Rows rows = {0, 0, 0};

    if (warp == 0) {
        Ring<S> stage;
        Ring<Q> words_of;
        int issued = 0;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            Picked<TOK> picked;
            if (kPicked) picked.look_up(a, rows.first, rows.count);
            const float *scale[(TOK + 31) / 32];
#pragma unroll
            for (int i = 0; i < (TOK + 31) / 32; ++i) {
                const int j = lane + 32 * i;
                const int64_t r = j >= rows.count ? -1 : kPicked ? source_row(a, rows.first + j) : rows.first + j;
                scale[i] = r >= 0 ? a.x_scales + r * a.x_scales_stride : nullptr;
            }
            const float *weight_scale = a.weight_scales + ((int64_t)rows.expert * features + feature / kBlock) * p.groups;
            for (int k = k0; k < k1; ++k, ++issued, stage.next(stages), words_of.next()) {
                const uint32_t s = stage.at;
                if (!(fine = bar_wait_warp(empty + 8 * s, stage.parity ^ 1))) break;
                const uint32_t bar = full + 8 * s, at = base + s * F::StageBytes, to = at + F::WeightBytes, words = scales + words_of.at * F::ScaleBytes;
                if (lane == 0) {
                    bar_expect(bar, F::WeightBytes + (kPicked ? 0 : F::RowBytes));
                    tensor_load(at, &weight, bar, k * kBlock, feature, rows.expert);
                    if (!kPicked) tensor_load(to, &x, bar, k * kBlock, rows.first);
                    copy_word(words + 4 * TOK, weight_scale + k, true);
                }
                if constexpr (kPicked) {
                    picked.copy(a, to, k);
                    bar_arrive_copies(bar);
                }
#pragma unroll
                for (int i = 0; i < (TOK + 31) / 32; ++i)
                    if (TOK >= 32 || lane < TOK)
                        copy_word(words + 4 * (lane + 32 * i), scale[i] ? scale[i] + (a.x_row_scales ? 0 : k) : a.x_scales, scale[i] != nullptr);
                bar_arrive_copies(scaled + 8 * words_of.at);
                __syncwarp();
            }
        }
        if (!fine)                                     // what is under way has to land before the block may end
            for (int n = stages, i = max(issued - n, 0); i < issued; ++i)
                (void)(bar_wait_warp(full + 8 * (i % n), i / n & 1) && bar_wait_warp(scaled + 8 * (i % Q), i / Q & 1));
    } else if (warp == 1) {
        const uint64_t operand = operand_of(base);
        const bool one = elected();
        Ring<S> stage;
        Ring<B> buffer;
        int n = 0;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            for (int k = k0; k < k1; ++k, ++n, stage.next(stages), buffer.next()) {
                if (!(fine = bar_wait_warp(full + 8 * stage.at, stage.parity, sums_empty + 8 * buffer.at, buffer.parity ^ 1))) break;
                tmem_after_sync();
                if (kPicked) written_for_mma();
                if (one) {
                    const uint64_t w = operand + stage.at * (F::StageBytes >> 4), r = w + (F::WeightBytes >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_e4m3(tmem + buffer.at * TOK, w + 2 * i, r + 2 * i, product_shape(kBlock, TOK), i > 0);
                    mma_commit(empty + 8 * stage.at);
                    mma_commit(sums_full + 8 * buffer.at);
                }
                __syncwarp();
            }
        }
        if (!fine)
            for (int i = max(n - B, 0); i < n; ++i) (void)bar_wait_warp(sums_full + 8 * (i % B), i / B & 1);
    } else {
        // a feature, and `Own` of the rows, to a thread
        constexpr int Own = F::Own;
        const int quarter = warp & 3, mine = quarter * 32 + lane, begin = (warp - 2) / 4 * Own;
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + begin;
        Ring<Q> words_of;
        Ring<B> buffer;
        for (int64_t u = blockIdx.x / cluster; fine; u += step) {
            rows = tile_of(u, feature);
            if (rows.count == 0 || (any && cluster > 1)) break;
            any = true;
            // which of the rows have one of x (a bit each)
            unsigned there[(Own + 31) / 32];
#pragma unroll
            for (int i = 0; i < (Own + 31) / 32; ++i) {
                const int row = begin + i * 32 + lane;
                there[i] = ~0u;
                if (kPicked) there[i] = __ballot_sync(~0u, row < rows.count && source_row(a, rows.first + row) >= 0);
            }
            unsigned long long sum[Own / 2];
#pragma unroll
            for (int j = 0; j < Own / 2; ++j) sum[j] = 0;
            for (int k = k0; k < k1; ++k, words_of.next(), buffer.next()) {
                if (!(fine = bar_wait_warp(scaled + 8 * words_of.at, words_of.parity, sums_full + 8 * buffer.at, buffer.parity))) break;
                tmem_after_sync();
                const float *words = reinterpret_cast<const float *>(shared + (scales - base)) + words_of.at * (F::ScaleBytes / 4);
                const unsigned long long sw = pair_of_floats(words[TOK], words[TOK]);
                constexpr int W = Own < 32 ? Own : 32;
#pragma unroll
                for (int j = 0; j < Own; j += W) {
                    float v[W];
                    tmem_load(from + buffer.at * TOK + j, v);
                    tmem_wait_loads(v);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 sx = *reinterpret_cast<const float4 *>(words + begin + j + i);
                        fma2(sum[(j + i) / 2], pair_of_floats(v[i], v[i + 1]), mul2(pair_of_floats(sx.x, sx.y), sw));
                        fma2(sum[(j + i) / 2 + 1], pair_of_floats(v[i + 2], v[i + 3]), mul2(pair_of_floats(sx.z, sx.w), sw));
                    }
                }
                tmem_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(sums_empty + 8 * buffer.at);
            }
            if (!fine) break;
            uint16_t *const here = static_cast<uint16_t *>(a.out) + (int64_t)rows.first * a.out_stride + feature + mine;
            const int high = feature + mine < a.out_dim ? rows.count : 0;
            const bool half = a.dtype == AR_F16;
            // (without a branch: one to a store took longer than the rest)
            auto store = [&](int row, float v) {
                const uint16_t h = __half_as_ushort(__float2half_rn(v)), b = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                asm volatile("{ .reg .pred p; setp.ne.b32 p, %2, 0; @p st.global.b16 [%0], %1; }" ::"l"(here + row * a.out_stride), "h"((uint16_t)(half ? h : b)), "r"((int)(row < high))
                             : "memory");
            };
            if (cluster > 1) {
                // Four rows of a feature side by side (or one, where a block has fewer) to the block whose rows they are; then this
                // block's rows of all blocks, added in their order.  One tile to a cluster.
                const int ways = __ffs(cluster) - 1, each = TOK >> ways, own_rows = Own >> ways, low = begin >> ways;      // this thread's: low .. low + own_rows - 1 of the block's
                const float *got = reinterpret_cast<const float *>(shared + (parts - base)) + mine;
                auto real = [&](int row) { return !kPicked || (row < rows.count && source_row(a, rows.first + row) >= 0); };
                if (each >= 4) {
                    uint32_t to = 0;
#pragma unroll
                    for (int j = 0; j < Own; j += 4) {
                        const int row = (begin + j) & (each - 1);
                        if (j == 0 || row == 0) to = cluster_address(parts, (begin + j) / each);
                        const float2 lo = floats_of(sum[j / 2]), hi = floats_of(sum[j / 2 + 1]);
                        cluster_send(to + ((rank * each + row) * kBlock + mine * 4) * 4, to + (sent - parts), make_float4(lo.x, lo.y, hi.x, hi.y));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < Own; ++j) {
                        const int row = j & (each - 1);
                        const uint32_t to = cluster_address(parts, j >> (each - 1));       // (each: 1 or 2)
                        const float2 v = floats_of(sum[j / 2]);
                        cluster_send(to + ((rank * each + row) * kBlock + mine) * 4, to + (sent - parts), j & 1 ? v.y : v.x);
                    }
                }
                if (!(fine = bar_wait_warp(sent, 0))) break;
                if (each >= 4) {
#pragma unroll 2
                    for (int i = 0; i < own_rows; i += 4) {
                        const float *from = got + (low + i) * kBlock + mine * 3;      // (four to a feature)
                        float4 w = *reinterpret_cast<const float4 *>(from);
#pragma unroll 4
                        for (int r = 1; r < cluster; ++r) {
                            const float4 v = *reinterpret_cast<const float4 *>(from + r * each * kBlock);
                            w = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
                        }
                        const int row = rank * each + low + i;
                        store(row, real(row) ? w.x : 0.0f);
                        store(row + 1, real(row + 1) ? w.y : 0.0f);
                        store(row + 2, real(row + 2) ? w.z : 0.0f);
                        store(row + 3, real(row + 3) ? w.w : 0.0f);
                    }
                } else {
                    for (int i = 0; i < each; ++i) {
                        float v = got[i * kBlock];
#pragma unroll 4
                        for (int r = 1; r < cluster; ++r) v += got[(r * each + i) * kBlock];
                        store(rank * each + i, real(rank * each + i) ? v : 0.0f);
                    }
                }
                break;
            }
#pragma unroll
            for (int j = 0; j < Own; j += 2) {
                const float2 v = floats_of(sum[j / 2]);
                store(begin + j, there[j / 32] >> (j & 31) & 1 ? v.x : 0.0f);
                store(begin + j + 1, there[j / 32] >> (j & 31) & 2 ? v.y : 0.0f);
            }
        }
    }
    if (!fine && lane == 0) atomicCAS(&g_few_status, 0, AR_ETIMEOUT);
    tmem_before_sync();
    // (a block that gave up waits until no other can send to it any more; one that did not has got all that is sent to it)
    if (__syncthreads_or(!fine) && cluster > 1) cluster_sync_all();
    tmem_after_sync();
    if (warp == 1) tmem_free(tmem, F::Columns);
}

// How many clusters of that many blocks run at the same time: those of a cluster share a part of the GPU, which holds a whole number
// of them (15 of 8 blocks, not 19, with a block to a multiprocessor; the runtime counts one to a multiprocessor).
template <int TOK, bool kPicked> cudaError_t clusters_at_once(int cluster, int *most) {
    using F = Few<TOK>;
    static int known[64][5] = {};          // (one more: 0 is not known, and none can be the answer)
    int dev = 0, log = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    while (1 << log < cluster) ++log;
    if (dev < 64 && (*most = *(volatile int *)&known[dev][log] - 1) >= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(F::Threads);
    cfg.dynamicSmemBytes = F::Smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(most, few_kernel<TOK, kPicked>, &cfg);
    *most *= F::Blocks;
    if (e == cudaSuccess && dev < 64) *(volatile int *)&known[dev][log] = *most + 1;
    return e;
}

template <int TOK, bool kPicked>
cudaError_t start_few_of(const Product &p, cudaStream_t s, int multiprocessors) {
    using F = Few<TOK>;
    const int64_t tiles = most_tiles(p.a, TOK), units = tiles * ((p.a.out_dim + kBlock - 1) / kBlock);
    const int row_tiles = p.a.offsets ? 0 : (int)tiles;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(few_kernel<TOK, kPicked>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::Smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_kernel<TOK, kPicked>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    CUtensorMap weight, x;
    if (!map_weight(&weight, p.a, kBlock) || !map_rows(&x, p.a, TOK)) return cudaErrorInvalidValue;
    const int64_t room = (int64_t)F::Blocks * multiprocessors;
    // Blocks to share a tile's channels, as long as all tiles' run at the same time and each has two groups or more.
    int cluster = 1;
    while (cluster < 16 && units * cluster * 2 <= room && p.groups >= cluster * 4) {
        int most = 0;
        e = clusters_at_once<TOK, kPicked>(cluster * 2, &most);
        if (e != cudaSuccess) return e;
        if (units > most) break;
        cluster *= 2;
    }
    const int64_t blocks = cluster > 1 ? units * cluster : std::min(units, room);
    return launch_next(few_kernel<TOK, kPicked>, dim3((unsigned)blocks), F::Threads, F::Smem, s, cluster > 1 ? cluster : 0, p, weight, x, cluster, row_tiles);
}

template <int TOK> cudaError_t start_few_of(const Product &p, cudaStream_t s, int multiprocessors) {
    return p.a.row_of ? start_few_of<TOK, true>(p, s, multiprocessors) : start_few_of<TOK, false>(p, s, multiprocessors);
}

}  // namespace

cudaError_t start_few(const Product &p, cudaStream_t s, int multiprocessors) {
    const ar_matmul_fp8_args &a = p.a;
    // Columns for the rows that a tile is likely to have: all of them, or twice an expert's share.
    const int64_t likely = a.offsets ? 2 * a.rows / a.experts : a.rows;
    const int tok = likely <= 16 ? 16 : likely <= 32 ? 32 : likely <= 64 ? 64 : 128;
    return tok == 16   ? start_few_of<16>(p, s, multiprocessors)
           : tok == 32 ? start_few_of<32>(p, s, multiprocessors)
           : tok == 64 ? start_few_of<64>(p, s, multiprocessors)
                       : start_few_of<128>(p, s, multiprocessors);
}

int take_few_status(int *code) {
    const int none = AR_OK;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_few_status, sizeof(int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_few_status, &none, sizeof(int));
    return launch_status(e);
}

}  // namespace tda
