// ar_matmul_fp8_many.cu -- products of many rows with an e4m3 weight: the matrix instructions' rate is what counts.
//
// Two blocks of a cluster, on two multiprocessors, share a tile of 256 rows and 256 features: each keeps its 128 rows (the
// lanes) and half of the features' operand, so that a group of 128 channels costs a block 32 KB of copies and as much reading of
// shared memory as writing, which is what 512 cycles of matrix instructions leave time for (a block alone with 128 x 256 would
// copy 48 KB).  Block 0 issues for both.  The instructions sum one group of channels; then eight warps, a row
// and 128 features to a thread, multiply by the two scales and add up in registers, while the next group's sums go to the
// other half of tensor memory.
//
// A tile of at most 128 rows (the end of an expert's) takes half of the instructions' time, three quarters of all: 64 rows to a block, whose
// features lie on twice the lanes.  Where the last round of tiles would occupy half of the pairs or less, its tiles are cut in two (256 x 8192 -> 8192
// 22 us, else 28; 8191 x 8192 -> 5120 232 and 240).
//
// GB300 graph replays: 8191 x 8192 -> 5120 229 us, 3.0 PFLOP/s (the tensor pipe is busy 68% of the time), 32792 rows of 64 experts, 2048 -> 4096
// features, 261 us; calls in a row, between which the clocks fall, 261 to 265 (2.6 PFLOP/s) and 288 to 296.  A step of 128 channels takes 720 to 760 cycles: the way of a group's sums, from the instructions' end through the
// eight warps until the other half of tensor memory is free again, is 820 cycles without any arithmetic.
//
// Blocks stay and go from tile to tile: a warp says which, the copies run ahead, and the next tile's first sums are
// under way while one is stored, 32 bytes of a row at a time.
#include <algorithm>

#include "ar_matmul_fp8.cuh"
#include "ar_tensor.cuh"

namespace tda {
namespace {

__device__ int g_many_status;

constexpr int kManyThreads = 384;             // a warpgroup for copies, instructions and tiles, two that add up
// Registers a thread: 168 at the start, 384 * 168 = 128 * 72 + 256 * 216.
constexpr int kRegistersMoving = 72, kRegistersAdding = 216;
constexpr int kTileRows = 256, kTileFeatures = 256;
// A stage is free when the matrix instructions have read it, its scales when they have been multiplied by: up to two groups later.
constexpr int kManyStages = 6, kManyScales = kManyStages + 2, kOperandBytes = kBlock * kBlock, kManyScaleBytes = (kBlock + 4) * 4, kTiles = 4;
constexpr int kFourScales = 3, kFourBytes = (kBlock + 2) * 16;      // (four groups' scales: those of 12 groups reach past two that are added and six that are copied)
constexpr int kScaleRoom = std::max(kFourScales * kFourBytes, kManyScales * kManyScaleBytes);
constexpr int kOddPitch = 34, kOddBytes = 32 * kOddPitch * 2;       // a warp's 32 rows of 32 results, where they leave by twos of bytes
constexpr int kManySmem = kManyStages * 2 * kOperandBytes + 8 * kOddBytes + kScaleRoom + kTiles * 16 + (2 * kManyStages + kManyScales + 4 + 2 * kTiles) * 8 + 16 + 1024;
constexpr int kRowTilesTogether = 8;

// What the pair does next: rows first .. first + count - 1 of the call (both blocks'), features from `feature` on.  Count 0: no more.
struct Tile {
    int expert, first, count, feature;
};

// Picked rows of x and their scales, side by side in the workspace: a warp to a row.  (The copy engine's own way to pick rows takes 0.6 us
// for 128 of them, and copies by threads take the time of the shared memory's instructions: either a tile would wait
// for them; 67 MB come and go in 25 us.)
__global__ void __launch_bounds__(256) pick_kernel(const ar_matmul_fp8_args a, uint8_t *rows, float *scales, int pitch, int groups) {
    after_the_stream();
    const int lane = threadIdx.x & 31;
    const int begin = a.offsets ? clamp_row(a.offsets[0], a.rows) : 0, end = a.offsets ? clamp_row(a.offsets[a.experts], a.rows) : (int)a.rows;
    for (int64_t row = begin + (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < end; row += (int64_t)gridDim.x * 8) {
        const int64_t from = source_row(a, row);
        if (from < 0) continue;            // (what is there is not used)
        const uint8_t *x = static_cast<const uint8_t *>(a.x) + from * a.x_stride;
        const int whole = a.dim / 16;
#pragma unroll 4
        for (int i = lane; i < whole; i += 32) reinterpret_cast<uint4 *>(rows + row * pitch)[i] = reinterpret_cast<const uint4 *>(x)[i];
        if (lane < a.dim % 16) rows[row * pitch + whole * 16 + lane] = x[whole * 16 + lane];
        for (int i = lane; i < groups; i += 32) scales[row * groups + i] = a.x_scales[from * a.x_scales_stride + i];
    }
}

// kOdd: rows of out that do not lie on 16 bytes.  (A kernel of its own: with both ways to store in one, the loops before them take a third
// longer, for want of registers.)
// kFours: scales come 16 bytes at a time, four groups' together, because the copies of single words (a line for each) take 4 to 10% of the time:
// 8191 x 8192 -> 5120 237 to 245 us against 260 to 265, 32792 rows of 64 experts 266 to 286 against 290 to 297, in a row of calls.
template <bool kOdd, bool kFours>
__global__ void __launch_bounds__(kManyThreads, 1) many_kernel(const __grid_constant__ Product p, const __grid_constant__ CUtensorMap weight,
                                                               const __grid_constant__ CUtensorMap x) {
    constexpr int S = kManyStages, Q = kFours ? kFourScales : kManyScales;
    extern __shared__ uint8_t raw[];
    const ar_matmul_fp8_args &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = (shared_address(raw) + 1023) & ~1023u;
    const uint32_t rows_at = base, weights = rows_at + S * kOperandBytes, odd_at = weights + S * kOperandBytes, scales = odd_at + 8 * kOddBytes, tiles_at = scales + kScaleRoom;
    // full: block 0's, both blocks' operands; scaled: the scales; empty: a stage's; sums_full, sums_empty (block 0's): the halves of
    // tensor memory; known, used: the next tiles
    const uint32_t full = tiles_at + kTiles * 16, scaled = full + S * 8, empty = scaled + Q * 8, sums_full = empty + S * 8, sums_empty = sums_full + 16;
    const uint32_t known = sums_empty + 16, used = known + kTiles * 8, tmem_at = used + kTiles * 8;
    uint8_t *const shared = raw + (base - shared_address(raw));
    volatile Tile *const tiles = reinterpret_cast<volatile Tile *>(shared + (tiles_at - base));
    const int rank = (int)cluster_rank();
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                bar_init(full + 8 * i, 1);
                bar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < Q; ++i) bar_init(scaled + 8 * i, 32);      // each lane's copies
            for (int i = 0; i < 2; ++i) {
                bar_init(sums_full + 8 * i, 1);
                bar_init(sums_empty + 8 * i, 16);
            }
            for (int i = 0; i < kTiles; ++i) {
                bar_init(known + 8 * i, 1);
                bar_init(used + 8 * i, 10);            // the copies' warp, the instructions' and the eight
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

    const int blocks = (a.out_dim + kBlock - 1) / kBlock;
    bool fine = true;
    Ring<kTiles> next;
    // The pair's next tile, for a warp that counts itself among `used`.
    auto next_tile = [&]() {
        if (!(fine = bar_wait_warp(known + 8 * next.at, next.parity))) return Tile{0, 0, 0, 0};
        const volatile Tile &t = tiles[next.at];
        const Tile tile = {t.expert, t.first, t.count, t.feature};
        __syncwarp();
        if (lane == 0) bar_arrive(used + 8 * next.at);
        next.next();
        return tile;
    };

    if (warp < 4) {
        registers_down<kRegistersMoving>();
        if (warp == 0) {
            const uint32_t full_of_0 = cluster_address(full, 0);
            Ring<S> stage;
            Ring<Q> words_of;
            int issued = 0, scales_asked = 0;
            while (fine) {
                const Tile tile = next_tile();
                if (tile.count == 0) break;
                // (half of them are read twice where the tile is short)
                const int own = tile.count <= kBlock ? kBlock / 2 : kBlock, first = tile.first + rank * own, count = min(tile.count - rank * own, own);
                const float *scale[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = lane + 32 * i;
                    scale[i] = j < count ? a.x_scales + (int64_t)(first + j) * a.x_scales_stride : nullptr;
                }
                // the weight's scales of both halves, by two lanes
                const int half = tile.feature / kBlock + lane;
                const float *weight_scale = lane < 2 && half < blocks ? a.weight_scales + ((int64_t)tile.expert * blocks + half) * p.groups : nullptr;
                for (int k = 0; k < p.groups; ++k, ++issued, stage.next()) {
                    const uint32_t s = stage.at;
                    if (!(fine = bar_wait_warp(empty + 8 * s, stage.parity ^ 1))) break;
                    const uint32_t bar = full_of_0 + 8 * s, to = rows_at + s * kOperandBytes, words = scales + words_of.at * (kFours ? kFourBytes : kManyScaleBytes);
                    if (lane == 0) {
                        if (rank == 0) bar_expect(full + 8 * s, 4 * kOperandBytes);
                        pair_tensor_load(weights + s * kOperandBytes, &weight, bar, k * kBlock, tile.feature + rank * kBlock, tile.expert);
                        pair_tensor_load(to, &x, bar, k * kBlock, first);
                    }
                    if constexpr (kFours) {
                        if (k % 4 == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) copy_piece(words + 16 * (lane + 32 * i), scale[i] ? scale[i] + k : a.x_scales, scale[i] ? 16 : 0);
                            if (lane < 2) copy_piece(words + 16 * (kBlock + lane), weight_scale ? weight_scale + k : a.weight_scales, weight_scale ? 16 : 0);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) copy_word(words + 4 * (lane + 32 * i), scale[i] ? scale[i] + (a.x_row_scales ? 0 : k) : a.x_scales, scale[i] != nullptr);
                        if (lane < 2) copy_word(words + 4 * (kBlock + lane), weight_scale ? weight_scale + k : a.weight_scales, weight_scale != nullptr);
                    }
                    if (!kFours || k % 4 == 0) {
                        bar_arrive_copies(scaled + 8 * words_of.at);
                        words_of.next();
                        ++scales_asked;
                    }
                    __syncwarp();
                }
            }
            if (!fine) {                                   // what is under way has to land before the blocks may end
                for (int i = max(scales_asked - Q, 0); i < scales_asked; ++i) (void)bar_wait_warp(scaled + 8 * (i % Q), i / Q & 1);
                if (rank == 0)
                    for (int i = max(issued - S, 0); i < issued; ++i) (void)bar_wait_warp(full + 8 * (i % S), i / S & 1);
            }
        } else if (warp == 1) {
            const uint64_t rows_operand = operand_of(rows_at), weights_operand = operand_of(weights);
            const bool one = elected();
            Ring<S> stage;
            Ring<2> half;
            int n = 0;
            while (fine) {
                const Tile tile = next_tile();
                if (tile.count == 0) break;
                if (rank != 0) continue;
                const uint32_t shape = product_shape(tile.count <= kBlock ? kBlock : kTileRows, kTileFeatures);
                // (the fewest instructions: a step of this loop has to be done before the matrix instructions of the last one are)
                for (int k = 0; k < p.groups; ++k, ++n, stage.next(), half.next()) {
                    if (!(fine = bar_wait_warp(full + 8 * stage.at, stage.parity, sums_empty + 8 * half.at, half.parity ^ 1))) break;
                    tmem_after_sync();
                    if (one) {
                        const uint64_t r = rows_operand + stage.at * (kOperandBytes >> 4), w = weights_operand + stage.at * (kOperandBytes >> 4);
                        const uint32_t to = tmem + half.at * kTileFeatures;
                        pair_mma_e4m3(to, r, w, shape, false);
                        pair_mma_e4m3(to, r + 2, w + 2, shape, true);
                        pair_mma_e4m3(to, r + 4, w + 4, shape, true);
                        pair_mma_e4m3(to, r + 6, w + 6, shape, true);
                        pair_mma_commit(empty + 8 * stage.at);
                        pair_mma_commit(sums_full + 8 * half.at);
                    }
                    __syncwarp();
                }
            }
            if (!fine)
                for (int i = max(n - 2, 0); i < n; ++i) (void)bar_wait_warp(sums_full + 8 * (i & 1), i >> 1 & 1);
        } else if (warp == 2) {
            // Which tiles: with one weight, 8 tiles of rows by all features, then the next 8 (what the GPU works on at a time is
            // a patch with few different rows and features, which L2 holds); else the experts' in their order.
            const int wide = (a.out_dim + kTileFeatures - 1) / kTileFeatures, pairs = gridDim.x / 2;
            const int64_t high = tiles_of_rows(a, kTileRows), whole = high * wide;
            const int64_t last = whole % pairs, cut = 2 * last <= pairs ? whole - last : whole, all = whole + (whole - cut);
            for (int64_t u = blockIdx.x / 2;; u += pairs) {
                Tile tile = {0, 0, 0, 0};
                if (u < all) {
                    const int64_t v = u < cut ? u : cut + ((u - cut) >> 1);
                    int64_t t;
                    if (a.offsets) {
                        t = v / wide;
                        tile.feature = (int)(v - t * wide) * kTileFeatures;
                    } else {
                        const int64_t band = v / (kRowTilesTogether * wide);
                        const int in = (int)(v - band * kRowTilesTogether * wide), h = (int)min((int64_t)kRowTilesTogether, high - band * kRowTilesTogether);
                        t = band * kRowTilesTogether + in % h;
                        tile.feature = in / h * kTileFeatures;
                    }
                    const Rows rows = rows_of_tile(a, t, kTileRows);
                    tile.expert = rows.expert;
                    tile.first = rows.first;
                    tile.count = rows.count;
                    if (u >= cut) {
                        const int skip = (u - cut) & 1 ? kBlock : 0;
                        tile.first += skip;
                        tile.count = min(tile.count - skip, kBlock);
                        if (tile.count <= 0) continue;
                    }
                }
                if (!(fine = bar_wait_warp(used + 8 * next.at, next.parity ^ 1))) break;
                if (lane == 0) {
                    volatile Tile &t = tiles[next.at];
                    t.expert = tile.expert;
                    t.first = tile.first;
                    t.count = tile.count;
                    t.feature = tile.feature;
                    bar_arrive(known + 8 * next.at);
                }
                next.next();
                if (tile.count == 0) break;
            }
        }
    } else {
        registers_up<kRegistersAdding>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t empty_of_0 = cluster_address(sums_empty, 0);
        const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0;      // stores of 32 bytes
        Ring<Q> words_of;
        Ring<2> sums;
        // (written out for either width: one loop that asks which keeps its sums in registers a third as fast)
        auto take = [&](const Tile &tile, auto short_tile) {
            // A short tile's 64 rows lie on two quarters of the lanes, its other 128 features on the other two.
            constexpr bool kShort = decltype(short_tile)::value;
            constexpr int kOwn = kShort ? kBlock / 2 : kBlock;      // rows of the block, and features of the thread
            const int first = tile.first + rank * kOwn, count = min(tile.count - rank * kOwn, kOwn);
            const int mine = (kShort ? quarter & 1 : quarter) * 32 + lane, block = kShort ? quarter >> 1 : half;
            const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + half * kOwn;
            const int feature = tile.feature + block * kBlock + (kShort ? half * kOwn : 0);
            const bool real = mine < count && source_row(a, first + mine) >= 0;
            unsigned long long sum[kOwn / 2];
#pragma unroll
            for (int j = 0; j < kOwn / 2; ++j) sum[j] = 0;
            for (int k = 0; k < p.groups; ++k, sums.next()) {
                if ((!kFours || k % 4 == 0) && !(fine = bar_wait_warp(scaled + 8 * words_of.at, words_of.parity))) return;
                const float *words = reinterpret_cast<const float *>(shared + (scales - base)) + words_of.at * ((kFours ? kFourBytes : kManyScaleBytes) / 4);
                const float f = kFours ? words[4 * mine + k % 4] * words[4 * (kBlock + block) + k % 4] : words[mine] * words[kBlock + block];
                if (!kFours || k % 4 == 3) words_of.next();
                if (!(fine = bar_wait_warp(sums_full + 8 * sums.at, sums.parity))) return;
                tmem_after_sync();
                // 16 columns are on their way while the 16 before are multiplied and added
                const unsigned long long both = pair_of_floats(f, f);
                const uint32_t at = from + sums.at * kTileFeatures;
                float v[2][16];
                tmem_load(at, v[0]);
                tmem_wait_loads(v[0]);
#pragma unroll
                for (int j = 0; j < kOwn / 16; ++j) {
                    if (j < kOwn / 16 - 1) tmem_load(at + (j + 1) * 16, v[(j + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        fma2(sum[j * 8 + i / 2], pair_of_floats(v[j & 1][i], v[j & 1][i + 1]), both);
                    if (j < kOwn / 16 - 1) tmem_wait_loads(v[(j + 1) & 1]);
                }
                tmem_before_sync();
                __syncwarp();
                if (lane == 0) cluster_bar_arrive(empty_of_0 + 8 * sums.at);
            }
            const int there = min(a.out_dim - feature, kOwn);
            if constexpr (kOdd) {
                // Rows that do not lie on 16 bytes: 32 features at a time by way of shared memory, a row to a store.
                uint16_t *const odd = reinterpret_cast<uint16_t *>(shared + (odd_at - base) + (warp - 4) * kOddBytes);
                const int low = mine - lane;
#pragma unroll
                for (int j = 0; j < kOwn; j += 32) {
                    if (j >= there) break;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 v = floats_of(sum[j / 2 + e]);
                        if (!real) v = make_float2(0, 0);
                        *reinterpret_cast<uint32_t *>(odd + lane * kOddPitch + 2 * e) = a.dtype == AR_F16 ? to_pair<__half>(v) : to_pair<__nv_bfloat16>(v);
                    }
                    __syncwarp();
                    if (j + lane < there)
                        for (int r = 0; r < 32 && low + r < count; ++r)
                            static_cast<uint16_t *>(a.out)[(int64_t)(first + low + r) * a.out_stride + feature + j + lane] = odd[r * kOddPitch + lane];
                    __syncwarp();
                }
                return;
            }
            if (mine >= count) return;
            uint16_t *const row = static_cast<uint16_t *>(a.out) + (int64_t)(first + mine) * a.out_stride + feature;
#pragma unroll
            for (int j = 0; j < kOwn; j += 16) {
                if (j >= there) break;
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float2 v = floats_of(sum[j / 2 + e]);
                    if (!real) v = make_float2(0, 0);
                    w[e] = a.dtype == AR_F16 ? to_pair<__half>(v) : to_pair<__nv_bfloat16>(v);
                }
                if (wide && j + 16 <= there) {
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + j), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                                 "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
                } else if (j + 16 <= there) {
                    *reinterpret_cast<uint4 *>(row + j) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(row + j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (j + e < there) row[j + e] = (uint16_t)(w[e / 2] >> (e & 1) * 16);
                }
            }
        };
        while (fine) {
            const Tile tile = next_tile();
            if (tile.count == 0) break;
            if (tile.count <= kBlock) take(tile, std::true_type());
            else take(tile, std::false_type());
            __syncwarp();
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
        for (const auto kernel : {many_kernel<false, false>, many_kernel<false, true>, many_kernel<true, false>, many_kernel<true, true>})
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kManySmem);
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    Product q = p;
    if (a.row_of) {
        const int64_t pitch = pitch_of(a);
        const int groups = a.x_row_scales ? 1 : p.groups;
        uint8_t *rows = static_cast<uint8_t *>(a.workspace);
        float *scales = reinterpret_cast<float *>(rows + a.rows * pitch);
        e = launch_next(pick_kernel, dim3((unsigned)std::min((a.rows + 7) / 8, (int64_t)8 * multiprocessors)), 256, 0, s, 0, a, rows, scales, (int)pitch, groups);
        if (e != cudaSuccess) return e;
        q.a.x = rows;
        q.a.x_stride = pitch;
        q.a.x_scales = scales;
        q.a.x_scales_stride = groups;
    }
    CUtensorMap weight, x;
    ar_matmul_fp8_args in_order = q.a;
    if (a.row_of) in_order.x_rows = a.rows;
    if (!map_weight(&weight, a, kBlock) || !map_rows(&x, in_order, kBlock)) return cudaErrorInvalidValue;
    const int64_t units = most_tiles(a, kTileRows) * ((a.out_dim + kTileFeatures - 1) / kTileFeatures), pairs = multiprocessors / 2;
    const bool odd = reinterpret_cast<uintptr_t>(a.out) % 16 != 0 || a.out_stride % 8 != 0;
    const bool fours = !a.x_row_scales && p.groups % 4 == 0 && q.a.x_scales_stride % 4 == 0 && !misaligned(q.a.x_scales, 16) && !misaligned(a.weight_scales, 16);
    const auto kernel = odd ? (fours ? many_kernel<true, true> : many_kernel<true, false>) : fours ? many_kernel<false, true> : many_kernel<false, false>;
    return launch_next(kernel, dim3((unsigned)(2 * std::min(2 * units, pairs))), kManyThreads, kManySmem, s, 2, q, weight, x);
}

int take_many_status(int *code) {
    const int none = AR_OK;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_many_status, sizeof(int));
    if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_many_status, &none, sizeof(int));
    return launch_status(e);
}

}  // namespace tda
