// ar_route.cu -- ar_route_experts: the router's choice and the rows by expert.
//
// The choice: a warp to a token, its logits in registers, `chosen` rounds of a maximum over the warp.  A
// logit's bits, turned so that whole numbers order them like the values, carry the order; among equal ones the
// lowest number wins a second vote.
//
// The rows: a stable counting sort of the pairs by expert in one cluster of 8 blocks, each with a
// run of the pairs, each warp of it with a part of that run: count by warp and expert, add up over warps and blocks
// (through the cluster's shared memory), then go over the pairs again, every pair's place being its expert's
// beginning, what earlier blocks and warps have of that expert, and its rank among the lanes with the same one.
#include <cooperative_groups.h>

#include <cfloat>

#include "ar_ffn.h"
#include "ar_kv4.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace tda;

constexpr int kMostExperts = 1024, kMostChosen = 32;
constexpr int kSortWarps = 32, kSortBlocks = 8;

template <typename T> __device__ __forceinline__ float logit(const void *p, int64_t i) { return Elem<T>::to_float(static_cast<const T *>(p)[i]); }
template <> __device__ __forceinline__ float logit<float>(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }

// Whole numbers in the values' order; 0 for what is never chosen.  (x + 0: -0 is 0.)
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint((x > FLT_MAX ? FLT_MAX : x) + 0.0f);
    return !(x > -INFINITY) ? 0 : b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }

// Lane l holds logits l, l + 32, ...
template <typename T, int V>
__global__ void __launch_bounds__(256) choose_kernel(const ar_route_experts_args a) {
    after_the_stream();
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (token >= a.tokens) return;
    uint32_t o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        o[i] = e < a.experts ? order_of(logit<T>(a.logits, token * a.logits_stride + e)) : 0;
    }
    float most = 0, sum = 0, own = 0;
    int id = -1;
    for (int j = 0; j < a.chosen; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, o[i]);
        best = __reduce_max_sync(~0u, best);
        if (best == 0) break;
        int e = kMostExperts;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (o[i] == best) e = i * 32 + lane;
        e = __reduce_min_sync(~0u, e);
        if (j == 0) {
            most = value_of(best);
            if (!a.normalize) {
#pragma unroll
                for (int i = 0; i < V; ++i) sum += o[i] ? expf(value_of(o[i]) - most) : 0.0f;
#pragma unroll
                for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
            }
        }
        const float w = expf(value_of(best) - most);
        if (a.normalize) sum += w;
        if (lane == j) {
            id = e;
            own = w;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * 32 + lane == e) o[i] = 0;
    }
    if (lane < a.chosen) {
        a.expert_ids[token * a.chosen + lane] = id;
        a.weights[token * a.chosen + lane] = id < 0 ? 0.0f : __fdiv_rn(own, sum);
    }
}

__global__ void __launch_bounds__(kSortWarps * 32) rows_kernel(const ar_route_experts_args a) {
    after_the_stream();
    extern __shared__ int sh[];
    const int E = a.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *count = sh;                            // [warps][E]: of each warp; then where its pairs of an expert begin
    int *total = sh + kSortWarps * E;           // [E]: of the block
    int *scan = total + E;                      // [warps]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank();
    const int64_t n = a.tokens * a.chosen;
    const int64_t share = ((n + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps) + 31) / 32 * 32;
    const int64_t begin = min(n, (rank * kSortWarps + warp) * share), end = min(n, begin + share);
    for (int i = threadIdx.x; i < kSortWarps * E; i += blockDim.x) count[i] = 0;
    __syncthreads();
    int *own = count + warp * E;
    for (int64_t i = begin; i < end; i += 32) {
        const int e = i + lane < end ? a.expert_ids[i + lane] : -1;
        const unsigned same = __match_any_sync(~0u, e);
        if (e >= 0 && lane == __ffs(same) - 1) own[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = count[w * E + e];
            count[w * E + e] = run;
            run += c;
        }
        total[e] = run;
    }
    cluster.sync();
    // one expert to a thread (at most 1024): what all blocks have of it, and those before this one
    const int e = threadIdx.x;
    int all = 0, before = 0;
    if (e < E)
        for (int b = 0; b < kSortBlocks; ++b) {
            const int c = cluster.map_shared_rank(total, b)[e];
            if (b < rank) before += c;
            all += c;
        }
    int run = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run += x;
    }
    if (lane == 31) scan[warp] = run;
    cluster.sync();         // (also: nobody reads another block's totals any more)
    int past = 0, sum = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) past += scan[w];
        sum += scan[w];
    }
    run += past;
    if (e < E) {
        if (rank == 0) a.offsets[e + 1] = run;
        for (int w = 0; w < kSortWarps; ++w) count[w * E + e] += run - all + before;
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[0] = 0;
    __syncthreads();
    for (int64_t i = begin; i < end; i += 32) {
        const int64_t at = i + lane;
        const int x = at < end ? a.expert_ids[at] : -1;
        const unsigned same = __match_any_sync(~0u, x);
        const int to = x >= 0 ? own[x] + __popc(same & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (x >= 0 && lane == __ffs(same) - 1) own[x] += __popc(same);
        __syncwarp();
        if (at < end) {
            a.place[at] = to;
            if (to >= 0) a.rows[to] = (int)(at / a.chosen);
        }
    }
    for (int64_t i = sum + (int64_t)rank * blockDim.x + threadIdx.x; i < n; i += kSortBlocks * blockDim.x) a.rows[i] = -1;
}

template <typename T>
cudaError_t choose(const ar_route_experts_args &a, cudaStream_t s) {
    const int v = (a.experts + 31) / 32;
    return launch_next(v <= 1 ? choose_kernel<T, 1> : v <= 2 ? choose_kernel<T, 2> : v <= 4 ? choose_kernel<T, 4>
                       : v <= 8 ? choose_kernel<T, 8> : v <= 16 ? choose_kernel<T, 16> : choose_kernel<T, 32>,
                       dim3((unsigned)((a.tokens + 7) / 8)), 256, 0, s, 0, a);
}

size_t sort_bytes(int experts) { return sizeof(int) * ((kSortWarps + 1) * (size_t)experts + kSortWarps); }

cudaError_t start(const ar_route_experts_args &a, cudaStream_t s) {
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sort_bytes(kMostExperts));
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    if (a.tokens > 0) {
        e = a.dtype == AR_F16 ? choose<__half>(a, s) : a.dtype == AR_BF16 ? choose<__nv_bfloat16>(a, s) : choose<float>(a, s);
        if (e != cudaSuccess) return e;
    }
    return launch_next(rows_kernel, dim3(kSortBlocks), kSortWarps * 32, sort_bytes(a.experts), s, kSortBlocks, a);
}

}  // namespace

extern "C" AR_API int ar_route_experts(const ar_route_experts_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_route_experts_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16 && a.dtype != AR_F32) return AR_EINVAL;
    if (a.tokens < 0 || a.experts < 1 || a.chosen < 1 || a.chosen > a.experts || (a.normalize & ~1)) return AR_EINVAL;
    if (a.experts > kMostExperts || a.chosen > kMostChosen || a.tokens > (1 << 30) / a.chosen) return AR_ETOOBIG;
    if (!a.offsets || misaligned(a.offsets, 4)) return AR_EINVAL;
    if (a.tokens > 0) {
        if (!a.logits || !a.weights || !a.expert_ids || !a.rows || !a.place) return AR_EINVAL;
        if (misaligned(a.logits, a.dtype == AR_F32 ? 4 : 2) || misaligned(a.weights, 4) || misaligned(a.expert_ids, 4) || misaligned(a.rows, 4) ||
            misaligned(a.place, 4))
            return AR_EINVAL;
    }
    return launch_status(start(a, stream));
}
