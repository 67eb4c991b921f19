// ar_route.cu -- ar_route_experts: the router's choice and the rows by expert.
//
// The choice: a warp to a token, its logits in registers.  A logit's bits, turned so that whole numbers order them like
// the values, carry the order; every lane knows its largest of the experts it has, and a round takes
// the largest of the warp (among equal ones the lowest lane's: the lanes have consecutive experts).
//
// The rows: a block takes up to 1024 pairs of consecutive tokens, counts them by expert, and a pair's place is its expert's
// beginning, what earlier blocks have of that expert, and how many of its own block's tokens before it have it (a
// bit of each expert's for each of the tokens, in shared memory).  One block does all where the pairs fit; else the counts
// go through the workspace, and a second launch adds up those of the blocks before.
//
// Past 256 blocks that adding up would be most of the work: the second launch is then a stable counting sort in one cluster of 8
// blocks, each with a run of the pairs, each warp of it with a part of that run: count by warp and expert, add up over warps
// and blocks (through the cluster's shared memory), then go over the pairs again.
//
// 8191 tokens to 8 of 256 experts take 17.1 us in GB300 graph replays (the choice 13 us by itself, two thirds of the cycles issue an
// instruction, some 800 to a token; the places 10), where the sort took 22 besides the choice; 5 tokens to 4 of 32, in one block, 2.2 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>

#include "ar_ffn.h"
#include "ar_kv4.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace tda;

constexpr int kMostExperts = 1024, kMostChosen = 32;
constexpr int kRouteThreads = 1024, kBlockPairs = 1024, kBlockWords = 8192, kMostBlocks = 256;
constexpr int kSortWarps = 32, kSortBlocks = 8;

template <typename T> __device__ __forceinline__ float value(T x) { return Elem<T>::to_float(x); }

// Whole numbers in the values' order; 0 for what is never chosen.  (x + 0: -0 is 0.)
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint((x > FLT_MAX ? FLT_MAX : x) + 0.0f);
    return !(x > -INFINITY) ? 0 : b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }

// What a logit is compared by: its order, and for types of 16 bits, whose order leaves the lower half free, the
// experts' order below it (so that no two are equal, and the largest says whose it is).  0: never chosen.
template <typename T> __device__ __forceinline__ uint32_t key_of(T x, int expert) {
    if constexpr (sizeof(T) == 4) {
        return order_of(x);
    } else {
        const uint32_t raw = *reinterpret_cast<const uint16_t *>(&x), b = raw == 0x8000 ? 0 : raw;
        return value(x) > -INFINITY ? (b & 0x8000 ? ~b : b | 0x8000) << 16 | (uint32_t)(0xffff - expert) : 0;
    }
}
template <typename T> __device__ __forceinline__ float number_of(uint32_t key) {
    if constexpr (sizeof(T) == 4) {
        return value_of(key);
    } else {
        const uint16_t raw = (uint16_t)(key & 0x80000000u ? key >> 16 & 0x7fff : ~(key >> 16));
        return fminf(value(*reinterpret_cast<const T *>(&raw)), FLT_MAX);
    }
}

// Lane l's logits V l .. V l + V - 1 of a token, in their order.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const ar_route_experts_args &a, int64_t token, bool vectors, uint32_t (&o)[V]) {
    const int first = (threadIdx.x & 31) * V;
    const T *p = static_cast<const T *>(a.logits) + token * a.logits_stride + first;
    constexpr int each = V * sizeof(T) < 16 ? V : 16 / (int)sizeof(T);       // values of a load
    if (vectors) {
#pragma unroll
        for (int i = 0; i < V; i += each) {
            union { uint4 q; uint2 d; uint32_t w; uint16_t h; T t[each]; } u;
            if (first + i < a.experts) {      // (whole loads: the number of experts is a multiple of `each`)
                if constexpr (each * sizeof(T) == 16) u.q = *reinterpret_cast<const uint4 *>(p + i);
                else if constexpr (each * sizeof(T) == 8) u.d = *reinterpret_cast<const uint2 *>(p + i);
                else if constexpr (each * sizeof(T) == 4) u.w = *reinterpret_cast<const uint32_t *>(p + i);
                else u.h = *reinterpret_cast<const uint16_t *>(p + i);
            }
#pragma unroll
            for (int e = 0; e < each; ++e) o[i + e] = first + i < a.experts ? key_of(u.t[e], first + i + e) : 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = first + i < a.experts ? key_of(p[i], first + i) : 0;
    }
}

// The experts of a token, by a warp whose lanes hold its keys: lane j < chosen returns the j-th's number (-1: none) and weight.
template <typename T, int V> __device__ __forceinline__ int choose(const ar_route_experts_args &a, uint32_t (&o)[V], float &weight) {
    const int lane = threadIdx.x & 31;
    uint32_t best = 0, own = 0, most = 0;
    int at = 0, id = -1;
    float all = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (sizeof(T) == 4 && o[i] > best) at = i;
        best = max(best, o[i]);
    }
    for (int j = 0; j < a.chosen; ++j) {
        const uint32_t top = __reduce_max_sync(~0u, best);
        if (top == 0) break;
        if (j == 0) {
            most = top;
            if (!a.normalize) {
                const float m = number_of<T>(top);
#pragma unroll
                for (int i = 0; i < V; ++i) all += o[i] ? expf(number_of<T>(o[i]) - m) : 0.0f;
            }
        }
        if constexpr (sizeof(T) == 4) {
            // (of equal logits the lowest lane's: it has the lowest numbers)
            const int src = __ffs(__ballot_sync(~0u, best == top)) - 1, e = src * V + __shfl_sync(~0u, at, src);
            if (lane == j) id = e;
            const int out = lane == src ? at : -1;
            best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i == out) o[i] = 0;
                if (o[i] > best) best = o[i], at = i;
            }
        } else {
            if (lane == j) id = 0xffff - (int)(top & 0xffff);
            best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (o[i] == top) o[i] = 0;
                best = max(best, o[i]);
            }
        }
        if (lane == j) own = top;
    }
    const float w = id < 0 ? 0.0f : expf(number_of<T>(own) - number_of<T>(most));
    float sum = a.normalize ? w : all;
#pragma unroll
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    weight = id < 0 ? 0.0f : __fdiv_rn(w, sum);
    return id;
}

// The pairs of one block: `ids` of them (-1: none); of each expert, which of the block's tokens have it, a bit each (`words`
// words to an expert), and `before`, the first of its rows in this block.
struct Pairs {
    int16_t ids[kBlockPairs];
    int before[kMostExperts];
    uint32_t has[kBlockWords];
    int scan[32];
};

__device__ __forceinline__ void clear_pairs(Pairs &s, int experts, int words) {
    for (int i = threadIdx.x; i < experts * words; i += kRouteThreads) s.has[i] = 0;
}
__device__ __forceinline__ void note_pair(Pairs &s, int id, int token, int words) {
    if (id >= 0) atomicOr(&s.has[id * words + (token >> 5)], 1u << (token & 31));
}
__device__ __forceinline__ int pairs_of(const Pairs &s, int expert, int words) {
    int n = 0;
    for (int w = 0; w < words; ++w) n += __popc(s.has[expert * words + w]);
    return n;
}

// Running sums over the experts of `own` (one expert to a thread): what earlier experts have, and all.
__device__ __forceinline__ int before_expert(Pairs &s, int own, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run += x;
    }
    if (lane == 31) s.scan[warp] = run;
    __syncthreads();
    static_assert(kRouteThreads == 32 * 32 && kMostExperts <= kRouteThreads, "a lane to each warp, a thread to each expert");
    int warps = s.scan[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, warps, d);
        if (lane >= d) warps += x;
    }
    const int earlier = __shfl_sync(~0u, warps, max(warp - 1, 0));
    all = __shfl_sync(~0u, warps, 31);
    return (warp > 0 ? earlier : 0) + run - own;
}

// Places and rows of the block's pairs, first .. first + n - 1 of the call.
__device__ __forceinline__ void place_pairs(const ar_route_experts_args &a, const Pairs &s, int64_t first, int n, int words) {
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
        const int e = s.ids[i], token = i / a.chosen;
        int to = -1;
        if (e >= 0) {
            to = s.before[e] + __popc(s.has[e * words + (token >> 5)] & ((1u << (token & 31)) - 1));
            for (int w = 0; w < token >> 5; ++w) to += __popc(s.has[e * words + w]);
            a.rows[to] = (int)(first / a.chosen) + token;
        }
        a.place[first + i] = to;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) choose_kernel(const ar_route_experts_args a, int tokens, int blocks, bool vectors) {
    __shared__ __align__(16) Pairs s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, a.tokens - first);
    const int words = (tokens + 31) / 32;
    if (blocks > 0) clear_pairs(s, a.experts, words);
    __syncthreads();
    after_the_stream();
    uint32_t o[V];
    if (warp < here) load_logits<T, V>(a, first + warp, vectors, o);
    for (int t = warp; t < here; t += kRouteThreads / 32) {
        float weight;
        const int id = choose<T, V>(a, o, weight);
        if (t + kRouteThreads / 32 < here) load_logits<T, V>(a, first + t + kRouteThreads / 32, vectors, o);
        if (lane < a.chosen) {
            const int64_t at = (first + t) * a.chosen + lane;
            a.expert_ids[at] = id;
            a.weights[at] = weight;
            if (blocks > 0) {
                s.ids[t * a.chosen + lane] = (int16_t)id;
                note_pair(s, id, t, words);
            }
        }
    }
    if (blocks == 0) return;
    __syncthreads();
    if (blocks > 1) {
        if (threadIdx.x < a.experts) a.workspace[(int64_t)blockIdx.x * a.experts + threadIdx.x] = pairs_of(s, threadIdx.x, words);
        return;
    }
    int all;
    const int begin = before_expert(s, threadIdx.x < a.experts ? pairs_of(s, threadIdx.x, words) : 0, all);
    if (threadIdx.x < a.experts) {
        s.before[threadIdx.x] = begin;
        a.offsets[threadIdx.x] = begin;
    }
    if (threadIdx.x == 0) a.offsets[a.experts] = all;
    __syncthreads();
    const int n = here * a.chosen;
    place_pairs(a, s, 0, n, words);
    for (int i = all + threadIdx.x; i < n; i += kRouteThreads) a.rows[i] = -1;
}

__global__ void __launch_bounds__(kRouteThreads) place_kernel(const ar_route_experts_args a, int tokens, int blocks) {
    __shared__ __align__(16) Pairs s;
    __shared__ int parts[2][kRouteThreads];
    const int words = (tokens + 31) / 32;
    clear_pairs(s, a.experts, words);
    __syncthreads();
    after_the_stream();
    const int64_t first = (int64_t)blockIdx.x * tokens * a.chosen, pairs = a.tokens * a.chosen;
    const int n = (int)min((int64_t)tokens * a.chosen, pairs - first);
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
        const int id = a.expert_ids[first + i];
        s.ids[i] = (int16_t)id;
        note_pair(s, id, i / a.chosen, words);
    }
    // as many threads to an expert as there are, each with some of the blocks
    const int wide = a.experts, each = kRouteThreads / wide, e = threadIdx.x % wide, part = threadIdx.x / wide;
    const int b0 = blocks * part / each, b1 = part < each ? blocks * (part + 1) / each : b0;
    int sum = 0, past = 0, all;
#pragma unroll 32
    for (int b = b0; b < b1; ++b) {
        const int c = a.workspace[(int64_t)b * wide + e];
        sum += c;
        if (b < blockIdx.x) past += c;
    }
    parts[0][threadIdx.x] = sum;
    parts[1][threadIdx.x] = past;
    __syncthreads();
    sum = past = 0;
    if (threadIdx.x < wide)
        for (int q = 0; q < each; ++q) {
            sum += parts[0][q * wide + threadIdx.x];
            past += parts[1][q * wide + threadIdx.x];
        }
    const int begin = before_expert(s, sum, all);
    if (threadIdx.x < wide) {
        s.before[threadIdx.x] = begin + past;
        if (blockIdx.x == 0) a.offsets[threadIdx.x] = begin;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = all;
    __syncthreads();
    place_pairs(a, s, first, n, words);
    for (int64_t i = all + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; i < pairs; i += (int64_t)gridDim.x * kRouteThreads) a.rows[i] = -1;
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
cudaError_t start_choice(const ar_route_experts_args &a, cudaStream_t s, int tokens, int blocks) {
    const int v = (a.experts + 31) / 32, each = v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8, bytes = std::min(each * (int)sizeof(T), 16), whole = bytes / (int)sizeof(T);
    const bool vectors = !misaligned(a.logits, bytes) && a.logits_stride % whole == 0 && a.experts % whole == 0;
    return launch_next(v <= 1 ? choose_kernel<T, 1> : v <= 2 ? choose_kernel<T, 2> : v <= 4 ? choose_kernel<T, 4>
                       : v <= 8 ? choose_kernel<T, 8> : v <= 16 ? choose_kernel<T, 16> : choose_kernel<T, 32>,
                       dim3((unsigned)((a.tokens + tokens - 1) / tokens)), kRouteThreads, 0, s, 0, a, tokens, blocks, vectors);
}

// Tokens to a block: 64 in one block, else enough for 128 blocks, and as many pairs and bits as a block can hold.
int tokens_of_block(const ar_route_experts_args &a) {
    const int64_t most = std::min(kBlockPairs / a.chosen, kBlockWords / a.experts * 32), want = std::max((a.tokens + 127) / 128, (int64_t)16);
    return (int)std::min(most, a.tokens <= 64 ? std::max<int64_t>(a.tokens, 1) : want);
}

size_t sort_bytes(int experts) { return sizeof(int) * ((kSortWarps + 1) * (size_t)experts + kSortWarps); }

cudaError_t start(const ar_route_experts_args &a, cudaStream_t s) {
    const int tokens = tokens_of_block(a);
    const int64_t blocks = (a.tokens + tokens - 1) / tokens;
    const bool sort = blocks == 0 || blocks > kMostBlocks;
    cudaError_t e = cudaSuccess;
    if (blocks) {
        const int counted = sort ? 0 : (int)blocks;
        e = a.dtype == AR_F16 ? start_choice<__half>(a, s, tokens, counted)
            : a.dtype == AR_BF16 ? start_choice<__nv_bfloat16>(a, s, tokens, counted) : start_choice<float>(a, s, tokens, counted);
        if (e != cudaSuccess || blocks == 1) return e;
    }
    if (!sort) return launch_next(place_kernel, dim3((unsigned)blocks), kRouteThreads, 0, s, 0, a, tokens, (int)blocks);
    static bool ready[64] = {};
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sort_bytes(kMostExperts));
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_next(rows_kernel, dim3(kSortBlocks), kSortWarps * 32, sort_bytes(a.experts), s, kSortBlocks, a);
}

}  // namespace

extern "C" AR_API size_t ar_route_experts_workspace(const ar_route_experts_args *args) {
    if (!args || args->tokens <= 0 || args->chosen < 1 || args->chosen > kMostChosen || args->experts < 1 || args->experts > kMostExperts) return 0;
    const int tokens = tokens_of_block(*args);
    const int64_t blocks = (args->tokens + tokens - 1) / tokens;
    return blocks > 1 && blocks <= kMostBlocks ? sizeof(int32_t) * (size_t)blocks * args->experts : 0;
}

extern "C" AR_API int ar_route_experts(const ar_route_experts_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_route_experts_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16 && a.dtype != AR_F32) return AR_EINVAL;
    if (a.tokens < 0 || a.experts < 1 || a.chosen < 1 || a.chosen > a.experts || (a.normalize & ~1)) return AR_EINVAL;
    if (a.experts > kMostExperts || a.chosen > kMostChosen || a.tokens > (1 << 30) / a.chosen) return AR_ETOOBIG;
    if (!a.offsets || misaligned(a.offsets, 4)) return AR_EINVAL;
    if (a.tokens > 0) {
        if (!a.logits || !a.weights || !a.expert_ids || !a.rows || !a.place || (!a.workspace && ar_route_experts_workspace(&a) > 0)) return AR_EINVAL;
        if (misaligned(a.logits, a.dtype == AR_F32 ? 4 : 2) || misaligned(a.weights, 4) || misaligned(a.expert_ids, 4) || misaligned(a.rows, 4) ||
            misaligned(a.place, 4) || misaligned(a.workspace, 4))
            return AR_EINVAL;
    }
    return launch_status(start(a, stream));
}
