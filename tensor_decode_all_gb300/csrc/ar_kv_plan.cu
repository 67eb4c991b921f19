// ar_kv_plan.cu -- ar_kv_plan: block tables and slot maps from the requests' lengths.
//
// Two running sums over the requests (new tokens, new pages) give every new token and page its place; each
// token then finds its request by bisection. Every block makes the whole sums for itself in shared memory (at
// most 8192 requests, a few passes of one block) and writes its share of the tokens; the blocks are one
// cluster, whose barrier stands between the reads of lens and *free_used and their writes, so that both may be
// updated in place.
//
// Bound by latency: 64 requests of a token each take 4.8 us on a GB300, 1000 requests with 23524 new tokens
// 9.0 (graph replays; the second writes 0.4 MB).
#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr int kPlanThreads = 1024;
constexpr int kPlanRequests = 8192;

struct Sums {
    long long tokens, pages;
};

__device__ __forceinline__ Sums warp_scan(Sums x) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long a = __shfl_up_sync(~0u, x.tokens, d), b = __shfl_up_sync(~0u, x.pages, d);
        if ((threadIdx.x & 31) >= d) {
            x.tokens += a;
            x.pages += b;
        }
    }
    return x;
}

__device__ __forceinline__ int pages_of(int64_t tokens, int page) { return (int)((tokens + page - 1) / page); }

// The last b with start[b] <= i, of n (start is non-decreasing, start[0] = 0 <= i).
__device__ __forceinline__ int find(const int *start, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const ar_kv_plan_args a) {
    extern __shared__ int sh[];
    int *len = sh, *token0 = sh + a.requests, *page0 = token0 + a.requests;
    __shared__ Sums warp_sums[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    after_the_stream();
    const int used = a.free_used[0];
    Sums carry = {0, 0};
    int bad = used < 0 ? 1 : 0;   // bit 0: AR_EINVAL, bit 1: AR_ETOOBIG
    for (int base = 0; base < a.requests; base += kPlanThreads) {
        const int b = base + threadIdx.x;
        const bool in = b < a.requests;
        const int n = in ? a.lens[b] : 0, m = in ? a.new_tokens[b] : 0;
        Sums x = {0, 0};
        if (n < 0 || m < 0 || (int64_t)n + m > 0x7fffffff) {
            bad |= 1;
        } else {
            const int had = pages_of(n, a.page), all = pages_of((int64_t)n + m, a.page);
            x = {m, all - had};
            if (all > a.table_width) bad |= 2;
            else if (m > 0 && n % a.page && a.table[(int64_t)b * a.table_stride + n / a.page] < 0) bad |= 1;
        }
        const Sums own = x;
        x = warp_scan(x);
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        if (warp == 0) warp_sums[lane] = warp_scan(warp_sums[lane]);
        __syncthreads();
        Sums before = carry;
        if (warp > 0) {
            before.tokens += warp_sums[warp - 1].tokens;
            before.pages += warp_sums[warp - 1].pages;
        }
        if (in) {
            // kept within 32 bits: past them the plan is refused and these are not read
            len[b] = n;
            token0[b] = (int)min(before.tokens + x.tokens - own.tokens, 0x7fffffffll);
            page0[b] = (int)min(before.pages + x.pages - own.pages, 0x7fffffffll);
        }
        carry.tokens += warp_sums[kPlanThreads / 32 - 1].tokens;
        carry.pages += warp_sums[kPlanThreads / 32 - 1].pages;
        __syncthreads();
    }
    if (carry.tokens > a.max_tokens) bad |= 2;
    if (carry.tokens > 0x7fffffff || (long long)used + carry.pages > 0x7fffffff) bad |= 1;
    const bool invalid = __syncthreads_or(bad & 1), big = __syncthreads_or(bad & 2);
    const int status = invalid ? AR_EINVAL : big ? AR_ETOOBIG : (long long)used + carry.pages > a.free_count ? AR_ENOMEM : AR_OK;
    const int tokens = status ? 0 : (int)carry.tokens, pages = status ? 0 : (int)carry.pages;

    // Every block of the cluster has read what follows may overwrite.
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");

    const unsigned first = blockIdx.x * kPlanThreads + threadIdx.x, stride = gridDim.x * kPlanThreads;
    for (int b = (int)first; b < a.requests; b += (int)stride) {
        const int end = b + 1 < a.requests ? token0[b + 1] : tokens;
        a.lens_out[b] = len[b] + (status ? 0 : end - token0[b]);
        a.cu[b] = status ? 0 : token0[b];
    }
    for (unsigned n = first; n < (unsigned)pages; n += stride) {
        const int i = (int)n, b = find(page0, a.requests, i);
        a.table[(int64_t)b * a.table_stride + pages_of(len[b], a.page) + i - page0[b]] = a.free_pages[used + i];
    }
    // Four tokens of a thread at a time: their loads are under way together.
    // (unsigned: a stride past the last of 2^31 stays above it)
    for (unsigned i0 = first; i0 < (unsigned)a.max_tokens; i0 += 4 * stride) {
        int b[4], p[4], in[4];
        int64_t id[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned i = i0 + e * stride;
            b[e] = p[e] = in[e] = -1;
            id[e] = 0;
            if (i < (unsigned)tokens) {
                b[e] = find(token0, a.requests, (int)i);
                p[e] = len[b[e]] + (int)i - token0[b[e]];
                const int col = p[e] / a.page, had = pages_of(len[b[e]], a.page);
                in[e] = p[e] - col * a.page;
                id[e] = col < had ? a.table[(int64_t)b[e] * a.table_stride + col] : a.free_pages[used + page0[b[e]] + col - had];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned i = i0 + e * stride;
            if (i < (unsigned)a.max_tokens) {
                a.slots[i] = id[e] * a.page + in[e];
                a.request[i] = b[e];
                a.position[i] = p[e];
            }
        }
    }
    if (first == 0) {
        a.cu[a.requests] = tokens;
        a.free_used_out[0] = used + pages;
        a.status[0] = status;
    }
}

}  // namespace

extern "C" AR_API int ar_kv_plan(const ar_kv_plan_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_kv_plan_args &a = *args;
    if (a.requests < 0 || a.table_width < 0 || a.page < kTileTokens || a.page % kTileTokens || a.max_tokens < 0 ||
        a.free_count < 0 || a.table_stride < a.table_width)
        return AR_EINVAL;
    if (a.requests > kPlanRequests) return AR_ETOOBIG;
    if (!a.free_used || !a.free_used_out || !a.status || !a.cu) return AR_EINVAL;
    if (a.requests > 0 && (!a.lens || !a.new_tokens || !a.lens_out || (!a.table && a.table_width > 0))) return AR_EINVAL;
    if (a.max_tokens > 0 && (!a.slots || !a.request || !a.position)) return AR_EINVAL;
    if (a.free_count > 0 && !a.free_pages) return AR_EINVAL;
    for (const void *p : {(const void *)a.lens, (const void *)a.new_tokens, (const void *)a.table, (const void *)a.free_pages,
                          (const void *)a.free_used, (const void *)a.lens_out, (const void *)a.cu, (const void *)a.request,
                          (const void *)a.position, (const void *)a.free_used_out, (const void *)a.status})
        if (misaligned(p, 4)) return AR_EINVAL;
    if (misaligned(a.slots, 8)) return AR_EINVAL;
    // One block while its threads have about one token each, else a cluster of 8.
    const int blocks = a.max_tokens > 2 * kPlanThreads ? 8 : 1;
    const size_t smem = (size_t)a.requests * 3 * sizeof(int);
    static bool ready[64] = {};      // the attribute is set once a device; racing threads set the same
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return launch_status(cudaErrorUnknown);
    if (!*(volatile bool *)&ready[dev]) {
        if (cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanRequests * 12) != cudaSuccess)
            return launch_status(cudaErrorUnknown);
        *(volatile bool *)&ready[dev] = true;
    }
    return launch_status(launch_next(plan_kernel, dim3((unsigned)blocks), kPlanThreads, smem, stream, (unsigned)blocks, a));
}
