// ar_silu_fp8.cu -- ar_silu_mul_fp8: the gated activation with e4m3 output and scales.
//
// One pass, 8 channels to a thread: 16 bytes of gates, 16 of factors, 8 of output.  Groups of a power of two up to 256 lie in
// 1 to 32 lanes of a warp, whose largest value goes round by shuffles; a row that is one group is a block's, its
// values kept in registers until the block's largest is known.
//
// 5 bytes a channel: 32767 rows of 1024 in groups of 128 take 30 us in GB300 graph replays, 5.6 TB/s or 84% of what a plain copy
// reaches; instructions are issued in three cycles of four, without the question for small gates it were 28.5 us.  61 rows of
// 3584, one scale each: 1.7 us.
#include <cuda_fp8.h>

#include <algorithm>

#include "ar_ffn.h"
#include "ar_kv4.cuh"
#include "ar_tensor.cuh"

namespace {

using namespace tda;

// The larger of two magnitudes (the first is 0 or more already); a NaN wins.
__device__ __forceinline__ float top_of(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// The same of a (0 or more already) and two others.
__device__ __forceinline__ float top_of(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// For gates below -8.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// Two at a time (the adds and products are instructions of two), for gates from -8 on, by the hardware's power of two and reciprocal.  The
// power's argument, up to 11.6, is rounded by 2^-21 and off by 2^-22.6 for log2(e)'s sake: exp(-g) is off by less than 2^-20.5
// with the instruction's own 2^-22, y by less than 2^-19.9.
__device__ __forceinline__ float2 quick_silu_mul(float2 g, float2 u) {
    float2 e, r;
    const unsigned long long gates = pair_of_floats(g.x, g.y);
    e = floats_of(mul2(gates, pair_of_floats(-1.4426950408889634f, -1.4426950408889634f)));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    r = floats_of(add2(pair_of_floats(e.x, e.y), pair_of_floats(1, 1)));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.y));
    return floats_of(mul2(mul2(gates, pair_of_floats(r.x, r.y)), pair_of_floats(u.x, u.y)));
}

// One value, the same bits as of two.  (Which form a value takes is its own gate's matter, so that a row has the same output wherever it lies.)
template <typename T> __device__ __forceinline__ float one_silu_mul(T gate, T factor) {
    const float g = Elem<T>::to_float(gate), u = Elem<T>::to_float(factor);
    return g < -8.0f ? silu_mul(g, u) : quick_silu_mul(make_float2(g, g), make_float2(u, u)).x;
}

// A group's scale from its largest value.  (A top up to 224 * 2^-149 rounds to 0 as well: what it leaves is 0 by the scale 1.)
__device__ __forceinline__ float divided_scale(float top) {
    const float scale = __fdiv_rn(top, 448.0f);
    return scale == 0 ? 1.0f : scale;
}

// The same, and what its values are multiplied by (0: they are divided).
__device__ __forceinline__ float2 scale_of(float top) {
    if (top > 0x1p-60f && top < 0x1p100f) return make_float2(top * (1.0f / 448.0f), __fdividef(448.0f, top));   // within 2 units of the last place of 1 / scale
    return make_float2(divided_scale(top), 0);
}

union Vec {
    uint4 v;
    uint32_t u[4];
};

// The 8 values of a thread, and the larger of `top` and theirs.
template <typename T> __device__ __forceinline__ float values(const Vec &g, const Vec &u, float (&y)[8], float top) {
    float low = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = pair_of<T>(g.u[e]), v = quick_silu_mul(a, pair_of<T>(u.u[e]));
        asm("min.f32 %0, %0, %1, %2;" : "+f"(low) : "f"(a.x), "f"(a.y));
        y[2 * e] = v.x;
        y[2 * e + 1] = v.y;
    }
    if (low < -8.0f) {          // (seldom; y is the smaller the more so)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = pair_of<T>(g.u[e]), b = pair_of<T>(u.u[e]);
            if (a.x < -8.0f) y[2 * e] = silu_mul(a.x, b.x);
            if (a.y < -8.0f) y[2 * e + 1] = silu_mul(a.y, b.y);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) top = top_of(top, y[2 * e], y[2 * e + 1]);
    return top;
}

__device__ __forceinline__ uint2 rounded(const float (&y)[8], float2 s) {
    uint32_t b[4];
    if (s.y != 0) {
        const unsigned long long factor = pair_of_floats(s.y, s.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __nv_cvt_float2_to_fp8x2(floats_of(mul2(pair_of_floats(y[2 * e], y[2 * e + 1]), factor)), __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            b[e] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[2 * e], s.x), __fdiv_rn(y[2 * e + 1], s.x)), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}

// (32767 rows of 1024: three vectors to a thread and 128 threads 30.0 us, two and 256 32.0, one and 256 34.5, four and 128 32.8)
constexpr int kGroupThreads = 128, kGroupVecs = 3;

// n / d for n below 2^31, by a product and a shift (d's multiplier is ceil(2^(32 + shift) / d) - 2^32, with the least shift that
// 2^shift >= d: the error is below n / 2^(32 + shift) < 1 / d).
struct Divisor {
    uint32_t d, factor, shift;
    explicit Divisor(uint32_t by) : d(by), shift(0) {
        while (((uint64_t)1 << shift) < by) ++shift;
        factor = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - by)) / by + 1);
    }
    __device__ uint32_t of(uint32_t n) const { return (__umulhi(n, factor) + n) >> shift; }
};

// `lanes` threads to a group, kGroupVecs vectors to a thread; a row's vectors are counted up to whole groups.
template <typename T>
__global__ void __launch_bounds__(kGroupThreads) groups_kernel(const ar_silu_mul_fp8_args a, int lanes, int groups, const Divisor row_vecs) {
    after_the_stream();
    const int vecs = a.dim / 8, padded = groups * lanes;
    const uint32_t all = (uint32_t)a.rows * padded;
    Vec g[kGroupVecs], u[kGroupVecs];
    int row[kGroupVecs], at[kGroupVecs];
#pragma unroll
    for (int i = 0; i < kGroupVecs; ++i) {
        const uint32_t n = (blockIdx.x * kGroupVecs + i) * kGroupThreads + threadIdx.x;
        row[i] = n < all ? (int)row_vecs.of(n) : -1;
        at[i] = (int)n - row[i] * padded;
        g[i].v = u[i].v = make_uint4(0, 0, 0, 0);
        if (row[i] >= 0 && at[i] < vecs) {
            const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + (int64_t)row[i] * a.x_stride) + at[i];
            g[i].v = __ldcs(x);
            u[i].v = __ldcs(x + vecs);
        }
    }
#pragma unroll
    for (int i = 0; i < kGroupVecs; ++i) {
        float y[8];
        float top = values<T>(g[i], u[i], y, 0.0f);
#pragma unroll
        for (int d = 16; d; d /= 2)
            if (d < lanes) top = top_of(top, __shfl_xor_sync(~0u, top, d));
        if (row[i] < 0 || at[i] >= vecs) continue;
        const float2 s = scale_of(top);
        reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + (int64_t)row[i] * a.dim)[at[i]] = rounded(y, s);
        if (at[i] % lanes == 0) a.scales[(int64_t)row[i] * groups + at[i] / lanes] = s.x;
    }
}

// A block to a row that is one group, V vectors to a thread.
template <typename T, int V>
__global__ void __launch_bounds__(1024) row_kernel(const ar_silu_mul_fp8_args a) {
    after_the_stream();
    __shared__ float tops[32];
    const int vecs = a.dim / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride);
    Vec g[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        g[i].v = u[i].v = make_uint4(0, 0, 0, 0);
        if (at < vecs) {
            g[i].v = __ldcs(x + at);
            u[i].v = __ldcs(x + vecs + at);
        }
    }
    float y[V][8], top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = values<T>(g[i], u[i], y[i], top);
#pragma unroll
    for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = lane < blockDim.x / 32 ? tops[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
    const float2 s = scale_of(top);
    uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.dim);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        if (at < vecs) out[at] = rounded(y[i], s);
    }
    if (threadIdx.x == 0) a.scales[row] = s.x;
}

// Blocks go from group to group, any size and alignment: once over it for the maximum, once for the output.
template <typename T>
__global__ void __launch_bounds__(128) any_group_kernel(const ar_silu_mul_fp8_args a) {
    after_the_stream();
    __shared__ float tops[4];
    const int group = a.group ? a.group : a.dim, groups = a.group ? (a.dim + group - 1) / group : 1;
    for (int64_t at = blockIdx.x; at < a.rows * groups; at += gridDim.x) {
        const int64_t row = at / groups;
        const int begin = (int)(at - row * groups) * group, end = min(a.dim, begin + group);
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
        float top = 0;
        for (int i = begin + threadIdx.x; i < end; i += 128) top = top_of(top, one_silu_mul(x[i], x[a.dim + i]));
#pragma unroll
        for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int i = 0; i < 4; ++i) top = top_of(top, tops[i]);
        const float2 s = scale_of(top);
        if (threadIdx.x == 0) a.scales[at] = s.x;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.dim;
        for (int i = begin + threadIdx.x; i < end; i += 128) {
            const float y = one_silu_mul(x[i], x[a.dim + i]);
            out[i] = __nv_cvt_float_to_fp8(s.y != 0 ? y * s.y : __fdiv_rn(y, s.x), __NV_SATFINITE, __NV_E4M3);
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t start(const ar_silu_mul_fp8_args &a, cudaStream_t s) {
    const int group = a.group ? a.group : a.dim, groups = a.group ? (a.dim + a.group - 1) / a.group : 1, vecs = a.dim / 8;
    // Vectors need rows on 16 bytes, and an output on 8.
    if (a.dim > 0 && a.dim % 8 == 0 && !misaligned(a.x, 16) && a.x_stride % 8 == 0 && !misaligned(a.out, 8)) {
        if (group <= 256 && group >= 8 && !(group & (group - 1))) {
            const int64_t all = a.rows * groups * (group / 8), each = kGroupThreads * kGroupVecs;
            if (all < 0x7fff0000)          // (2^34 channels)
                return launch_next(groups_kernel<T>, dim3((unsigned)((all + each - 1) / each)), kGroupThreads, 0, s, 0, a, group / 8, groups,
                                   Divisor((uint32_t)(groups * (group / 8))));
        } else if (groups == 1 && vecs <= 4096) {
            const int v = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4, threads = ((vecs + v - 1) / v + 31) / 32 * 32;
            return launch_next(v == 1 ? row_kernel<T, 1> : v == 2 ? row_kernel<T, 2> : row_kernel<T, 4>, dim3((unsigned)a.rows), threads, 0, s, 0, a);
        }
    }
    return launch_next(any_group_kernel<T>, dim3((unsigned)std::min(a.rows * groups, (int64_t)1 << 20)), 128, 0, s, 0, a);
}

}  // namespace

extern "C" AR_API int ar_silu_mul_fp8(const ar_silu_mul_fp8_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_silu_mul_fp8_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.rows < 0 || a.dim < 0 || a.group < 0 || a.group > a.dim) return AR_EINVAL;
    if (a.rows > 1 << 30 || a.dim > 1 << 20) return AR_ETOOBIG;
    if (a.rows == 0) return AR_OK;
    if (!a.scales || (a.dim > 0 && (!a.x || !a.out)) || misaligned(a.x, 2) || misaligned(a.scales, 4)) return AR_EINVAL;
    return launch_status(a.dtype == AR_F16 ? start<__half>(a, stream) : start<__nv_bfloat16>(a, stream));
}
