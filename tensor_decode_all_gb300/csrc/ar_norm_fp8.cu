// ar_norm_fp8.cu -- ar_add_norm_fp8: residual, RMS norm and e4m3 output with scales.
//
// One pass: a block takes a row and keeps h = x + residual in registers.  Since
// y = h * w * inv with inv = 1 / sqrt(mean + eps) common to the row, the largest |y|
// of a group is inv times its largest |h * w|: the sum of squares and the maxima
// come out of one round through shared memory, and no value is read or computed twice.
//
// Bound by memory: 7 bytes an element (x, residual, h and the e4m3 output).  In
// GB300 graph replays 8192 rows of 8192 take 70.0 us, 6.7 TB/s or 99% of what a plain
// copy reaches; 8192 of 5120 with groups of 128 45.9 us, 6.4 TB/s; 8 rows of 8192 2.1 us.
// A block that went from row to row with the next row's loads ahead needed
// 85 registers and was slower (82.9 us, or spilled); many short blocks do the same overlap.
// Rows that do not lie on 16 bytes and groups that a warp's lanes do not divide take a
// kernel that goes through shared memory, a third as fast.
#include <cuda_fp8.h>

#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr int kNormThreads = 256;
constexpr int kNormDim = 32768;
constexpr int kFewRows = 304;             // two blocks to a multiprocessor

__device__ __forceinline__ float block_sum(float v, float *buf) {
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kNormThreads / 32; ++i) v += buf[i];
    __syncthreads();
    return v;
}

// The larger of two magnitudes; a NaN wins.
__device__ __forceinline__ float top_of(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// The same of a (0 or more already) and two others.
__device__ __forceinline__ float top_of(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// A group's scale from its largest |y|.  (Up to 224 * 2^-149 it rounds to 0 as well: what it leaves is 0 by the scale 1.)
__device__ __forceinline__ float divided_scale(float top) {
    const float scale = __fdiv_rn(top, 448.0f);
    return scale == 0 ? 1.0f : scale;
}

// y / scale, by the scale's reciprocal where that is finite.
__device__ __forceinline__ float quotient(float y, float scale, float reciprocal) {
    return scale < 0x1p-100f ? __fdiv_rn(y, scale) : y * reciprocal;
}

// Vectors of 8 channels, V to a thread: vector i * blockDim.x + threadIdx.x.  Lanes: threads that share a
// group (a power of two up to 32; 0: the row is one group).
template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024) norm_rows_kernel(const ar_add_norm_fp8_args a, int lanes) {
    __shared__ float2 buf[32];
    const int vecs = a.dim / 8, warps = blockDim.x / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    union Vec { uint4 v; uint32_t u[4]; };
    Vec xv[V], rv[V], wv[V];
    auto load = [&](int64_t row) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride);
        const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.residual) + row * a.residual_stride);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = i * blockDim.x + threadIdx.x;
            xv[i].v = rv[i].v = make_uint4(0, 0, 0, 0);
            if (at < vecs) {
                xv[i].v = __ldcs(x + at);
                if (a.residual) rv[i].v = __ldcs(r + at);
            }
        }
    };
    after_the_stream();
    const int64_t row = blockIdx.x;
    load(row);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        // (an ordinary load: this kernel may have begun before the one that writes the weight has ended)
        wv[i].v = at < vecs ? static_cast<const uint4 *>(a.weight)[at] : make_uint4(0, 0, 0, 0);
    }
    const int groups = lanes ? (vecs + lanes - 1) / lanes : 1;
    float h[V][8], top[V], sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        top[i] = 0;
        Vec out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x2 = pair_of<T>(xv[i].u[e]), w2 = pair_of<T>(wv[i].u[e]);
            float2 v = x2;
            if (a.residual) {
                const float2 r2 = pair_of<T>(rv[i].u[e]);
                v.x += r2.x;
                v.y += r2.y;
            }
            out.u[e] = to_pair<T>(v);
            sum = fmaf(v.x, v.x, sum);
            sum = fmaf(v.y, v.y, sum);
            h[i][2 * e] = v.x * w2.x;
            h[i][2 * e + 1] = v.y * w2.y;
            top[i] = top_of(top[i], h[i][2 * e], h[i][2 * e + 1]);
        }
        const int at = i * blockDim.x + threadIdx.x;
        if (a.residual_out && at < vecs)
            reinterpret_cast<uint4 *>(static_cast<T *>(a.residual_out) + row * a.residual_out_stride)[at] = out.v;
    }
    float most = 0;
    if (lanes == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) most = top_of(most, top[i]);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        sum += __shfl_xor_sync(~0u, sum, d);
        if (lanes == 0) {
            most = top_of(most, __shfl_xor_sync(~0u, most, d));
        } else if (d < lanes) {
#pragma unroll
            for (int i = 0; i < V; ++i) top[i] = top_of(top[i], __shfl_xor_sync(~0u, top[i], d));
        }
    }
    if (lane == 0) buf[warp] = make_float2(sum, most);
    __syncthreads();
    // every warp adds the warps' sums for itself, in the same order
    const float2 part = lane < warps ? buf[lane] : make_float2(0, 0);
    sum = part.x;
    most = part.y;
#pragma unroll
    for (int d = 16; d; d /= 2) {
        sum += __shfl_xor_sync(~0u, sum, d);
        most = top_of(most, __shfl_xor_sync(~0u, most, d));
    }
    const float inv = rsqrtf(__fdiv_rn(sum, (float)a.dim) + a.eps);
    uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.dim);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        const float m = lanes ? top[i] : most;
        float scale = m * inv * (1.0f / 448.0f), q = __fdividef(448.0f, m);       // h * q: within 2 units of the last place of y / scale
        if (!(m > 0x1p-60f && m < 0x1p100f && inv > 0)) {
            // zeros, the ends of the range (inv / scale may be past it), infinities; rows whose sum of squares is infinite: y = 0
            scale = divided_scale(m * inv);
            q = 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = __fdiv_rn(h[i][e] * inv, scale);
        }
        if (!(inv == inv)) scale = q = inv;
        if (at < vecs) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                b[e] = __nv_cvt_float2_to_fp8x2(make_float2(h[i][2 * e] * q, h[i][2 * e + 1] * q), __NV_SATFINITE, __NV_E4M3);
            __stcs(out + at, make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16));
            if (lanes ? at % lanes == 0 : at == 0) a.scales[row * groups + (lanes ? at / lanes : 0)] = scale;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const ar_add_norm_fp8_args a) {
    after_the_stream();
    extern __shared__ float h[];
    __shared__ float buf[kNormThreads / 32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *r = a.residual ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
    T *ro = a.residual_out ? static_cast<T *>(a.residual_out) + row * a.residual_out_stride : nullptr;
    const T *w = static_cast<const T *>(a.weight);
    uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.dim;
    float sum = 0;
    for (int i = threadIdx.x; i < a.dim; i += kNormThreads) {
        float v = Elem<T>::to_float(x[i]);
        if (r) v += Elem<T>::to_float(r[i]);
        if (ro) ro[i] = Elem<T>::from_float(v);
        h[i] = v;
        sum = fmaf(v, v, sum);
    }
    sum = block_sum(sum, buf);
    const float inv = rsqrtf(__fdiv_rn(sum, (float)a.dim) + a.eps);
    const int group = a.group ? a.group : a.dim, groups = group ? (a.dim + group - 1) / group : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (groups == 1) {
        float top = 0;
        for (int i = threadIdx.x; i < a.dim; i += kNormThreads) {
            h[i] = h[i] * inv * Elem<T>::to_float(w[i]);
            top = top_of(top, h[i]);
        }
#pragma unroll
        for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
        if (lane == 0) buf[warp] = top;
        __syncthreads();
        for (int i = 0; i < kNormThreads / 32; ++i) top = top_of(top, buf[i]);
        const float scale = divided_scale(top), q = __fdiv_rn(1.0f, scale);
        if (threadIdx.x == 0) a.scales[row] = scale;
        for (int i = threadIdx.x; i < a.dim; i += kNormThreads) out[i] = __nv_cvt_float_to_fp8(quotient(h[i], scale, q), __NV_SATFINITE, __NV_E4M3);
    } else {
        for (int g = warp; g < groups; g += kNormThreads / 32) {
            const int end = min(a.dim, (g + 1) * group);
            float top = 0;
            for (int i = g * group + lane; i < end; i += 32) {
                h[i] = h[i] * inv * Elem<T>::to_float(w[i]);
                top = top_of(top, h[i]);
            }
#pragma unroll
            for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
            const float scale = divided_scale(top), q = __fdiv_rn(1.0f, scale);
            if (lane == 0) a.scales[row * groups + g] = scale;
            for (int i = g * group + lane; i < end; i += 32) out[i] = __nv_cvt_float_to_fp8(quotient(h[i], scale, q), __NV_SATFINITE, __NV_E4M3);
        }
    }
}

bool aligned16(const void *p, int64_t stride) { return !misaligned(p, 16) && stride % 8 == 0; }

template <typename T>
cudaError_t start(const ar_add_norm_fp8_args &a, cudaStream_t s) {
    // Threads that share a group of the vector kernel; -1: it cannot take the call.
    int lanes = -1;
    if (a.dim > 0 && a.dim % 8 == 0 && aligned16(a.x, a.x_stride) && aligned16(a.residual, a.residual_stride) && aligned16(a.weight, 0) &&
        aligned16(a.residual_out, a.residual_out_stride) && !misaligned(a.out, 8)) {
        if (a.group == 0 || a.group == a.dim) lanes = 0;
        else if (a.group == 8 || a.group == 16 || a.group == 32 || a.group == 64 || a.group == 128 || a.group == 256) lanes = a.group / 8;
    }
    if (lanes >= 0) {
        const int vecs = a.dim / 8;
        // Vectors to a thread: more of them keep as many loads in flight with fewer warps to meet (8192 x
        // 8192, one scale a row: four 70.6 us, two 77.5; 16384 x 4096, groups of 128: four 72.6, two 76.6, one
        // 90.5), fewer make a short row's way shorter where there are no others to wait for (64 x 4096: two
        // 2.8 us, four 3.2).
        const int v = vecs <= 128 ? 1 : vecs < 512 || (vecs <= 1024 && a.rows <= kFewRows) ? 2 : 4;
        const int threads = ((vecs + v - 1) / v + 31) / 32 * 32;
        return launch_next(v == 1 ? norm_rows_kernel<T, 1> : v == 2 ? norm_rows_kernel<T, 2> : norm_rows_kernel<T, 4>, dim3((unsigned)a.rows),
                           threads, 0, s, 0, a, lanes);
    }
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !*(volatile bool *)&ready[dev])) {
        e = cudaFuncSetAttribute(norm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormDim * 4);
        if (e == cudaSuccess && dev < 64) *(volatile bool *)&ready[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_next(norm_kernel<T>, dim3((unsigned)a.rows), kNormThreads, (size_t)a.dim * 4, s, 0, a);
}

}  // namespace

extern "C" AR_API int ar_add_norm_fp8(const ar_add_norm_fp8_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_add_norm_fp8_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.rows < 0 || a.dim < 0 || a.group < 0 || a.group > a.dim || !(a.eps >= 0)) return AR_EINVAL;
    if (a.dim > kNormDim || a.rows > 0x7fffffff) return AR_ETOOBIG;
    if (a.rows == 0) return AR_OK;
    if (!a.scales || (a.dim > 0 && (!a.x || !a.weight || !a.out))) return AR_EINVAL;
    if (misaligned(a.x, 2) || misaligned(a.residual, 2) || misaligned(a.weight, 2) || misaligned(a.residual_out, 2) ||
        misaligned(a.scales, 4))
        return AR_EINVAL;
    return launch_status(a.dtype == AR_F16 ? start<__half>(a, stream) : start<__nv_bfloat16>(a, stream));
}
