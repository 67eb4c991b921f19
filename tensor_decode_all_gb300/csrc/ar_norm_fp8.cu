// ar_norm_fp8.cu -- ar_add_norm_fp8: residual, RMS norm and e4m3 output with scales.
//
// One block takes a row: h = x + residual goes to shared memory while its
// squares are summed, then y = h * rsqrt(mean + eps) * weight is taken group by
// group, a warp each, for the group's maximum and its quotients.
#include <cuda_fp8.h>

#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr int kNormThreads = 256;
constexpr int kNormDim = 32768;

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
    return __uint_as_float(max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const ar_add_norm_fp8_args a) {
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
    const int group = a.group ? a.group : a.dim, groups = (a.dim + group - 1) / group;
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
        const float scale = top == 0 ? 1.0f : __fdiv_rn(top, 448.0f), q = __fdiv_rn(1.0f, scale);
        if (threadIdx.x == 0) a.scales[row] = scale;
        for (int i = threadIdx.x; i < a.dim; i += kNormThreads) out[i] = __nv_cvt_float_to_fp8(h[i] * q, __NV_SATFINITE, __NV_E4M3);
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
            const float scale = top == 0 ? 1.0f : __fdiv_rn(top, 448.0f), q = __fdiv_rn(1.0f, scale);
            if (lane == 0) a.scales[row * groups + g] = scale;
            for (int i = g * group + lane; i < end; i += 32) out[i] = __nv_cvt_float_to_fp8(h[i] * q, __NV_SATFINITE, __NV_E4M3);
        }
    }
}

template <typename T>
cudaError_t start(const ar_add_norm_fp8_args &a, cudaStream_t s) {
    const size_t smem = (size_t)a.dim * 4;
    const cudaError_t e = cudaFuncSetAttribute(norm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormDim * 4);
    if (e != cudaSuccess) return e;
    norm_kernel<T><<<(unsigned)a.rows, kNormThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

extern "C" AR_API int ar_add_norm_fp8(const ar_add_norm_fp8_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_add_norm_fp8_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.rows < 0 || a.dim < 0 || a.group < 0 || a.group > a.dim || !(a.eps >= 0)) return AR_EINVAL;
    if (a.dim > kNormDim || a.rows > 0x7fffffff) return AR_ETOOBIG;
    if (a.rows == 0 || a.dim == 0) return AR_OK;
    if (!a.x || !a.weight || !a.out || !a.scales) return AR_EINVAL;
    if (misaligned(a.x, 2) || misaligned(a.residual, 2) || misaligned(a.weight, 2) || misaligned(a.residual_out, 2) ||
        misaligned(a.scales, 4))
        return AR_EINVAL;
    return launch_status(a.dtype == AR_F16 ? start<__half>(a, stream) : start<__nv_bfloat16>(a, stream));
}
