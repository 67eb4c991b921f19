// ar_silu_fp8.cu -- ar_silu_mul_fp8: the gated activation with e4m3 output and scales.
#include <cuda_fp8.h>

#include <algorithm>

#include "ar_ffn.h"
#include "ar_kv4.cuh"

namespace {

using namespace tda;

// The larger of two magnitudes (the first is 0 or more already); a NaN wins.
__device__ __forceinline__ float top_of(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

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
        for (int i = begin + threadIdx.x; i < end; i += 128) top = top_of(top, silu_mul(Elem<T>::to_float(x[i]), Elem<T>::to_float(x[a.dim + i])));
#pragma unroll
        for (int d = 16; d; d /= 2) top = top_of(top, __shfl_xor_sync(~0u, top, d));
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int i = 0; i < 4; ++i) top = top_of(top, tops[i]);
        const float scale = top == 0 ? 1.0f : __fdiv_rn(top, 448.0f);
        if (threadIdx.x == 0) a.scales[at] = scale;
        uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.dim;
        for (int i = begin + threadIdx.x; i < end; i += 128)
            out[i] = __nv_cvt_float_to_fp8(__fdiv_rn(silu_mul(Elem<T>::to_float(x[i]), Elem<T>::to_float(x[a.dim + i])), scale), __NV_SATFINITE, __NV_E4M3);
        __syncthreads();
    }
}

template <typename T>
cudaError_t start(const ar_silu_mul_fp8_args &a, cudaStream_t s) {
    const int64_t groups = a.rows * (a.group ? (a.dim + a.group - 1) / a.group : 1);
    return launch_next(any_group_kernel<T>, dim3((unsigned)std::min(groups, (int64_t)1 << 20)), 128, 0, s, 0, a);
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
