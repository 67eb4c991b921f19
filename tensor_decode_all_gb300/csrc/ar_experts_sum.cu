// ar_experts_sum.cu -- ar_experts_sum: the weighted sum of each token's rows.
#include <algorithm>

#include "ar_ffn.h"
#include "ar_kv4.cuh"

namespace {

using namespace tda;

// A thread to a channel, any alignment.
template <typename T>
__global__ void __launch_bounds__(256) any_sum_kernel(const ar_experts_sum_args a) {
    after_the_stream();
    const int64_t token = blockIdx.x;
    for (int c = blockIdx.y * 256 + threadIdx.x; c < a.dim; c += 256 * gridDim.y) {
        float sum = 0;
        for (int j = 0; j < a.chosen; ++j) {
            const int p = a.place[token * a.chosen + j];
            if (p >= 0 && p < a.rows) sum = fmaf(a.weights[token * a.chosen + j], Elem<T>::to_float(static_cast<const T *>(a.x)[p * a.x_stride + c]), sum);
        }
        static_cast<T *>(a.out)[token * a.out_stride + c] = Elem<T>::from_float(sum);
    }
}

template <typename T>
cudaError_t start(const ar_experts_sum_args &a, cudaStream_t s) {
    return launch_next(any_sum_kernel<T>, dim3((unsigned)a.tokens, (unsigned)std::min(64, (a.dim + 255) / 256)), 256, 0, s, 0, a);
}

}  // namespace

extern "C" AR_API int ar_experts_sum(const ar_experts_sum_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_experts_sum_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.rows < 0 || a.tokens < 0 || a.dim < 0 || a.chosen < 0) return AR_EINVAL;
    if (a.rows > 1 << 30 || a.tokens > 1 << 30 || a.dim > 1 << 20 || a.chosen > 1024) return AR_ETOOBIG;
    if (a.tokens == 0 || a.dim == 0) return AR_OK;
    if (!a.out || (a.rows > 0 && !a.x) || (a.chosen > 0 && (!a.weights || !a.place))) return AR_EINVAL;
    if (misaligned(a.x, 2) || misaligned(a.out, 2) || misaligned(a.weights, 4) || misaligned(a.place, 4)) return AR_EINVAL;
    return launch_status(a.dtype == AR_F16 ? start<__half>(a, stream) : start<__nv_bfloat16>(a, stream));
}
