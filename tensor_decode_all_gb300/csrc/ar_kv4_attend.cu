// ar_kv4_attend.cu -- ar_kv4_attend: attention over the 4-bit paged cache.
//
// A warp takes one query row: its lanes share a token's channels, and the
// tokens go by one at a time under a running maximum and sum.
#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr size_t kWorkspaceBytes = 1 << 20;

struct Attend {
    ar_kv4_attend_args a;
    int vec;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) attend_kernel(const Attend c) {
    constexpr int G = D / kGroup, C = D / 32;    // lane l holds channels of group j: 32 j + l, for j < G
    const ar_kv4_attend_args &a = c.a;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (item >= (int64_t)a.tokens * a.q_heads) return;
    const int row = (int)(item / a.q_heads), head = (int)(item % a.q_heads), kv = head / (a.q_heads / a.kv_heads);
    int *status = static_cast<int *>(a.workspace);
    // the row's request
    int b = row, first = row, end = row + 1;
    if (a.cu) {
        for (b = 0; b < a.requests; ++b)
            if (a.cu[b] <= row && row < a.cu[b + 1]) break;
        if (b == a.requests) return;
        first = a.cu[b];
        end = a.cu[b + 1];
        if (end > a.tokens && lane == 0) *status = AR_EINVAL;
    }
    int n = a.lens[b];
    if (n < 0 || n > (int64_t)a.table_width * a.page) {
        if (lane == 0) *status = AR_EINVAL;
        n = n < 0 ? 0 : a.table_width * a.page;
    }
    const int p = n - (end - first) + (row - first);
    const T *q = static_cast<const T *>(a.q) + row * a.q_token_stride + head * a.q_head_stride;
    float qv[C], o[C] = {}, m = -INFINITY, l = 0;
#pragma unroll
    for (int j = 0; j < C; ++j) qv[j] = Elem<T>::to_float(q[32 * j + lane]) * a.scale;
    for (int tok = 0; tok <= p; ++tok) {
        if (a.window && tok <= p - a.window && tok >= a.sinks) continue;
        const int id = a.table[(int64_t)b * a.table_stride + tok / a.page];
        if (id < 0 || id >= a.pages) {
            if (lane == 0) *status = AR_EINVAL;
            continue;
        }
        const uint8_t *tile = static_cast<const uint8_t *>(a.pool) +
                              (((int64_t)id * a.kv_heads + kv) * (a.page / kTileTokens) + tok % a.page / kTileTokens) * tile_bytes(D);
        const int r = tok % kTileTokens;
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(tile);
        const uint16_t *vh = reinterpret_cast<const uint16_t *>(tile + tile_v(D));
        const uint16_t *ks = reinterpret_cast<const uint16_t *>(tile + tile_ks(D)), *vs = reinterpret_cast<const uint16_t *>(tile + tile_vs(D));
        float s = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int u = kw[k_word(G, r, lane / 8, j)] >> (4 * (lane % 8)) & 15;
            s = fmaf(qv[j], (float)(u - 8) * bf16_bits(ks[r * G + j]), s);
        }
#pragma unroll
        for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
        const float m2 = fmaxf(m, s), keep = expf(m - m2), e = expf(s - m2);
        l = fmaf(l, keep, e);
        m = m2;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int u = vh[2 * v_word(G, r, lane / 4, j) + (r & 1)] >> (4 * (lane % 4)) & 15;
            o[j] = fmaf(o[j], keep, e * ((float)(u - 8) * bf16_bits(vs[r * G + j])));
        }
    }
    T *out = static_cast<T *>(a.out) + row * a.out_token_stride + head * a.out_head_stride;
#pragma unroll
    for (int j = 0; j < C; ++j) out[32 * j + lane] = Elem<T>::from_float(l > 0 ? __fdiv_rn(o[j], l) : l == l ? 0.0f : l);
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.q_heads + head] = l > 0 ? m + logf(l) : l == l ? -INFINITY : l;
}

template <typename T>
cudaError_t start(const Attend &c, cudaStream_t s) {
    const int64_t blocks = ((int64_t)c.a.tokens * c.a.q_heads + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (c.a.head_dim == 64) attend_kernel<T, 64><<<(unsigned)blocks, 128, 0, s>>>(c);
    else if (c.a.head_dim == 128) attend_kernel<T, 128><<<(unsigned)blocks, 128, 0, s>>>(c);
    else attend_kernel<T, 256><<<(unsigned)blocks, 128, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace

extern "C" {

AR_API size_t ar_kv4_workspace_bytes(void) { return kWorkspaceBytes; }

AR_API int ar_kv4_workspace_init(void *workspace, ar_stream_t stream) {
    if (!workspace || misaligned(workspace, 256)) return AR_EINVAL;
    return launch_status(cudaMemsetAsync(workspace, 0, 4096, stream));
}

AR_API int ar_kv4_status(const void *workspace) {
    int status = 0;
    if (!workspace) return AR_EINVAL;
    if (cudaMemcpy(&status, workspace, sizeof status, cudaMemcpyDeviceToHost) != cudaSuccess) return launch_status(cudaErrorUnknown);
    return status;
}

AR_API int ar_kv4_attend(const ar_kv4_attend_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    Attend c;
    c.a = *args;
    const ar_kv4_attend_args &a = c.a;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return AR_EINVAL;
    if (a.tokens < 0 || a.requests < 0 || a.q_heads < 1 || a.kv_heads < 1 || a.q_heads % a.kv_heads || a.max_new < 0 ||
        a.page < kTileTokens || a.page % kTileTokens || a.table_width < 0 || a.table_stride < a.table_width || a.window < 0 ||
        a.sinks < 0 || a.pages < 0 || !(a.scale - a.scale == 0) || (!a.cu && a.tokens != a.requests))
        return AR_EINVAL;
    if (a.requests > 8192) return AR_ETOOBIG;
    if (a.tokens == 0) return AR_OK;
    if (!a.q || !a.out || !a.workspace || a.requests < 1 || !a.lens || (!a.table && a.table_width > 0) || (!a.pool && a.pages > 0))
        return AR_EINVAL;
    if (misaligned(a.q, 2) || misaligned(a.out, 2) || misaligned(a.lse, 4) || misaligned(a.pool, 16) || misaligned(a.table, 4) ||
        misaligned(a.lens, 4) || misaligned(a.cu, 4) || misaligned(a.workspace, 256))
        return AR_EINVAL;
    c.vec = rows_aligned(a.q, a.q_token_stride, a.q_head_stride) && rows_aligned(a.out, a.out_token_stride, a.out_head_stride);
    return launch_status(a.dtype == AR_F16 ? start<__half>(c, stream) : start<__nv_bfloat16>(c, stream));
}

}  // extern "C"
