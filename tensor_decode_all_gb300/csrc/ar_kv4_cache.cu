// ar_kv4_cache.cu -- ar_kv4_append and ar_kv4_load: rows of K and V to 4 bits
// in the paged cache, and back.
//
// append, per group of 32 channels:  scale = bf16(max|x| / 7),  n = rint(x / scale).
// The division by 7 and by the scale are IEEE ones, so that a plain
// implementation in binary32 writes the same bytes.
#include "ar_kv4.cuh"

namespace {

using namespace tda;

struct Rows {
    void *k, *v;
    uint8_t *pool;
    const int64_t *slots;
    int64_t k_token, k_head, v_token, v_head, slots_in_pool, tokens;
    int heads, page, vec;
};

// Where a slot's tile of a head starts; the slot is inside the pool.
template <int D>
__device__ __forceinline__ uint8_t *tile_of(const Rows &a, int64_t slot, int head) {
    const int64_t page = slot / a.page, in = slot % a.page;
    return a.pool + ((page * a.heads + head) * (a.page / kTileTokens) + in / kTileTokens) * tile_bytes(D);
}

// A thread takes 8 channels of one token and head: one K word, two halves of V
// words; the 4 threads of a group share its maximum by shuffles.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_kernel(Rows a) {
    constexpr int G = D / kGroup, kPer = D / 8;
    const int64_t row = (int64_t)blockIdx.x * (256 / kPer) + threadIdx.x / kPer;
    const int c = threadIdx.x % kPer, j = c / 4, t = c % 4;
    const int64_t token = row / a.heads;
    const int head = (int)(row % a.heads);
    if (token >= a.tokens) return;          // whole rows leave together, and a group is within one
    const int64_t slot = a.slots[token];
    if (slot < 0 || slot >= a.slots_in_pool) return;
    const int r = (int)(slot % kTileTokens);
    uint8_t *tile = tile_of<D>(a, slot, head);
    const unsigned mask = 0xfu << ((threadIdx.x & 31) & ~3);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const T *src = static_cast<const T *>(side ? a.v : a.k) + token * (side ? a.v_token : a.k_token) +
                       head * (side ? a.v_head : a.k_head) + 8 * c;
        float x[8];
        load8(src, a.vec != 0, x);
        // The largest magnitude as bits, so that a NaN (above every number) wins.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(mask, top, 1));
        top = max(top, __shfl_xor_sync(mask, top, 2));
        const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.0f));
        const float s = __bfloat162float(scale);
        uint32_t n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = rintf(__fdiv_rn(x[i], s));
            // fmax and fmin turn NaN into a bound, so NaN (and 0 / 0) is asked for first
            n[i] = (uint32_t)(f == f ? (int)fminf(fmaxf(f, -7.0f), 7.0f) + 8 : 8);
        }
        if (side == 0) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= n[i] << (4 * i);
            reinterpret_cast<uint32_t *>(tile)[k_word(G, r, t, j)] = w;
        } else {
            uint16_t *base = reinterpret_cast<uint16_t *>(tile + tile_v(D));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                base[2 * v_word(G, r, 2 * t + h, j) + (r & 1)] =
                    (uint16_t)(n[4 * h] | n[4 * h + 1] << 4 | n[4 * h + 2] << 8 | n[4 * h + 3] << 12);
        }
        if (t == 0)
            reinterpret_cast<__nv_bfloat16 *>(tile + (side ? tile_vs(D) : tile_ks(D)))[r * G + j] = scale;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) load_kernel(Rows a) {
    constexpr int G = D / kGroup, kPer = D / 8;
    const int64_t row = (int64_t)blockIdx.x * (256 / kPer) + threadIdx.x / kPer;
    const int c = threadIdx.x % kPer, j = c / 4, t = c % 4;
    const int64_t token = row / a.heads;
    const int head = (int)(row % a.heads);
    if (token >= a.tokens) return;
    const int64_t slot = a.slots[token];
    const bool in = slot >= 0 && slot < a.slots_in_pool;
    const int r = (int)(slot & (kTileTokens - 1));
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        T *dst = static_cast<T *>(side ? a.v : a.k) + token * (side ? a.v_token : a.k_token) +
                 head * (side ? a.v_head : a.k_head) + 8 * c;
        float x[8] = {};
        if (in) {
            const uint8_t *tile = tile_of<D>(a, slot, head);
            uint32_t w;
            if (side == 0) {
                w = reinterpret_cast<const uint32_t *>(tile)[k_word(G, r, t, j)];
            } else {
                const uint16_t *base = reinterpret_cast<const uint16_t *>(tile + tile_v(D));
                w = base[2 * v_word(G, r, 2 * t, j) + (r & 1)] |
                    (uint32_t)base[2 * v_word(G, r, 2 * t + 1, j) + (r & 1)] << 16;
            }
            const float s = bf16_bits(reinterpret_cast<const uint16_t *>(tile + (side ? tile_vs(D) : tile_ks(D)))[r * G + j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)((int)(w >> (4 * i) & 15) - 8) * s;
        }
        store8(dst, a.vec != 0, x);
    }
}

int check(const ar_kv4_rows_args *p) {
    if (!p) return AR_EINVAL;
    if (p->dtype != AR_F16 && p->dtype != AR_BF16) return AR_EINVAL;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return AR_EINVAL;
    if (p->tokens < 0 || p->kv_heads < 1 || p->page < kTileTokens || p->page % kTileTokens || p->pages < 0)
        return AR_EINVAL;
    if (p->tokens == 0) return AR_OK;
    if (!p->k || !p->v || !p->slots || (!p->pool && p->pages > 0)) return AR_EINVAL;
    if (misaligned(p->k, 2) || misaligned(p->v, 2) || misaligned(p->slots, 8) || misaligned(p->pool, 16)) return AR_EINVAL;
    if (p->tokens > (int64_t)1 << 31 || p->pages > (int64_t)1 << 31 || p->kv_heads > 1 << 16) return AR_EINVAL;
    return AR_OK;
}

template <typename T, int D>
cudaError_t start(const Rows &a, bool append, cudaStream_t s) {
    const int64_t per = 256 / (D / 8), blocks = (a.tokens * a.heads + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (append) append_kernel<T, D><<<(unsigned)blocks, 256, 0, s>>>(a);
    else load_kernel<T, D><<<(unsigned)blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t start(const Rows &a, int D, bool append, cudaStream_t s) {
    return D == 64 ? start<T, 64>(a, append, s) : D == 128 ? start<T, 128>(a, append, s) : start<T, 256>(a, append, s);
}

int rows(const ar_kv4_rows_args *p, bool append, cudaStream_t s) {
    const int rc = check(p);
    if (rc || p->tokens == 0) return rc;
    Rows a;
    a.k = p->k; a.v = p->v; a.pool = static_cast<uint8_t *>(p->pool); a.slots = p->slots;
    a.k_token = p->k_token_stride; a.k_head = p->k_head_stride;
    a.v_token = p->v_token_stride; a.v_head = p->v_head_stride;
    a.slots_in_pool = p->pages * p->page; a.tokens = p->tokens;
    a.heads = p->kv_heads; a.page = p->page;
    a.vec = rows_aligned(p->k, a.k_token, a.k_head) && rows_aligned(p->v, a.v_token, a.v_head);
    return launch_status(p->dtype == AR_F16 ? start<__half>(a, p->head_dim, append, s)
                                            : start<__nv_bfloat16>(a, p->head_dim, append, s));
}

}  // namespace

extern "C" {

AR_API int ar_kv4_append(const ar_kv4_rows_args *args, ar_stream_t stream) { return rows(args, true, stream); }

AR_API int ar_kv4_load(const ar_kv4_rows_args *args, ar_stream_t stream) { return rows(args, false, stream); }

}  // extern "C"
