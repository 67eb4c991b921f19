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
    const int64_t page = (uint64_t)slot >> 32 ? slot / a.page : (int64_t)((uint32_t)slot / (uint32_t)a.page), in = slot - page * a.page;
    return a.pool + ((page * a.heads + head) * (a.page / kTileTokens) + in / kTileTokens) * tile_bytes(D);
}

// G words from or to consecutive addresses, in the widest accesses.
template <int G>
__device__ __forceinline__ void put_words(uint32_t *p, const uint32_t (&w)[G]) {
    if constexpr (G == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

template <int G>
__device__ __forceinline__ void get_words(const uint32_t *p, uint32_t (&w)[G]) {
    if constexpr (G == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    }
}

// N consecutive elements (4 or 8), one access where the rows lie on 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void get_row(const T *p, bool vec, float (&x)[N]) {
    union { uint4 v; uint2 u; T e[8]; } w;
    if (!vec) {
#pragma unroll
        for (int i = 0; i < N; ++i) w.e[i] = p[i];
    } else if constexpr (N == 8) {
        w.v = __ldcs(reinterpret_cast<const uint4 *>(p));
    } else {
        w.u = __ldcs(reinterpret_cast<const uint2 *>(p));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Elem<T>::to_float(w.e[i]);
}

template <typename T, int N>
__device__ __forceinline__ void put_row(T *p, bool vec, const float (&x)[N]) {
    union { uint4 v; uint2 u; T e[8]; } w;
#pragma unroll
    for (int i = 0; i < N; ++i) w.e[i] = Elem<T>::from_float(x[i]);
    if (!vec) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = w.e[i];
    } else if constexpr (N == 8) {
        *reinterpret_cast<uint4 *>(p) = w.v;
    } else {
        *reinterpret_cast<uint2 *>(p) = w.u;
    }
}

// A group's scale and N of its channels as nibbles; Lanes threads (First to First * Lanes / 2 apart) hold the group.
template <int N, int Lanes, int First>
__device__ __forceinline__ uint32_t quantise(const float (&x)[N], __nv_bfloat16 &scale) {
    // The largest magnitude as bits, so that a NaN (above every number) wins.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int d = First; d < First * Lanes; d *= 2) top = max(top, __shfl_xor_sync(~0u, top, d));
    scale = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.0f));
    const float s = __bfloat162float(scale);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float f = rintf(__fdiv_rn(x[i], s));
        // fmax and fmin turn NaN into a bound, so NaN (and 0 / 0) is asked for first
        const uint32_t n = (uint32_t)(f == f ? (int)fminf(fmaxf(f, -7.0f), 7.0f) + 8 : 8);
        w |= n << (4 * i);
    }
    return w;
}

constexpr int kRowThreads = 128;

// What a warp works on: 8 tokens of one head, K or V.  The lanes take the tokens
// as the tile's words lie, so that 8 consecutive tokens of a tile are
// read and written in whole lines: for K lane (r, t) has token r, channels 32 j + 8 t .. + 7
// of every group j; for V lane (g, t) has tokens 2 t and 2 t + 1, channels 32 j + 4 g .. + 3.
struct Job {
    int64_t token0;
    int head, lane;
    bool v, any;
};

__device__ __forceinline__ Job job_of(const Rows &a) {
    Job w;
    const int64_t n = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
    w.lane = threadIdx.x & 31;
    w.v = n & 1;
    const int64_t rest = n >> 1, octet = rest / a.heads;
    w.head = (int)(rest - octet * a.heads);
    w.token0 = octet * 8;
    w.any = w.token0 < a.tokens;
    return w;
}

__device__ __forceinline__ int64_t slot_at(const Rows &a, int64_t token) {
    const int64_t slot = token >= 0 && token < a.tokens ? a.slots[token] : -1;
    return slot < a.slots_in_pool ? slot : -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(Rows a) {
    constexpr int G = D / kGroup;
    const Job w = job_of(a);
    if (!w.any) return;
    if (!w.v) {
        const int r8 = w.lane / 4, t = w.lane % 4;
        const int64_t token = w.token0 + r8, slot = slot_at(a, token);
        const bool in = slot >= 0;
        const T *src = static_cast<const T *>(a.k) + (in ? token : 0) * a.k_token + w.head * a.k_head + 8 * t;
        uint32_t words[G];
        __nv_bfloat16 scales[G];
        float x[G][8];
#pragma unroll
        for (int j = 0; j < G; ++j) get_row(src + 32 * j, a.vec != 0, x[j]);
#pragma unroll
        for (int j = 0; j < G; ++j) words[j] = quantise<8, 4, 1>(x[j], scales[j]);
        if (!in) return;
        uint8_t *tile = tile_of<D>(a, slot, w.head);
        const int r = (int)(slot % kTileTokens);
        put_words(reinterpret_cast<uint32_t *>(tile) + k_word(G, r, t, 0), words);
        // lane t has the t-th share of the scales
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (j % 4 == t) reinterpret_cast<__nv_bfloat16 *>(tile + tile_ks(D))[r * G + j] = scales[j];
        return;
    }
    const int g = w.lane / 4, t = w.lane % 4;
    // Two tokens whose slots are 2 p and 2 p + 1 share words: the one at the even slot writes both, wherever in the 8 it
    // stands.  Of a run, that is one of every lane's two; other tokens write their halves of the words.
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        const int64_t token = w.token0 + 2 * t + c, slot = slot_at(a, token);
        const bool even = slot >= 0 && slot % 2 == 0;
        const bool pair = even && slot_at(a, token + 1) == slot + 1;
        const bool follows = slot >= 0 && !even && slot_at(a, token - 1) == slot - 1;
        const bool in = slot >= 0 && !follows;
        if (!__any_sync(~0u, in)) continue;
        uint32_t words[2][G];
        __nv_bfloat16 scales[2][G];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const T *src = static_cast<const T *>(a.v) + (in ? token + (pair ? p : 0) : 0) * a.v_token + w.head * a.v_head + 4 * g;
            float x[G][4];
#pragma unroll
            for (int j = 0; j < G; ++j) get_row(src + 32 * j, a.vec != 0, x[j]);
#pragma unroll
            for (int j = 0; j < G; ++j) words[p][j] = quantise<4, 8, 4>(x[j], scales[p][j]);
        }
        if (!in) continue;
        uint8_t *tile = tile_of<D>(a, slot, w.head);
        const int r = (int)(slot % kTileTokens);
        uint32_t *dst = reinterpret_cast<uint32_t *>(tile + tile_v(D)) + v_word(G, r, g, 0);
        __nv_bfloat16 *vs = reinterpret_cast<__nv_bfloat16 *>(tile + tile_vs(D)) + r * G;
        if (pair) {
            uint32_t both[G];
#pragma unroll
            for (int j = 0; j < G; ++j) both[j] = words[0][j] | words[1][j] << 16;
            put_words(dst, both);
        } else {
#pragma unroll
            for (int j = 0; j < G; ++j) reinterpret_cast<uint16_t *>(dst + j)[r & 1] = (uint16_t)words[0][j];
        }
        // lane g has the g-th scale of both tokens
#pragma unroll
        for (int j = 0; j < G; ++j)
            if (j == g) {
                vs[j] = scales[0][j];
                if (pair) vs[G + j] = scales[1][j];
            }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) load_kernel(Rows a) {
    constexpr int G = D / kGroup;
    const Job w = job_of(a);
    if (!w.any) return;
    if (!w.v) {
        const int t = w.lane % 4;
        const int64_t token = w.token0 + w.lane / 4, slot = slot_at(a, token);
        if (token >= a.tokens) return;
        T *dst = static_cast<T *>(a.k) + token * a.k_token + w.head * a.k_head + 8 * t;
        uint32_t words[G] = {};
        float s[G] = {};
        if (slot >= 0) {
            const uint8_t *tile = tile_of<D>(a, slot, w.head);
            const int r = (int)(slot % kTileTokens);
            get_words(reinterpret_cast<const uint32_t *>(tile) + k_word(G, r, t, 0), words);
#pragma unroll
            for (int j = 0; j < G; ++j) s[j] = bf16_bits(reinterpret_cast<const uint16_t *>(tile + tile_ks(D))[r * G + j]);
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = slot >= 0 ? (float)((int)(words[j] >> (4 * i) & 15) - 8) * s[j] : 0.0f;
            put_row(dst + 32 * j, a.vec != 0, x);
        }
        return;
    }
    const int g = w.lane / 4, t = w.lane % 4;
    // A lane's two tokens, if they share words, need them once: the second read of the same words is from the first level cache.
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int64_t token = w.token0 + 2 * t + c, slot = slot_at(a, token);
        if (token >= a.tokens) return;
        T *dst = static_cast<T *>(a.v) + token * a.v_token + w.head * a.v_head + 4 * g;
        uint32_t words[G] = {};
        float s[G] = {};
        if (slot >= 0) {
            const uint8_t *tile = tile_of<D>(a, slot, w.head);
            const int r = (int)(slot % kTileTokens);
            get_words(reinterpret_cast<const uint32_t *>(tile + tile_v(D)) + v_word(G, r, g, 0), words);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                words[j] >>= 16 * (r & 1);
                s[j] = bf16_bits(reinterpret_cast<const uint16_t *>(tile + tile_vs(D))[r * G + j]);
            }
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = slot >= 0 ? (float)((int)(words[j] >> (4 * i) & 15) - 8) * s[j] : 0.0f;
            put_row(dst + 32 * j, a.vec != 0, x);
        }
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
    const int64_t per = kRowThreads / 32, blocks = ((a.tokens + 7) / 8 * a.heads * 2 + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (append) append_kernel<T, D><<<(unsigned)blocks, kRowThreads, 0, s>>>(a);
    else load_kernel<T, D><<<(unsigned)blocks, kRowThreads, 0, s>>>(a);
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
