// ar_kv4_cache.cu -- ar_kv4_append and ar_kv4_load: rows of K and V to 4 bits in the paged cache, and back.
//
// append, per group of 32 channels:  scale = bf16(max|x| / 7),  n = rint(x / scale). Both quotients are
// rounded as IEEE division rounds them, so that a plain implementation in binary32 writes the same bytes.
//
// A warp takes 8 tokens of one head, K or V, its lanes as the tile's words lie, so that a run of tokens is
// read and written in whole lines.  Measured on a GB300 (graph replays): 8191 tokens of 8 heads of 128, append
// 14.5 us (43 MB), load 8.7; 64 tokens 3.0 and 2.5 us.  Bound by the rounding's instructions (0.64 a cycle and
// scheduler), not by its 6.3 us of memory: with a division to a value 32.6 us, with a scale made by every lane
// 16.9.
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

// N consecutive elements (4 or 8) as pairs, one access where the rows lie on 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void get_row(const T *p, bool vec, uint32_t (&x)[N / 2]) {
    if (!vec) {
        const unsigned short *e = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) x[i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
    } else if constexpr (N == 8) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        x[0] = v.x; x[1] = v.y;
    }
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

// The scales of M groups whose channels lie in 2^Bits lanes, First apart: the maxima are reduced while they
// are dealt out, so that a lane ends with M >> Bits of the groups (or shares one), makes their scales, and the
// others get them by shuffles.  Group m is made in lane m * 2^Bits / M of the 2^Bits.
template <typename T, int M, int Bits, int First>
struct Scales {
    static constexpr int kOwn = M >> Bits ? M >> Bits : 1;
    __nv_bfloat16 scale[kOwn];      // of groups own .. own + kOwn - 1
    float s[kOwn], r[kOwn];
    int own;
    bool first;                     // of the lanes that made the same group

    // top: largest magnitudes of this lane's share by their bits, two elements to a word (a NaN is above every
    // number)
    __device__ __forceinline__ Scales(uint32_t (&top)[M], int lane) {
        int n = M;
        own = 0;
        first = true;
#pragma unroll
        for (int b = Bits - 1; b >= 0; --b) {
            const bool up = lane & (First << b);
            if (n > 1) {
                n /= 2;
#pragma unroll
                for (int i = 0; i < M / 2; ++i)
                    if (i < n) {
                        const uint32_t give = up ? top[i] : top[i + n], keep = up ? top[i + n] : top[i];
                        top[i] = __vmaxu2(keep, __shfl_xor_sync(~0u, give, First << b));
                    }
                own += up ? n : 0;
            } else {
                top[0] = __vmaxu2(top[0], __shfl_xor_sync(~0u, top[0], First << b));
                first &= !up;
            }
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            scale[i] = __float2bfloat16_rn(__fdiv_rn(pair_of<T>(max(top[i] & 0xffffu, top[i] >> 16)).x, 7.0f));
            s[i] = __bfloat162float(scale[i]);
            r[i] = __frcp_rn(s[i]);
        }
    }
    // group m's scale and its reciprocal; base: the lane with the lowest number of the 2^Bits
    __device__ __forceinline__ float2 of(int m, int base) const {
        const int from = base + (m << Bits) / M * First;
        return make_float2(__shfl_sync(~0u, s[m % kOwn], from), __shfl_sync(~0u, r[m % kOwn], from));
    }
};

// N channels of a group as nibbles.
template <typename T, int N>
__device__ __forceinline__ uint32_t quantise(const uint32_t (&pairs)[N / 2], float2 sr) {
    const float s = sr.x, r = sr.y;
    float x[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 v = pair_of<T>(pairs[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
    uint32_t w = 0;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        // x / s rounded as IEEE division rounds it, from the rounded 1 / s and one exact remainder (P.
        // Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  |x /
        // s| < 7.02, so the sum with 1.5 * 2^23 rounds it half to even into the low bits.
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float q = x[i] * r, n = fmaf(fmaf(-q, s, x[i]), r, q) + (12582912.0f + 8.0f);
            w |= (__float_as_uint(n) & 15u) << (4 * i);
        }
    } else {
        // zeros, the type's ends, infinities and NaN: a pair at a time, the pairs moving up (an index that
        // varies would put them into local memory)
        uint32_t p[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = pairs[i];
#pragma unroll 1
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = pair_of<T>(p[0]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = rintf(__fdiv_rn(e ? v.y : v.x, s));
                // fmax and fmin turn NaN into a bound, so NaN is asked for first; a scale that rounded to 0 has n = 0
                const uint32_t n = (uint32_t)(f == f && s != 0 ? (int)fminf(fmaxf(f, -7.0f), 7.0f) + 8 : 8);
                w = w >> 4 | n << (4 * N - 4);
            }
#pragma unroll
            for (int k = 0; k + 1 < N / 2; ++k) p[k] = p[k + 1];
        }
    }
    return w;
}

template <int N>
__device__ __forceinline__ uint32_t top_of(const uint32_t (&pairs)[N]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = __vmaxu2(top, pairs[i] & 0x7fff7fffu);
    return top;
}

// Nibble i of w as u - 8: under the exponent of 2^23 it is a whole number, and one subtraction is exact.
__device__ __forceinline__ float nibble(uint32_t w, int i) { return __uint_as_float((w >> (4 * i) & 15u) | 0x4b000000u) - (8388608.0f + 8.0f); }

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
    after_the_stream();
    const Job w = job_of(a);
    if (!w.any) return;
    if (!w.v) {
        const int r8 = w.lane / 4, t = w.lane % 4;
        const int64_t token = w.token0 + r8, slot = slot_at(a, token);
        const bool in = slot >= 0;
        // (the row does not wait for its slot)
        const T *src = static_cast<const T *>(a.k) + (token < a.tokens ? token : 0) * a.k_token + w.head * a.k_head + 8 * t;
        uint32_t words[G], x[G][4], top[G];
#pragma unroll
        for (int j = 0; j < G; ++j) get_row<T, 8>(src + 32 * j, a.vec != 0, x[j]);
#pragma unroll
        for (int j = 0; j < G; ++j) top[j] = top_of(x[j]);
        const Scales<T, G, 2, 1> scales(top, w.lane);
#pragma unroll
        for (int j = 0; j < G; ++j) words[j] = quantise<T, 8>(x[j], scales.of(j, w.lane & ~3));
        if (!in) return;
        uint8_t *tile = tile_of<D>(a, slot, w.head);
        const int r = (int)(slot % kTileTokens);
        put_words(reinterpret_cast<uint32_t *>(tile) + k_word(G, r, t, 0), words);
        __nv_bfloat16 *ks = reinterpret_cast<__nv_bfloat16 *>(tile + tile_ks(D)) + r * G + scales.own;
#pragma unroll
        for (int i = 0; i < scales.kOwn; ++i)
            if (scales.first) ks[i] = scales.scale[i];
        return;
    }
    const int g = w.lane / 4, t = w.lane % 4;
    // Two tokens whose slots are 2 p and 2 p + 1 share words.  Where both are this warp's, next to each other,
    // the lane of the first writes whole words: tokens 2 t and 2 t + 1 of a lane in a run that begins at an
    // even slot, 2 t + 1 and the next lane's first in one that begins at an odd slot.  Other tokens write
    // their halves of the words.
    int64_t slot[3];
    uint32_t words[3][G], x[2][G][2], top[2 * G];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int64_t token = w.token0 + 2 * t + c;
        slot[c] = slot_at(a, token);
        const T *src = static_cast<const T *>(a.v) + (token < a.tokens ? token : 0) * a.v_token + w.head * a.v_head + 4 * g;
#pragma unroll
        for (int j = 0; j < G; ++j) get_row<T, 4>(src + 32 * j, a.vec != 0, x[c][j]);
    }
#pragma unroll
    for (int m = 0; m < 2 * G; ++m) top[m] = top_of(x[m / G][m % G]);
    const Scales<T, 2 * G, 3, 4> scales(top, w.lane);
#pragma unroll
    for (int m = 0; m < 2 * G; ++m) words[m / G][m % G] = quantise<T, 4>(x[m / G][m % G], scales.of(m, t));
    const int64_t after = __shfl_down_sync(~0u, slot[0], 1, 4), before = __shfl_up_sync(~0u, slot[1], 1, 4);
    slot[2] = t < 3 ? after : -1;
#pragma unroll
    for (int j = 0; j < G; ++j) words[2][j] = __shfl_down_sync(~0u, words[0][j], 1, 4);
    // the scales that this lane made: of token own / G
    const int64_t theirs = scales.own < G ? slot[0] : slot[1];
    if (theirs >= 0 && scales.first) {
        __nv_bfloat16 *vs = reinterpret_cast<__nv_bfloat16 *>(tile_of<D>(a, theirs, w.head) + tile_vs(D)) + theirs % kTileTokens * G + scales.own % G;
#pragma unroll
        for (int i = 0; i < scales.kOwn; ++i) vs[i] = scales.scale[i];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int64_t here = slot[c], prior = c ? slot[0] : t > 0 ? before : -1;
        const bool even = here % 2 == 0, pair = even && slot[c + 1] == here + 1;
        if (here < 0 || (!even && prior == here - 1)) continue;       // (the latter: the token before has written it)
        uint8_t *tile = tile_of<D>(a, here, w.head);
        const int r = (int)(here % kTileTokens);
        uint32_t *dst = reinterpret_cast<uint32_t *>(tile + tile_v(D)) + v_word(G, r, g, 0);
        if (pair) {
            uint32_t both[G];
#pragma unroll
            for (int j = 0; j < G; ++j) both[j] = words[c][j] | words[c + 1][j] << 16;
            put_words(dst, both);
        } else {
#pragma unroll
            for (int j = 0; j < G; ++j) reinterpret_cast<uint16_t *>(dst + j)[r & 1] = (uint16_t)words[c][j];
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) load_kernel(Rows a) {
    constexpr int G = D / kGroup;
    after_the_stream();
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
            for (int i = 0; i < 8; ++i) x[i] = slot >= 0 ? nibble(words[j], i) * s[j] : 0.0f;
            put_row(dst + 32 * j, a.vec != 0, x);
        }
        return;
    }
    // A lane's two tokens, if they share words, need them once: the second read of the same words is from the
    // first level cache.
    const int g = w.lane / 4, t = w.lane % 4;
    uint32_t words[2][G];
    float s[2][G];
    bool in[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int64_t slot = slot_at(a, w.token0 + 2 * t + c);
        in[c] = slot >= 0;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            words[c][j] = 0;
            s[c][j] = 0;
        }
        if (in[c]) {
            const uint8_t *tile = tile_of<D>(a, slot, w.head);
            const int r = (int)(slot % kTileTokens);
            get_words(reinterpret_cast<const uint32_t *>(tile + tile_v(D)) + v_word(G, r, g, 0), words[c]);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                words[c][j] >>= 16 * (r & 1);
                s[c][j] = bf16_bits(reinterpret_cast<const uint16_t *>(tile + tile_vs(D))[r * G + j]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int64_t token = w.token0 + 2 * t + c;
        if (token >= a.tokens) continue;
        T *dst = static_cast<T *>(a.v) + token * a.v_token + w.head * a.v_head + 4 * g;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = in[c] ? nibble(words[c][j], i) * s[c][j] : 0.0f;
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
    return launch_next(append ? append_kernel<T, D> : load_kernel<T, D>, dim3((unsigned)blocks), kRowThreads, 0, s, 0, a);
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
