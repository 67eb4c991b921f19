// ar_kv4.cuh -- the 4-bit cache's tile layout and small helpers of the
// operators of include/ar_ops.h.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ar_ops.h"

namespace tda {

constexpr int kTileTokens = 16;   // tokens of a tile
constexpr int kGroup = 32;        // channels that share a scale

__host__ __device__ constexpr int tile_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int tile_v(int D) { return 8 * D; }
__host__ __device__ constexpr int tile_ks(int D) { return 16 * D; }
__host__ __device__ constexpr int tile_vs(int D) { return 17 * D; }

// The 32-bit word that holds token r's K channels 32*j + 8*t .. + 7 (nibble i: channel + i).
__host__ __device__ constexpr int k_word(int G, int r, int t, int j) { return (r * 4 + t) * G + j; }
// The word whose half r % 2 holds token r's V channels 32*j + 4*g .. + 3.
__host__ __device__ constexpr int v_word(int G, int r, int g, int j) {
    return ((r >> 3) * 32 + g * 4 + ((r & 7) >> 1)) * G + j;
}

template <typename T> struct Elem;
template <> struct Elem<__half> {
    static __device__ float to_float(__half x) { return __half2float(x); }
    static __device__ __half from_float(float x) { return __float2half_rn(x); }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ float bf16_bits(uint32_t bits) { return __uint_as_float(bits << 16); }

// Both elements of a pair, and a pair of two rounded elements.
template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<__half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ uint32_t to_pair(float2 v) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Whether rows at p with these strides (elements of 2 bytes) all start on 16 bytes.
inline bool rows_aligned(const void *p, int64_t a, int64_t b) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && a % 8 == 0 && b % 8 == 0;
}

inline bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Every kernel of these operators is launched as a programmatic dependent of the work before it on its stream:
// its blocks may come to the GPU while that work ends, which hides the launch, and wait here, before they
// touch any memory, until it has ended and its writes are visible.  The next such kernel may come as soon as
// all blocks of this one have.
__device__ __forceinline__ void after_the_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
inline cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, unsigned cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The launch's own error, not one left by an earlier call of the program.
inline int launch_status(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    (void)cudaGetLastError();
    return AR_ECUDA;
}

}  // namespace tda
