// ar_matmul_fp8.cu -- ar_matmul_fp8: the checks of a call, the choice of its kernel, and the kernel that takes any alignment.
#include <cuda_fp8.h>

#include <algorithm>

#include "ar_matmul_fp8.cuh"

namespace {

using namespace tda;

// ---------------------------------------------------- rows of any alignment
//
// Tiles of 64 rows and 64 features, 4 warps.  Bytes go through registers to shared memory as fp16 (which holds every
// e4m3 value), the products are mma.sync's: rows that are not on 16 bytes cannot be moved by bulk copies, and
// no weight that is kept for its speed is laid out like that.  1000 rows of 4095 channels times 2048 features take 228 us, 8 of 8191 times 1280
// 170 (by single bytes, and without the next group's on their way, 619 and 227).

constexpr int kSide = 64, kPitch = kBlock + 8;   // (8 more halves to a row: no two of a fragment's rows share banks)

__device__ __forceinline__ uint32_t widened(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}

// 64 channels of a row from the channel on: one row to two threads.  Inside a row whole words are read, and of each two the four bytes
// that begin where the channels do; at its ends single bytes.
struct Piece {
    uint32_t w[17], shift;
    bool inside;
    __device__ __forceinline__ void load(const uint8_t *row, int channel, int dim, bool there) {
        inside = there && channel >= 4 && channel + 68 <= dim;
        if (!inside) return;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + channel);
        const uint32_t *words = reinterpret_cast<const uint32_t *>(at & ~(uintptr_t)3);
        shift = (uint32_t)(at & 3) * 8;
#pragma unroll
        for (int i = 0; i < 17; ++i) w[i] = words[i];
    }
    __device__ __forceinline__ void store(__half *to, const uint8_t *row, int channel, int dim, bool there) const {
        if (inside) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t b = __funnelshift_r(w[i], w[i + 1], shift);
                *reinterpret_cast<uint2 *>(to + 4 * i) = make_uint2(widened(b & 0xffff), widened(b >> 16));
            }
            return;
        }
        for (int i = 0; i < 64; i += 2) {
            const int c = channel + i;
            const uint32_t lo = there && c < dim ? row[c] : 0, hi = there && c + 1 < dim ? row[c + 1] : 0;
            *reinterpret_cast<uint32_t *>(to + i) = widened(lo | hi << 8);
        }
    }
};

__global__ void __launch_bounds__(128) any_rows_kernel(const Product p) {
    after_the_stream();
    __shared__ __half xs[kSide][kPitch], ws[kSide][kPitch];
    const ar_matmul_fp8_args &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const Rows rows = rows_of_tile(a, blockIdx.x, kSide);
    if (rows.count == 0) return;
    const int feature = blockIdx.y * kSide;
    const uint8_t *x = static_cast<const uint8_t *>(a.x), *w = static_cast<const uint8_t *>(a.weight) + rows.expert * a.expert_stride;
    const int mine = threadIdx.x >> 1;
    const int64_t from = mine < rows.count ? source_row(a, rows.first + mine) : -1;
    int64_t source[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + g + 8 * h;
        source[h] = r < rows.count ? source_row(a, rows.first + r) : -1;
    }
    const float *scale_w = a.weight_scales + ((int64_t)rows.expert * ((a.out_dim + kBlock - 1) / kBlock) + feature / kBlock) * p.groups;
    float acc[8][4] = {};
    const uint8_t *const own_x = x + max(from, (int64_t)0) * a.x_stride, *const own_w = w + (int64_t)(feature + mine) * a.weight_stride;
    const bool has_w = feature + mine < a.out_dim;
    const int half = (threadIdx.x & 1) * 64;
    Piece next_x, next_w;
    next_x.load(own_x, half, a.dim, from >= 0);
    next_w.load(own_w, half, a.dim, has_w);
    for (int k = 0; k < p.groups; ++k) {
        const int channel = k * kBlock + half;
        next_x.store(&xs[mine][half], own_x, channel, a.dim, from >= 0);
        next_w.store(&ws[mine][half], own_w, channel, a.dim, has_w);
        __syncthreads();
        // (the next group's are on their way during this one's products)
        next_x.load(own_x, channel + kBlock, a.dim, from >= 0);
        next_w.load(own_w, channel + kBlock, a.dim, has_w);
        float part[8][4] = {};
#pragma unroll
        for (int s = 0; s < kBlock; s += 16) {
            uint32_t f[4];
            const int r = warp * 16 + g;
            f[0] = *reinterpret_cast<uint32_t *>(&xs[r][s + 2 * t]);
            f[1] = *reinterpret_cast<uint32_t *>(&xs[r + 8][s + 2 * t]);
            f[2] = *reinterpret_cast<uint32_t *>(&xs[r][s + 2 * t + 8]);
            f[3] = *reinterpret_cast<uint32_t *>(&xs[r + 8][s + 2 * t + 8]);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const uint32_t b0 = *reinterpret_cast<uint32_t *>(&ws[n * 8 + g][s + 2 * t]), b1 = *reinterpret_cast<uint32_t *>(&ws[n * 8 + g][s + 2 * t + 8]);
                asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                             : "+f"(part[n][0]), "+f"(part[n][1]), "+f"(part[n][2]), "+f"(part[n][3])
                             : "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]), "r"(b0), "r"(b1));
            }
        }
        const float sw = scale_w[k];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float s = source[h] >= 0 ? a.x_scales[source[h] * a.x_scales_stride + (a.x_row_scales ? 0 : k)] * sw : 0.0f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                acc[n][2 * h] = fmaf(part[n][2 * h], s, acc[n][2 * h]);
                acc[n][2 * h + 1] = fmaf(part[n][2 * h + 1], s, acc[n][2 * h + 1]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + g + 8 * h;
        if (r >= rows.count) continue;
        const int64_t at = (rows.first + r) * a.out_stride;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            for (int e = 0; e < 2; ++e) {
                const int c = feature + n * 8 + 2 * t + e;
                if (c >= a.out_dim) continue;
                const float v = source[h] >= 0 ? acc[n][2 * h + e] : 0.0f;
                if (a.dtype == AR_F16) static_cast<__half *>(a.out)[at + c] = __float2half_rn(v);
                else static_cast<__nv_bfloat16 *>(a.out)[at + c] = __float2bfloat16_rn(v);
            }
    }
}

cudaError_t start_any(const Product &p, cudaStream_t s) {
    const int64_t tiles = most_tiles(p.a, kSide);
    return launch_next(any_rows_kernel, dim3((unsigned)tiles, (unsigned)((p.a.out_dim + kSide - 1) / kSide)), 128, 0, s, 0, p);
}

// ------------------------------------------------- what the copy engine sees

using Encode = decltype(&cuTensorMapEncodeTiled);

// The driver's function; nullptr where there is none.
Encode encoder() {
    static Encode f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess || found != cudaDriverEntryPointSuccess)
            p = nullptr;
        (void)cudaGetLastError();
        return reinterpret_cast<Encode>(p);
    }();
    return f;
}

bool encode(CUtensorMap *m, const void *at, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    static const cuuint32_t ones[3] = {1, 1, 1};
    const Encode f = encoder();
    auto call = [&] {
        return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(at), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (!f) return false;
    CUresult r = call();
    // (a host thread that has made no call yet that needs a context has none: unlike the runtime's, the driver's function does not make it current)
    int dev = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = call();
    return r == CUDA_SUCCESS;
}

// Whether the copy engine can take these rows: on 16 bytes, one after another.
bool copyable(const void *at, int64_t rows, int64_t stride, int64_t dim) {
    return !misaligned(at, 16) && (rows == 1 || (stride % 16 == 0 && stride >= dim && stride < (int64_t)1 << 39));
}

bool fast(const Product &p) {
    const ar_matmul_fp8_args &a = p.a;
    // (picked rows are found by 32 bits)
    if (a.row_of && a.x_rows > 1 && a.x_rows > ((int64_t)16 << 32) / std::max(a.x_stride, (int64_t)1)) return false;
    return a.dim > 0 && a.x_rows > 0 && copyable(a.x, a.x_rows, a.x_stride, a.dim) && copyable(a.weight, a.out_dim, a.weight_stride, a.dim) &&
           copyable(a.weight, a.experts, a.expert_stride, a.dim) && encoder();
}

int multiprocessors_of_device() {
    static int known[64] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (n = *(volatile int *)&known[dev])) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) *(volatile int *)&known[dev] = n;
    return n;
}

// Which of the fast kernels: the one that takes less time by its steps (groups of 128 channels that follow each other) in the tiles that follow each
// other, in units of 10 ns: with 128 rows to a block 0.5 us a step and 4 us besides, 6.3 where clusters share the channels; with 256 to a pair
// 0.39 and 4.5, and 3 more to a tile whose results leave by twos of bytes.  128 rows of 8192 times 8192 features took 21 us against 27,
// 256 35 against 27; 384 rows times 1280 features 14.8 against 26; 97 rows of 816 times 10853 8.3 against 11.3.  Up to 64 rows (32 to an expert)
// the weights' bytes count, and the first is always faster (64 rows: 18 against 27; 32 experts of 32 rows 48 against 53, of 64
// rows 76 against 54).
bool takes_many(const ar_matmul_fp8_args &a) {
    const int64_t experts = a.offsets ? a.experts : 1, rows = (a.rows + experts - 1) / experts, groups = (a.dim + kBlock - 1) / kBlock;
    if (rows <= (a.offsets ? 32 : 64)) return false;
    const int known = multiprocessors_of_device(), multiprocessors = known > 1 ? known : 152;
    auto up = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
    const int64_t tiles = experts * up(rows, 128) * up(a.out_dim, 128), pairs = experts * up(rows, 256) * up(a.out_dim, 256);
    int64_t share = 1;
    while (share < 16 && tiles * share * 2 <= multiprocessors && groups >= share * 4) share *= 2;
    const bool odd = misaligned(a.out, 16) || a.out_stride % 8 != 0;
    return 450 + up(pairs, multiprocessors / 2) * (39 * groups + (odd ? 300 : 0)) < (share > 1 ? 630 : 400) + 50 * up(tiles * share, multiprocessors) * up(groups, share);
}

}  // namespace

namespace tda {

bool map_weight(CUtensorMap *m, const ar_matmul_fp8_args &a, int box) {
    // (strides that nothing is found by are any multiple of 16)
    const int64_t row = a.out_dim > 1 ? a.weight_stride : (a.dim + 15) / 16 * 16, expert = a.experts > 1 ? a.expert_stride : row * a.out_dim;
    const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.out_dim, (cuuint64_t)a.experts}, strides[2] = {(cuuint64_t)row, (cuuint64_t)expert};
    const cuuint32_t boxes[3] = {kBlock, (cuuint32_t)box, 1};
    return encode(m, a.weight, 3, dims, strides, boxes);
}

bool map_rows(CUtensorMap *m, const ar_matmul_fp8_args &a, int box) {
    const int64_t row = a.x_rows > 1 ? a.x_stride : (a.dim + 15) / 16 * 16;
    const cuuint64_t dims[2] = {(cuuint64_t)a.dim, (cuuint64_t)a.x_rows}, strides[1] = {(cuuint64_t)row};
    const cuuint32_t boxes[2] = {kBlock, (cuuint32_t)box};
    return encode(m, a.x, 2, dims, strides, boxes);
}

}  // namespace tda

extern "C" AR_API int ar_matmul_fp8(const ar_matmul_fp8_args *args, ar_stream_t stream) {
    if (!args) return AR_EINVAL;
    const ar_matmul_fp8_args &a = *args;
    if (a.dtype != AR_F16 && a.dtype != AR_BF16) return AR_EINVAL;
    if (a.rows < 0 || a.x_rows < 0 || a.out_dim < 0 || a.dim < 0 || a.experts < 1 || (a.x_row_scales & ~1)) return AR_EINVAL;
    if ((!a.offsets && a.experts != 1) || (!a.row_of && a.x_rows != a.rows)) return AR_EINVAL;
    constexpr int64_t most = 1 << 30;
    if (a.rows > most || a.x_rows > most || a.dim > 1 << 20 || a.out_dim > 1 << 20 || a.experts > 1024) return AR_ETOOBIG;
    if (a.rows == 0 || a.out_dim == 0) return AR_OK;
    if (!a.out || (a.dim > 0 && (!a.weight || !a.weight_scales || (a.x_rows > 0 && (!a.x || !a.x_scales))))) return AR_EINVAL;
    if (misaligned(a.x_scales, 4) || misaligned(a.weight_scales, 4) || misaligned(a.out, 2) || misaligned(a.offsets, 4) || misaligned(a.row_of, 4) || misaligned(a.workspace, 16))
        return AR_EINVAL;
    Product p;
    p.a = a;
    p.groups = (a.dim + kBlock - 1) / kBlock;
    if (!fast(p)) return launch_status(start_any(p, stream));
    const int multiprocessors = multiprocessors_of_device();
    if (multiprocessors < 2) return AR_ECUDA;
    if (takes_many(a) && (!a.row_of || a.workspace)) return launch_status(start_many(p, stream, multiprocessors));
    return launch_status(start_few(p, stream, multiprocessors));
}

extern "C" AR_API size_t ar_matmul_fp8_workspace(const ar_matmul_fp8_args *args) {
    if (!args || !args->row_of || args->rows <= 0 || args->dim <= 0 || args->experts < 1 || !takes_many(*args)) return 0;
    const size_t groups = args->x_row_scales ? 1 : ((size_t)args->dim + kBlock - 1) / kBlock;
    return (size_t)args->rows * ((size_t)pitch_of(*args) + groups * sizeof(float));
}

extern "C" AR_API int ar_matmul_fp8_status(void) {
    int few = AR_OK, many = AR_OK;
    const int rc = take_few_status(&few), other = take_many_status(&many);
    return rc ? rc : other ? other : few ? few : many;
}
