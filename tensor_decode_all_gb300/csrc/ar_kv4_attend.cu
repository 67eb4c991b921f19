// ar_kv4_attend.cu -- ar_kv4_attend: attention over the 4-bit paged cache.
//
// A block of four warps takes rows of one request and kv head (8 NT query rows:
// new tokens x heads of the group) over a run of the request's tokens; runs of
// all requests are cut evenly over the blocks of one resident grid, and what a
// cut separates is joined by the last block to arrive.
//
// The products are S^T = K Q^T and O^T = V^T P^T (mma.m16n8k16, fp16 operands,
// binary32 sums), with the tokens (channels) as the 16 rows and the query rows
// as the 8 columns, so that a group of 8 heads fills the instruction.  K and V
// enter as the whole numbers they are: a nibble under fp16's exponent of 1024
// is 1024 + u, and one subtraction gives u - 8 exactly.  K's scales multiply
// the sums of each group of 32 channels, V's the weights, both in binary32.
//
// Softmax runs in base 2 under a reference M per row, common to a warp, that moves
// only when a score passes it by 2^6: p = 2^(s - M).  M also holds the exponent of the largest V
// scale seen, so that a weight p * scale stays within fp16 with 2^-14 of
// it still a normal number, whatever the scales.
//
// Each warp reads its tokens on its own: a ring of stages in shared memory,
// filled by bulk copies (a tile is 18 D contiguous bytes) one stage or more ahead.
#include <type_traits>

#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr int kWarps = 4;
constexpr int kThreads4 = kWarps * 32;
constexpr int kMaxRequests = 8192;
constexpr int kMaxGrid = 1024;            // blocks a workspace has room for
constexpr float kNoScore = -3.0e38f;      // below every score; finite, so that differences are numbers
constexpr int kHead = 8;                  // weights stand near 2^kHead ...
constexpr int kLead = 6;                  // ... and may pass it by 2^kLead before the reference moves

// Workspace: [0] status; from 4096: counters, one to a block; from 16384: two partial results to a block.
constexpr size_t kCounterAt = 4096, kPartAt = 16384;
constexpr size_t kWorkspaceBytes = kPartAt + (16u << 20);

struct Attend {
    ar_kv4_attend_args a;
    int group;        // query heads of a kv head
    int vec_q, vec_o;
    int min_chunks;   // least chunks worth a block of their own
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t b0, const uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats to fp16, the first in the low half.
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The 8 nibbles of w as fp16 pairs u - 8: nibbles (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void nibbles_to_half(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t k1024 = 0x64006400u;
    const __half2 m1032 = __half2half2(__ushort_as_half(0xe408));   // -1032
    const __half2 m72 = __half2half2(__ushort_as_half(0xd480));     // -72
    const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));     // 1 / 16
    const uint32_t w8 = w >> 8;
    uint32_t x[4];
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x[0]) : "r"(w), "r"(k1024));
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(x[1]) : "r"(w), "r"(k1024));
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x[2]) : "r"(w8), "r"(k1024));
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(x[3]) : "r"(w8), "r"(k1024));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 v = *reinterpret_cast<__half2 *>(&x[i]);
        // 1024 + u, or 1024 + 16 u: both ways exact
        v = (i & 1) ? __hfma2(v, r16, m72) : __hadd2(v, m1032);
        h[i] = *reinterpret_cast<uint32_t *>(&v);
    }
}

// N words from shared memory in the widest accesses (the address is a multiple of 4 N, up to 16).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    }
}

template <int D_, int NT_, int CT_, int S_>
struct Shape {
    static constexpr int D = D_;              // head dim
    static constexpr int NT = NT_;            // 8-row tiles of query rows
    static constexpr int CT = CT_;            // tiles of a chunk, the unit of work and a stage of the ring
    static constexpr int S = S_;              // stages
    static constexpr int G = D / kGroup;
    static constexpr int Tokens = CT * kTileTokens;
    static constexpr int Rows = 8 * NT;
    static constexpr bool QShared = NT > 2;   // q operands in shared memory, for want of registers
    static constexpr int Stage = CT * tile_bytes(D);
    static constexpr int Ring = kWarps * S * Stage;
    static constexpr int OStride = D + 4;     // floats of a row in the exchange: conflict-free for 16-byte stores
    static constexpr int Exchange = kWarps * Rows * (OStride + 2) * 4;
    static constexpr int QBytes = QShared ? D / 16 * NT * 32 * 8 : 0;
    static constexpr int Data = Ring > Exchange ? Ring : Exchange;
    static constexpr int Smem = Data + QBytes;
    static constexpr size_t PartFloats = (size_t)Rows * (D + 2);   // rows, then their references and sums
    static constexpr size_t Fit = (kWorkspaceBytes - kPartAt) / (2 * PartFloats * 4);
    static constexpr int MaxGrid = Fit < kMaxGrid ? (int)Fit : kMaxGrid;
};

// What a request asks for.
struct Request {
    int len, first, count;   // tokens, first row of q, rows
    int blocks, chunks;      // row blocks; chunks of a row block (an upper bound where there are several)
};

template <class C>
__device__ __forceinline__ Request request_of(const Attend &c, int b) {
    const ar_kv4_attend_args &a = c.a;
    Request r;
    int *status = static_cast<int *>(a.workspace);
    r.len = a.lens[b];
    r.first = a.cu ? a.cu[b] : b;
    const int end = a.cu ? a.cu[b + 1] : b + 1;
    const long long room = (long long)a.table_width * a.page;
    if (r.len < 0 || r.len > room || r.first < 0 || end < r.first || end > a.tokens) {
        atomicCAS(status, 0, AR_EINVAL);
        r.len = min(max(r.len, 0), (int)min(room, 0x7fffffffll));
        r.first = min(max(r.first, 0), a.tokens);
    }
    r.count = max(min(end, a.tokens) - r.first, 0);
    r.blocks = (int)(((long long)r.count * c.group + C::Rows - 1) / C::Rows);
    const int all = max((r.len + C::Tokens - 1) / C::Tokens, 1);
    r.chunks = all;
    if (a.window) {
        const int sink = (int)min((long long)all, ((long long)a.sinks + C::Tokens - 1) / C::Tokens);
        if (r.blocks <= 1) {
            const int low = max(r.len - r.count - a.window + 1, 0) / C::Tokens;
            r.chunks = all - low + min(sink, low);
        } else {
            r.chunks = (int)min((long long)all, sink + ((long long)a.window + C::Rows) / C::Tokens + 2);
        }
    }
    return r;
}

// Wait for a stage's copies, with a limit (about a second, and a millisecond
// once one has run out), after which the status says so and the caller goes on
// with what is there.
__device__ __forceinline__ void wait_stage(uint32_t bar, uint32_t parity, bool &late, int *status) {
    for (int i = 0; i < (late ? 1 << 10 : 1 << 20); ++i) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return;
    }
    late = true;
    atomicCAS(status, 0, AR_ETIMEOUT);
}

template <typename T, class C>
__global__ void __launch_bounds__(kThreads4) attend_kernel(const __grid_constant__ Attend c) {
    constexpr int D = C::D, NT = C::NT, CT = C::CT, S = C::S, G = C::G, Rows = C::Rows;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) unsigned long long bars[kWarps * S];
    __shared__ long long sums[kWarps];
    __shared__ int start_b, is_last;
    __shared__ long long start_off;
    const ar_kv4_attend_args &a = c.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int *status = static_cast<int *>(a.workspace);

    // Running sum over the requests' chunks: every block finds its share by itself.
    long long u0, u1;
    long long per;
    {
        const int each = (a.requests + kThreads4 - 1) / kThreads4;
        const int b0 = min((int)threadIdx.x * each, a.requests), b1 = min(b0 + each, a.requests);
        long long own = 0;
        for (int b = b0; b < b1; ++b) {
            const Request r = request_of<C>(c, b);
            own += (long long)r.blocks * r.chunks * a.kv_heads;
        }
        long long run = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long x = __shfl_up_sync(~0u, run, d);
            if (lane >= d) run += x;
        }
        if (lane == 31) sums[warp] = run;
        if (threadIdx.x < kWarps * S)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&bars[threadIdx.x])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) run += sums[w];
            total += sums[w];
        }
        per = max((total + gridDim.x - 1) / gridDim.x, (long long)c.min_chunks);
        u0 = min(per * blockIdx.x, total);
        u1 = min(u0 + per, total);
        if (u0 >= u1) return;
        long long at = run - own;
        if (at <= u0 && u0 < run) {
            for (int b = b0; b < b1; ++b) {
                const Request r = request_of<C>(c, b);
                const long long units = (long long)r.blocks * r.chunks * a.kv_heads;
                if (u0 < at + units) {
                    start_b = b;
                    start_off = u0 - at;
                    break;
                }
                at += units;
            }
        }
        __syncthreads();
    }
    int b = start_b;
    long long off = start_off;
    uint8_t *ring = smem + warp * S * C::Stage;
    const uint32_t ring_addr = smem_addr(ring), bar_addr = smem_addr(&bars[warp * S]);
    bool late = false;
    uint32_t filled = 0, used = 0;   // stages filled and used by this warp, over all its segments

    for (long long u = u0; u < u1;) {
        const Request r = request_of<C>(c, b);
        const long long units = (long long)r.blocks * r.chunks * a.kv_heads;
        if (off >= units) {
            if (++b >= a.requests) break;   // only if the lengths changed meanwhile
            off = 0;
            continue;
        }
        // The segment: one kv head and row block, chunks c0 .. c0 + take of it.
        const int seg = (int)(off / r.chunks), c0 = (int)(off % r.chunks);
        const int take = (int)min((long long)(r.chunks - c0), u1 - u);
        const int kv = seg / r.blocks, row0 = seg % r.blocks * Rows;
        const int rows = min(Rows, r.count * c.group - row0);
        const int pos0 = r.len - r.count;                                // position of the first new token
        const int pos_lo = pos0 + row0 / c.group, pos_hi = pos0 + (row0 + rows - 1) / c.group;
        const int low = a.window ? max(pos_lo - a.window + 1, 0) : 0;   // first token in a window
        const int low_chunk = low / C::Tokens;
        const int sink_chunks = a.window ? (int)min((long long)low_chunk, ((long long)a.sinks + C::Tokens - 1) / C::Tokens) : 0;
        const int chunks = pos_hi < 0 ? 0 : sink_chunks + pos_hi / C::Tokens - low_chunk + 1;
        const int cb = min(c0 + take, chunks);
        const int mine = cb - c0 > warp ? (cb - c0 - warp + kWarps - 1) / kWarps : 0;   // chunks c0 + warp + 4 k of it

        // -- the producer's side: page ids of 32 / CT chunks at a time, a batch ahead
        const int last_tile = pos_hi < 0 ? -1 : pos_hi / kTileTokens;
        const int32_t *table = a.table + (long long)b * a.table_stride;
        constexpr int kBatch = 32 / CT;
        auto chunk_id = [&](int k) {
            const int i = c0 + warp + kWarps * k;
            return i < sink_chunks ? i : low_chunk + i - sink_chunks;
        };
        auto page_ids = [&](int k) -> int {
            k += lane / CT;
            if (k >= mine) return 0;
            const int tile = chunk_id(k) * CT + lane % CT;
            return tile <= last_tile ? table[tile * kTileTokens / a.page] : 0;
        };
        int ids = page_ids(0), ids_next = page_ids(kBatch);
        int sent = 0;
        auto send = [&]() {
            if (sent >= mine) return;
            if (sent && sent % kBatch == 0) {
                ids = ids_next;
                ids_next = page_ids(sent + kBatch);
            }
            const int stage = filled % S;
            const int tile = chunk_id(sent) * CT + lane;
            int id = __shfl_sync(~0u, ids, sent % kBatch * CT + lane % CT);
            const bool get = lane < CT && tile <= last_tile;
            const unsigned n = __popc(__ballot_sync(~0u, get));
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar_addr + 8 * stage),
                             "r"(n * (unsigned)tile_bytes(D)) : "memory");
            __syncwarp();
            if (get) {
                if (id < 0 || id >= a.pages) {
                    atomicCAS(status, 0, AR_EINVAL);
                    id = 0;
                }
                const uint8_t *src = static_cast<const uint8_t *>(a.pool) +
                                     (((long long)id * a.kv_heads + kv) * (a.page / kTileTokens) + tile % (a.page / kTileTokens)) *
                                         tile_bytes(D);
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 ring_addr + stage * C::Stage + lane * tile_bytes(D)),
                             "l"(src), "r"((unsigned)tile_bytes(D)), "r"(bar_addr + 8 * stage)
                             : "memory");
            }
            ++sent;
            ++filled;
        };
        for (int i = 0; i < S; ++i) send();

        // -- q: column g of tile n is row row0 + 8 n + g; fp16 of q / 2^e, e the row's own for bfloat16
        uint32_t qf[C::QShared ? 1 : NT][D / 16][2];
        uint2 *q_shared = reinterpret_cast<uint2 *>(smem + C::Data);
        float mult[NT][2];            // what a sum of products is worth, in base 2: columns 2 t and 2 t + 1
        int pos[NT][2];               // their positions
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = row0 + 8 * n + g;
            const bool in = row < row0 + rows;
            float x[G][8];
            uint32_t top = 0;
            const T *src = static_cast<const T *>(a.q) + (long long)(r.first + (in ? row / c.group : 0)) * a.q_token_stride +
                           (long long)(kv * c.group + (in ? row % c.group : 0)) * a.q_head_stride + 8 * t;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                if (in) {
                    load8(src + 32 * j, c.vec_q != 0, x[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[j][i]) & 0x7fffffffu);
            }
            float unit = 1, worth = a.scale * 1.4426950408889634f;
            if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                // 2^e <= top, and 2^-e a normal number; zeros, infinities and NaN stay as they are
                int e = (int)(top >> 23) - 127;
                if (top == 0 || e == 128) e = 0;
                e = max(min(e, 126), -126);
                unit = __uint_as_float((uint32_t)(127 - e) << 23);
                worth *= __uint_as_float((uint32_t)(127 + e) << 23);
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = pack_half(x[j][i] * unit, x[j][i + 4] * unit);
                if constexpr (C::QShared) {
                    if (warp == n % kWarps) {
                        q_shared[((2 * j) * NT + n) * 32 + lane] = make_uint2(h[0], h[1]);
                        q_shared[((2 * j + 1) * NT + n) * 32 + lane] = make_uint2(h[2], h[3]);
                    }
                } else {
                    qf[n][2 * j][0] = h[0]; qf[n][2 * j][1] = h[1];
                    qf[n][2 * j + 1][0] = h[2]; qf[n][2 * j + 1][1] = h[3];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mult[n][i] = __shfl_sync(~0u, worth, (2 * t + i) * 4);
                pos[n][i] = min(pos0 + (row0 + 8 * n + 2 * t + i) / c.group, pos_hi);
            }
        }
        if constexpr (C::QShared) __syncthreads();

        float o[D / 16][NT][4];
        float ref[NT][2], l[NT][2];
        int vexp = -80;                      // exponent of the largest V scale so far, at least -80
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][n][i] = 0;
            ref[n][0] = ref[n][1] = kNoScore;
            l[n][0] = l[n][1] = 0;
        }

        for (int k = 0; k < mine; ++k) {
            const int stage = used % S;
            wait_stage(bar_addr + 8 * stage, (used / S) & 1, late, status);
            const uint8_t *data = ring + stage * C::Stage;
            const int tok0 = chunk_id(k) * C::Tokens;
            // Whether every row sees every token of the chunk.
            const bool full = tok0 + C::Tokens - 1 <= pos_lo &&
                              (!a.window || tok0 > pos_hi - a.window || tok0 <= a.sinks - C::Tokens);

            // scores
            float x[CT][NT][4];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint8_t *tile = data + ct * tile_bytes(D);
                uint32_t w0[G], w1[G], sc0[G / 2], sc1[G / 2];
                load_words(tile + lane * G * 4, w0);
                load_words(tile + (32 + lane) * G * 4, w1);
                load_words(tile + tile_ks(D) + g * G * 2, sc0);
                load_words(tile + tile_ks(D) + (g + 8) * G * 2, sc1);
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    uint32_t h0[4], h1[4];
                    nibbles_to_half(w0[j], h0);
                    nibbles_to_half(w1[j], h1);
                    const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
                    const float s0 = __uint_as_float(j & 1 ? sc0[j / 2] & 0xffff0000u : sc0[j / 2] << 16);
                    const float s1 = __uint_as_float(j & 1 ? sc1[j / 2] & 0xffff0000u : sc1[j / 2] << 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float acc[4] = {0, 0, 0, 0};
                        if constexpr (C::QShared) {
                            const uint2 q0 = q_shared[((2 * j) * NT + n) * 32 + lane], q1 = q_shared[((2 * j + 1) * NT + n) * 32 + lane];
                            mma16816(acc, a0, q0.x, q0.y);
                            mma16816(acc, a1, q1.x, q1.y);
                        } else {
                            mma16816(acc, a0, qf[n][2 * j][0], qf[n][2 * j][1]);
                            mma16816(acc, a1, qf[n][2 * j + 1][0], qf[n][2 * j + 1][1]);
                        }
                        if (j == 0) {
                            x[ct][n][0] = acc[0] * s0; x[ct][n][1] = acc[1] * s0;
                            x[ct][n][2] = acc[2] * s1; x[ct][n][3] = acc[3] * s1;
                        } else {
                            x[ct][n][0] = fmaf(acc[0], s0, x[ct][n][0]); x[ct][n][1] = fmaf(acc[1], s0, x[ct][n][1]);
                            x[ct][n][2] = fmaf(acc[2], s1, x[ct][n][2]); x[ct][n][3] = fmaf(acc[3], s1, x[ct][n][3]);
                        }
                    }
                }
            }
            // V scales: the largest exponent among tokens that some row sees
            int vmax = 0;
#pragma unroll
            for (int i = 0; i < CT * D / 128; ++i) {
                const int wd = i * 32 + lane, ct = wd / (D / 4), in = wd % (D / 4);
                uint32_t w = *reinterpret_cast<const uint32_t *>(data + ct * tile_bytes(D) + tile_vs(D) + in * 4);
                if (!full) {
                    const int tok = tok0 + ct * kTileTokens + in / (G / 2);
                    if (tok > pos_hi || (a.window && tok <= pos_lo - a.window && tok >= a.sinks)) w = 0;
                }
                const int e0 = (w >> 7) & 255, e1 = (w >> 23) & 255;
                vmax = max(vmax, max(e0 == 255 ? 0 : e0, e1 == 255 ? 0 : e1));
            }
            bool move = vmax - 127 > vexp;
            // relative to the reference; what a row does not see is -infinity
            const float most = (float)(kHead + kLead - vexp);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[ct][n][i] *= mult[n][i & 1];
                        if (!full) {
                            const int tok = tok0 + ct * kTileTokens + g + (i & 2) * 4, p = pos[n][i & 1];
                            const bool see = tok <= p && (!a.window || tok > p - a.window || tok < a.sinks);
                            x[ct][n][i] = see ? x[ct][n][i] : -INFINITY;
                        }
                        move |= x[ct][n][i] - ref[n][i & 1] > most;
                    }
            if (__any_sync(~0u, move)) {
                vmax = __reduce_max_sync(~0u, vmax);
                vexp = max(vexp, vmax - 127);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float top = kNoScore;
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) top = fmaxf(top, fmaxf(x[ct][n][i], x[ct][n][i + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                        // the reference never falls: a lower one would let earlier weights overflow
                        const float now = top > kNoScore ? fmaxf(ref[n][i], top + (float)(vexp - kHead)) : ref[n][i];
                        const float keep = exp2_approx(ref[n][i] - now);
                        ref[n][i] = now;
                        l[n][i] *= keep;
#pragma unroll
                        for (int m = 0; m < D / 16; ++m) {
                            o[m][n][i] *= keep;
                            o[m][n][i + 2] *= keep;
                        }
                    }
            }
            // weights, and the sum over V
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint8_t *tile = data + ct * tile_bytes(D);
                uint32_t w0[G], w1[G], sc0[G / 2], sc1[G / 2];
                load_words(tile + tile_v(D) + lane * G * 4, w0);
                load_words(tile + tile_v(D) + (32 + lane) * G * 4, w1);
                load_words(tile + tile_vs(D) + g * G * 2, sc0);
                load_words(tile + tile_vs(D) + (g + 8) * G * 2, sc1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[ct][n][i] = exp2_approx(x[ct][n][i] - ref[n][i & 1]);
                    l[n][0] += x[ct][n][0] + x[ct][n][2];
                    l[n][1] += x[ct][n][1] + x[ct][n][3];
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    uint32_t h0[4], h1[4];
                    nibbles_to_half(w0[j], h0);
                    nibbles_to_half(w1[j], h1);
                    const uint32_t a0[4] = {h0[0], h0[1], h1[0], h1[1]}, a1[4] = {h0[2], h0[3], h1[2], h1[3]};
                    const float s0 = __uint_as_float(j & 1 ? sc0[j / 2] & 0xffff0000u : sc0[j / 2] << 16);
                    const float s1 = __uint_as_float(j & 1 ? sc1[j / 2] & 0xffff0000u : sc1[j / 2] << 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float p[4] = {x[ct][n][0] * s0, x[ct][n][1] * s0, x[ct][n][2] * s1, x[ct][n][3] * s1};
                        if (!full) {
                            // a scale that no row of ours may see can be anything
#pragma unroll
                            for (int i = 0; i < 4; ++i) p[i] = x[ct][n][i] == 0 ? 0 : p[i];
                        }
                        const uint32_t b0 = transpose8x8(pack_half(p[0], p[1])), b1 = transpose8x8(pack_half(p[2], p[3]));
                        mma16816(o[2 * j][n], a0, b0, b1);
                        mma16816(o[2 * j + 1][n], a1, b0, b1);
                    }
                }
            }
            ++used;
            __syncwarp();      // every lane has read the stage
            send();
        }

        // -- join the warps: each one's reference, sum and rows through shared memory
        __syncthreads();
        float *xo = reinterpret_cast<float *>(smem), *xm = xo + kWarps * Rows * C::OStride;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[n][i] += __shfl_xor_sync(~0u, l[n][i], d);
                const int col = 8 * n + 2 * t + i;
                if (g == 0) {
                    xm[(warp * Rows + col) * 2] = ref[n][i];
                    xm[(warp * Rows + col) * 2 + 1] = l[n][i];
                }
#pragma unroll
                for (int j = 0; j < G; ++j)
                    *reinterpret_cast<float4 *>(&xo[(warp * Rows + col) * C::OStride + 32 * j + 4 * g]) =
                        make_float4(o[2 * j][n][i], o[2 * j][n][i + 2], o[2 * j + 1][n][i], o[2 * j + 1][n][i + 2]);
            }
        }
        __syncthreads();
        // The segment's other blocks, if any.
        const long long s0 = u - c0;
        const int first = (int)(s0 / per), parts = (int)((s0 + r.chunks - 1) / per) - first + 1;
        float *part_base = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kPartAt);
        float *part = part_base + (2 * (size_t)blockIdx.x + (first == (int)blockIdx.x ? 1 : 0)) * C::PartFloats;
        auto finish = [&](int col, int quad, float4 v, float m, float sum) {
            const int row = row0 + col;
            const float inv = sum > 0 ? __fdiv_rn(1.0f, sum) : sum == sum ? 0.0f : sum;
            const long long token = r.first + row / c.group;
            const int head = kv * c.group + row % c.group;
            T *dst = static_cast<T *>(a.out) + token * a.out_token_stride + (long long)head * a.out_head_stride + 4 * quad;
            union { uint2 u; T e[4]; } w;
            w.e[0] = Elem<T>::from_float(v.x * inv); w.e[1] = Elem<T>::from_float(v.y * inv);
            w.e[2] = Elem<T>::from_float(v.z * inv); w.e[3] = Elem<T>::from_float(v.w * inv);
            if (c.vec_o) {
                *reinterpret_cast<uint2 *>(dst) = w.u;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[i] = w.e[i];
            }
            if (quad == 0 && a.lse)
                a.lse[token * a.q_heads + head] =
                    sum > 0 ? (m + log2f(sum)) * 0.6931471805599453f : sum == sum ? -INFINITY : sum;
        };
        for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads4) {
            const int col = i / (D / 4), quad = i % (D / 4);
            float m = kNoScore;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, xm[(w * Rows + col) * 2]);
            float4 v = make_float4(0, 0, 0, 0);
            float sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_approx(xm[(w * Rows + col) * 2] - m);
                const float4 y = *reinterpret_cast<const float4 *>(&xo[(w * Rows + col) * C::OStride + 4 * quad]);
                sum = fmaf(xm[(w * Rows + col) * 2 + 1], f, sum);
                v.x = fmaf(y.x, f, v.x); v.y = fmaf(y.y, f, v.y); v.z = fmaf(y.z, f, v.z); v.w = fmaf(y.w, f, v.w);
            }
            if (parts == 1) {
                finish(col, quad, v, m, sum);
            } else {
                *reinterpret_cast<float4 *>(part + col * D + 4 * quad) = v;
                if (quad == 0) {
                    part[Rows * D + 2 * col] = m;
                    part[Rows * D + 2 * col + 1] = sum;
                }
            }
        }
        if (parts > 1) {
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                unsigned *counter = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(a.workspace) + kCounterAt) + first;
                is_last = atomicAdd(counter, 1) == (unsigned)parts - 1;
                if (is_last) *counter = 0;   // for the next call
                __threadfence();
            }
            __syncthreads();
            if (is_last) {
                // in the order of the parts, whoever came last
                auto at = [&](int i) { return part_base + (i == 0 ? 2 * (size_t)first + 1 : 2 * (size_t)(first + i)) * C::PartFloats; };
                for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads4) {
                    const int col = i / (D / 4), quad = i % (D / 4);
                    float m = kNoScore, sum = 0;
                    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
                    for (int k = 0; k < parts; ++k) {
                        const float *p = at(k);
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p + Rows * D + 2 * col));
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(p + col * D + 4 * quad));
                        const float m2 = fmaxf(m, ml.x), f0 = exp2_approx(m - m2), f1 = exp2_approx(ml.x - m2);
                        m = m2;
                        sum = fmaf(sum, f0, ml.y * f1);
                        v.x = fmaf(v.x, f0, y.x * f1); v.y = fmaf(v.y, f0, y.y * f1);
                        v.z = fmaf(v.z, f0, y.z * f1); v.w = fmaf(v.w, f0, y.w * f1);
                    }
                    finish(col, quad, v, m, sum);
                }
            }
        }
        __syncthreads();   // the ring is free for the next segment's copies
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        u += take;
        off += take;
    }
}

template <typename T, class C>
int start(const Attend &c, cudaStream_t s) {
    const void *kernel = reinterpret_cast<const void *>(attend_kernel<T, C>);
    // blocks resident at once on this device, asked once (0: not asked yet; racing threads store the same)
    static int resident[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return launch_status(cudaErrorUnknown);
    int grid = *(volatile int *)&resident[dev];
    if (grid == 0) {
        int per_sm = 0, sms = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads4, C::Smem) != cudaSuccess || per_sm < 1 ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return launch_status(cudaErrorUnknown);
        grid = min(per_sm * sms, C::MaxGrid);
        *(volatile int *)&resident[dev] = grid;
    }
    // No more blocks than the longest contexts the table can hold would fill.
    const long long chunks = ((long long)c.a.table_width * c.a.page + C::Tokens - 1) / C::Tokens;
    const long long blocks = ((long long)c.a.tokens * c.group + C::Rows - 1) / C::Rows + c.a.requests;
    const long long most = (blocks * max(chunks, 1ll) * c.a.kv_heads + c.min_chunks - 1) / c.min_chunks;
    void *args[] = {const_cast<Attend *>(&c)};
    return launch_status(cudaLaunchKernel(kernel, dim3((unsigned)min((long long)grid, most)), dim3(kThreads4), args, C::Smem, s));
}

template <typename T>
int start(const Attend &c, cudaStream_t s) {
    const long long rows = (long long)max(c.a.max_new, 1) * c.group;
    switch (c.a.head_dim) {
        case 64:
            if (rows <= 8) return start<T, Shape<64, 1, 2, 4>>(c, s);
            if (rows <= 16) return start<T, Shape<64, 2, 2, 4>>(c, s);
            return start<T, Shape<64, 4, 2, 4>>(c, s);
        case 128:
            if (rows <= 8) return start<T, Shape<128, 1, 2, 3>>(c, s);
            if (rows <= 16) return start<T, Shape<128, 2, 2, 3>>(c, s);
            return start<T, Shape<128, 4, 1, 4>>(c, s);
        default:
            if (rows <= 8) return start<T, Shape<256, 1, 1, 3>>(c, s);
            return start<T, Shape<256, 2, 1, 3>>(c, s);
    }
}

}  // namespace

extern "C" {

AR_API size_t ar_kv4_workspace_bytes(void) { return kWorkspaceBytes; }

AR_API int ar_kv4_workspace_init(void *workspace, ar_stream_t stream) {
    if (!workspace || misaligned(workspace, 256)) return AR_EINVAL;
    return launch_status(cudaMemsetAsync(workspace, 0, kPartAt, stream));
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
    if (a.requests > kMaxRequests) return AR_ETOOBIG;
    if (a.tokens == 0) return AR_OK;
    if (!a.q || !a.out || !a.workspace || a.requests < 1 || !a.lens || (!a.table && a.table_width > 0) ||
        (a.table_width > 0 && (!a.pool || a.pages < 1)))
        return AR_EINVAL;
    if (misaligned(a.q, 2) || misaligned(a.out, 2) || misaligned(a.lse, 4) || misaligned(a.pool, 16) || misaligned(a.table, 4) ||
        misaligned(a.lens, 4) || misaligned(a.cu, 4) || misaligned(a.workspace, 256))
        return AR_EINVAL;
    c.group = a.q_heads / a.kv_heads;
    // A window or sinks that cover the table limit nothing; smaller ones and the rows stay where sums fit 32 bits.
    const long long room = (long long)a.table_width * a.page;
    if (a.window >= room || a.sinks >= room) c.a.window = 0;
    if ((long long)a.tokens * c.group > 1 << 30 || c.a.window > 1 << 30) return AR_ETOOBIG;
    c.vec_q = rows_aligned(a.q, a.q_token_stride, a.q_head_stride);
    c.vec_o = rows_aligned(a.out, a.out_token_stride, a.out_head_stride);
    c.min_chunks = kWarps;
    return a.dtype == AR_F16 ? start<__half>(c, stream) : start<__nv_bfloat16>(c, stream);
}

}  // extern "C"
