// ar_kv4_attend.cu -- ar_kv4_attend: attention over the 4-bit paged cache.
//
// A warp takes 8 or 16 query rows (new tokens x heads) of one request and kv head over a run of the request's
// tokens, with its own ring of stages in shared memory and no other warp to wait for.  The runs cut the chunks
// of all requests, heads and row blocks, laid end to end, into equal shares, one to a warp of a resident grid;
// where a cut separates a row's tokens the partial results go to the workspace, and a second, small kernel
// joins them in order.
//
// The products are S^T = K Q^T and O^T = V^T P^T (mma.m16n8k16, fp16 operands, binary32 sums), with the tokens
// (channels) as the 16 rows and the query rows as the 8 columns, so that a group of 8 heads fills the
// instruction.  (tcgen05 has 64 rows at least, and wants its operands in shared memory: each nibble would be
// written there at four times its size and read once.)  K and V enter as the whole numbers u - 8 that they are: a
// nibble u in the mantissa of a power of two is that power plus u, and one exact instruction to a pair takes the
// rest off.  (Taking K's out of the sums instead, by where the accumulators start, loses bits, up to 8 where most
// of a group is 0, and the product of an infinite scale with a sum that is 0; it was not faster: 69 us for 68.)  K's
// scales multiply the sums of each group of 32 channels, V's the weights, both in binary32; weight x scale is
// rounded once, to fp16.
//
// Softmax runs in base 2 under a reference M per row, common to a warp, that moves only when a score passes it
// by 2^6: p = 2^(s - M), and the usual step costs a vote in place of a reduction.  M also holds the exponent
// of the largest V scale seen, so that a weight p * scale stays below fp16's largest number, and is a normal one
// down to 2^-22 of the largest scale (a smaller one is off by 2^-33 of that, where the largest p is 1).
//
// Each warp reads its tokens on its own: a ring of stages in shared memory, filled by bulk copies (a tile is
// 18 D contiguous bytes) a stage ahead, the next segment's first stages before the last one's results are
// written.
//
// Measured on a GB300 (graph replays): 64 requests of 16385 to 32768 tokens, 8 kv heads of 8, D 128: 306 us,
// 6.0 TB/s of cache or 88% of what a plain copy reaches; 64 ragged ones of 517 to 8001: 68 us, 69%; 128 ragged
// with a window of 1024 and D 64: 32 us; one of 1003 tokens and one kv head: 9.7 us.  The short ones are bound
// by the instructions they issue: 318 for a tile of 16 tokens and one head of 128, 0.60 a cycle and scheduler,
// two of five on the ALU pipe, which takes one every other cycle; DRAM carries the bytes that have to be read
// and no more, and the matrix instructions take a quarter of the time.  12 warps a multiprocessor: 16 with 126
// registers each were 12% slower.
#include "ar_kv4.cuh"

namespace {

using namespace tda;

constexpr int kMaxRequests = 8192;
constexpr int kWarps = 4;                 // warps of a block; each works alone
constexpr float kNoScore = -3.0e38f;      // below every score; finite, so that differences are numbers
constexpr int kHead = 8;                  // weights stand near 2^kHead ...
constexpr int kLead = 6;                  // ... and may pass it by 2^kLead before the reference moves
// Chunks that beginning a segment is worth in the shares: its latency and its results.  64 ragged requests,
// and a window of 17 chunks a segment: 1: 71.9 and 38.6 us, 2: 70.2 and 34.1, 3: 69.4 and 33.0, 4: 71.4 and
// 33.5, 6: 71.5 and 34.6.
constexpr int kStart = 3;

// Workspace: status, a record for each warp, and two partial results to a warp.
struct Record {
    int parts;                      // of the segment that begins in the warp and ends in another; 0: there is none
    int rows, kv, row0, first;      // as in Segment
    int unused[3];
};
constexpr int kMaxWarps = 2048;
constexpr size_t kRecordAt = 256, kPartAt = kRecordAt + kMaxWarps * sizeof(Record);
constexpr size_t kWorkspaceBytes = kPartAt + (24u << 20);
static_assert(kPartAt % 256 == 0, "partial results start on a line");

struct Attend {
    ar_kv4_attend_args a;
    int group;        // query heads of a kv head
    int vec_q, vec_o;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma16816(d, a, b0, b1, d[0], d[1], d[2], d[3]);
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

// The 8 nibbles of w as fp16 pairs u - 8: nibbles (0, 4), (1, 5), (2, 6), (3, 7).  A whole number under the exponent
// of 2^10 is 1024 + itself, so one logical instruction makes a pair and one exact operation takes the rest off
// (Y. J. Kim, R. Henry, R. Fahim, H. H. Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into
// Cloud Scale Production", 2022).
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

template <int D_, int NT_, int CT_, int CI_, int S_, int Blocks_>
struct Shape {
    static constexpr int D = D_;              // head dim
    static constexpr int NT = NT_;            // 8-row tiles of query rows
    static constexpr int CT = CT_;            // tiles of a chunk, the unit of work and a stage of the ring
    static constexpr int CI = CI_;            // tiles multiplied together, see the shapes below
    static constexpr int S = S_;              // stages
    static constexpr int Blocks = Blocks_;    // of an SM, for which registers are kept
    static constexpr int G = D / kGroup;
    static constexpr int Tokens = CT * kTileTokens;
    static constexpr int Rows = 8 * NT;
    static constexpr int Stage = CT * tile_bytes(D);
    static constexpr int Smem = kWarps * S * Stage;
    static constexpr size_t PartFloats = (size_t)Rows * (D + 2);   // rows, then their references and sums
};

// What a request asks for.
struct Request {
    int len, first, count;   // tokens, first row of q, rows
    int blocks, chunks;      // row blocks; chunks of a row block (an upper bound where there are several)
    // A row block's length in the row of shares: a segment costs as much as kStart chunks beside its own.
    __device__ long long length() const { return chunks + kStart; }
    __device__ long long total(int kv_heads) const { return blocks * length() * kv_heads; }
};

template <class C>
__device__ __forceinline__ Request request_of(const Attend &c, int b) {
    const ar_kv4_attend_args &a = c.a;
    Request r;
    r.len = a.lens[b];
    r.first = a.cu ? a.cu[b] : b;
    const int end = a.cu ? a.cu[b + 1] : b + 1;
    const long long room = (long long)a.table_width * a.page;
    if (r.len < 0 || r.len > room || r.first < 0 || end < r.first || end > a.tokens) {
        atomicCAS(static_cast<int *>(a.workspace), 0, AR_EINVAL);
        r.len = min(max(r.len, 0), (int)min(room, 0x7fffffffll));
        r.first = min(max(r.first, 0), a.tokens);
    }
    r.count = max(min(end, a.tokens) - r.first, 0);
    r.blocks = (r.count * c.group + C::Rows - 1) / C::Rows;
    const int all = max((int)(((long long)r.len + C::Tokens - 1) / C::Tokens), 1);
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

// A segment: a run of the chunks of one row block of one kv head of a request.
struct Segment {
    int rows, kv, row0, first;      // query rows, kv head, first row (token x group), first row of q of the request
    int pos0, pos_lo, pos_hi;       // position of the request's first new token, of the rows' first and last
    int c0, chunks;                 // chunks c0 .. c0 + chunks - 1 of those that its rows see
    int sink_chunks, low_chunk;     // chunk i is i below sink_chunks, i + low_chunk - sink_chunks from there on
    int request, end_tile;          // its tiles that hold tokens end there
    int whole, begins;              // all of its row block; its beginning
};

__device__ __forceinline__ int chunk_at(int i, int sink_chunks, int low_chunk) {
    return i < sink_chunks ? i : low_chunk + i - sink_chunks;
}

__device__ __forceinline__ long long now_ns() {
    long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of that parity to end, with a limit (four seconds) after
// which the status says so and the answer is false.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int *status) {
    long long begun = 0;
    for (;;) {
        uint32_t done;
        for (int i = 0; i < 64; ++i) {
            asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                         : "=r"(done) : "r"(bar), "r"(parity) : "memory");
            if (done) return true;
        }
        const long long t = now_ns();
        if (begun == 0) begun = t;
        if (t - begun > 4000000000ll) break;
    }
    atomicCAS(status, 0, AR_ETIMEOUT);
    return false;
}

// A row's result: divided by its sum, rounded; 0 and -infinity where nothing was seen.
template <typename T>
__device__ __forceinline__ void store_row(const Attend &c, long long token, int head, int channel, float4 v, float m, float sum) {
    const ar_kv4_attend_args &a = c.a;
    const float inv = sum > 0 ? __fdiv_rn(1.0f, sum) : sum == sum ? 0.0f : sum;
    T *dst = static_cast<T *>(a.out) + token * a.out_token_stride + (long long)head * a.out_head_stride + channel;
    union { uint2 u; T e[4]; } w;
    w.e[0] = Elem<T>::from_float(v.x * inv); w.e[1] = Elem<T>::from_float(v.y * inv);
    w.e[2] = Elem<T>::from_float(v.z * inv); w.e[3] = Elem<T>::from_float(v.w * inv);
    if (c.vec_o) {
        *reinterpret_cast<uint2 *>(dst) = w.u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = w.e[i];
    }
    if (channel == 0 && a.lse)
        a.lse[token * a.q_heads + head] = sum > 0 ? (m + log2f(sum)) * 0.6931471805599453f : sum == sum ? -INFINITY : sum;
}

template <typename T, class C>
__global__ void __launch_bounds__(kWarps * 32, C::Blocks) attend_kernel(const __grid_constant__ Attend c) {
    constexpr int D = C::D, NT = C::NT, CT = C::CT, CI = C::CI, S = C::S, G = C::G;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) unsigned long long bars[kWarps * S];
    __shared__ long long sums[kWarps], start_off[kWarps], start_u[kWarps];   // where each warp's walk stands
    __shared__ int start_b[kWarps];
    __shared__ Segment segments[kWarps][2];
    const ar_kv4_attend_args &a = c.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int *status = static_cast<int *>(a.workspace);

    // Running sum over the requests' chunks: every warp finds its share by itself.
    long long u0, u1, per;
    after_the_stream();
    {
        const int each = (a.requests + kWarps * 32 - 1) / (kWarps * 32);
        const int b0 = min((int)threadIdx.x * each, a.requests), b1 = min(b0 + each, a.requests);
        long long own = 0;
        for (int b = b0; b < b1; ++b) {
            const Request r = request_of<C>(c, b);
            own += r.total(a.kv_heads);
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
        const long long warps = (long long)gridDim.x * kWarps;
        per = max((total + warps - 1) / warps, 1ll);
        // (the block's first share tells whether there is any)
        const long long first = per * kWarps * blockIdx.x;
        if (first < total) {
            long long at = run - own;
            if (at < first + per * kWarps && run > first) {
                for (int b = b0; b < b1; ++b) {
                    const Request r = request_of<C>(c, b);
                    const long long units = r.total(a.kv_heads);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const long long u = first + per * w;
                        if (at <= u && u < at + units) {
                            start_b[w] = b;
                            start_off[w] = u - at;
                            start_u[w] = u;
                        }
                    }
                    at += units;
                }
            }
        }
        u0 = min(first + per * warp, total);
        u1 = min(u0 + per, total);
        __syncthreads();
    }
    const int self = blockIdx.x * kWarps + warp;
    Record *record = reinterpret_cast<Record *>(static_cast<uint8_t *>(a.workspace) + kRecordAt) + self;
    if (lane == 0) record->parts = 0;
    if (u0 >= u1) return;

    // ---- the copies' side: walks the segments, at most one ahead of the products
    uint8_t *ring = smem + warp * S * C::Stage;
    const uint32_t ring_addr = smem_addr(ring), bar_addr = smem_addr(&bars[warp * S]);
    const int tiles_page = a.page / kTileTokens;
    constexpr int kBatch = 32 / CT;
    uint32_t filled = 0, used = 0;       // stages filled and used, over all segments
    int walked = 0;                      // segments walked to
    // Of the segment walked to last: its chunks and how many of them are sent.  Lane l has the address of tile
    // l % CT of its chunk l / CT of a batch, and reads the page ids of the batch after.
    int p_chunks = 0, sent = 0, batch_tile = 0, batch_id = 0;
    const uint8_t *src = nullptr;
    unsigned have = 0;                   // lanes whose tile exists
    auto read_ids = [&](int k) {
        const Segment &s = segments[warp][(walked - 1) & 1];
        k += lane / CT;
        batch_tile = k < p_chunks ? chunk_at(s.c0 + k, s.sink_chunks, s.low_chunk) * CT + lane % CT : s.end_tile;
        batch_id = batch_tile < s.end_tile ? a.table[(long long)s.request * a.table_stride + batch_tile / tiles_page] : 0;
    };
    auto walk = [&]() -> bool {
        __syncwarp();                    // every lane is done with the segment whose place this takes
        int b = start_b[warp];
        long long off = start_off[warp], u = start_u[warp];
        Segment s;
        for (;;) {
            if (u >= u1 || b >= a.requests) return false;     // (the latter only if the lengths changed meanwhile)
            const Request r = request_of<C>(c, b);
            if (off >= r.total(a.kv_heads)) {
                ++b;
                off = 0;
                continue;
            }
            const int length = (int)r.length();
            const int index = off >> 32 ? (int)(off / length) : (int)((unsigned)off / (unsigned)length);
            const int from = (int)(off - (long long)index * length), take = (int)min((long long)(length - from), u1 - u);
            const long long last = u - from + length - 1;
            u += take;
            off += take;
            if (from + take <= kStart) continue;              // no chunk of it
            s.kv = index / r.blocks;
            s.row0 = (index - s.kv * r.blocks) * C::Rows;
            s.rows = min(C::Rows, r.count * c.group - s.row0);
            s.first = r.first;
            s.request = b;
            s.pos0 = r.len - r.count;
            s.pos_lo = s.pos0 + s.row0 / c.group;
            s.pos_hi = s.pos0 + (s.row0 + s.rows - 1) / c.group;
            s.end_tile = s.pos_hi < 0 ? 0 : s.pos_hi / kTileTokens + 1;
            s.low_chunk = a.window ? max(s.pos_lo - a.window + 1, 0) / C::Tokens : 0;
            s.sink_chunks = a.window ? (int)min((long long)s.low_chunk, ((long long)a.sinks + C::Tokens - 1) / C::Tokens) : 0;
            const int seen = s.pos_hi < 0 ? 0 : s.sink_chunks + s.pos_hi / C::Tokens - s.low_chunk + 1;
            s.c0 = max(from - kStart, 0);
            s.chunks = max(min(from + take - kStart, seen) - s.c0, 0);
            s.begins = from <= kStart;
            s.whole = s.begins && from + take == length;
            if (lane == 0 && s.begins && !s.whole) {
                // it goes on in other warps
                record->rows = s.rows; record->kv = s.kv; record->row0 = s.row0; record->first = s.first;
                record->parts = (int)((last >> 32 ? last / per : (unsigned)last / (unsigned)per) - self) + 1;
            }
            break;
        }
        __syncwarp();                    // every lane has read where the walk stood
        if (lane == 0) {
            segments[warp][walked & 1] = s;
            start_b[warp] = b;
            start_off[warp] = off;
            start_u[warp] = u;
        }
        __syncwarp();
        ++walked;
        p_chunks = s.chunks;
        sent = 0;
        read_ids(0);
        return true;
    };
    auto send = [&]() {
        const int in = sent % kBatch * CT;    // first lane of the chunk
        if (in == 0) {
            const Segment &s = segments[warp][(walked - 1) & 1];
            const bool get = batch_tile < s.end_tile;
            have = __ballot_sync(~0u, get);
            int id = batch_id;
            if (get && (id < 0 || id >= a.pages)) {
                atomicCAS(status, 0, AR_EINVAL);
                id = 0;
            }
            src = static_cast<const uint8_t *>(a.pool) +
                  (((long long)id * a.kv_heads + s.kv) * tiles_page + batch_tile % tiles_page) * tile_bytes(D);
            read_ids(sent + kBatch);
        }
        const uint32_t stage = filled % S, bar = bar_addr + 8 * stage, n = __popc((have >> in) & ((1u << CT) - 1));
        if (lane == in)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n * tile_bytes(D)) : "memory");
        __syncwarp();
        if ((unsigned)(lane - in) < n)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             ring_addr + stage * C::Stage + (lane - in) * tile_bytes(D)),
                         "l"(src), "r"((unsigned)tile_bytes(D)), "r"(bar)
                         : "memory");
        ++sent;
        ++filled;
    };

    // q of a segment: column g of tile n is row row0 + 8 n + g; lane t has channels 32 j + 8 t .. + 7
    uint4 raw[NT][G];
    auto read_q = [&](const Segment &s) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = s.row0 + 8 * n + g;
            const bool in = 8 * n + g < s.rows;
            const T *qs = static_cast<const T *>(a.q) + (long long)(s.first + (in ? row / c.group : 0)) * a.q_token_stride +
                          (long long)(s.kv * c.group + (in ? row % c.group : 0)) * a.q_head_stride + 8 * t;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                union { uint4 v; T e[8]; } x;
                x.v = make_uint4(0, 0, 0, 0);
                if (in) {
                    if (c.vec_q) {
                        x.v = *reinterpret_cast<const uint4 *>(qs + 32 * j);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x.e[i] = qs[32 * j + i];
                    }
                }
                raw[n][j] = x.v;
            }
        }
    };

    // ---- the products' side
    uint2 qf[NT][D / 16];
    float mult[NT][2];                    // what a sum of products is worth, in base 2: columns 2 t and 2 t + 1
    float o[D / 16][NT][4];
    float ref[NT][2], l[NT][2];
    int vexp = 0;                         // exponent of the largest V scale so far, at least -80
    float most = 0, vnext = 0;            // what moves the reference: a score, a scale
    int at = -1, next = 0, end = 0;       // the segment multiplied, its next chunk and its end
    int full0 = 0, full1 = 0, full2 = 0;  // every row sees all of its chunks below full0, and from full1 to full2
    auto seg = [&]() -> const Segment & { return segments[warp][at & 1]; };

    // CI tiles of a chunk.  Full: every row sees every token of it.
    auto multiply = [&](auto is_full, const uint8_t *data, int tok0) {
        constexpr bool Full = decltype(is_full)::value;
        float x[CI][NT][4];
#pragma unroll
        for (int ct = 0; ct < CI; ++ct) {
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
                    float acc[4];
                    const uint2 q0 = qf[n][2 * j], q1 = qf[n][2 * j + 1];
                    mma16816(acc, a0, q0.x, q0.y, 0.0f, 0.0f, 0.0f, 0.0f);
                    mma16816(acc, a1, q1.x, q1.y);
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
        // V scales: the largest among tokens that some row sees, infinities and NaN left out
        float vtop = 0;
#pragma unroll
        for (int i = 0; i < (CI * D + 127) / 128; ++i) {
            const int wd = (i * 32 + lane) % (CI * D / 4), ct = wd / (D / 4), in = wd % (D / 4);   // (16 words: each twice)
            uint32_t w = *reinterpret_cast<const uint32_t *>(data + ct * tile_bytes(D) + tile_vs(D) + in * 4);
            if constexpr (!Full) {
                const int tok = tok0 + ct * kTileTokens + in / (G / 2);
                if (tok > seg().pos_hi || (a.window && tok <= seg().pos_lo - a.window && tok >= a.sinks)) w = 0;
            }
            vtop = fmaxf(vtop, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w))));
        }
        // scores under the reference; what a row does not see is -infinity
        if constexpr (!Full) {
#pragma unroll
            for (int ct = 0; ct < CI; ++ct)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = seg().row0 + 8 * n + 2 * t + (i & 1), p = min(seg().pos0 + row / c.group, seg().pos_hi);
                        const int tok = tok0 + ct * kTileTokens + g + (i & 2) * 4;
                        const bool see = tok <= p && (!a.window || tok > p - a.window || tok < a.sinks);
                        x[ct][n][i] = see ? x[ct][n][i] * mult[n][i & 1] : -INFINITY;
                    }
        }
        float y[CI][NT][4];
        float above = kNoScore;
#pragma unroll
        for (int ct = 0; ct < CI; ++ct)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[ct][n][i] = Full ? fmaf(x[ct][n][i], mult[n][i & 1], -ref[n][i & 1]) : x[ct][n][i] - ref[n][i & 1];
                    above = fmaxf(above, y[ct][n][i]);
                }
        if (__any_sync(~0u, vtop >= vnext || above > most)) {
            if (!(vtop < INFINITY)) {
                // an infinite scale spoils its own group; the others keep theirs
                vtop = 0;
#pragma unroll 1
                for (int i = 0; i < 2 * ((CI * D + 127) / 128); ++i) {
                    const int half = (i / 2 * 32 + lane) % (CI * D / 4) * 2 + i % 2, ct = half / (D / 2), in = half % (D / 2),
                              tok = tok0 + ct * kTileTokens + in / G;
                    const float v = fabsf(bf16_bits(*reinterpret_cast<const uint16_t *>(data + ct * tile_bytes(D) + tile_vs(D) + in * 2)));
                    const bool see = Full || (tok <= seg().pos_hi && (!a.window || tok > seg().pos_lo - a.window || tok < a.sinks));
                        if (see && v < INFINITY) vtop = fmaxf(vtop, v);
                }
            }
            vexp = max(vexp, (int)(__reduce_max_sync(~0u, __float_as_uint(vtop)) >> 23) - 127);
            most = (float)(kHead + kLead - vexp);
            vnext = __uint_as_float((uint32_t)(vexp + 128) << 23);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = kNoScore;
#pragma unroll
                    for (int ct = 0; ct < CI; ++ct) top = fmaxf(top, fmaxf(x[ct][n][i], x[ct][n][i + 2]));
                    if constexpr (Full) {
                        // (a product with a negative scale turns the order around)
                        float low = -kNoScore;
#pragma unroll
                        for (int ct = 0; ct < CI; ++ct) low = fminf(low, fminf(x[ct][n][i], x[ct][n][i + 2]));
                        top = fmaxf(top * mult[n][i], low * mult[n][i]);
                    }
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    // the reference never falls: a lower one would let earlier weights overflow
                    const float now = top > kNoScore ? fmaxf(ref[n][i], top + (float)(vexp - kHead)) : ref[n][i];
                    // With V's exponent the reference can move by more than binary32 has exponents (V of zeros before
                    // V of 2^60), while the sums, far from 1 themselves, stay within: so by the factor's root, twice.
                    const float root = exp2_approx((ref[n][i] - now) * 0.5f);
                    ref[n][i] = now;
                    l[n][i] = l[n][i] * root * root;
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        o[m][n][i] = o[m][n][i] * root * root;
                        o[m][n][i + 2] = o[m][n][i + 2] * root * root;
                    }
#pragma unroll
                    for (int ct = 0; ct < CI; ++ct)
#pragma unroll
                        for (int h = i; h < 4; h += 2)
                            y[ct][n][h] = Full ? fmaf(x[ct][n][h], mult[n][i], -now) : x[ct][n][h] - now;
                }
        }
        // weights, and the sum over V
#pragma unroll
        for (int ct = 0; ct < CI; ++ct) {
            const uint8_t *tile = data + ct * tile_bytes(D);
            uint32_t w0[G], w1[G], sc0[G / 2], sc1[G / 2];
            load_words(tile + tile_v(D) + lane * G * 4, w0);
            load_words(tile + tile_v(D) + (32 + lane) * G * 4, w1);
            load_words(tile + tile_vs(D) + g * G * 2, sc0);
            load_words(tile + tile_vs(D) + (g + 8) * G * 2, sc1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (what a row does not see is known by a negative zero from a weight too small to hold)
                    const bool hidden = !Full && y[ct][n][i] == -INFINITY;
                    y[ct][n][i] = hidden ? -0.0f : exp2_approx(y[ct][n][i]);
                }
                l[n][0] += y[ct][n][0] + y[ct][n][2];
                l[n][1] += y[ct][n][1] + y[ct][n][3];
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
                    float p[4] = {y[ct][n][0] * s0, y[ct][n][1] * s0, y[ct][n][2] * s1, y[ct][n][3] * s1};
                    if constexpr (!Full) {
                        // a scale that a row does not see can be anything
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = __float_as_uint(y[ct][n][i]) == 0x80000000u ? 0 : p[i];
                    }
                    const uint32_t b0 = transpose8x8(pack_half(p[0], p[1])), b1 = transpose8x8(pack_half(p[2], p[3]));
                    mma16816(o[2 * j][n], a0, b0, b1);
                    mma16816(o[2 * j + 1][n], a1, b0, b1);
                }
            }
        }
    };


    for (;;) {
        // Fill the free stages, going on into the next segment; at the start one, so that every warp's first
        // data come early.
#pragma unroll 1
        while (filled - used < (at < 0 ? 1 : S)) {
            if (sent < p_chunks) send();
            else if (walked - 1 > at || !walk()) break;
        }
#pragma unroll 1
        while (next < end) {
            const uint32_t stage = used % S;
            if (__any_sync(~0u, !bar_wait(bar_addr + 8 * stage, (used / S) & 1, status))) {
                // A copy that does not come: the warp waits for its others (with the same limit), so that none
                // lands in a stage that is filled anew or after the block has gone, and leaves its share undone.
#pragma unroll 1
                for (uint32_t k = used; k != filled; ++k) (void)bar_wait(bar_addr + 8 * (k % S), (k / S) & 1, status);
                return;
            }
            const uint8_t *data = ring + stage * C::Stage;
            if (next < full0 || (next >= full1 && next < full2)) {
#pragma unroll 1
                for (int i = 0; i < CT; i += CI) multiply(std::true_type(), data + i * tile_bytes(D), 0);
            } else {
                const Segment &s = seg();
                const int tok0 = chunk_at(next, s.sink_chunks, s.low_chunk) * C::Tokens;
#pragma unroll 1
                for (int i = 0; i < CT; i += CI) {
                    const int from = tok0 + i * kTileTokens, to = from + CI * kTileTokens - 1;
                    // (a step that no row sees is left out)
                    if (from <= s.pos_hi && (!a.window || to > s.pos_lo - a.window || from < a.sinks))
                        multiply(std::false_type(), data + i * tile_bytes(D), from);
                }
            }
            ++next;
            ++used;
            __syncwarp();      // every lane has read the stage
            if (sent >= p_chunks) break;
            send();
        }
        if (next < end) continue;

        // The segment's end.  The next one's q comes while the results go.
        const bool more = at + 1 < walked;
        if (more) read_q(segments[warp][(at + 1) & 1]);
        if (at >= 0) {
            const Segment &seg = segments[warp][at & 1];
            // -- results: to their rows, or one part of them to the workspace
            float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kPartAt) +
                          (2 * (size_t)self + (seg.begins ? 1 : 0)) * C::PartFloats;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) l[n][i] += __shfl_xor_sync(~0u, l[n][i], d);
                    const int col = 8 * n + 2 * t + i, row = seg.row0 + col;
                    if (col < seg.rows) {
                        const long long token = seg.first + row / c.group;
                        const int head = seg.kv * c.group + row % c.group;
#pragma unroll
                        for (int j = 0; j < G; ++j) {
                            const float4 v = make_float4(o[2 * j][n][i], o[2 * j][n][i + 2], o[2 * j + 1][n][i], o[2 * j + 1][n][i + 2]);
                            const int channel = 32 * j + 4 * g;
                            if (seg.whole) store_row<T>(c, token, head, channel, v, ref[n][i], l[n][i]);
                            else *reinterpret_cast<float4 *>(part + col * D + channel) = v;
                        }
                        if (!seg.whole && g == 0) *reinterpret_cast<float2 *>(part + C::Rows * D + 2 * col) = make_float2(ref[n][i], l[n][i]);
                    }
                }
            }
        }
        if (!more) break;
        ++at;
        next = seg().c0;
        end = next + seg().chunks;
        full0 = a.window ? min(seg().sink_chunks, a.sinks / C::Tokens) : 0;
        full1 = seg().pos_hi < a.window || !a.window ? seg().sink_chunks - seg().low_chunk
                                                     : seg().sink_chunks - seg().low_chunk + (seg().pos_hi - a.window) / C::Tokens + 1;
        full2 = seg().pos_lo < 0 ? 0 : seg().sink_chunks - seg().low_chunk + (int)(((long long)seg().pos_lo + 1) / C::Tokens);

        // -- operands of q: fp16 of q / 2^e, e the row's own for bfloat16
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[G][8];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                union { uint4 v; T e[8]; } w;
                w.v = raw[n][j];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[j][i] = Elem<T>::to_float(w.e[i]);
                    top = max(top, __float_as_uint(x[j][i]) & 0x7fffffffu);
                }
            }
            float unit = 1, worth = a.scale * 1.4426950408889634f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
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
                qf[n][2 * j] = make_uint2(h[0], h[1]);
                qf[n][2 * j + 1] = make_uint2(h[2], h[3]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) mult[n][i] = __shfl_sync(~0u, worth, (2 * t + i) * 4);
        }

        vexp = -80;
        most = kHead + kLead + 80;
        vnext = __uint_as_float((uint32_t)(128 - 80) << 23);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][n][i] = 0;
            ref[n][0] = ref[n][1] = kNoScore;
            l[n][0] = l[n][1] = 0;
        }
    }
}

// Joins the parts of the segment that begins in a warp, in their order.  A
// block to a warp's record and, by Spread, to one of its rows: then groups of D / 4
// threads share out the parts, for where a few rows have many.

template <typename T, class C, bool Spread, int kJoinThreads = Spread ? 256 : 128>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Attend c) {
    constexpr int D = C::D, Quads = D / 4, Groups = Spread ? kJoinThreads / Quads : 1;
    __shared__ float4 rows[Groups][Quads];
    __shared__ float2 facts[Groups];
    // (no early word to the kernel after: an attention's blocks would take the multiprocessors from this one's)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint8_t *ws = static_cast<const uint8_t *>(c.a.workspace);
    const Record r = reinterpret_cast<const Record *>(ws + kRecordAt)[blockIdx.x];
    if (r.parts == 0 || (Spread && (int)blockIdx.y >= r.rows)) return;
    // part 0 lies in its warp's second place, the others in their warps' first
    const float *base = reinterpret_cast<const float *>(ws + kPartAt) + (2 * (size_t)blockIdx.x + 1) * C::PartFloats;
    const int group = Spread ? threadIdx.x / Quads : 0;
    for (int i = Spread ? blockIdx.y * Quads + threadIdx.x % Quads : threadIdx.x; i < r.rows * Quads; i += kJoinThreads) {
        const int col = i / Quads, quad = i % Quads;
        float m = kNoScore, sum = 0;
        float4 v = make_float4(0, 0, 0, 0);
        constexpr int kAtOnce = 8;
        // The first `count` parts under one reference.  Factors by their roots, twice: the references can be further
        // apart than binary32 has exponents, the sums not.
        auto add = [&](const float2 (&ml)[kAtOnce], const float4 (&y)[kAtOnce], int count) {
            float m2 = m;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e)
                if (e < count) m2 = fmaxf(m2, ml[e].x);
            const float r0 = exp2_approx((m - m2) * 0.5f);
            m = m2;
            sum = sum * r0 * r0;
            v.x = v.x * r0 * r0; v.y = v.y * r0 * r0; v.z = v.z * r0 * r0; v.w = v.w * r0 * r0;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                if (e >= count) break;
                const float r = exp2_approx((ml[e].x - m2) * 0.5f);
                sum = fmaf(ml[e].y * r, r, sum);
                v.x = fmaf(y[e].x * r, r, v.x); v.y = fmaf(y[e].y * r, r, v.y);
                v.z = fmaf(y[e].z * r, r, v.z); v.w = fmaf(y[e].w * r, r, v.w);
            }
        };
        for (int k = group; k < r.parts; k += kAtOnce * Groups) {
            float2 ml[kAtOnce];
            float4 y[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int part = k + e * Groups;
                const float *p = part ? base + (2 * (size_t)part - 1) * C::PartFloats : base;
                if (part < r.parts) {
                    ml[e] = __ldcg(reinterpret_cast<const float2 *>(p + C::Rows * D + 2 * col));
                    y[e] = __ldcg(reinterpret_cast<const float4 *>(p + col * D + 4 * quad));
                }
            }
            add(ml, y, (r.parts - k + Groups - 1) / Groups);
        }
        if constexpr (Spread) {
            rows[group][quad] = v;
            if (quad == 0) facts[group] = make_float2(m, sum);
            __syncthreads();
            if (group > 0) return;
#pragma unroll
            for (int k = 1; k < Groups; k += kAtOnce) {
                float2 ml[kAtOnce];
                float4 y[kAtOnce];
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e) {
                    if (k + e < Groups) {
                        ml[e] = facts[k + e];
                        y[e] = rows[k + e][quad];
                    }
                }
                add(ml, y, Groups - k);
            }
        }
        const int row = r.row0 + col;
        store_row<T>(c, (long long)r.first + row / c.group, r.kv * c.group + row % c.group, 4 * quad, v, m, sum);
        if constexpr (Spread) return;
    }
}

// Up to this many segments a row's parts are many (one request of 262139 tokens: 228 to a row), and a block
// takes one row and shares them out; beyond, a block takes all rows of a record (that request with one kv
// head, parts in one line: 116 us, shared out: 38).
constexpr int kSpreadSegments = 64;

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
            cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kWarps * 32, C::Smem) != cudaSuccess || per_sm < 1 ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return launch_status(cudaErrorUnknown);
        const int fit = (int)((kWorkspaceBytes - kPartAt) / (2 * kWarps * C::PartFloats * 4));
        grid = min(per_sm * sms, min(fit, kMaxWarps / kWarps));
        *(volatile int *)&resident[dev] = grid;
    }
    // No more blocks than the longest contexts the table can hold would fill.
    const long long chunks = max(((long long)c.a.table_width * c.a.page + C::Tokens - 1) / C::Tokens, 1ll);
    const long long blocks = ((long long)c.a.tokens * c.group + C::Rows - 1) / C::Rows + c.a.requests;
    const long long most = (blocks * (chunks + kStart) * c.a.kv_heads + kWarps - 1) / kWarps;
    grid = (int)min((long long)grid, most);
    cudaError_t e = launch_next(attend_kernel<T, C>, dim3((unsigned)grid), kWarps * 32, C::Smem, s, 0, c);
    if (e == cudaSuccess && chunks > 1) {     // one chunk is never split
        const bool spread = (long long)c.a.requests * c.a.kv_heads <= kSpreadSegments;
        const dim3 blocks((unsigned)(grid * kWarps), spread ? C::Rows : 1);
        e = spread ? launch_next(join_kernel<T, C, true>, blocks, 256, 0, s, 0, c) : launch_next(join_kernel<T, C, false>, blocks, 128, 0, s, 0, c);
    }
    return launch_status(e);
}

template <typename T>
int start(const Attend &c, cudaStream_t s) {
    const long long rows = (long long)max(c.a.max_new, 1) * c.group;
    // Chunks of 64 tokens in two or three stages, 3 blocks an SM with one row tile (with chunks of 32 tokens
    // 75 us where this takes 70, 64 ragged requests).  Steps of two tiles: of one 71 us, of four 76, which do
    // not fit the instruction cache.  Two row tiles have room for 2 blocks and steps of one tile (drafts of up
    // to 6 tokens: 51 us, of two 54); three and four row tiles, with q in shared memory, took 69 and 99.
    switch (c.a.head_dim) {
        case 64: return rows <= 8 ? start<T, Shape<64, 1, 4, 2, 3, 3>>(c, s) : start<T, Shape<64, 2, 4, 1, 3, 3>>(c, s);
        case 128: return rows <= 8 ? start<T, Shape<128, 1, 4, 2, 2, 3>>(c, s) : start<T, Shape<128, 2, 4, 1, 2, 2>>(c, s);
        default: return start<T, Shape<256, 1, 1, 1, 5, 2>>(c, s);
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
    if (a.q == a.out) return AR_EINVAL;      // other blocks may still read q when a row is written
    if (!a.q || !a.out || !a.workspace || a.requests < 1 || !a.lens || (!a.table && a.table_width > 0) ||
        (a.table_width > 0 && (!a.pool || a.pages < 1)))
        return AR_EINVAL;
    if (misaligned(a.q, 2) || misaligned(a.out, 2) || misaligned(a.lse, 4) || misaligned(a.pool, 16) || misaligned(a.table, 4) ||
        misaligned(a.lens, 4) || misaligned(a.cu, 4) || misaligned(a.workspace, 256))
        return AR_EINVAL;
    c.group = a.q_heads / a.kv_heads;
    // A window or sinks that cover the table limit nothing; smaller ones and the rows stay where sums fit 32
    // bits.
    const long long room = (long long)a.table_width * a.page;
    if (a.window >= room || a.sinks >= room) c.a.window = 0;
    if ((long long)a.tokens * c.group > 1 << 30 || c.a.window > 1 << 30 || (long long)a.tokens * a.q_heads > 0x7fffffff)
        return AR_ETOOBIG;
    c.vec_q = rows_aligned(a.q, a.q_token_stride, a.q_head_stride);
    c.vec_o = rows_aligned(a.out, a.out_token_stride, a.out_head_stride);
    return a.dtype == AR_F16 ? start<__half>(c, stream) : start<__nv_bfloat16>(c, stream);
}

}  // extern "C"
