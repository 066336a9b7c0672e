// Paged decode attention over the 4-bit pool: out = softmax(q . K scale) V for one query token per
// sequence, each kv head shared by a group of query heads.
//
// The bound is HBM: 20 HD bytes per 16 tokens and kv head. Both products run on mma.sync m16n8k16
// with the 4-bit codes as the A operand and up to 8 query heads as the 8 columns, and no code is
// ever decoded: (word & 0x000f000f) is a pair of subnormal f16 numbers c 2^-24, which the matrix unit
// multiplies exactly, (word & 0x00f000f0) a pair 16 times that and (word & 0x00ff00ff) the sum of both;
// the upper bytes come down by a byte permutation. The scales stay outside:
//   S^T = K Q^T: one f32 sum per (key, head) and 32-element block, sum_i q_i c_i, then
//         s = sum_b d_b sum_b + sum_b m_b (sum_i q_i), the last product one m16n8k8 MMA of the minima
//         with the q sums in two f16 parts, in units (kSumUnit) that keep both in the normal range: 22 bits
//         of every sum, however small beside the head's largest |q| (as subnormal parts, in the codes'
//         units, a score of small sums was off by 2^-8 of itself; the times are the same). q is brought to
//         [2^14, 2^15) by a power of two (exact), elements that meet the 16-fold codes are divided by 16.
//   O^T = V^T P^T: p d_b takes the part of p, as two f16 numbers (22 bits; p alone in f16 would cost
//         as much again as the rounding of the output), the minima are one more MMA whose fifth row
//         of ones gives the sum of p.
// Up to 4 heads: columns 4-7 repeat heads 0-3 and carry the low parts, so the second part is free;
// otherwise each value product runs twice.
//
// The softmax reference is lazy: p = 2^(x - ref) with ref raised (and the sums rescaled) only when
// some x exceeds it by 14 binades, so most tiles need one vote instead of a maximum over lanes.
//
// Codes are not negative: the sums of scaled codes and of minima grow while the values that they stand
// for cancel, and the matrix unit truncates what it adds. Every 8 tiles the minima's sums therefore move
// into the value sums (settle), which keeps the error at that of the output's rounding at any length.
//
// Work is a flat list of places: the tiles (16 tokens of one kv head and one group of up to 8 heads) of
// each segment (a sequence's kv head and group) and kEntry places for entering and leaving it. The list is
// cut into equal windows, one per CTA (two on an SM), whatever the lengths; the 8 warps of a CTA take its
// tiles in turn, each through its own ring of bulk copies, which runs on across the borders of sequences.
// At a border the warps' sums are joined in shared memory. A segment's part that a CTA does not hold whole
// is written to the workspace, and the CTA that takes the last ticket joins the parts in order.
//
// Measured (HD 128, contexts 128 - 8192, 32 heads on 8, batch 32): 47 us, 3.7 TB/s; 8 heads per kv head and
// contexts of 20000 - 40960, batch 16: 70 us, 4.4 TB/s (a copy reaches 6.8). About 360 instructions a tile,
// half of them on the pipe that takes one in two cycles, 55% of the issue slots, 16 warps on an SM (128
// registers each): what bounds it is the latency of a tile's instructions and, for a few tiles a warp, the
// chain length - table - record - join - parts (9.3 us for 2048 tokens). Copies alone take 36 and 59 us.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "ql_internal.h"
#include "ql_kv4_attn.h"
#include "ql_kv4_rec.cuh"

namespace ql {
namespace {

constexpr int kHeads = 8;                 // query heads per tile
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStages = 4;                // tiles of a warp in flight
constexpr int kCtasPerSm = 2;
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float kTop = 14.f;              // log2 of the largest weight before the reference moves
constexpr float kSumUnit = 0x1p-5f;       // of a block's sum of q as an f16 operand: up to 2^20 units, and both of its parts in the normal range
constexpr int kSettle = 8;                // tiles of a warp between two settlings of the sums, a power of two
constexpr int kEntry = 20;                // what a segment costs besides its tiles, in tiles (about 3 us; 10: 6% slower on ragged batches)
constexpr int kLeast = 2 * kWarps;            // the shortest window (2048 tokens on 8 kv heads: 9.5 us, with kWarps 10.2)

constexpr size_t kSlotBytes = (size_t)(128 / 16 + 1) * 32 * sizeof(float4);   // a stored state at HD 128

struct Params {
    const __half* q;
    const uint8_t* pool;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* positions;
    const int32_t* active;
    int batch, n_heads, n_kv, group, chunks;   // chunks: parts of up to 8 heads of a group
    long long maxb, num_blocks;
    float scale_log2;
    bool early;
    __half* out;
    float* slots;       // [2 gridDim.x] stored states: a CTA's part of the segment it starts in and of the one it ends in
    int* tickets;       // [gridDim.x], zero between launches
};

// The matrix instructions are volatile: a plain asm may be moved into a branch that some lanes take.
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with C = z (a quad of zeros).
__device__ __forceinline__ void mma16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, const float (&z)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}
__device__ __forceinline__ void mma8_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0, const float (&z)[4]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%8,%9,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(b0), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}
// The transpose of an 8 x 8 f16 matrix held one row pair per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T>
__device__ __forceinline__ T lds(uint32_t a);
template <>
__device__ __forceinline__ uint32_t lds<uint32_t>(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
template <>
__device__ __forceinline__ uint2 lds<uint2>(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
template <>
__device__ __forceinline__ uint4 lds<uint4>(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
// N consecutive words of a row: one load
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t a) {
    if constexpr (N == 4) {
        const uint4 v = lds<uint4>(a);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = lds<uint2>(a);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = lds<uint32_t>(a);
    }
}

// Wait for phase `parity` of an mbarrier: false after 2 s.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred q;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        if (bar_test(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < kWaitNs);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    return bar_test(bar, parity) || bar_wait_slow(bar, parity);
}

// A warp's running state: the value sums in units of 2^-24 (rows of the lower half c, of the upper half
// c + 16 c' with the code c' of their own: whole bytes, which need no mask), the minima's
// sums (row b < NB) and the weights' sum (row 4), and the references of this lane's two heads.
template <int HD>
struct State {
    float o[HD / 16][4];
    float z[4];
    float ref[2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        z[0] = z[1] = z[2] = z[3] = 0.f;
        ref[0] = ref[1] = -FLT_MAX;
    }
    __device__ __forceinline__ void scale(float f0, float f1) {
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
            o[i][0] *= f0;
            o[i][1] *= f1;
            o[i][2] *= f0;
            o[i][3] *= f1;
        }
        z[0] *= f0;
        z[1] *= f1;
    }
    // The minima's sums move to the value sums. Codes are not negative, so both grow where the values they
    // stand for cancel; the matrix unit truncates what it adds, by more the larger the sum.
    __device__ __forceinline__ void settle(int lane) {
#pragma unroll
        for (int b = 0; b < HD / 32; ++b) {
            const float z0 = __shfl_sync(0xffffffffu, z[0], 4 * b + (lane & 3)), z1 = __shfl_sync(0xffffffffu, z[1], 4 * b + (lane & 3));
#pragma unroll
            for (int i = 2 * b; i < 2 * b + 2; ++i) {
                o[i][0] = fmaf(z0, 0x1p-24f, o[i][0]);
                o[i][1] = fmaf(z1, 0x1p-24f, o[i][1]);
                o[i][2] = fmaf(z0, 0x1p-20f + 0x1p-24f, o[i][2]);
                o[i][3] = fmaf(z1, 0x1p-20f + 0x1p-24f, o[i][3]);
            }
        }
        if (lane < HD / 8) z[0] = z[1] = 0.f;
    }
    // rows of float4 per lane: 0 .. HD / 16 - 1 the value sums, then minima's sums and references
    __device__ __forceinline__ void put(float4* to) const {
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) to[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        to[HD / 16 * 32] = make_float4(z[0], z[1], ref[0], ref[1]);
    }
    // add a state stored by put
    __device__ __forceinline__ void join(const float4* from) {
        const float4 t = from[HD / 16 * 32];
        const float r0 = fmaxf(ref[0], t.z), r1 = fmaxf(ref[1], t.w);
        const float a0 = exp2_fast(ref[0] - r0), a1 = exp2_fast(ref[1] - r1);
        const float b0 = exp2_fast(t.z - r0), b1 = exp2_fast(t.w - r1);
        ref[0] = r0;
        ref[1] = r1;
        z[0] = fmaf(t.x, b0, z[0] * a0);
        z[1] = fmaf(t.y, b1, z[1] * a1);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
            const float4 v = from[i * 32];
            o[i][0] = fmaf(v.x, b0, o[i][0] * a0);
            o[i][1] = fmaf(v.y, b1, o[i][1] * a1);
            o[i][2] = fmaf(v.z, b0, o[i][2] * a0);
            o[i][3] = fmaf(v.w, b1, o[i][3] * a1);
        }
    }
};

// One row of several states joined: value sums v, minima's sums and references t.
struct Slice {
    float4 v, t;
    __device__ __forceinline__ void join(float4 w, float4 u) {
        const float r0 = fmaxf(t.z, u.z), r1 = fmaxf(t.w, u.w);
        const float a0 = exp2_fast(t.z - r0), a1 = exp2_fast(t.w - r1);
        const float b0 = exp2_fast(u.z - r0), b1 = exp2_fast(u.w - r1);
        t = make_float4(fmaf(u.x, b0, t.x * a0), fmaf(u.y, b1, t.y * a1), r0, r1);
        v = make_float4(fmaf(w.x, b0, v.x * a0), fmaf(w.y, b1, v.y * a1), fmaf(w.z, b0, v.z * a0), fmaf(w.w, b1, v.w * a1));
    }
};

// The length of sequence b: 0 for an inactive one or one that does not fit its table.
__device__ __forceinline__ int seq_len(const Params& p, int b) {
    if (p.active && p.active[b] == 0) return 0;
    const long long len = p.context_lens ? (long long)p.context_lens[b] : (long long)p.positions[b] + 1;
    return len < 0 || len > p.maxb * 16 ? 0 : (int)len;
}

// A segment: the tiles blk0 .. blk1 - 1 (of nb) of one (sequence, kv head, chunk of heads) that lie in a
// CTA's window of the list, the CTA's tiles rel and on. In the list a segment is kEntry places for entering
// and leaving it, then its tiles; at: the place of tile 0 in the window (negative where the window starts
// behind it). The same in every lane.
struct Segment {
    int b, s, len, nb, blk0, blk1, rel, at;
    __device__ __forceinline__ bool last(int window) const { return at + nb + kEntry >= window; }
    __device__ __forceinline__ void next(const Params& p, int S, int window) {
        rel += blk1 - blk0;
        at += nb + kEntry;
        if (++s == S) {
            s = 0;
            do {
                ++b;
                len = seq_len(p, b);
            } while (len == 0);
            nb = (len + 15) >> 4;
        }
        blk0 = 0;
        blk1 = min(nb, window - at);
    }
};

// a / b below 2^20, without the call that a division of 64 bits is
__device__ __forceinline__ int quotient(long long a, long long b) {
    int q = (int)__fdividef((float)a, (float)b);
    while (q * b > a) --q;
    while ((q + 1) * b <= a) ++q;
    return q;
}

template <int HD, bool DUP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_attn_kernel(Params p, DevError* err) {
    using R = Kv4<HD>;
    using St = State<HD>;
    constexpr int NB = R::NB, MT = HD / 16, REC = R::BYTES, ROWS = (MT + 1) * 32;
    constexpr int STAGE = REC + 16;                          // a record and the barrier that its copy completes on
    constexpr int MERGE = 9;                                 // parts loaded at a time: those of 128 tiles, and one more
    static_assert(MT <= kWarps, "");
    extern __shared__ __align__(128) unsigned char smem[];   // [warp][stage], then 4 states
    __shared__ Segment ahead[kWarps];                        // where each warp's copies are
    __shared__ struct {                                      // a part written: its CTAs, its (sequence, s)
        int c0, c1, b, s;
    } part[2];                                               // of the segment that the window starts in, of the one it ends in
    __shared__ int complete[2];                              // the part was its segment's last
    const int tid = threadIdx.x;
    int lane;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));       // kept in a register, not read again and again
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the same in every lane, and known to be
    const int gq = lane >> 2, tq = lane & 3;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * STAGE, ring_end = ring + kStages * STAGE;
    float4* const joins = reinterpret_cast<float4*>(smem + kWarps * kStages * STAGE);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(ring + i * STAGE + REC) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (!p.early) pdl_wait();   // every CTA waits before it ends, so that what follows is behind what went before

    // the whole list's length, then this CTA's run of it and the segment that it starts in; a batch of up to
    // 32 takes one round of loads
    const int S = p.n_kv * p.chunks;
    int len0 = 0;
    long long total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        const int len = b < p.batch ? seq_len(p, b) : 0;
        if (b0 == 0) len0 = len;
        if (b < p.batch && len == 0 && blockIdx.x == 0 && warp == 0 && !(p.active && p.active[b] == 0)) {
            const long long l = p.context_lens ? (long long)p.context_lens[b] : (long long)p.positions[b] + 1;
            if (l != 0) record_device_error(err, kErrAttnLength, b, l);
        }
        total += __reduce_add_sync(0xffffffffu, len > 0 ? kEntry + ((len + 15) >> 4) : 0);
    }
    total *= S;
    // the CTAs' windows: total / gridDim.x places, rounded up (by a little more where that is past 32 bits)
    int per = (total >> 31) == 0 ? (int)(((uint32_t)total + gridDim.x - 1) / gridDim.x) : (int)__fdividef((float)total, (float)gridDim.x);
    if ((total >> 31) != 0) per += (per >> 18) + 1;
    per = max(per, kLeast);
    const long long lo = (long long)blockIdx.x * per;
    if (lo >= total) {
        pdl_wait();
        return;
    }
    const int window = (int)(lo + per < total ? per : total - lo);
    Segment sg;
    {
        long long before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int b = b0 + lane;
            const int len = b0 == 0 ? len0 : b < p.batch ? seq_len(p, b) : 0;
            long long incl = (long long)(len > 0 ? kEntry + ((len + 15) >> 4) : 0) * S;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned here = __ballot_sync(0xffffffffu, before + incl > lo);
            if (here) {
                const int l = __ffs(here) - 1;
                sg.b = b0 + l;
                sg.len = __shfl_sync(0xffffffffu, len, l);
                sg.nb = (sg.len + 15) >> 4;
                const long long in = lo - (before + __shfl_sync(0xffffffffu, incl, l) - (long long)(kEntry + sg.nb) * S);
                sg.s = quotient(in, kEntry + sg.nb);
                sg.at = kEntry - (int)(in - (long long)sg.s * (kEntry + sg.nb));
                sg.blk0 = max(0, -sg.at);
                sg.blk1 = min(sg.nb, window - sg.at);
                sg.rel = 0;
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }

    if (sg.blk1 <= sg.blk0) {   // no tile in the window
        pdl_wait();
        return;
    }

    // ---- q's rows for the products' columns
    uint2 qr[NB][2];
    auto load_q = [&](const Segment& g) {
        const int kv = p.chunks == 1 ? g.s : g.s / p.chunks, c = g.s - kv * p.chunks;
        const int nh = min(kHeads, p.group - c * kHeads), h = DUP ? gq & 3 : gq;
        const __half* src = p.q + ((size_t)g.b * p.n_heads + kv * p.group + c * kHeads + (h < nh ? h : 0)) * HD + 4 * tq;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            for (int k = 0; k < 2; ++k) {   // q is 4-byte aligned
                const uint32_t* at = reinterpret_cast<const uint32_t*>(src + 32 * b + 16 * k);
                qr[b][k] = make_uint2(__ldg(at), __ldg(at + 1));
            }
        }
    };

    // ---- the ring: the tiles of this warp (numbers warp, warp + 8, ... of the run), in order
    int pblk, pend;                    // the next tile to copy and the end of its segment; pend 0: none left
    uint32_t pofs;                     // its kv head's place in a block
    int ids, later;                    // block ids: lane l has that of the warp's tile with number 8 l + warp's part in pblk's 256; the next 256
    const uint32_t rec_stride = (uint32_t)p.n_kv * REC;
    const uint32_t elected = lane == 0;
    const unsigned long long policy = l2_evict_first();   // the context is read once per step
    auto blocks = [&](int from) {
        const int at = (from & ~(32 * kWarps - 1)) + kWarps * lane + (from & (kWarps - 1));
        return at < pend ? __ldg(p.block_tables + (size_t)ahead[warp].b * p.maxb + at) : -1;
    };
    auto enter = [&](const Segment& g) {   // the warp's first tile in segment g, if it has one
        pblk = g.blk0 + ((warp - g.rel) & (kWarps - 1));
        pend = g.blk1;
        pofs = (uint32_t)(p.chunks == 1 ? g.s : g.s / p.chunks) * REC;
    };
    auto look = [&]() {
        const Segment& g = ahead[warp];   // its q rows on their way to L2
        const int kv = p.chunks == 1 ? g.s : g.s / p.chunks, c = g.s - kv * p.chunks;
        if (c * kHeads + (lane >> 2) < p.group)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                p.q + ((size_t)g.b * p.n_heads + kv * p.group + c * kHeads + (lane >> 2)) * HD + (lane & 3) * (HD / 4)));
        ids = blocks(pblk);
        later = blocks(pblk + 32 * kWarps);
    };
    auto cross = [&]() {               // past the segment's end: the next one with a tile of this warp
        Segment g = ahead[warp];
        do {
            if (g.last(window)) {
                pend = 0;
                ids = -1;
                return;
            }
            g.next(p, S, window);
            enter(g);
        } while (pblk >= pend);
        __syncwarp();
        if (lane == 0) ahead[warp] = g;
        __syncwarp();
        look();
    };
    unsigned bad = 0;                  // stages without a record (a block id outside the pool, or a failed wait)
    bool dead = false;                 // a wait ran out: no more copies
    // copy the next tile to the stage at rec; what is rare is behind one vote
    auto issue = [&](uint32_t rec) {
        if (pend == 0) return;   // none left
        const int phys = __shfl_sync(0xffffffffu, ids, pblk / kWarps);
        const bool in = (unsigned)phys < (unsigned)p.num_blocks, go = in && bad == 0;
        const uint8_t* const from = p.pool + ((size_t)(unsigned)phys * rec_stride + pofs);
        asm volatile(
            "{\n .reg .pred e;\n setp.ne.u32 e, %5, 0;\n"
            "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
            "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%2], [%3], %1, [%0], %4;\n}" ::"r"(
                rec + REC),
            "r"(REC), "r"(rec), "l"(from), "l"(policy), "r"(go ? elected : 0u)
            : "memory");
        pblk += kWarps;
        if (!__any_sync(0xffffffffu, !go || pblk >= pend || (pblk & (31 * kWarps)) == 0)) return;
        if (!go) {
            const unsigned bit = 1u << ((rec - ring) / STAGE);
            bad = in && !dead ? bad & ~bit : bad | bit;
            if (lane == 0) {
                if (in && !dead) {
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(rec + REC), "r"(REC) : "memory");
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, "
                        "[%3], %4;" ::"r"(rec), "l"(from), "r"(REC), "r"(rec + REC), "l"(policy)
                        : "memory");
                } else {
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(rec + REC) : "memory");
                    if (!dead) record_device_error(err, kErrAttnBlock, (long long)ahead[warp].b * p.maxb + pblk - kWarps, phys);
                }
            }
            __syncwarp();
        }
        if (pblk >= pend) cross();
        else if ((pblk & (31 * kWarps)) == 0) {
            ids = later;
            later = blocks(pblk + 32 * kWarps);
        }
    };
    if (lane == 0) ahead[warp] = sg;
    __syncwarp();
    enter(sg);
    if (pblk < pend) look();
    else cross();
    bool waited = !p.early;
#pragma unroll 1
    for (int i = 0; i < kStages && pend != 0; ++i) {
        if (!waited && pblk >= ahead[warp].nb - 1) {   // the block that holds the newest row
            pdl_wait();
            waited = true;
        }
        issue(ring + i * STAGE);
    }
    if (!waited) pdl_wait();

    St st;
    float zero[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
    uint32_t rec = ring, parity = 0;   // the stage of this warp's next tile, and its barrier's phase
    // lane constants: shared-memory offsets within a record
    const int krow = ((gq >> 1) & 3) | ((gq & 1) << 2);   // the key of this lane's row of the score product
    const uint32_t offK = R::KC + krow * (HD / 2) + 4 * NB * tq;
    const uint32_t offKD = R::KD + krow * NB * 2, offKM = R::KM + krow * NB * 2 + (NB == 4 ? 4 * (tq & 1) : 0);
    const uint32_t offV = R::VC + tq * (HD / 2) + R::vunit(tq, gq);
    const uint32_t offVD = R::VD + tq * NB * 8, offVM = R::VM + tq * NB * 8 + 4 * (gq & (NB - 1));

    // ---- the end of a segment: row w of the joined state (value sums of 16 elements) is warp w's
    const bool has = warp < MT;
    const int row = has ? warp : 0;
    int parts = 0, arrival = 0;   // parts written (1: of the segment the window starts in, 2: of the one it ends in); the first's ticket (thread 0)
    bool deferred = false;        // that ticket is still to be looked at
    auto emit = [&](const Slice& sl, int b, int s) {
        if (!has) return;
        const int kv = p.chunks == 1 ? s : s / p.chunks, c = s - kv * p.chunks;
        const int nh = min(kHeads, p.group - c * kHeads), hc = 2 * tq, eb = warp >> 1;
        const float l0 = __shfl_sync(0xffffffffu, sl.t.x, 16 + tq), l1 = __shfl_sync(0xffffffffu, sl.t.y, 16 + tq);
        const float i0 = l0 > 0.f ? 1.f / l0 : 0.f, i1 = l1 > 0.f ? 1.f / l1 : 0.f;
        const float z0 = __shfl_sync(0xffffffffu, sl.t.x, 4 * eb + tq), z1 = __shfl_sync(0xffffffffu, sl.t.y, 4 * eb + tq);
        __half* o = p.out + ((size_t)b * p.n_heads + kv * p.group + c * kHeads + hc) * HD + 16 * warp + gq;
        if (hc < nh) {
            o[0] = __float2half_rn(fmaf(sl.v.x, 0x1p24f, z0) * i0);
            o[8] = __float2half_rn(fmaf(sl.v.z - sl.v.x, 0x1p20f, z0) * i0);
        }
        if (hc + 1 < nh) {
            o[HD] = __float2half_rn(fmaf(sl.v.y, 0x1p24f, z1) * i1);
            o[HD + 8] = __float2half_rn(fmaf(sl.v.w - sl.v.y, 0x1p20f, z1) * i1);
        }
    };

    for (;;) {
        const int nh = min(kHeads, p.group - (p.chunks == 1 ? 0 : sg.s % p.chunks) * kHeads);
        st.clear();
        float top = kTop;               // log2 of the largest weight
        __half2 dlim = __float2half2_rn(2.f);   // the largest value scale that goes with it
        int blk = sg.blk0 + ((warp - sg.rel) & (kWarps - 1));
        // ---- q as the B operand of the score product
        uint32_t ql[NB][2], qh[NB][2], qz = 0;
        float fac[2];
        if (blk < sg.blk1) {
            const int h = DUP ? gq & 3 : gq;
            load_q(sg);
            __half2 m2 = __float2half2_rn(0.f);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    qr[b][k].x = h < nh ? qr[b][k].x : 0u;
                    qr[b][k].y = h < nh ? qr[b][k].y : 0u;
                    m2 = __hmax2(m2, __hmax2(__habs2(h2(qr[b][k].x)), __habs2(h2(qr[b][k].y))));
                }
            }
            float mx = fmaxf(__low2float(m2), __high2float(m2));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^e brings the largest |q| of the head to [2^14, 2^15): two factors, each an f16 number; exact but
            // for what e = -1 (a largest |q| of 2^15 or more) takes from numbers below 2^-13
            const int e = mx > 0.f && mx < INFINITY ? 14 - ((int)(__float_as_uint(mx) >> 23) - 127) : 0;
            const int e0 = min(e, 14);
            const __half2 up0 = __float2half2_rn(__uint_as_float((uint32_t)(e0 + 127) << 23));
            const __half2 up1 = __float2half2_rn(__uint_as_float((uint32_t)(min(e - e0, 14) + 127) << 23));
            const __half2 up2 = __float2half2_rn(__uint_as_float((uint32_t)(max(e - 28, 0) + 127) << 23));
            const __half2 sixteenth = __float2half2_rn(0.0625f);
            float qs[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float s = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2 x = __hmul2(__hmul2(__hmul2(h2(qr[b][k].x), up0), up1), up2);
                    const __half2 y = __hmul2(__hmul2(__hmul2(h2(qr[b][k].y), up0), up1), up2);
                    s += __low2float(x) + __high2float(x) + (__low2float(y) + __high2float(y));
                    const __half2 lo = __lows2half2(x, y), hi = __highs2half2(x, y);
                    (k ? qh : ql)[b][0] = u32(k ? __hmul2(lo, sixteenth) : lo);
                    (k ? qh : ql)[b][1] = u32(k ? __hmul2(hi, sixteenth) : hi);
                }
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                qs[b] = s * kSumUnit;   // 2^15 at most
            }
            // the sums' high and low f16 parts (22 bits, but 2^-25 at least), opposite the minima of blocks 2 (tq & 1),
            // 2 (tq & 1) + 1
            const float sa = NB == 4 && (tq & 1) ? qs[NB - 2] : qs[0], sb = NB == 4 && (tq & 1) ? qs[NB - 1] : qs[1];
            const __half2 hi2 = __floats2half2_rn(sa, sb);
            const float2 hf = __half22float2(hi2);
            const __half2 lo2 = __floats2half2_rn(sa - hf.x, sb - hf.y);
            qz = NB == 4 ? u32(tq < 2 ? hi2 : lo2) : tq == 0 ? u32(hi2) : tq == 1 ? u32(lo2) : 0u;
            const float f = p.scale_log2 * __uint_as_float((uint32_t)(24 - e + 127) << 23);
            fac[0] = __shfl_sync(0xffffffffu, f, 8 * tq);
            fac[1] = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
        }
        // ---- the tiles, each in three steps
        // scores: S^T of the record at rec, rows keys krow, krow + 8 of this lane, columns heads 2 tq, 2 tq + 1
        auto score = [&](uint32_t rec, float (&s)[4]) {
            uint32_t wa[NB], wb[NB], da[NB / 2], db[NB / 2];
            lds_words(wa, rec + offK);
            lds_words(wb, rec + offK + 8 * (HD / 2));
            lds_words(da, rec + offKD);
            lds_words(db, rec + offKD + 16 * NB);
            mma8_first(s, lds<uint32_t>(rec + offKM), lds<uint32_t>(rec + offKM + 16 * NB), qz, zero);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] *= 0x1p-24f / kSumUnit;   // to the codes' units
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float a[4];
                const uint32_t wa8 = __byte_perm(wa[b], 0u, 0x4341), wb8 = __byte_perm(wb[b], 0u, 0x4341);
                const uint32_t la8 = wa8 & 0x000f000fu, lb8 = wb8 & 0x000f000fu;
                mma16_first(a, wa[b] & 0x000f000fu, wb[b] & 0x000f000fu, la8, lb8, ql[b][0], ql[b][1], zero);
                // the upper codes of the upper bytes as a difference (exact): another pipe than the masks'
                mma16(a, wa[b] & 0x00f000f0u, wb[b] & 0x00f000f0u, u32(__hsub2(h2(wa8), h2(la8))), u32(__hsub2(h2(wb8), h2(lb8))), qh[b][0], qh[b][1]);
                const float2 d0 = __half22float2(h2(da[b / 2])), d1 = __half22float2(h2(db[b / 2]));
                const float x0 = b & 1 ? d0.y : d0.x, x1 = b & 1 ? d1.y : d1.x;
                s[0] = fmaf(x0, a[0], s[0]);
                s[1] = fmaf(x0, a[1], s[1]);
                s[2] = fmaf(x1, a[2], s[2]);
                s[3] = fmaf(x1, a[3], s[3]);
            }
        };
        // weights: p = 2^(s fac - ref) in two f16 parts, keys down the columns of the B operand
        uint32_t ph[2], plo[2];
        auto weigh = [&](uint32_t rec, int blk_, float (&s)[4]) {
            float t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = fmaf(s[k], fac[k & 1], -st.ref[k & 1]);
            const int left = sg.len - 16 * blk_;
            if (left < 16 || bad != 0) {   // slots past the context, or a block that is not there: any bytes
                const int valid = (bad >> ((rec - ring) / STAGE)) & 1u ? 0 : left;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if ((k < 2 ? krow : krow + 8) >= valid) {
                        t[k] = -INFINITY;
                        s[k] = NAN;   // left out of every maximum
                    }
                }
                // their value scales and minima become 0 (slot lane & 15: VD for lanes 0-15, VM for the others)
                const uint32_t at = rec + (lane < 16 ? R::VD : R::VM) + 2 * R::vscale(lane & 15, 0);
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    asm volatile("{\n .reg .pred q;\n setp.ge.s32 q, %1, %2;\n @q st.shared.u16 [%0], %3;\n}" ::"r"(at + 4 * b),
                                 "r"(lane & 15), "r"(valid), "h"((uint16_t)0) : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy into this stage
                __syncwarp();
            }
            // the value scales of slots tq, tq + 4 and tq + 8, tq + 12
            uint32_t vd[2][NB];
            lds_words(vd[0], rec + offVD);
            lds_words(vd[1], rec + offVD + 4 * NB);
            uint32_t large = 0;   // a scale of 2 or more (or a NaN) has bit 14 set
#pragma unroll
            for (int b = 0; b < NB; ++b) large |= vd[0][b] | vd[1][b];
            const float over = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
            if (__any_sync(0xffffffffu, over > top || (large & 0x40004000u) != 0)) {
                __half2 dmax = __hmax2(h2(vd[0][0]), h2(vd[1][0]));
#pragma unroll
                for (int b = 1; b < NB; ++b) dmax = __hmax2(dmax, __hmax2(h2(vd[0][b]), h2(vd[1][b])));
                if (__any_sync(0xffffffffu, over > top || !__hble2(dmax, dlim))) {
                    float m0 = fmaxf(s[0] * fac[0], s[2] * fac[0]), m1 = fmaxf(s[1] * fac[1], s[3] * fac[1]);
                    float dw = fmaxf(__low2float(dmax), __high2float(dmax));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                    }
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) dw = fmaxf(dw, __shfl_xor_sync(0xffffffffu, dw, o));
                    // p and p d stay below 2^15: the largest scale is at most 2^(15 - top). Above 2^14 (top = 1) every tile
                    // with such a scale comes here, and has weights of 2^-5 at most then
                    const float old = top;
                    float lim = __low2float(dlim);
                    while (top > 1.f && dw > lim) {
                        top -= 1.f;
                        lim *= 2.f;
                    }
                    dlim = __float2half2_rn(lim);
                    // the largest weight so far becomes 2^(top - 6): room for 6 binades before the next move
                    const float r0 = fmaxf(st.ref[0] + (old - top), m0 - top + 6.f), r1 = fmaxf(st.ref[1] + (old - top), m1 - top + 6.f);
                    st.scale(exp2_fast(st.ref[0] - r0), exp2_fast(st.ref[1] - r1));
                    st.ref[0] = r0;
                    st.ref[1] = r1;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (t[k] != -INFINITY) t[k] = fmaf(s[k], fac[k & 1], -st.ref[k & 1]);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float p0 = exp2_fast(t[2 * k]), p1 = exp2_fast(t[2 * k + 1]);
                const __half2 hi2 = __floats2half2_rn(p0, p1);
                const float2 hf = __half22float2(hi2);
                ph[k] = transposed(u32(hi2));
                plo[k] = transposed(u32(__floats2half2_rn(p0 - hf.x, p1 - hf.y)));
            }
        };
        // values: O^T, A rows elements gq (+ 8, as whole bytes) of a 16-element half block, its columns the slots
        auto value = [&](uint32_t rec) {
            uint32_t v[4][NB / 2], vd[2][NB];
            lds_words(vd[0], rec + offVD);
            lds_words(vd[1], rec + offVD + 4 * NB);
            const uint32_t vm0 = lds<uint32_t>(rec + offVM), vm1 = lds<uint32_t>(rec + offVM + 4 * NB);   // minima of block gq
#pragma unroll
            for (int k = 0; k < 4; ++k) lds_words(v[k], rec + offV + k * 4 * (HD / 2));
            const bool low = DUP && gq >= 4;
            {
                const uint32_t one = gq == 4 ? 0x3c003c00u : 0u;
                const uint32_t a0 = gq < NB ? vm0 : one, a2 = gq < NB ? vm1 : one;
                mma16(st.z, a0, 0u, a2, 0u, low ? plo[0] : ph[0], low ? plo[1] : ph[1]);
                if (!DUP) mma16(st.z, a0, 0u, a2, 0u, plo[0], plo[1]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t ph_[2], pl_[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2 d = h2(vd[k][b]);
                    const __half2 hi2 = __hmul2(h2(ph[k]), d);
                    // the product's rounding, exactly, and the low part's product
                    const __half2 lo2 = __hfma2(h2(plo[k]), d, __hfma2(h2(ph[k]), d, __hneg2(hi2)));
                    ph_[k] = low ? u32(lo2) : u32(hi2);
                    pl_[k] = u32(lo2);
                }
                const uint32_t x = __byte_perm(v[0][b / 2], v[1][b / 2], b & 1 ? 0x7632 : 0x5410);
                const uint32_t y = __byte_perm(v[2][b / 2], v[3][b / 2], b & 1 ? 0x7632 : 0x5410);
                const uint32_t x8 = __byte_perm(x, 0u, 0x4341), y8 = __byte_perm(y, 0u, 0x4341);
                const uint32_t x0 = x & 0x000f000fu, x1 = x & 0x00ff00ffu, y0 = y & 0x000f000fu, y1 = y & 0x00ff00ffu;
                const uint32_t x2 = x8 & 0x000f000fu, y2 = y8 & 0x000f000fu;
                mma16(st.o[2 * b], x0, x1, y0, y1, ph_[0], ph_[1]);
                mma16(st.o[2 * b + 1], x2, x8, y2, y8, ph_[0], ph_[1]);
                if (!DUP) {
                    mma16(st.o[2 * b], x0, x1, y0, y1, pl_[0], pl_[1]);
                    mma16(st.o[2 * b + 1], x2, x8, y2, y8, pl_[0], pl_[1]);
                }
            }
        };
        auto arrived = [&]() {   // the record at rec
            if (!__all_sync(0xffffffffu, bar_test(rec + REC, parity)) && !__all_sync(0xffffffffu, bar_wait_slow(rec + REC, parity))) {
                if (!dead && lane == 0) record_device_error(err, kErrAttnStage, sg.b, blk);
                dead = true;
                bad = ~0u;
            }
            __syncwarp();
        };
        auto advance = [&]() {
            rec += STAGE;
            if (rec == ring_end) {
                rec = ring;
                parity ^= 1u;
            }
        };
        // the scores of a tile beside the values of the one before it: two independent chains
        if (blk < sg.blk1) {
            float s[4];
            arrived();
            score(rec, s);
            weigh(rec, blk, s);
#pragma unroll 1
            for (blk += kWarps; blk < sg.blk1; blk += kWarps) {
                const uint32_t old = rec;
                advance();
                arrived();
                score(rec, s);
                value(old);
                __syncwarp();   // every lane is done with the record
                issue(old);
                weigh(rec, blk, s);
                if ((blk & (kSettle * kWarps - kWarps)) == 0) st.settle(lane);
            }
            value(rec);
            __syncwarp();
            issue(rec);
            advance();
        }
        if (DUP) {   // the low parts' columns join the high ones
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[i][k] += __shfl_xor_sync(0xffffffffu, st.o[i][k], 2);
            st.z[0] += __shfl_xor_sync(0xffffffffu, st.z[0], 2);
            st.z[1] += __shfl_xor_sync(0xffffffffu, st.z[1], 2);
        }
        // ---- the warps' states join: 4 to 7 with 0 to 3, then row w of those four by warp w
        float4* mine = joins + (size_t)(warp & 3) * ROWS + lane;
        __syncthreads();
        if (warp >= 4) st.put(mine);
        __syncthreads();
        if (warp < 4) {
            st.join(mine);
            __syncwarp();
            st.put(mine);
        }
        __syncthreads();
        Slice sl;
        sl.v = joins[row * 32 + lane];
        sl.t = joins[MT * 32 + lane];
#pragma unroll
        for (int k = 1; k < 4; ++k) sl.join(joins[k * ROWS + row * 32 + lane], joins[k * ROWS + MT * 32 + lane]);
        if (sg.blk1 - sg.blk0 == sg.nb) emit(sl, sg.b, sg.s);
        else {
            const int end = sg.blk0 == 0 ? 1 : 0;
            float4* to = reinterpret_cast<float4*>(p.slots) + (2 * (size_t)blockIdx.x + end) * ROWS + lane;
            if (has) __stcg(to + row * 32, sl.v);
            if (warp == 0) __stcg(to + MT * 32, sl.t);
            const bool more = !sg.last(window);
            const int c0 = quotient(lo + sg.at, per), c1 = quotient(lo + sg.at + sg.nb - 1, per);
            __syncthreads();
            if (tid == 0) {   // releases the CTA's part (ordered by the barrier)
                part[end] = {c0, c1, sg.b, sg.s};
                int n;
                if (more) {   // the answer is not looked at before the end
                    asm volatile("atom.add.release.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(p.tickets + c0) : "memory");
                    arrival = n;
                } else {      // acquires the others' parts, where theirs came before
                    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(p.tickets + c0) : "memory");
                    complete[end] = n == c1 - c0;
                }
            }
            if (more) deferred = true;
            parts |= 1 + end;
        }
        if (sg.last(window)) break;
        sg.next(p, S, window);
    }
    pdl_trigger();   // not before: the next grid's CTAs would take the room of this one's (a decode step of 36 layers 26 us longer)
    if (parts) {   // (the same in every thread)
        if (tid == 0) {
            if (deferred) {
                complete[0] = arrival == part[0].c1 - part[0].c0;
                asm volatile("fence.acq_rel.gpu;" ::: "memory");
            }
            if ((parts & 1) && complete[0]) p.tickets[part[0].c0] = 0;   // armed for the next launch
            if ((parts & 2) && complete[1]) p.tickets[part[1].c0] = 0;
        }
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (!(parts >> i & 1) || !complete[i]) continue;
            // this CTA's part came last: all of them, in order
            const int c0 = part[i].c0, c1 = part[i].c1;
            Slice sl;
#pragma unroll 1
            for (int k0 = c0; k0 <= c1; k0 += MERGE) {
                float4 v[MERGE], t[MERGE];
#pragma unroll
                for (int k = 0; k < MERGE; ++k) {
                    const int c = min(k0 + k, c1);
                    const float4* from = reinterpret_cast<const float4*>(p.slots) + (2 * (size_t)c + (c == c0 ? 1 : 0)) * ROWS + lane;
                    v[k] = __ldcg(from + row * 32);
                    t[k] = __ldcg(from + MT * 32);
                }
#pragma unroll
                for (int k = 0; k < MERGE; ++k) {
                    if (k0 + k > c1) break;
                    if (k0 + k == c0) {
                        sl.v = v[k];
                        sl.t = t[k];
                    } else sl.join(v[k], t[k]);
                }
            }
            emit(sl, part[i].b, part[i].s);
        }
    }
    if (dead) {   // copies may still be in flight: wait for them (again with a limit) before leaving
        for (int i = 0; i < kStages; ++i) {
            bar_wait(rec + REC, parity);
            rec += STAGE;
            if (rec == ring_end) {
                rec = ring;
                parity ^= 1u;
            }
        }
    }
}

template <int HD>
constexpr size_t attn_smem() {
    return (size_t)kWarps * kStages * (Kv4<HD>::BYTES + 16) + (size_t)(kWarps / 2) * (HD / 16 + 1) * 32 * sizeof(float4);
}

int attn_grid() { return kCtasPerSm * num_sms(); }

template <int HD, bool DUP>
cudaError_t attn_go(const Params& p, int grid, cudaStream_t s, bool pdl, DevError* err) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem_once(kv4_attn_kernel<HD, DUP>, attn_smem<HD>(), done);
    return e == cudaSuccess ? launch(kv4_attn_kernel<HD, DUP>, dim3((unsigned)grid), dim3(kThreads), attn_smem<HD>(), s, pdl, p, err)
                            : e;
}

}  // namespace

size_t kv4_attn_workspace_bytes() {
    const size_t g = (size_t)attn_grid();
    return 2 * g * kSlotBytes + g * sizeof(int);
}

int kv4_attn_launch(const Kv4AttnArgs& a, cudaStream_t s, bool pdl) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "4-bit attention: no device error record");
    const int grid = attn_grid();
    Params p = {};
    p.q = a.q;
    p.pool = a.pool;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.positions = a.positions;
    p.active = a.active;
    p.batch = a.batch;
    p.n_heads = a.n_heads;
    p.n_kv = a.n_kv_heads;
    p.group = a.n_heads / a.n_kv_heads;
    p.chunks = (p.group + kHeads - 1) / kHeads;
    p.maxb = a.max_blocks_per_seq;
    p.num_blocks = a.num_blocks;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.early = pdl && a.early;
    p.out = a.out;
    p.slots = static_cast<float*>(a.workspace);
    p.tickets = reinterpret_cast<int*>(static_cast<char*>(a.workspace) + 2 * (size_t)grid * kSlotBytes);
    const bool dup = p.group <= 4;
    const cudaError_t e = a.head_dim == 128
                              ? (dup ? attn_go<128, true>(p, grid, s, pdl, err) : attn_go<128, false>(p, grid, s, pdl, err))
                              : (dup ? attn_go<64, true>(p, grid, s, pdl, err) : attn_go<64, false>(p, grid, s, pdl, err));
    return e == cudaSuccess ? QL_OK : cuda_error(e, "4-bit attention launch");
}

}  // namespace ql

extern "C" size_t ql_paged_attn_kv4_workspace_bytes(int64_t batch, int n_heads, int n_kv_heads, int head_dim,
                                                    int64_t max_blocks_per_seq) {
    if (batch < 1 || n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || (head_dim != 64 && head_dim != 128) ||
        max_blocks_per_seq < 1)
        return 0;
    return ql::kv4_attn_workspace_bytes();
}

extern "C" int ql_paged_attn_decode_kv4(const void* d_q, const void* d_pool, const int32_t* d_block_tables,
                                        const int32_t* d_context_lens, int64_t batch, int n_heads, int n_kv_heads,
                                        int head_dim, int block_size, int64_t max_blocks_per_seq, int64_t num_blocks,
                                        float scale, void* d_out, void* d_workspace, size_t workspace_bytes,
                                        void* stream) {
    using namespace ql;
    const char* nm = "ql_paged_attn_decode_kv4";
    QL_REQUIRE(d_q && d_pool && d_block_tables && d_context_lens && d_out && d_workspace, std::string(nm) + ": null pointer");
    QL_REQUIRE(head_dim == 64 || head_dim == 128, std::string(nm) + ": head_dim must be 64 or 128");
    QL_REQUIRE(block_size == 16, std::string(nm) + ": block_size must be 16");
    QL_REQUIRE(n_heads > 0 && n_heads <= (1 << 20) && n_kv_heads > 0 && n_heads % n_kv_heads == 0,
               std::string(nm) + ": n_heads must be a multiple of n_kv_heads, 2^20 at most");
    QL_REQUIRE(batch >= 1 && batch <= 65535 && batch * n_heads < (1ll << 31) / 128, std::string(nm) + ": batch out of range");
    QL_REQUIRE(max_blocks_per_seq >= 1 && max_blocks_per_seq < kKv4MaxBlocks && num_blocks >= 1 && num_blocks < (1ll << 31),
               std::string(nm) + ": bad table or pool size");
    QL_REQUIRE(batch * max_blocks_per_seq < (1ll << 38) / n_heads, std::string(nm) + ": batch * max_blocks_per_seq out of range");
    QL_REQUIRE((reinterpret_cast<uintptr_t>(d_pool) & 15) == 0 && (reinterpret_cast<uintptr_t>(d_workspace) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(d_q) & 3) == 0 && (reinterpret_cast<uintptr_t>(d_out) & 3) == 0,
               std::string(nm) + ": the pool and the workspace must be 16-byte aligned, q and the output 4-byte aligned");
    QL_REQUIRE((reinterpret_cast<uintptr_t>(d_block_tables) & 3) == 0 && (reinterpret_cast<uintptr_t>(d_context_lens) & 3) == 0,
               std::string(nm) + ": misaligned block tables or lengths");
    QL_REQUIRE(workspace_bytes >= kv4_attn_workspace_bytes(),
               std::string(nm) + ": workspace too small");
    Kv4AttnArgs a = {};
    a.q = static_cast<const __half*>(d_q);
    a.pool = static_cast<const uint8_t*>(d_pool);
    a.block_tables = d_block_tables;
    a.context_lens = d_context_lens;
    a.batch = (int)batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.scale = scale;
    a.out = static_cast<__half*>(d_out);
    a.workspace = d_workspace;
    a.workspace_bytes = workspace_bytes;
    return kv4_attn_launch(a, static_cast<cudaStream_t>(stream), true);
}
