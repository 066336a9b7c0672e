// Latent attention of a prompt chunk over the paged cache, in the expanded form:
//
//  1. mla_expand_kernel: every head's keys k = Wk_h c and values v = Wv_h c of the whole context, f16, by a tcgen05 product over
//     the cache's rows (256 tokens x 256 outputs a pair of CTAs), and the rotated key parts laid out beside them;
//  2. mla_chunk_kernel: causal attention of 256 queries of one head by a pair of CTAs, the online softmax over tiles of 128 keys in
//     two independent halves of the tiles (even and odd), so that one half's products run beside the other's weights;
//  3. mla_chunk_join_kernel, where units are cut: their parts joined.
#include "ql_batched.h"
#include "ql_mla_tc.cuh"

#include <algorithm>

namespace ql {
namespace mla {

constexpr int kQ = 128;     // queries of a CTA, keys of a tile
constexpr float kLow = 5.f; // log2 of the least that a row's largest weight may be with the reference that most rows begin with

// ---------------------------------------------------------------- keys and values
struct ExpandParams {
    CUtensorMap tc;         // the pool: [token][rank + 64]
    CUtensorMap tw;         // weights: [head, row][rank]
    CUtensorMap tk, tv;     // keys, values: [head, token][D], boxes of 32 tokens x 64
    const __half* pool;
    const int32_t* table;
    const int32_t* position;
    __half* turned;         // [cap][64]
    int* live;              // [cap / 128]: a bit per block of 16 tokens: it is in the pool
    long long maxb, num_blocks, cap;
    int n, H;
    DevError* err;
    unsigned long long ns;
};

// Tokens of the context with the chunk, 0 where the position does not fit the table.
__device__ __forceinline__ long long context(const int32_t* position, int n, long long maxb) {
    const long long p = __ldcg(position);
    return p >= 0 && p + n <= maxb * kBlock ? p + n : 0;
}

// A warp's 32 tokens, a lane each (`live`: its block is in the pool): whether a value of the lane's latent vector is NaN or an infinity.
template <int R>
__device__ __forceinline__ bool latent_broken(const __half* pool, bool live, int id, long long tok, int lane) {
    bool broken = false;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {   // a row at a time, by the whole warp
        const bool is = __shfl_sync(0xffffffffu, live, i);
        const long long row = (long long)__shfl_sync(0xffffffffu, id, i) * kBlock + __shfl_sync(0xffffffffu, (int)(tok % kBlock), i);
        bool bad = false;
#pragma unroll
        for (int k = 0; k < R / 256; ++k) {
            const uint4 v = is ? __ldg(reinterpret_cast<const uint4*>(pool + row * (R + kRope)) + 32 * k + lane) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) bad |= (u[j] & 0x7c00u) == 0x7c00u || (u[j] & 0x7c000000u) == 0x7c000000u;
        }
        const bool any = __any_sync(0xffffffffu, bad);
        if (lane == i) broken = any;
    }
    return broken;
}

// A pair of CTAs multiplies 256 tokens (128 in each) with 256 weight rows (half of them in each): 64 bytes a cycle and SM
// of operands read from shared memory, where a CTA alone reads 96 beside the 128 that it would have to take in from L2 (one CTA a
// product of 128 x 256: 53.6 us for 4096 tokens and 32 heads, bound by L2). The tokens stay in shared memory for all the heads of
// a pair's share of the work; the weights stream through a ring. 32 heads of 128, rank 512: 8192 tokens 46 us (1.49 PFLOP/s), 4096 tokens 31 us.
// A product of 256 x 256 x 512 takes 4700 cycles of the 4100 that its instructions need; the first one's operands arrive 5 us after the launch,
// and 14 (or 7) rounds of 76 pairs do not come out even. Not bound by the weights' reads (without half of them: 1.5 us less) nor by the stores
// alone (6 us less without any). Keys and values are rounded to f16, as the attention's operands have to be; sums are f32.
template <int D, int R>
struct ExpandCfg {
    static constexpr int HEADS = 128 / D;                  // heads of a product: 256 outputs
    static constexpr int KC = R / 64;                      // runs of 64 latent values
    static constexpr int STAGES = R == 512 ? 5 : 8, AB = 128 * 128, BB = 128 * 128, OB = 32 * 128;   // OB: 64 outputs of a warp's 32 tokens
    // (with rank 512 a fifth stage is worth more than eight storing warps' room: 49.7 instead of 52.6 us; with 256, 11.5 instead of 13)
    static constexpr int kOut = R == 512 ? 4 : 8, kCopy = kOut, kProduct = kOut + 1, THREADS = (kOut + 2) * 32;   // warps
    static constexpr size_t SMEM = (size_t)KC * AB + (size_t)STAGES * BB + kOut * OB;
    // what has landed in either CTA is reported to rank 0's barriers, what has been read to both CTAs'
    static constexpr int kAFull = 0, kBFull = KC, kBEmpty = kBFull + STAGES, kAEmpty = kBEmpty + STAGES, kDFull = kAEmpty + KC, kDEmpty = kDFull + 2, kDone = kDEmpty + 2, kBars = kDone + 1;
    static_assert(SMEM + 2048 <= 232448, "shared memory");
};

// The pair's copies in flight, after an abort.
template <typename C>
__device__ __noinline__ void settle_expand(uint32_t bar, uint32_t issued, DevError* err, unsigned long long ns) {
    if (cluster_rank() == 0 && threadIdx.x == 32 * C::kCopy) {
        const Waits alone = {err, nullptr, ns};
        settle_ring(bar + C::kAFull * 8, C::KC, issued, C::AB, alone, 702);
        settle_ring(bar + C::kBFull * 8, C::STAGES, issued + 4, C::BB, alone, 703);
    }
    __syncthreads();
    cluster_sync();
}

template <int D, int R>
__global__ void __launch_bounds__(ExpandCfg<D, R>::THREADS, 1) __cluster_dims__(2, 1, 1) mla_expand_kernel(const __grid_constant__ ExpandParams p) {
    using C = ExpandCfg<D, R>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[C::kBars];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ int issued[2];   // copies of the tokens' runs, of the weights
    const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t bar = su32(bars), as = su32(smem), bs = as + C::KC * C::AB;
    if (t == 0) {
        for (int i = 0; i < C::kBars; ++i) bar_init(bar + i * 8, i == C::kDEmpty || i == C::kDEmpty + 1 ? 2 * C::kOut : 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tc);
        prefetch_map(&p.tw);
    }
    if (warp == C::kProduct) tmem_alloc2<512>(&tmem_at);
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, tmem_at, 0);
    const PairWaits wt = {{p.err, &abort_flag, p.ns}};
    const Waits alone = {p.err, nullptr, p.ns};
    pdl_wait();
    pdl_trigger();   // not before this CTA has its tensor memory: the attention, which takes all of it, waits for this grid's end
    const long long L = context(p.position, p.n, p.maxb);
    if (L == 0 && t == 0 && blockIdx.x == 0) record_device_error(p.err, kErrAttnLength, 0, __ldg(p.position));
    // this pair's run of (256 tokens, 256 outputs), the tokens outside
    const int hgs = (p.H + C::HEADS - 1) / C::HEADS, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int units = (int)((L + 255) / 256) * hgs, each = units / pairs, more = units % pairs;   // (below 2^22)
    const int u0 = __shfl_sync(0xffffffffu, pair * each + min(pair, more), 0), u1 = __shfl_sync(0xffffffffu, u0 + each + (pair < more), 0);

    const uint32_t there = in_cta(bar, 0);
    if (warp == C::kCopy) {
        // ------------------------------------------------ copies: a block of 16 tokens a lane, the weights by lane 0
        const long long nblk = (L + kBlock - 1) / kBlock;
        int held = -1, loads = 0, it = 0, runs = 0;
        bool ok = true;
        int tp = u0 / hgs, hg = u0 - tp * hgs;
        for (int u = u0; u < u1 && ok; ++u, hg = hg + 1 == hgs ? 0 : hg + 1, tp += hg == 0) {
            const bool fresh = tp != held;
            int row = 0;
            if (fresh) {
                const long long at = (long long)tp * 16 + 8 * rank + lane;
                bool live = false;
                int id = -1;
                if (lane < 8 && at < nblk) {
                    id = __ldg(p.table + at);
                    live = id >= 0 && id < p.num_blocks;
                    if (!live && hg == 0) record_device_error(p.err, kErrAttnBlock, at, id);
                }
                const unsigned mask = __ballot_sync(0xffffffffu, live);
                if (lane == 0 && hg == 0) p.live[2 * tp + rank] = (int)mask;
                row = live ? id * kBlock : (int)(p.num_blocks * kBlock);   // outside: zeros
                held = tp;
                ++loads;
            }
            for (int c = 0; c < C::KC; ++c) {   // (behind a wait that failed nothing is armed or issued)
                const int s = it % C::STAGES;
                if (fresh) {   // a run of the tokens' values makes room as its last product ends
                    ok = loads < 2 || warp_wait(bar + (C::kAEmpty + c) * 8, (uint32_t)loads & 1u, wt, 700);
                    if (!ok) break;
                    ++runs;
                    if (lane == 0 && rank == 0) bar_expect(bar + (C::kAFull + c) * 8, 2 * C::AB);
                    __syncwarp();
                    if (lane < 8) copy2_box2(as + c * C::AB + lane * 2048, &p.tc, 64 * c, row, there + (C::kAFull + c) * 8);
                }
                ok = it < C::STAGES || warp_wait(bar + (C::kBEmpty + s) * 8, (uint32_t)(it / C::STAGES - 1) & 1u, wt, 701);
                if (!ok) break;
                ++it;
                if (lane == 0) {
                    if (rank == 0) bar_expect(bar + (C::kBFull + s) * 8, 2 * C::BB);
                    copy2_box2(bs + s * C::BB, &p.tw, 64 * c, hg * 256 + 128 * rank, there + (C::kBFull + s) * 8);
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            issued[0] = runs;
            issued[1] = it;
        }
    } else if (warp == C::kProduct) {
        // ------------------------------------------------ products of both CTAs, issued by rank 0
        constexpr uint32_t I = instr(256, 256, false, false);
        const uint32_t one = elect_one();
        const uint64_t ad = operand(as, 16, 1024, 2), bd = operand(bs, 16, 1024, 2);
        int hg = u0 % hgs, loads = 0, s = 0;
        uint32_t phase = 0;                     // of the ring's stage s
        bool ok = rank == 0;
        for (int n = 0; n < u1 - u0 && ok; ++n) {
            const bool fresh = n == 0 || hg == 0;
            hg = hg + 1 == hgs ? 0 : hg + 1;
            const bool last = hg == 0 && n + 1 < u1 - u0;
            loads += fresh;
            for (int c = 0; c < C::KC; ++c) {
                if (fresh) ok = warp_wait(bar + (C::kAFull + c) * 8, (uint32_t)(loads - 1) & 1u, wt, 711);
                ok = ok && warp_wait(bar + (C::kBFull + s) * 8, phase, wt, 712);
                if (c == 0 && n >= 2) ok = ok && warp_wait(bar + (C::kDEmpty + (n & 1)) * 8, (uint32_t)((n >> 1) - 1) & 1u, wt, 710);
                if (!ok) break;
                fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma2_ss(one, tb + 256 * (n & 1), ad + ((c * C::AB + 32 * k) >> 4), bd + ((s * C::BB + 32 * k) >> 4), I, c > 0 || k > 0);
                mma2_commit(one, bar + (C::kBEmpty + s) * 8);
                if (last) mma2_commit(one, bar + (C::kAEmpty + c) * 8);
                if (++s == C::STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            mma2_commit(one, bar + (C::kDFull + (n & 1)) * 8);
        }
        if (rank == 0) {
            mma2_commit(one, bar + C::kDone * 8);
            warp_wait(bar + C::kDone * 8, 0u, alone, 715);
        }
    } else {
        // ------------------------------------------------ a token a thread: its 256 outputs, or 128 of them, rounded and stored
        unsigned char* stage = smem + C::KC * C::AB + C::STAGES * C::BB + warp * C::OB + lane * 128;
        int n = 0;
        bool broken = false;   // A token of the chunk whose latent vector holds NaN or an infinity: NaN as key for those who see it, 0 as value
                               // for those whose weight of it is 0.
        int tp = u0 / hgs, hg = u0 - tp * hgs;
        for (int u = u0; u < u1; ++u, ++n, hg = hg + 1 == hgs ? 0 : hg + 1, tp += hg == 0) {
            const int b = n & 1;
            const long long tok = (long long)tp * 256 + 128 * rank + 32 * (warp & 3) + lane;
            const bool in = tok < L;   // rows behind the context are zeros: what its last block holds there must not meet the weights
            const bool fresh = n == 0 || hg == 0;
            int id = -1;
            if (fresh && in) id = __ldg(p.table + tok / kBlock);
            const bool live = id >= 0 && id < p.num_blocks;
            if (fresh) broken = __any_sync(0xffffffffu, live && tok > L - p.n) && latent_broken<R>(p.pool, live, id, tok, lane);
            if (hg == 0 && warp < 4) { // the rotated part as it is
                const uint4* src = reinterpret_cast<const uint4*>(p.pool + ((long long)(live ? id : 0) * kBlock + tok % kBlock) * (R + kRope) + R);
                uint4* dst = reinterpret_cast<uint4*>(p.turned + tok * kRope);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            }
            if (!warp_wait(bar + (C::kDFull + b) * 8, (uint32_t)(n >> 1) & 1u, wt, 720)) break;
            fence_after();
            const uint32_t acc = tb + 256 * b + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
            for (int c = warp >> 2;; c += C::kOut / 4) {   // 64 outputs: rounded into shared memory, copied out from there
                const int h = hg * C::HEADS + 64 * c / (2 * D), e = 64 * c % (2 * D);
                const bool is = c < 4 && h < p.H, last = !is || c + C::kOut / 4 >= 4;
                float f[64];
                if (is) {
                    tmem_ld32(acc + 64 * c, f);
                    tmem_ld32(acc + 64 * c + 32, f + 32);
                    wait_ld();
                    tie32(f);
                    tie32(f + 32);
                }
                if (last) {   // the sums are free for the next unit but one
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_cluster(there + (C::kDEmpty + b) * 8);
                }
                if (!is) break;
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < 64; ++i) most = fmaxf(most, fabsf(f[i]));
                if (in && most >= 65520.f) {
                    record_device_error(p.err, kErrLatentKey, tok, h);
                    // a value as the largest that f16 holds: an infinity would meet the weights of 0 of queries that do not see it
                    if (e >= D) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) f[i] = fabsf(f[i]) < INFINITY ? fminf(fmaxf(f[i], -65504.f), 65504.f) : f[i];
                    }
                }
                if (broken) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) f[i] = e < D ? NAN : 0.f;
                }
                if (lane == 0) stores_read();   // the copy before this one
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(stage + ((i ^ (lane & 7)) << 4)) =
                        in ? make_uint4(pack_half(f[8 * i], f[8 * i + 1]), pack_half(f[8 * i + 2], f[8 * i + 3]), pack_half(f[8 * i + 4], f[8 * i + 5]),
                                        pack_half(f[8 * i + 6], f[8 * i + 7]))
                           : make_uint4(0u, 0u, 0u, 0u);
                fence_async();
                __syncwarp();
                if (lane == 0) store_box2(e < D ? &p.tk : &p.tv, e % D, (int)((long long)h * p.cap + tok), su32(stage));
                if (last) break;
            }
        }
        if (lane == 0) stores_done();
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    cluster_sync();   // no product, report or commit is left that touches the other CTA
    if (abort_flag) settle_expand<C>(su32(bars), su32(issued), p.err, p.ns);   // (the same in both)
    if (warp == C::kProduct) {
        fence_after();
        tmem_free2<512>(tb);
    }
}

// ---------------------------------------------------------------- attention
struct ChunkParams {
    CUtensorMap tq;         // queries: [head][token][D + 64]
    CUtensorMap tk;         // keys: [head, token][D]
    CUtensorMap tv;         // values: [head, token][D]
    CUtensorMap tt;         // rotated parts: [token][64]
    const int* live;
    const int32_t* table;
    const int32_t* position;
    __half* out;            // [n][H][D]
    float* parts;           // cut: [window + unit][query of the unit][D]
    float2* stats;          // [window + unit][query]: reference (log2), sum of the weights
    long long maxb, num_blocks, cap;
    int n, H, pairs, cut;
    float scale_log2;
    DevError* err;
    unsigned long long ns;
};

// A pair of CTAs takes 256 queries of one head, 128 in each, and shares every tile of keys and values: each CTA brings 64 of a
// tile's 128 keys and half of its values' columns. A CTA alone takes 80 KB from L2 for every 10.5 MFLOP, and 152 of them
// are held up by L2 (1.4 us a tile of 128 queries and 128 keys; its products take 0.66).
// The pairs stay for the whole grid's work. A unit of it is (256 queries, head); units are ordered by their length and
// dealt out to and fro, so that all pairs end together, and a unit's queries, first tiles and scores arrive while the one before is finished.
// Where there are few (cut), all units' tiles in a row are cut into a window a pair instead, and parts of a unit joined afterwards (against a number
// of parts that is the same for all units: 777 tokens after 1234, 20 heads of 64, 37.1 -> 32.8 us; 256 after 30000, 32 heads of 128, 284 -> 275;
// 256 after 7936, 40 heads, 116.5 -> 105; 1000 after 1000, 8 heads, 27.3 -> 28.4).
// A causal prompt of 4096 tokens, 32 heads of 128: 129 us, 1.33 PFLOP/s of what the mask leaves. A tile of 256 x 128 takes 1640 - 1740 cycles, its
// products 1280: with two halves in turn each has a chain of scores (800), maximum (450), exponentials (800), values (600) and the way between the
// warps (600) for two tiles. From unit to unit go 4 thousand cycles more. The weights are f16 (the product's operand, up to 2^15), their sums f32.
// Without gain: weights before their maximum is known, judged by their sum (registers spill: 156 -> 170 us a prompt).
template <int D, int NQ>
struct ChunkCfg {
    static constexpr int CH = (D + kRope) / 64, RUN = kQ * 128;      // a run of 64 values of 128 rows
    // Buffers of queries (NQ) and tiles in flight share the room. With units in turn a second buffer is worth a tile with 128 values (a 4096-token
    // prompt 151.9 -> 150.5 us), with a window or two a pair it is not (256 tokens after 7936 83.2 -> 85.2); with 64 there is room for both.
    static constexpr int KRUN = 64 * 128, STAGES = D == 128 && NQ == 2 ? 3 : 4;
    static constexpr int QB = CH * RUN, KB = CH * KRUN, VB = kQ * D; // V: 128 keys x D / 2 columns
    static constexpr size_t SMEM = NQ * QB + STAGES * (KB + VB);
    static constexpr uint32_t OCOL = 256, COLS = 512;                // tensor memory: two S (P over them), two O
    // what has landed in either CTA, and the weights of both, are reported to rank 0's barriers, what the products have read or
    // written to both CTAs'; a unit's sums are left to its own CTA's
    static constexpr int kQFull = 0, kQEmpty = NQ, kKFull = 2 * NQ, kKEmpty = kKFull + STAGES, kVFull = kKEmpty + STAGES, kVEmpty = kVFull + STAGES,
                         kSFull = kVEmpty + STAGES, kPReady = kSFull + 2, kOFree = kPReady + 2, kSums = kOFree + 1, kDone = kSums + 2, kBars = kDone + 1;
};

// Four lanes' four 16-byte units each, transposed: unit r of lane i becomes what was unit i of lane r.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & o) continue;
            const uint4 give = up ? u[k] : u[k + o];
            uint4 got;
            got.x = __shfl_xor_sync(0xffffffffu, give.x, o);
            got.y = __shfl_xor_sync(0xffffffffu, give.y, o);
            got.z = __shfl_xor_sync(0xffffffffu, give.z, o);
            got.w = __shfl_xor_sync(0xffffffffu, give.w, o);
            if (up) u[k] = got;
            else u[k + o] = got;
        }
    }
}

constexpr int kSoft = 16, kCopy = 16, kProduct = 17, kChunkThreads = 18 * 32;   // warps: softmax, copies, products

// The units' tiles in a row, for `cut`: unit b H + h has the block of queries that is the b-th from the end, and `enter` places before its tiles for
// what it costs to enter and leave it. From one block to the one before it there are two tiles less.
constexpr int kLeast = 8;   // tiles of a window at least: shorter ones make more parts than they save (4 heads after 16000: 39.9 us with 8, 42 with 4)
struct Row {
    int H, blocks, past, longest, enter, window;
    __device__ Row(int n, int H, int before, int pairs)
        : H(H), blocks((n + 2 * kQ - 1) / (2 * kQ)), past((before + kQ - 1) / kQ), longest((before + n + kQ - 1) / kQ), enter(4) {
        window = max((start(blocks) + pairs - 1) / pairs, kLeast);
        // One block of queries: windows that end where heads end, if they are little longer (256 queries after 7936, 32 heads: 32 tiles of one
        // head each are 1.2 us shorter than 28 of two; the 6 tiles that "little" stands for rest on this one shape).
        if (blocks == 1 && H <= pairs) {
            const int k = pairs / H, even = max((longest + k - 1) / k, kLeast);
            if (even <= window + 6) {
                window = even;
                enter = k * even - longest;
            }
        }
    }
    __device__ int tiles(int b) const { return b == 0 ? longest : 2 * (blocks - b) + past; }
    __device__ int start(int b) const { return b == 0 ? 0 : H * (longest + enter + (b - 1) * (past + enter + 2 * blocks - b)); }   // of the block's first head
    __device__ int start(int b, int h) const { return start(b) + h * (tiles(b) + enter); }
};

// The pair's copies in flight, after an abort.
template <typename C, int NQ>
__device__ __noinline__ void settle_chunk(uint32_t bar, uint32_t issued, DevError* err, unsigned long long ns) {
    if (cluster_rank() == 0 && threadIdx.x == 32 * kCopy) {
        const Waits alone = {err, nullptr, ns};
        settle_ring(bar + C::kQFull * 8, NQ, issued, C::QB, alone, 802);
        settle_ring(bar + C::kKFull * 8, C::STAGES, issued + 4, C::KB, alone, 803);
        settle_ring(bar + C::kVFull * 8, C::STAGES, issued + 8, C::VB, alone, 804);
    }
    __syncthreads();
    cluster_sync();
}

template <int D, int NQ>
__global__ void __launch_bounds__(kChunkThreads, 1) __cluster_dims__(2, 1, 1) mla_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = ChunkCfg<D, NQ>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[C::kBars];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ int issued[3];   // copies of queries, keys, values
    __shared__ int rows_now;    // read once, so that all warps run the same tiles
    __shared__ float tops[2][2][kQ], sums[2][2][2][kQ], refs[2][2][kQ];   // (sums and refs of two units in turn)
    const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t bar = su32(bars), qs = su32(smem), ks = qs + NQ * C::QB, vs = ks + C::STAGES * C::KB;
    if (t == 0) {
        for (int i = 0; i < C::kBars; ++i) bar_init(bar + i * 8, (i >= C::kPReady && i <= C::kOFree) || i == C::kSums || i == C::kSums + 1 ? kSoft : 1);
        abort_flag = 0;
        rows_now = (int)context(p.position, p.n, p.maxb);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tq);
        prefetch_map(&p.tk);
        prefetch_map(&p.tv);
        prefetch_map(&p.tt);
    }
    if (warp == kProduct) tmem_alloc2<C::COLS>(&tmem_at);
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, tmem_at, 0), there = in_cta(bar, 0);
    const PairWaits wt = {{p.err, &abort_flag, p.ns}};
    const Waits alone = {p.err, nullptr, p.ns};
    const long long L = rows_now;
    // whether a block of the context is missing (its keys are then left out): the rare case is told apart here, once, beside the
    // kernel before this one, and not at every tile
    bool gap = false;
    for (long long i = t; i < (L + kBlock - 1) / kBlock; i += kChunkThreads) {
        const int id = __ldcg(p.table + i);
        gap |= id < 0 || id >= p.num_blocks;
    }
    gap = __syncthreads_or(gap);
    const int before = L ? (int)(L - p.n) : 0;
    const int blocks = (p.n + 2 * kQ - 1) / (2 * kQ), units = L ? blocks * p.H : 0, pairs = gridDim.x / 2, pair = blockIdx.x / 2;

    // u / d for u < 2^22, `by` the rounded 1 / d
    const float by_heads = 1.f / (float)p.H;
    auto quotient = [](int u, int d, float by) {
        int k = (int)((float)u * by);
        k -= k * d > u;
        return k + ((k + 1) * d <= u);
    };
    const Row in_a_row(p.n, p.H, before, pairs);
    const int lo = pair * in_a_row.window, hi = lo + in_a_row.window;
    int first_unit = 0;
    if (p.cut) {   // the one that holds place lo
        int b = 0;
        while (b + 1 < blocks && in_a_row.start(b + 1) <= lo) ++b;
        first_unit = b * p.H + min((lo - in_a_row.start(b)) / (in_a_row.tiles(b) + in_a_row.enter), p.H);
    }
    pdl_wait();
    pdl_trigger();
    // The k-th unit of this pair: the head, the first query, where a part of it goes (-1: the whole unit), its first tile and their number
    // (of a part: possibly none); false behind the last.
    struct Unit {
        int h, first, slot, j0, tiles;
    };
    auto unit = [&](int k, Unit& w) {
        // (to and fro: where the last row of units is short, the pairs that have one there are those of the row's end)
        const int u = p.cut ? first_unit + k : k * pairs + (k & 1 ? pairs - 1 - pair : pair);
        if (u >= units) return false;
        const int b = quotient(u, p.H, by_heads);
        w.h = u - b * p.H;
        w.first = (blocks - 1 - b) * 2 * kQ;
        w.slot = -1;
        w.j0 = 0;
        w.tiles = in_a_row.tiles(b);    // that the last of the unit's queries sees
        if (p.cut) {
            const int start = in_a_row.start(b, w.h);
            if (start >= hi) return false;
            const int all = w.tiles, j1 = min(hi - start - in_a_row.enter, all);
            w.j0 = max(lo - start - in_a_row.enter, 0);
            w.tiles = j1 - w.j0;
            if (w.tiles < all) w.slot = pair + u;
        }
        return true;
    };
    auto work = [&](auto each) {
        Unit w;
        for (int k = 0; unit(k, w) && each(w, k); ++k) {}
    };
    int jt = 0, un = 0;   // tiles and units with tiles so far

    if (warp == kCopy) {
        // ------------------------------------------------ copies: this CTA's queries and its halves of the tiles
        if (lane == 0) {
            bool ok = true;
            int asked = 0, keys = 0, vals = 0;   // units whose queries have been asked for, tiles (behind a wait that failed nothing is armed or issued)
            auto queries = [&](const Unit& w) {
                const int b = asked % NQ;
                ok = asked < NQ || bar_wait(bar + (C::kQEmpty + b) * 8, (uint32_t)(asked / NQ - 1) & 1u, wt, 799);
                if (!ok) return;
                if (rank == 0) bar_expect(bar + (C::kQFull + b) * 8, 2 * C::QB);
                for (int c = 0; c < C::CH; ++c)
                    copy2_box3(qs + b * C::QB + c * C::RUN, &p.tq, 64 * c, w.first + kQ * rank, w.h, there + (C::kQFull + b) * 8);
                ++asked;
            };
            work([&](const Unit& w, int k) {
                const int h = w.h, j0 = w.j0, tiles = w.tiles;
                if (tiles <= 0) return true;
                if (asked == 0) queries(w);
                for (int j = 0; j < tiles && ok; ++j) {
                    const int s = vals % C::STAGES, at = (j0 + j) * kQ, row = (int)((long long)h * p.cap) + at;
                    const uint32_t ph = (uint32_t)(vals / C::STAGES - 1) & 1u, kf = there + (C::kKFull + s) * 8, vf = there + (C::kVFull + s) * 8;
                    ok = vals < C::STAGES || bar_wait(bar + (C::kKEmpty + s) * 8, ph, wt, 800);
                    if (!ok) break;
                    ++keys;
                    if (rank == 0) bar_expect(bar + (C::kKFull + s) * 8, 2 * C::KB);
                    for (int c = 0; c < D / 64; ++c) copy2_box2(ks + s * C::KB + c * C::KRUN, &p.tk, 64 * c, row + 64 * rank, kf);
                    copy2_box2(ks + s * C::KB + D / 64 * C::KRUN, &p.tt, 0, at + 64 * rank, kf);
                    ok = vals < C::STAGES || bar_wait(bar + (C::kVEmpty + s) * 8, ph, wt, 801);
                    if (!ok) break;
                    ++vals;
                    if (rank == 0) bar_expect(bar + (C::kVFull + s) * 8, 2 * C::VB);
                    copy2_box2(vs + s * C::VB, &p.tv, D / 2 * rank, row, vf);
                    if (j == (NQ == 2 ? min(1, tiles - 1) : tiles - 1)) {   // the next unit's queries, spread over the rows of all heads, come from far
                        Unit next;
                        int i = k + 1;
                        bool is;
                        while ((is = unit(i, next)) && next.tiles <= 0) ++i;
                        if (is) queries(next);
                    }
                }
                return ok;
            });
            issued[0] = asked;
            issued[1] = keys;
            issued[2] = vals;
        }
        __syncwarp();
    } else if (warp == kProduct) {
        // ------------------------------------------------ products of both CTAs: the scores of a tile before the values of the one before it
        if (rank == 0) {
            constexpr uint32_t IS = instr(2 * kQ, kQ, false, false), IO = instr(2 * kQ, D, false, true);
            const uint32_t one = elect_one();
            const uint64_t qd = operand(qs, 16, 1024, 2), kd = operand(ks, 16, 1024, 2);
            const uint64_t vd = operand(vs, 16, D * 8, D == 128 ? 2 : 4);   // a run of D / 2 columns
            // The values of tile i, the j-th of unit u - 1: behind the next tile's scores, be they another unit's (with one buffer of queries those
            // have to wait, and the values do not).
            auto values = [&](int i, int j, int u) {
                const int s = i % C::STAGES;
                if (!warp_wait(bar + (C::kVFull + s) * 8, (uint32_t)(i / C::STAGES) & 1u, wt, 812)) return false;
                if (!warp_wait(bar + (C::kPReady + (i & 1)) * 8, (uint32_t)(i >> 1) & 1u, wt, 813)) return false;
                if (j == 0 && u > 1 && !warp_wait(bar + C::kOFree * 8, (uint32_t)u & 1u, wt, 815)) return false;   // (u - 2: the unit before)
                fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma2_ts(one, tb + C::OCOL + (i & 1) * D, tb + (i & 1) * kQ + 8 * k, vd + s * (C::VB >> 4) + ((k * 16 * D) >> 4), IO, j > 1 || k > 0);
                mma2_commit(one, bar + (C::kVEmpty + s) * 8);
                return true;
            };
            int last_j = 0;
            bool ok = true;
            work([&](const Unit& w, int) {
                const int tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
                if (tiles <= 0) return true;
                const int b = un % NQ;
                bool held = jt > 0;   // the tile before's values
                if (NQ == 1 && held) {
                    ok = values(jt - 1, last_j, un);
                    held = false;
                }
                ok = ok && warp_wait(bar + (C::kQFull + b) * 8, (uint32_t)(un / NQ) & 1u, wt, 810);
                if (!ok) return false;
                ++un;
                for (int j = 0; j < tiles; ++j) {
                    const int s = jt % C::STAGES;
                    ok = warp_wait(bar + (C::kKFull + s) * 8, (uint32_t)(jt / C::STAGES) & 1u, wt, 811);
                    if (!ok) return false;
                    fence_after();
#pragma unroll
                    for (int k = 0; k < 4 * C::CH; ++k)
                        mma2_ss(one, tb + (jt & 1) * kQ, qd + b * (C::QB >> 4) + (((k >> 2) * C::RUN + (k & 3) * 32) >> 4),
                                kd + s * (C::KB >> 4) + (((k >> 2) * C::KRUN + (k & 3) * 32) >> 4), IS, k > 0);
                    mma2_commit(one, bar + (C::kKEmpty + s) * 8);
                    mma2_commit(one, bar + (C::kSFull + (jt & 1)) * 8);
                    if (j + 1 == tiles) mma2_commit(one, bar + (C::kQEmpty + b) * 8);
                    ok = !held || values(jt - 1, last_j, j > 0 ? un : un - 1);
                    if (!ok) return false;
                    held = true;
                    last_j = j;
                    ++jt;
                }
                return true;
            });
            if (ok && jt > 0) values(jt - 1, last_j, un);
            mma2_commit(one, bar + C::kDone * 8);
            warp_wait(bar + C::kDone * 8, 0u, alone, 814);
        }
    } else {
        // ------------------------------------------------ softmax: eight warps have the even tiles, eight the odd ones; of the eight, four
        // have keys 0 - 63 of a tile and four the rest; a thread has one query. The eight run the same tiles whatever their waits
        // return, so that their named barriers always meet. The two eights meet on mbarriers, by bounded waits: once one has failed nothing
        // keeps them within a unit of each other.
        const int g = warp >> 3, hf = (warp >> 2) & 1, q = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, sc = tb + lanes + g * kQ, oc = tb + lanes + C::OCOL + g * D;
        const float2 scale = make_float2(p.scale_log2, p.scale_log2);
        work([&](const Unit& w, int) {
            const int tiles = max(w.tiles, 0), q0 = w.first + kQ * (int)rank, rows = p.n - q0;   // (some, all or none of 128)
            const int last = before + q0 + q - 64 * hf;        // the last key this query sees, counted from this thread's first
            const int off = (jt & 1) ^ g;                      // this half's first tile of the unit
            const int mine = tiles > off ? (tiles - off + 1) >> 1 : 0;
            // the values up to the unit's tile i are in O
            auto done = [&](int i) {
                const int j = jt + i;
                warp_wait(bar + (C::kVEmpty + j % C::STAGES) * 8, (uint32_t)(j / C::STAGES) & 1u, wt, 822);
                fence_after();
            };
            // The weights' reference, log2: -kLow where the row's first scores allow it (the largest lies between 0 and kLag - kLow then), else
            // kLift below their largest; from then on it is moved where a score passes kLag above it. Weights of up to 2^kLag are as exact in f16 as
            // smaller ones, and O has to be scaled only then.
            float m = -kLow, l = 0.f;
            bool set = false;
            for (int i = 0; i < mine; ++i) {
                const int at = (w.j0 + off + 2 * i) * kQ, j = jt + off + 2 * i;
                warp_wait(bar + (C::kSFull + g) * 8, (uint32_t)(j >> 1) & 1u, wt, 821);
                fence_after();
                float x[64];
                tmem_ld32(sc + 64 * hf, x);
                tmem_ld32(sc + 64 * hf + 32, x + 32);
                wait_ld();
                tie32(x);
                tie32(x + 32);
                if (at + kQ - 1 > before + q0 || gap) {   // the same for the CTA
                    const int seen = last - at;
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c > seen ? -INFINITY : x[c];
                    if (gap) {
                        const int live = __ldg(p.live + w.j0 + off + 2 * i) >> (4 * hf);
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (!((live >> b) & 1)) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) x[16 * b + c] = -INFINITY;
                            }
                    }
                }
                float most[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < 64; ++c) most[c & 3] = fmaxf(most[c & 3], x[c]);
                float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) * p.scale_log2;
                // (The barrier also keeps the weights, which take the scores' place, behind the other four warps' loads. Whether a row is
                // set is known to both halves of its keys only as far as each has seen it: they settle it together where either asks.)
                unsigned raise;
                asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.or.pred b, %2, 256, a;\n selp.u32 %0, 1, 0, b;\n}"
                             : "=r"(raise) : "r"((unsigned)(top > m + kLag || (!set && top < 0.f))), "r"(1 + g) : "memory");
                if (raise) {
                    tops[g][hf][q] = top;
                    asm volatile("barrier.cta.sync %0, 256;" ::"r"(1 + g) : "memory");
                    top = fmaxf(top, tops[g][hf ^ 1][q]);
                    // (O is scaled for all of the rows, so that each may as well have its reference where it would be set)
                    const bool move = top > -INFINITY && (top > m + kLift || (!set && top < 0.f));
                    const float now = move ? top - kLift : m, f = set ? ex2(m - now) : 0.f;
                    m = now;
                    set |= top > -INFINITY;
                    l *= f;
                    if (i > 0) {
                        done(off + 2 * i - 2);
#pragma unroll 1
                        for (int c = hf * (D / 32); c < (hf + 1) * (D / 32); ++c) {
                            float v[16];
                            uint32_t u[16];
                            tmem_load<16>(oc + 16 * c, v);
#pragma unroll
                            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(v[k] * f);
                            tmem_st16(oc + 16 * c, u);
                        }
                    }
                } else set = true;
                const float2 ref = make_float2(-m, -m);
                float2 sum[4] = {};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t u[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 e = fma2(make_float2(x[32 * c + 2 * k], x[32 * c + 2 * k + 1]), scale, ref);
                        const float2 w = make_float2(ex2(e.x), ex2(e.y));
                        sum[k & 3] = add2(sum[k & 3], w);
                        u[k] = pack_half(w.x, w.y);
                    }
                    tmem_st16(sc + 32 * hf + 16 * c, u);
                }
                const float2 s2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += s2.x + s2.y;
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_cluster(there + (C::kPReady + g) * 8);
            }
            // Both halves of the tiles joined by the eight warps that had the last tile, half of the values each four; the other
            // eight leave what they know and go on to the next unit.
            const bool whole = w.slot < 0;
            float ma = -1e30f, mb = -1e30f, total = 0.f;
            if (tiles > 0) {
                const int lastg = (jt + tiles - 1) & 1, turn = un & 1;
                const uint32_t left = bar + (C::kSums + turn) * 8, phase = (uint32_t)(un >> 1) & 1u;
                sums[turn][g][hf][q] = l;
                refs[turn][g][q] = set ? m : -1e30f;          // (the same from both halves of the keys)
                ++un;
                __syncwarp();
                if (lane == 0) bar_arrive(left);
                if (g != lastg) {
                    jt += tiles;
                    return true;
                }
                warp_wait(left, phase, wt, 823);
                ma = refs[turn][0][q];
                mb = refs[turn][1][q];
                const float top = fmaxf(ma, mb);
                total = (sums[turn][0][0][q] + sums[turn][0][1][q]) * ex2(ma - top) + (sums[turn][1][0][q] + sums[turn][1][1][q]) * ex2(mb - top);
                if (tiles > 1) done(tiles - 2);
                done(tiles - 1);
            } else return true;   // (the join does not look for a part here)
            const float top = fmaxf(ma, mb), inv = !whole ? 1.f : total == 0.f ? 0.f : 1.f / total;
            const float ca = ex2(ma - top) * inv, cb = ex2(mb - top) * inv;
            const bool even = tiles > (jt & 1), odd = tiles > (1 ^ (jt & 1));   // which of the two O hold something of this unit
            // Four lanes store 64 bytes of one query together (one lane a query: rows far apart, which held up the warps for 3500 cycles).
            const int r0 = q & ~3, part = q & 3;
            const size_t step = (size_t)p.H * D, row0 = (size_t)(q0 + r0) * step + (size_t)w.h * D;
            auto values = [&](int d0, float* x, float* y) {   // 16 of them, both halves of the tiles together
                constexpr int N = 16;
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = y[k] = 0.f;
                if (even) tmem_raw<N>(tb + lanes + C::OCOL + d0, x);
                if (odd) tmem_raw<N>(tb + lanes + C::OCOL + D + d0, y);
                wait_ld();
                tie<N>(x);
                tie<N>(y);
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = fmaf(y[k], cb, x[k] * ca);
            };
            auto read = [&] {   // both O are read: the next unit's values may go there
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_cluster(there + C::kOFree * 8);
            };
            if (whole) {
                uint32_t packed[D / 4];   // (all of them before the first store: the next unit waits for O)
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float x[16], y[16];
                    values(hf * (D / 2) + 16 * c, x, y);
#pragma unroll
                    for (int k = 0; k < 8; ++k) packed[8 * c + k] = pack_half(x[2 * k], x[2 * k + 1]);
                }
                read();
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint4 u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) u[k] = make_uint4(packed[16 * c + 4 * k], packed[16 * c + 4 * k + 1], packed[16 * c + 4 * k + 2], packed[16 * c + 4 * k + 3]);
                    transpose4(u, lane);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r0 + r < rows) *reinterpret_cast<uint4*>(p.out + row0 + r * step + hf * (D / 2) + 32 * c + 8 * part) = u[r];
                }
            } else {
                float* dst = p.parts + ((size_t)w.slot * 2 * kQ + kQ * rank + r0) * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float x[16], y[16];
                    const int d0 = hf * (D / 2) + 16 * c;
                    values(d0, x, y);
                    if (c == D / 32 - 1) read();
                    uint4 u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        u[k] = make_uint4(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]), __float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3]));
                    transpose4(u, lane);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r0 + r < rows) *reinterpret_cast<uint4*>(dst + r * D + d0 + 4 * part) = u[r];
                }
            }
            if (!whole && hf == 0 && q < rows) p.stats[(size_t)w.slot * 2 * kQ + kQ * rank + q] = make_float2(top, total);
            jt += tiles;
            return true;
        });
    }
    fence_before();
    __syncthreads();
    cluster_sync();   // no product, report or commit is left that touches the other CTA
    if (abort_flag) settle_chunk<C, NQ>(su32(bars), su32(issued), p.err, p.ns);   // (the same in both)
    if (warp == kProduct) {
        fence_after();
        tmem_free2<C::COLS>(tb);
    }
}

// A warp a query and head, four parts' loads together; which parts there are is worked out before the wait. Bound by latency: 3 us behind the
// attention (7 alone) for 256 queries of 32 heads in two parts.
template <int D>
__global__ void __launch_bounds__(256) mla_chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    const int i = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;   // (below 2^22)
    const int L = (int)context(p.position, p.n, p.maxb);
    const int row = i / p.H, h = i - row * p.H;
    const Row in_a_row(p.n, p.H, max(L - p.n, 0), p.pairs);
    const int b = in_a_row.blocks - 1 - row / (2 * kQ), start = in_a_row.start(b, h) + in_a_row.enter;
    const int w0 = start / in_a_row.window, count = (start + in_a_row.tiles(b) - 1) / in_a_row.window - w0 + 1;
    const size_t at = (size_t)(w0 + b * p.H + h) * 2 * kQ + row % (2 * kQ);
    pdl_wait();
    pdl_trigger();
    if (row >= p.n || L == 0 || count == 1) return;   // (a whole unit is in its place)
    constexpr int V = D / 32, AT_ONCE = 4;
    float top = -INFINITY, total = 0.f, x[V] = {};
    for (int s0 = 0; s0 < count; s0 += AT_ONCE) {   // four parts at a time
        float2 st[AT_ONCE];
        float v[AT_ONCE][V];
#pragma unroll
        for (int s = 0; s < AT_ONCE; ++s) {
            const size_t part = at + (size_t)(s0 + s) * 2 * kQ;
            st[s] = s0 + s < count ? __ldcg(p.stats + part) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 a = s0 + s < count ? __ldcg(reinterpret_cast<const float2*>(p.parts + part * D + lane * V + k)) : make_float2(0.f, 0.f);
                v[s][k] = a.x;
                v[s][k + 1] = a.y;
            }
        }
        float now = top;
#pragma unroll
        for (int s = 0; s < AT_ONCE; ++s) now = fmaxf(now, st[s].x);
        const float f0 = top == now ? 1.f : ex2(top - now);
        total *= f0;
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] *= f0;
        top = now;
#pragma unroll
        for (int s = 0; s < AT_ONCE; ++s) {
            if (st[s].y == 0.f) continue;   // no key, and no part
            const float f = ex2(st[s].x - top);
            total += st[s].y * f;
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = fmaf(v[s][k], f, x[k]);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int k = 0; k < V; k += 2)
        *reinterpret_cast<__half2*>(p.out + (size_t)i * D + lane * V + k) = __floats2half2_rn(x[k] * inv, x[k + 1] * inv);
}

// ---------------------------------------------------------------- host
// Few queries go through the absorbed form, each for itself over the cache: a query costs it the context's rows once per 64 heads,
// where the expanded form first makes every head's keys and values. Both grow with the context, which the host does not know.
// Expanded / absorbed in us, 32 heads of 128, rank 512, after 8000 tokens: 84 / 18 (1 token), 84 / 27 (8), 85 / 55 (32), 85 / 80 (48);
// with no context 18 / 12, 19 / 13, 19 / 18, 20 / 25. 128 heads after 8000: 333 / 123 (32), 344 / 339 (96); with no context
// 24 / 27 (16), 24 / 41 (32). 8 heads of 64, rank 256, after 8000: 24 / 15 (4), 24 / 24 (16).
// Under a table of at most 1024 tokens the context cannot grow dear: 4 heads of 64, rank 256, after 0 and 900 tokens 12 / 10 and 16 / 13 (16),
// 16 of 128, rank 512, 15 / 15 and 21 / 20 (32), 32 of 64 14 / 14 and 20 / 17 (16).
static bool few(int64_t n, int H, int D, int64_t maxb) { return n <= 32 && (n * 128 <= (int64_t)H * D || (maxb <= 64 && n * H <= 512)); }

constexpr int kMostPairs = 80;   // pairs of CTAs with a window each
struct ChunkShape {
    bool cut;
    long long cap;                                       // rows of the keys and values a head
    size_t v, turned, live, stats, parts, total;         // offsets in the workspace
};
static ChunkShape chunk_shape(int64_t n, int H, int D, int64_t maxb) {
    ChunkShape s = {};
    s.cap = (maxb * kBlock + 255) / 256 * 256;
    // Few units are cut evenly over the pairs where that costs less, for the longest context that the table holds: rounds of 76 units and the
    // end of each (about 2 tiles), against their share, a second entry and the join. (76 pairs: 152 SMs. The workspace's size, which this decides,
    // is asked for without a device; where another number of pairs is launched the cut is a worse one, not a wrong one.)
    const int64_t units = (n + 2 * kQ - 1) / (2 * kQ) * H, tiles = s.cap / kQ;
    s.cut = units < 152 && (units * (tiles + 2) + 75) / 76 + 5 < (units + 75) / 76 * (tiles + 2);
    auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    s.v = up((size_t)H * s.cap * D * 2);
    s.turned = 2 * s.v;
    s.live = s.turned + up((size_t)s.cap * kRope * 2);
    s.stats = s.live + up((size_t)tiles * 4);
    s.parts = s.stats + (s.cut ? up((size_t)(kMostPairs + units) * 2 * kQ * 8) : 0);
    s.total = s.parts + (s.cut ? up((size_t)(kMostPairs + units) * 2 * kQ * D * 4) : 0);
    return s;
}

// Bytes of the workspace that a call uses; 0 where its sizes are out of range.
static size_t chunk_need(int64_t n, int H, int D, int R, int64_t maxb) {
    if (!shape_ok(D, R) || n < 1 || n > 65535 || H < 1 || H > 1024 || n * H >= (1 << 22) || maxb < 1 || maxb > (1 << 16)) return 0;
    return few(n, H, D, maxb) ? absorbed_workspace(n, H, R) : chunk_shape(n, H, D, maxb).total;
}

// Clusters of two CTAs of a kernel that the current device holds at once, looked up once.
template <typename K>
static int pairs_at_once(K kernel, int threads, size_t smem, std::atomic<int>* known, int* out) {
    int dev = 0;
    QL_TRY_CUDA(cudaGetDevice(&dev));
    *out = dev < 64 ? known[dev].load() : 0;
    if (*out > 0) return QL_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    QL_TRY_CUDA(cudaOccupancyMaxActiveClusters(out, kernel, &cfg));
    if (*out < 1) return set_error(QL_ECUDA, "ql_mla_attn_chunk: the GPU does not hold a pair of its CTAs");
    if (dev < 64) known[dev].store(*out);
    return QL_OK;
}

// The attention's shared memory allowed and its pairs counted, once.
template <int D, int NQ>
static int attention_ready(int* pairs) {
    static std::atomic<unsigned long long> done{0};
    static std::atomic<int> most[64];
    QL_TRY_CUDA(allow_smem_once(mla_chunk_kernel<D, NQ>, ChunkCfg<D, NQ>::SMEM, done));
    return pairs_at_once(mla_chunk_kernel<D, NQ>, kChunkThreads, ChunkCfg<D, NQ>::SMEM, most, pairs);
}

template <int D, int R>
static int chunk_go(const AttnIn& a, const ChunkShape& sh, cudaStream_t s) {
    using E = ExpandCfg<D, R>;
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "ql_mla_attn_chunk: no device error record");
    static std::atomic<unsigned long long> done{0};
    QL_TRY_CUDA(allow_smem_once(mla_expand_kernel<D, R>, E::SMEM, done));
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    ExpandParams ep = {};
    ChunkParams cp = {};
    const uint64_t row = (R + kRope) * 2;
    {
        const uint64_t d[2] = {R + kRope, (uint64_t)a.num_blocks * kBlock}, st[1] = {row};
        const uint32_t b[2] = {64, kBlock};
        if (int rc = f16_tensor_map(a.pool, 2, d, st, b, &ep.tc)) return rc;
    }
    {
        const uint64_t d[2] = {R, (uint64_t)a.H * 2 * D}, st[1] = {R * 2};
        const uint32_t b[2] = {64, 128};
        if (int rc = f16_tensor_map(a.w, 2, d, st, b, &ep.tw)) return rc;
    }
    {
        const uint64_t w = (D + kRope) * 2, d[3] = {D + kRope, (uint64_t)a.rows, (uint64_t)a.H}, st[2] = {a.H * w, w};
        const uint32_t b[3] = {64, kQ, 1};
        if (int rc = f16_tensor_map(a.q, 3, d, st, b, &cp.tq)) return rc;
    }
    {
        const uint64_t d[2] = {D, (uint64_t)a.H * sh.cap}, st[1] = {D * 2};
        const uint32_t b[2] = {64, 64}, v[2] = {D / 2, kQ};
        if (int rc = f16_tensor_map(ws, 2, d, st, b, &cp.tk)) return rc;
        if (int rc = f16_tensor_map(ws + sh.v, 2, d, st, v, &cp.tv)) return rc;
        const uint32_t o[2] = {64, 32};
        if (int rc = f16_tensor_map(ws, 2, d, st, o, &ep.tk)) return rc;
        if (int rc = f16_tensor_map(ws + sh.v, 2, d, st, o, &ep.tv)) return rc;
    }
    {
        const uint64_t d[2] = {kRope, (uint64_t)sh.cap}, st[1] = {kRope * 2};
        const uint32_t b[2] = {64, 64};
        if (int rc = f16_tensor_map(ws + sh.turned, 2, d, st, b, &cp.tt)) return rc;
    }
    ep.pool = static_cast<const __half*>(a.pool);
    ep.table = cp.table = a.table;
    ep.position = cp.position = a.lens;
    ep.turned = reinterpret_cast<__half*>(ws + sh.turned);
    ep.live = reinterpret_cast<int*>(ws + sh.live);
    cp.live = ep.live;
    ep.maxb = cp.maxb = a.maxb;
    ep.num_blocks = cp.num_blocks = a.num_blocks;
    ep.cap = cp.cap = sh.cap;
    ep.n = cp.n = (int)a.rows;
    ep.H = cp.H = a.H;
    ep.err = cp.err = err;
    ep.ns = cp.ns = 2000000000ull;
    cp.out = static_cast<__half*>(a.out);
    cp.parts = reinterpret_cast<float*>(ws + sh.parts);
    cp.stats = reinterpret_cast<float2*>(ws + sh.stats);
    cp.cut = sh.cut;
    cp.scale_log2 = a.scale * 1.44269504088896340736f;
    // as many pairs as the GPU holds at once, and as there can be work for
    static std::atomic<int> most[64];
    int pairs = 0, pairs2 = 0;
    if (int rc = pairs_at_once(mla_expand_kernel<D, R>, E::THREADS, E::SMEM, most, &pairs)) return rc;
    constexpr int ONE = D == 128 ? 1 : 2;   // buffers of queries where units are cut
    if (int rc = sh.cut ? attention_ready<D, ONE>(&pairs2) : attention_ready<D, 2>(&pairs2)) return rc;
    pairs = (int)std::min<int64_t>(pairs, sh.cap / 256 * ((a.H + E::HEADS - 1) / E::HEADS));
    pairs2 = sh.cut ? std::min(pairs2, kMostPairs) : (int)std::min<int64_t>(pairs2, (a.rows + 2 * kQ - 1) / (2 * kQ) * a.H);
    cp.pairs = pairs2;
    cudaError_t e = launch(mla_expand_kernel<D, R>, dim3(2 * (unsigned)pairs), dim3(E::THREADS), E::SMEM, s, true, ep);
    if (e == cudaSuccess)
        e = sh.cut ? launch(mla_chunk_kernel<D, ONE>, dim3(2 * (unsigned)pairs2), dim3(kChunkThreads), ChunkCfg<D, ONE>::SMEM, s, true, cp)
                   : launch(mla_chunk_kernel<D, 2>, dim3(2 * (unsigned)pairs2), dim3(kChunkThreads), ChunkCfg<D, 2>::SMEM, s, true, cp);
    if (e == cudaSuccess && sh.cut)
        e = launch(mla_chunk_join_kernel<D>, dim3((unsigned)((a.rows * a.H + 7) / 8)), dim3(256), 0, s, true, cp);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "ql_mla_attn_chunk");
}

}  // namespace mla
}  // namespace ql

extern "C" size_t ql_mla_chunk_workspace_bytes(int64_t n_tokens, int n_heads, int head_dim, int rank, int64_t max_blocks_per_seq) {
    // Fewer tokens may be cut, or take the other form: the most that any number up to n_tokens needs.
    size_t most = ql::mla::chunk_need(n_tokens, n_heads, head_dim, rank, max_blocks_per_seq);
    if (most == 0) return 0;
    for (int64_t n = 2 * ql::mla::kQ; n < n_tokens && n / (2 * ql::mla::kQ) * n_heads < 152; n += 2 * ql::mla::kQ)
        most = std::max(most, ql::mla::chunk_need(n, n_heads, head_dim, rank, max_blocks_per_seq));
    for (int64_t n = std::min<int64_t>(n_tokens, 32); n > 0; --n)
        most = std::max(most, ql::mla::chunk_need(n, n_heads, head_dim, rank, max_blocks_per_seq));
    return most;
}

extern "C" int ql_mla_attn_chunk(const void* d_q, const void* d_w_kv, const void* d_pool, const int32_t* d_block_table,
                                 const int32_t* d_position, int64_t n_tokens, int n_heads, int head_dim, int rank, int rope_dim,
                                 int block_size, int64_t max_blocks_per_seq, int64_t num_blocks, float scale, void* d_out,
                                 void* d_workspace, size_t workspace_bytes, void* stream) {
    using namespace ql;
    using namespace ql::mla;
    const AttnIn a = {d_q, d_w_kv, d_pool, d_block_table, d_position, n_tokens, 1, max_blocks_per_seq, num_blocks, n_heads, head_dim, rank,
                      rope_dim, block_size, scale, d_out, d_workspace, workspace_bytes};
    if (int rc = attn_check("ql_mla_attn_chunk", a, chunk_need(n_tokens, n_heads, head_dim, rank, max_blocks_per_seq))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (few(n_tokens, n_heads, head_dim, max_blocks_per_seq)) return absorbed_launch(a, true, s);
    const ChunkShape sh = chunk_shape(n_tokens, n_heads, head_dim, max_blocks_per_seq);
    if (head_dim == 128) return rank == 512 ? chunk_go<128, 512>(a, sh, s) : chunk_go<128, 256>(a, sh, s);
    return rank == 512 ? chunk_go<64, 512>(a, sh, s) : chunk_go<64, 256>(a, sh, s);
}
