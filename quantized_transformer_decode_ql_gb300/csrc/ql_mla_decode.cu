// Latent attention of one new token per sequence over the paged cache, in three launches:
//
//  1. mla_absorb_kernel: q'_h = Wk_h^T q_h, the heads' queries against the latents themselves, as f16 (up to 32 heads: as a
//     pair of f16, 22 bits, which enter the scores' product as 64 heads);
//  2. mla_decode_kernel: the batch's tiles of 64 keys cut into equal windows, one per SM (the lengths are on the device only), a
//     window's tiles on the 5th-generation tensor cores, each tile read once for up to 64 heads: S^T = K q'^T (64 keys x heads),
//     the online softmax, O^T += V^T P (rank x heads), K the tile's rows and V their first `rank` values, the same bytes in
//     shared memory;
//  3. mla_join_kernel: a sequence's parts joined, o as a pair of f16, out_h = Wv_h o_h.
#include "ql_batched.h"
#include "ql_mla_tc.cuh"

namespace ql {
namespace mla {

constexpr int kTile = 64;       // keys of a tile
constexpr int kEnter = 1;       // tiles that entering a sequence costs a window (its query, its part written): charged in the split
constexpr int kMaxWin = 160;    // windows at most

__host__ __device__ inline int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Tiles of a sequence; 0 for an idle slot and for a length outside the table.
__device__ __forceinline__ int tiles_checked(int len, long long cap) { return len > 0 && len <= cap ? tiles_of(len) : 0; }

// The lengths of the batch's rows: an array, or those of a chunk's queries (row b sees one key more than row b - 1; -1 where
// the chunk does not fit the table).
struct Lengths {
    const int32_t* lens;
    const int32_t* position;   // null: lens
    int batch;
    long long cap;             // longest length
    __device__ int operator()(int b) const {
        if (position == nullptr) return __ldcg(lens + b);
        const long long p = __ldcg(position);
        return p >= 0 && p + batch <= cap ? (int)p + b + 1 : -1;
    }
};

// ---------------------------------------------------------------- the absorbed queries
struct AbsorbParams {
    const __half* q;       // [batch][H][D + 64]
    const __half* w;       // [H][2 D][R]
    __half* qc;            // [batch][halves][H][R + 64]
    int batch, H, halves;  // halves: 2 where the rest of each rounding is kept, too
    DevError* err;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One head, 64 of the rank columns, up to 64 rows of the batch. 4 warps, 16 columns each, f16 products with f32 sums (a batch's few rows
// fill no larger tile). The weights (16 KB) are asked into L2 before the previous kernel's end and read behind it, since that kernel may be
// what wrote them (read before it: 0.7 us less at one row). Bound by their way from L2 and the launch: about 3.5 us for 32 heads of 128,
// rank 512, at 1 to 32 rows (without shared memory, each lane its own rows: 3 us longer at 32).
template <int D, int R>
__global__ void __launch_bounds__(128) mla_absorb_kernel(const __grid_constant__ AbsorbParams p) {
    constexpr int WP = 72, QP = D + 8;    // row pitches in shared memory: 16-byte parts of 8 rows in different banks
    __shared__ __align__(16) __half ws[128 * WP];      // weights, then the outputs: [half][row]
    __shared__ __align__(16) __half qs[64 * QP];
    const int slices = R / 64, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int h = blockIdx.x / slices, r0 = (blockIdx.x % slices) * 64, b0 = blockIdx.y * 64;
    const __half* w = p.w + (size_t)h * 2 * D * R + r0;
    for (int i = t; i < D; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + (size_t)i * R));
    pdl_wait();
    pdl_trigger();
    for (int i = t; i < D * 8; i += 128) cp16(su32(ws + (i >> 3) * WP + (i & 7) * 8), w + (size_t)(i >> 3) * R + (i & 7) * 8);
    const int rows = min(64, p.batch - b0);
    constexpr int QC = D / 8;
    for (int i = t; i < 64 * QC; i += 128) {
        const int b = i / QC, c = i % QC;
        if (b < rows) cp16(su32(qs + b * QP + c * 8), p.q + ((size_t)(b0 + b) * p.H + h) * (D + kRope) + c * 8);
        else *reinterpret_cast<uint4*>(qs + b * QP + c * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const size_t rest = (size_t)p.H * (R + kRope);         // from a value to the rest of its rounding
    if (r0 == 0)   // the rotated part as it is
        for (int i = t; i < rows * 8; i += 128) {
            const int b = b0 + (i >> 3);
            __half* dst = p.qc + ((size_t)b * p.halves * p.H + h) * (R + kRope) + R + (i & 7) * 8;
            *reinterpret_cast<uint4*>(dst) = __ldg(reinterpret_cast<const uint4*>(p.q + ((size_t)b * p.H + h) * (D + kRope) + D + (i & 7) * 8));
            if (p.halves == 2) *reinterpret_cast<uint4*>(dst + rest) = make_uint4(0u, 0u, 0u, 0u);
        }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    uint32_t b[D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k)   // (k 0-7, n 0-7), (k 8-15, n 0-7), (k 0-7, n 8-15), (k 8-15, n 8-15)
        ldsm4t(b[k], su32(ws + (16 * k + (lane & 15)) * WP + 16 * warp + 8 * (lane >> 4)));
    __syncthreads();
    for (int m = 0; m < rows; m += 16) {
        float c[2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4];
            ldsm4(a, su32(qs + (m + (lane & 15)) * QP + 16 * k + 8 * (lane >> 4)));
            mma16(c[0], a[0], a[1], a[2], a[3], b[k][0], b[k][1]);
            mma16(c[1], a[0], a[1], a[2], a[3], b[k][2], b[k][3]);
        }
        bool large[2] = {};             // in the lane's two rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // n tile i / 2, row group i % 2
            const int r = m + (lane >> 2) + 8 * (i & 1);
            const float x = c[i >> 1][2 * (i & 1)], y = c[i >> 1][2 * (i & 1) + 1];
            if (r < rows) {
                __half* dst = ws + r * WP + 16 * warp + 8 * (i >> 1) + 2 * (lane & 3);
                const __half2 v = __floats2half2_rn(x, y);
                *reinterpret_cast<__half2*>(dst) = v;
                if (p.halves == 2) *reinterpret_cast<__half2*>(dst + 64 * WP) = __floats2half2_rn(x - __low2float(v), y - __high2float(v));
                large[i & 1] |= !(fabsf(x) < 65520.f && fabsf(y) < 65520.f);
            }
        }
        if (large[0] || large[1]) record_device_error(p.err, kErrLatentQuery, b0 + m + (lane >> 2) + (large[0] ? 0 : 8), h);
    }
    __syncthreads();
    for (int i = t; i < rows * 8 * p.halves; i += 128) {   // 128 bytes a row and half
        const int half = i >= rows * 8, r = (i - half * rows * 8) >> 3, c = i & 7;
        *reinterpret_cast<uint4*>(p.qc + ((size_t)(b0 + r) * p.halves * p.H + h) * (R + kRope) + half * rest + r0 + 8 * c) =
            *reinterpret_cast<const uint4*>(ws + (64 * half + r) * WP + 8 * c);
    }
}

// ---------------------------------------------------------------- the attention
template <int R, int NH>
struct Cfg {
    static constexpr int CH = (R + kRope) / 64;         // runs of 64 values (128 bytes) of a row
    static constexpr int GROUP = CH * 1024;             // 8 rows: [run][row][128 bytes], swizzled
    static constexpr int TILE = 8 * GROUP;
    static constexpr int HALVES = NH == 32 ? 2 : 1, NQ = NH * HALVES;   // of the queries: 64 columns of scores either way
    static constexpr int QB = CH * NQ * 128;            // [run][half][head][128 bytes]
    static constexpr int PB = kTile * NH * 2;           // [key][head]
    static constexpr int STAGES = R == 512 ? 2 : 4;
    static constexpr int PBUF = R == 512 && NH == 64 ? 1 : 2;
    static constexpr int MT = R / 128;                  // blocks of 128 latent values
    static constexpr uint32_t SCOL = MT * NH;           // tensor memory: O^T of each block, then two S^T
    static constexpr uint32_t COLS = SCOL + 2 * NQ <= 128 ? 128 : SCOL + 2 * NQ <= 256 ? 256 : 512;
    static constexpr size_t SMEM = (size_t)STAGES * TILE + QB + PBUF * PB;
    // a stage is freed block by block (kKEmpty + 4 stage + block): the next copies start while the values are still multiplied
    static constexpr int kKFull = 0, kKEmpty = STAGES, kSFull = 5 * STAGES, kPReady = kSFull + 2, kQFull = kPReady + 2, kQEmpty = kQFull + 1,
                         kDone = kQEmpty + 1, kBars = kDone + 1;
    static constexpr uint32_t PSW = NH == 64 ? 2 : 4;   // P's rows of 2 NH bytes: 128- or 64-byte swizzle
    static constexpr int HN = NH / 2;                   // heads of a softmax group of four warps (four groups of 16 for 64 heads: 4 us longer, 8 x 4000 - 16000 with 96 heads)
    static constexpr int kSoftWarps = NH / HN * 4, kCopyWarp = kSoftWarps, kScoreWarp = kSoftWarps + 1, kValueWarp = kSoftWarps + 2,
                         THREADS = (kSoftWarps + 3) * 32;
    static_assert(SCOL + 2 * NQ <= 512, "tensor memory");
    static_assert(SMEM + 2048 <= 232448, "shared memory");
};

struct DecodeParams {
    CUtensorMap tk;        // the pool: [group of 8 rows][run][row][64 values]
    CUtensorMap tq;        // absorbed queries: [sequence][run][half][head][64 values]
    const int32_t* tables;
    Lengths lens;
    float* parts;          // [head group][window + sequence][per][R]
    float2* stats;         // [head group][window + sequence][per]: reference (log2) and sum of the weights
    long long maxb, cap, num_blocks;   // maxb: entries from a row's table to the next (0: one table)
    int batch, H, windows, groups, per;   // per: heads of a part, NH or all that there are
    float scale_log2;
    DevError* err;
    unsigned long long ns;
};

// N columns of a warp's lower 16 lanes reduced (N = 16: lanes 16-31 end with nothing of use; N = 32: they hold neutral values):
// lane j < N ends with column j's.
template <bool MAX, int N>
__device__ __forceinline__ float reduce_columns(float (&v)[N], int lane) {
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            const float got = __shfl_xor_sync(0xffffffffu, give, o);
            v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    return v[0];
}

// The window: places [lo, hi) of all; `first` holds place lo, which starts at place `start`.
struct Window {
    int lo, hi, first, start;
};

// Every CTA cuts the batch by itself, from the lengths: it starts before the absorbed queries are there, and so this and its
// first tiles' copies cost nothing. (Lengths, tables and the cache are older than the kernel that makes the queries, which lets this
// one start only once it has waited for what came before it; they are read from L2, past whatever an SM may still hold.)
template <int THREADS>
__device__ Window make_window(const DecodeParams& p, int win) {
    constexpr int WARPS = THREADS / 32;
    __shared__ int sums[2][WARPS];
    __shared__ int found[2];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    auto places = [&](int b) {
        const int len = b < p.batch ? p.lens(b) : 0, n = tiles_checked(len, p.cap);
        if (len != 0 && n == 0 && blockIdx.x == 0) record_device_error(p.err, kErrAttnLength, b, len);
        return n ? n + kEnter : 0;
    };
    if (p.batch <= 32) {   // every warp by itself
        const int n = places(lane);
        int end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, o);
            end += lane >= o ? v : 0;
        }
        const int total = __shfl_sync(0xffffffffu, end, 31), W = max(1, (total + p.windows - 1) / p.windows);
        const int lo = win * W, hi = min(lo + W, total);
        const unsigned in = __ballot_sync(0xffffffffu, n && end - n <= lo && lo < end);
        const int first = in ? __ffs(in) - 1 : 0;
        __syncthreads();
        return {lo, hi, first, __shfl_sync(0xffffffffu, end - n, first)};
    }
    const int mine = places(t);
    int sum = mine;
    for (int b = t + THREADS; b < p.batch; b += THREADS) sum += places(b);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[0][warp] = sum;
    if (t == 0) found[0] = found[1] = 0;
    __syncthreads();
    int total = 0;
    for (int i = 0; i < WARPS; ++i) total += sums[0][i];
    const int W = max(1, (total + p.windows - 1) / p.windows);
    const int lo = win * W, hi = min(lo + W, total);
    int before = 0;
    for (int b0 = 0, k = 1; b0 < p.batch && before <= lo; b0 += THREADS, k ^= 1) {
        const int b = b0 + t, n = b0 == 0 ? mine : places(b);
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, o);
            at += lane >= o ? v : 0;
        }
        if (lane == 31) sums[k][warp] = at;
        __syncthreads();   // (the sums of two steps ago, and the total, are read)
        int all = 0;
        for (int i = 0; i < WARPS; ++i) {
            if (i == warp) at += before + all - n;
            all += sums[k][i];
        }
        if (lo < hi && n && at <= lo && lo < at + n) {
            found[0] = b;
            found[1] = at;
        }
        before += all;
    }
    __syncthreads();
    return {lo, hi, found[0], found[1]};
}

// After an abort, behind a barrier of the CTA: whoever gave up, the copies in flight land before the CTA leaves.
template <typename C>
__device__ __noinline__ void settle_decode(uint32_t bar, const int* issued, DevError* err, unsigned long long ns) {
    if (threadIdx.x != 32 * C::kCopyWarp) return;
    const Waits alone = {err, nullptr, ns};
    const int it = issued[0], sg = issued[2];
    if (issued[1]) bar_forgo(bar + (C::kKFull + (it - 1) % C::STAGES) * 8, issued[1] * 2 * C::GROUP);
    for (int i = max(0, it - C::STAGES); i < it; ++i)
        bar_wait(bar + (C::kKFull + i % C::STAGES) * 8, (uint32_t)(i / C::STAGES) & 1u, alone, 300);
    if (sg > 0) bar_wait(bar + C::kQFull * 8, (uint32_t)(sg - 1) & 1u, alone, 301);
}

// One CTA an SM, a window of the batch's tiles each. Two stages of 64 keys (73.7 KB each at rank 512) and the queries fill shared memory; a
// stage is freed a block of 16 keys at a time. Scores have the keys as rows and the heads as columns, so that a softmax thread keeps one key's
// heads in registers and stores its weights as the value product's B operand.
//  16 x 20000 - 40960, 64 heads, rank 512: 106 us of the call's 116, 5.3 TB/s. A tile takes 2.0 us, 1.75 where the cache is in L2: HBM's latency
//    and the chain of scores, softmax and values through two stages bound it together.
//  32 x 128 - 8192, 32 heads: 38.6 us of 47.7; 5.5 - 5.9 TB/s in the loop, where copies of such tiles alone reach 6.6.
template <int R, int NH>
__global__ void __launch_bounds__(Cfg<R, NH>::THREADS, 1) mla_decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = Cfg<R, NH>;
    constexpr int HN = C::HN;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[C::kBars];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    __shared__ int issued[3];   // tiles, blocks that the last one lacks, queries
    __shared__ int live_blocks[C::STAGES];
    __shared__ __align__(16) float ref[NH];          // the weights' reference of each head, log2, negated
    __shared__ float factor[NH], column[4][NH];
    __shared__ __align__(16) int4 turns[2];          // the softmax groups' sequence
    const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
    const uint32_t bar = su32(bars), ks = su32(smem), qs = ks + C::STAGES * C::TILE, ps = qs + C::QB;
    if (t == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            bar_init(bar + (C::kKFull + s) * 8, 1);
            for (int k = 0; k < 4; ++k) bar_init(bar + (C::kKEmpty + 4 * s + k) * 8, 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(bar + (C::kSFull + s) * 8, 1);
            bar_init(bar + (C::kPReady + s) * 8, C::kSoftWarps);
        }
        bar_init(bar + C::kQFull * 8, 1);
        bar_init(bar + C::kQEmpty * 8, 1);
        bar_init(bar + C::kDone * 8, 2);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tk);
        prefetch_map(&p.tq);
    }
    if (warp == C::kScoreWarp) tmem_alloc<C::COLS>(&tmem_at);
    fence_before();
    const int hg = blockIdx.x % p.groups, win = blockIdx.x / p.groups;
    const Window window = make_window<C::THREADS>(p, win);   // (and a barrier of the CTA)
    fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, tmem_at, 0);
    const Waits wt = {p.err, &abort_flag, p.ns};
    const Waits alone = {p.err, nullptr, p.ns};

    // The window's next sequence and its tiles [t0, t1); false behind the last.
    int next_b = window.first, start = window.lo < window.hi ? window.start : window.hi;
    auto next = [&](int4& s) {
        while (next_b < p.batch && start < window.hi) {
            const int b = next_b++, len = p.lens(b), n = tiles_checked(len, p.cap);
            if (n == 0) continue;
            const int t0 = max(window.lo - start - kEnter, 0), t1 = min(window.hi - start - kEnter, n);
            start += n + kEnter;
            if (t0 < t1) {
                s = make_int4(b, len, __shfl_sync(0xffffffffu, t0, 0), __shfl_sync(0xffffffffu, t1, 0));
                return true;
            }
        }
        return false;
    };
    auto sequences = [&](auto each) {   // `each` returns false to stop
        int4 s;
        while (next(s) && each(s.x, s.y, s.z, s.w)) {}
    };
    auto empty = [&](int i, int block) { return bar + (C::kKEmpty + 4 * (i % C::STAGES) + block) * 8; };
    auto turn = [&](int i) { return (uint32_t)(i / C::STAGES) & 1u; };   // parity of tile i's stage

    int it = 0, sg = 0;   // tiles and sequences so far
    if (warp == C::kCopyWarp) {
        // ------------------------------------------------ copies: lanes 0-3 bring the tile's four blocks
        int missing = 0;   // blocks of the last tile whose bytes are expected and not asked for
        sequences([&](int b, int len, int t0, int t1) {
            auto query = [&] {
                if (lane == 0) {
                    bar_expect(bar + C::kQFull * 8, C::QB);
                    copy_box5(qs, &p.tq, 0, hg * NH, 0, 0, b, bar + C::kQFull * 8);
                }
                ++sg;
            };
            bool first = sg == 0;
            if (!first) {
                if (!warp_wait(bar + C::kQEmpty * 8, (uint32_t)(sg - 1) & 1u, wt, 100)) return false;
                query();
            }
            const int nblk = (len + kBlock - 1) / kBlock;
            const int32_t* table = p.tables + (size_t)b * p.maxb;
            auto load_id = [&](int tt) { return lane < 4 && 4 * tt + lane < nblk ? __ldcg(table + 4 * tt + lane) : -1; };
            int id = load_id(t0);
            for (int tt = t0; tt < t1; ++tt, ++it) {
                if (first && it == C::STAGES) {   // the absorbed queries are the previous kernel's; what the cache holds is older
                    pdl_wait();
                    pdl_trigger();
                    query();
                    first = false;
                }
                const int s = it % C::STAGES;
                const bool in = lane < 4 && 4 * tt + lane < nblk, live = in && id >= 0 && id < p.num_blocks;
                if (in && !live && hg == 0) record_device_error(p.err, kErrAttnBlock, b * p.maxb + 4 * tt + lane, id);
                const unsigned mask = __ballot_sync(0xffffffffu, live) & 15u;
                const int now = live ? 2 * id : 2 * (int)p.num_blocks;   // outside: zeros
                if (tt + 1 < t1) id = load_id(tt + 1);
                // The stage's last phase is complete before it is armed again, also where a wait has failed (weights of its tile are then
                // reported, and its blocks given back, whatever has arrived).
                bool ok = it < C::STAGES || warp_wait(bar + (C::kKFull + s) * 8, turn(it - C::STAGES), wt, 204), sent = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // (behind a wait that failed nothing is armed or asked for)
                    ok = ok && (it < C::STAGES || warp_wait(empty(it, k), turn(it - C::STAGES), wt, 200 + k));
                    if (k == 0 && lane == 0) {
                        live_blocks[s] = (int)mask;
                        fence_async();   // rows cleared through the generic proxy before the copies into them
                    }
                    __syncwarp();
                    if (lane == k && ok) {
                        if (k == 0) bar_expect(bar + (C::kKFull + s) * 8, C::TILE);
                        copy_box4(ks + s * C::TILE + k * 2 * C::GROUP, &p.tk, 0, 0, 0, now, bar + (C::kKFull + s) * 8);
                        sent = true;
                    }
                    __syncwarp();
                }
                if (!ok) {
                    const int blocks = __popc(__ballot_sync(0xffffffffu, sent));
                    missing = blocks ? 4 - blocks : 0;
                    it += blocks > 0;
                    return false;
                }
            }
            if (first) {
                pdl_wait();
                pdl_trigger();
                query();
            }
            return true;
        });
        if (lane == 0) {
            issued[0] = it;
            issued[1] = missing;
            issued[2] = sg;
        }
    } else if (warp == C::kScoreWarp) {
        // ------------------------------------------------ S^T = K q'^T, two tiles ahead of their values at most
        constexpr uint32_t I = instr(64, C::NQ, false, false);
        const uint32_t one = elect_one();
        const uint64_t kd = operand(ks, 16, C::GROUP, 2), qd = operand(qs, 16, 1024, 2);
        sequences([&](int, int, int t0, int t1) {
            if (!warp_wait(bar + C::kQFull * 8, (uint32_t)sg & 1u, wt, 401)) return false;
            ++sg;
            for (int tt = t0; tt < t1; ++tt, ++it) {
                if (it >= 2 && !warp_wait(bar + (C::kPReady + (it & 1)) * 8, (uint32_t)((it >> 1) - 1) & 1u, wt, 402)) return false;   // its S is read
                if (!warp_wait(bar + (C::kKFull + it % C::STAGES) * 8, turn(it), wt, 403)) return false;
                fence_after();
                const uint64_t k0 = kd + (it % C::STAGES) * (C::TILE >> 4);
#pragma unroll
                for (int k = 0; k < 4 * C::CH; ++k)
                    mma_ss(one, tb + C::SCOL + (it & 1) * C::NQ, k0 + (((k >> 2) * 1024 + (k & 3) * 32) >> 4),
                           qd + (((k >> 2) * C::NQ * 128 + (k & 3) * 32) >> 4), I, k > 0);
                mma_commit(one, bar + (C::kSFull + (it & 1)) * 8);
                if (tt + 1 == t1) mma_commit(one, bar + C::kQEmpty * 8);
            }
            return true;
        });
        mma_commit(one, bar + C::kDone * 8);   // every product has ended before the tensor memory is given back
        warp_wait(bar + C::kDone * 8, 0u, alone, 500);
    } else if (warp == C::kValueWarp) {
        // ------------------------------------------------ O^T += V^T P
        constexpr uint32_t I = instr(128, NH, true, true);
        const uint32_t one = elect_one();
        const uint64_t vd = operand(ks, 1024, C::GROUP, 2), pd = operand(ps, 16, 8 * NH * 2, C::PSW);
        sequences([&](int, int, int t0, int t1) {
            for (int tt = t0; tt < t1; ++tt, ++it) {
                if (!warp_wait(bar + (C::kPReady + (it & 1)) * 8, (uint32_t)(it >> 1) & 1u, wt, 404)) return false;
                fence_after();
                const uint64_t v = vd + (it % C::STAGES) * (C::TILE >> 4), w = pd + (it % C::PBUF) * (C::PB >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int m = 0; m < C::MT; ++m)
                        mma_ss(one, tb + m * NH, v + ((2 * k * C::GROUP + 2 * m * 1024) >> 4), w + ((k * 16 * NH * 2) >> 4), I, tt > t0 || k > 0);
                    mma_commit(one, empty(it, k));
                }
            }
            return true;
        });
        mma_commit(one, bar + C::kDone * 8);
        warp_wait(bar + C::kDone * 8, 0u, alone, 501);
    } else {
        // ------------------------------------------------ softmax: warps 4 g .. 4 g + 3 have half of the heads; a lane has a key, warp w
        // of four the keys 16 w .. 16 w + 15 (M = 64: the scores fill 16 of a warp's 32 lanes).
        // The four warps run the same tiles whatever their waits return, and take them from one of them (lengths that change during the
        // launch, an error of the caller's, would else tell them apart), so that their barriers always meet.
        const int g = warp >> 2, w4 = warp & 3, h0 = g * HN, tg = t & 127;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const int key = 16 * w4 + (lane & 15);
        const bool mine = lane < 16;
        auto meet = [&] { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory"); };
        for (;;) {
            if (w4 == 0) {
                int4 s;
                if (!next(s)) s.x = -1;
                if (lane == 0) turns[g] = s;
            }
            meet();
            const int4 now = turns[g];
            const int b = now.x, len = now.y, t0 = __shfl_sync(0xffffffffu, now.z, 0), t1 = __shfl_sync(0xffffffffu, now.w, 0);
            if (b < 0) break;
            float l[HN];
#pragma unroll
            for (int h = 0; h < HN; ++h) l[h] = 0.f;
            for (int tt = t0; tt < t1; ++tt, ++it) {
                const int s = it % C::STAGES;
                warp_wait(bar + (C::kKFull + s) * 8, turn(it), wt, 600);   // live_blocks, and the rows to clear
                const int left = len - tt * kTile;                       // keys of this tile
                const bool seen = mine && key < left && ((live_blocks[s] >> w4) & 1);
                if (left < kTile && (left & 15)) {   // what the last block holds behind the sequence must not meet the products
                    const int end = (left + 15) & ~15;
                    for (int i = t; i < (end - left) * C::CH * 8; i += 32 * C::kSoftWarps) {
                        const int row = left + i / (C::CH * 8), c = i % (C::CH * 8);
                        *reinterpret_cast<uint4*>(smem + s * C::TILE + (row >> 3) * C::GROUP + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                warp_wait(bar + (C::kSFull + (it & 1)) * 8, (uint32_t)(it >> 1) & 1u, wt, 601);
                fence_after();
                const uint32_t sc = tb + lanes + C::SCOL + (it & 1) * C::NQ + h0;
                const float2 scale = make_float2(p.scale_log2, p.scale_log2);
                float x[HN];
                float over = -INFINITY;
                auto scores = [&](float* s) {
                    if constexpr (C::HALVES == 2) {
                        float r[HN];
                        tmem_raw<HN>(sc, s);
                        tmem_raw<HN>(sc + NH, r);
                        wait_ld();
                        tie<HN>(s);
                        tie<HN>(r);
#pragma unroll
                        for (int h = 0; h < HN; h += 2) {
                            const float2 a = add2(make_float2(s[h], s[h + 1]), make_float2(r[h], r[h + 1]));
                            s[h] = a.x;
                            s[h + 1] = a.y;
                        }
                    } else tmem_load<HN>(sc, s);
                };
                auto exponents = [&] {   // x: how far the scores lie above their heads' references
                    scores(x);
                    if (seen) {
#pragma unroll
                        for (int h = 0; h < HN; h += 4) {
                            const float4 r = *reinterpret_cast<const float4*>(ref + h0 + h);
                            const float2 a = fma2(make_float2(x[h], x[h + 1]), scale, make_float2(r.x, r.y));
                            const float2 c = fma2(make_float2(x[h + 2], x[h + 3]), scale, make_float2(r.z, r.w));
                            x[h] = a.x;
                            x[h + 1] = a.y;
                            x[h + 2] = c.x;
                            x[h + 3] = c.y;
                            over = fmaxf(over, fmaxf(fmaxf(a.x, a.y), fmaxf(c.x, c.y)));
                        }
                    }
                };
                // The reference follows the running maximum by steps: weights of up to 2^kLag are as exact in f16 as
                // smaller ones, and O has to be scaled only when a score passes that.
                unsigned raise = 1;
                if (tt > t0) {
                    exponents();
                    asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.or.pred b, %2, 128, a;\n selp.u32 %0, 1, 0, b;\n}"
                                 : "=r"(raise) : "r"((unsigned)(over > kLag)), "r"(1 + g) : "memory");
                }
                if (raise) {
                    {
                        float v[HN];
                        scores(v);
#pragma unroll
                        for (int i = 0; i < HN; ++i) v[i] = seen ? v[i] * p.scale_log2 : -INFINITY;
                        const float most = reduce_columns<true, HN>(v, lane);
                        if (lane < HN) column[w4][h0 + lane] = most;
                    }
                    meet();
                    if (tg < HN) {
                        const int h = h0 + tg;
                        const float most = fmaxf(fmaxf(column[0][h], column[1][h]), fmaxf(column[2][h], column[3][h]));
                        // a finite reference where no key is left, so that the next tile's weights stay numbers
                        const float old = tt == t0 ? -1e30f : -ref[h], now = fmaxf(old, most - kLift);
                        factor[h] = tt == t0 ? 0.f : ex2(old - now);
                        ref[h] = -now;
                    }
                    meet();
                    if (tt > t0) {
#pragma unroll
                        for (int h = 0; h < HN; ++h) l[h] *= factor[h0 + h];
                        warp_wait(empty(it - 1, 3), turn(it - 1), wt, 602);   // O holds the tiles before this one
                        fence_after();
#pragma unroll 1
                        for (int m = 0; m < C::MT; ++m) {
                            float v[HN];
                            uint32_t u[HN];
                            tmem_load<HN>(tb + lanes + m * NH + h0, v);
#pragma unroll
                            for (int i = 0; i < HN; ++i) u[i] = __float_as_uint(v[i] * factor[h0 + i]);
                            if constexpr (HN == 32) tmem_st32(tb + lanes + m * NH + h0, u);
                            else tmem_st16(tb + lanes + m * NH + h0, u);
                        }
                        wait_st();
                    }
                    exponents();
                }
                // the tile before last (or, with one buffer, the last) has taken its weights
                if (it >= C::PBUF) warp_wait(empty(it - C::PBUF, 3), turn(it - C::PBUF), wt, 603);
                unsigned char* row = smem + C::STAGES * C::TILE + C::QB + (it % C::PBUF) * C::PB + key * NH * 2;
                const int sw = NH == 64 ? key & 7 : (key >> 1) & 3;
                if (mine) {   // (a key that is not seen, its scores never looked at, weighs 0)
#pragma unroll
                    for (int h = 0; h < HN; h += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 w = seen ? make_float2(ex2(x[h + i]), ex2(x[h + i + 1])) : make_float2(0.f, 0.f);
                            const float2 sum = add2(make_float2(l[h + i], l[h + i + 1]), w);
                            l[h + i] = sum.x;
                            l[h + i + 1] = sum.y;
                            u[i / 2] = pack_half(w.x, w.y);
                        }
                        *reinterpret_cast<uint4*>(row + ((((h0 + h) >> 3) ^ sw) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar + (C::kPReady + (it & 1)) * 8);
            }
            // the part: O^T's lanes are latent values, its columns heads
            const int heads = min(NH, p.H - hg * NH);
            const size_t part = ((size_t)hg * (p.windows + p.batch) + win + b) * p.per;
            {
                float v[HN];
#pragma unroll
                for (int i = 0; i < HN; ++i) v[i] = mine ? l[i] : 0.f;
                const float sum = reduce_columns<false, HN>(v, lane);
                if (lane < HN) column[w4][h0 + lane] = sum;
            }
            meet();
            if (tg < HN && h0 + tg < heads) {
                const int h = h0 + tg;
                p.stats[part + h] = make_float2(-ref[h], column[0][h] + column[1][h] + column[2][h] + column[3][h]);
            }
            warp_wait(empty(it - 1, 3), turn(it - 1), wt, 604);
            fence_after();
#pragma unroll 1
            for (int m = 0; m < C::MT; ++m) {
                float v[HN];
                tmem_load<HN>(tb + lanes + m * NH + h0, v);
                float* o = p.parts + (part + h0) * R + 128 * m + 32 * w4 + lane;
#pragma unroll
                for (int i = 0; i < HN; ++i)
                    if (h0 + i < heads) o[i * R] = v[i];
            }
            fence_before();
            meet();   // before the next sequence's reference and columns
        }
    }
    // (the copying warp of a window with tiles has waited already)
    pdl_wait();
    pdl_trigger();
    fence_before();
    __syncthreads();
    if (abort_flag) settle_decode<C>(su32(bars), issued, p.err, p.ns);
    if (warp == C::kScoreWarp) {
        fence_after();
        tmem_free<C::COLS>(tb);
    }
}

// ---------------------------------------------------------------- parts joined, values projected
struct JoinParams {
    const __half* w;       // [H][2 D][R]
    Lengths lens;
    const float* parts;
    const float2* stats;
    __half* out;           // [batch][H][D]
    long long cap;
    int batch, H, windows, per, rows;   // rows: sequences of a cluster, 1, 2, 4 or 8
};

// A cluster of four CTAs takes one head and `rows` sequences. Each CTA joins the parts of a quarter of the latent values, hands
// them to the other three through distributed shared memory, and multiplies all of them with a quarter of the head's value
// rows (they are B fragments of m16n8k16: a lane's 16 bytes are 8 consecutive values of one row; which k they stand for is the
// products' own business as long as A's are the same). What the lengths alone decide is worked out before the wait on the
// attention; behind it the parts and their statistics are loaded at once.
// o enters the product as two f16 numbers (22 bits): as one, its rounding alone would be as large as the output's.
// Bound by latency (lengths, statistics, parts, the cluster's barrier, weights): 4 us for one sequence of 32 heads, 6 for 32 (a CTA a head
// instead of a cluster: 3 us more at one).
constexpr int kJoinThreads = 256, kJoinCtas = 4, kJoinRows = 8;
template <int D, int R, int NH>
__global__ void __launch_bounds__(kJoinThreads, 4) __cluster_dims__(kJoinCtas, 1, 1) mla_join_kernel(const __grid_constant__ JoinParams p) {
    constexpr int OP = R + 32, PER = R / kJoinCtas / 4, GROUPS = kJoinThreads / PER;   // threads of a sequence's quarter (4 values each)
    constexpr int NT = D / kJoinCtas / 8, KW = 8 / NT, KS = R / 32 / KW;               // 8-row tiles of a CTA, warps and steps of one
    constexpr int AT_ONCE = 4;                                                         // parts a thread loads at a time
    __shared__ __align__(16) __half os[2][kJoinRows * OP];   // o, its upper and lower halves
    __shared__ __align__(16) float4 share[GROUPS][PER];
    __shared__ float scale[kJoinRows][kMaxWin];
    __shared__ float sums[8][kJoinRows][8];
    __shared__ int first[kJoinRows], count[kJoinRows], places[2][8];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quarter = blockIdx.x % kJoinCtas, h = blockIdx.x / kJoinCtas;
    const int b0 = blockIdx.y * p.rows, nt = warp / KW, kw = warp % KW;
    const int d0 = quarter * (D / kJoinCtas) + 8 * nt;       // this warp's value rows
    const int hg = h / NH;
    const size_t base = (size_t)hg * (p.windows + p.batch);
    // this CTA's value rows into L2 while the attention still runs
    for (int i = t; i < D / kJoinCtas * (R / 64); i += kJoinThreads)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w + ((size_t)h * 2 * D + D + quarter * (D / kJoinCtas)) * R + (size_t)i * 64));
    // every CTA of the cluster has started before another writes into it (waited for below)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    {
        // the places of all sequences and of those before this cluster's, as the attention counts them
        int all = 0, before = 0;
        for (int b = t; b < p.batch; b += kJoinThreads) {
            const int n = tiles_checked(p.lens(b), p.cap);
            all += n ? n + kEnter : 0;
            before += n && b < b0 ? n + kEnter : 0;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        if (lane == 0) {
            places[0][warp] = all;
            places[1][warp] = before;
        }
        __syncthreads();
        if (t < kJoinRows) {   // (lanes 0-7 of one warp)
            all = before = 0;
            for (int i = 0; i < 8; ++i) {
                all += places[0][i];
                before += places[1][i];
            }
            const int W = max(1, (all + p.windows - 1) / p.windows), b = b0 + t;
            const int n = t < p.rows && b < p.batch ? tiles_checked(p.lens(b), p.cap) : 0, mine = n ? n + kEnter : 0;
            int at = mine;
#pragma unroll
            for (int o = 1; o < kJoinRows; o <<= 1) {
                const int v = __shfl_up_sync(0xffu, at, o);
                at += t >= o ? v : 0;
            }
            at += before - mine + kEnter;
            // (inside the workspace whatever the lengths do meanwhile)
            const int w0 = n ? min(at / W, p.windows - 1) : 0;
            first[t] = w0 + b;
            count[t] = n ? min((at + n - 1) / W, p.windows - 1) - w0 + 1 : 0;
        }
        __syncthreads();
    }
    const int g = t / PER, at = t % PER;
    const int split = GROUPS / p.rows, r0 = g / split;   // groups of a sequence (powers of two; at least one)
    const float4* src = reinterpret_cast<const float4*>(p.parts + ((base + first[r0]) * p.per + h % NH) * R + quarter * (R / kJoinCtas)) + at;
    const float2* stats = p.stats + (base + first[warp] + lane) * p.per + h % NH;
    const size_t next = (size_t)split * (p.per * (R / 4));
    const int c0 = count[r0];
    pdl_wait();
    pdl_trigger();
    float4 v[AT_ONCE];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            v[i] = i0 + i * split < c0 ? __ldcg(src + (size_t)i0 * (p.per * (R / 4)) + i * next) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(g % split);
    {
        const int r = warp, c = count[r];
        constexpr int MORE = kMaxWin / 32;
        float2 s[MORE];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < MORE; ++i) {
            s[i] = 32 * i + lane < c ? __ldcg(stats + 32 * i * p.per) : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, s[i].x);
        }
        if (c > 0) {
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
            for (int i = 0; i < MORE; ++i) {
                s[i].x = ex2(s[i].x - m);
                l += s[i].y * s[i].x;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // no key left: 0; NaN stays
#pragma unroll
            for (int i = 0; i < MORE; ++i)
                if (32 * i + lane < c) scale[r][32 * i + lane] = s[i].x * inv;
        }
    }
    __syncthreads();
    auto put = [&](int r, float4 a) {    // 4 values of o to all four CTAs
        const float x[4] = {a.x, a.y, a.z, a.w};
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i] - __half2float(__float2half_rn(x[i]));
        const uint32_t u[2][2] = {{pack_half(x[0], x[1]), pack_half(x[2], x[3])}, {pack_half(y[0], y[1]), pack_half(y[2], y[3])}};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t here = su32(os[i] + r * OP + quarter * (R / kJoinCtas) + 4 * at);
#pragma unroll
            for (int c = 0; c < kJoinCtas; ++c) {
                uint32_t there;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(c));
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(there), "r"(u[i][0]), "r"(u[i][1]) : "memory");
            }
        }
    };
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = g % split; i0 < c0; i0 += AT_ONCE * split) {
        if (i0 >= AT_ONCE * split) load(i0);
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const float f = i0 + i * split < c0 ? scale[r0][i0 + i * split] : 0.f;
            a.x = fmaf(v[i].x, f, a.x);
            a.y = fmaf(v[i].y, f, a.y);
            a.z = fmaf(v[i].z, f, a.z);
            a.w = fmaf(v[i].w, f, a.w);
        }
    }
    if (split > 1) {
        share[g][at] = a;
        __syncthreads();
        a = share[g < p.rows ? g * split : 0][at];
        for (int i = 1; i < split; ++i) {
            const float4 x = share[g < p.rows ? g * split + i : 0][at];
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (g < p.rows || split == 1) put(g, a);   // (with one group a sequence, g is the sequence)
    uint4 w[KS];
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < KS; ++k)
        w[k] = __ldg(reinterpret_cast<const uint4*>(p.w + ((size_t)h * 2 * D + D + d0 + (lane >> 2)) * R + 32 * (kw * KS + k) + 8 * (lane & 3)));
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    float c[4][4] = {};   // four chains of products
    const int r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // rows 8-15 of the products are not used; rows that are not there keep to themselves
            const uint4 x = *reinterpret_cast<const uint4*>(os[half] + r * OP + 32 * (kw * KS + k) + 8 * j);
            mma16(c[half], x.x, 0u, x.y, 0u, w[k].x, w[k].y);
            mma16(c[2 + half], x.z, 0u, x.w, 0u, w[k].z, w[k].w);
        }
    sums[warp][r][2 * j] = (c[0][0] + c[2][0]) + (c[1][0] + c[3][0]);
    sums[warp][r][2 * j + 1] = (c[0][1] + c[2][1]) + (c[1][1] + c[3][1]);
    __syncthreads();
    if (kw == 0 && count[r]) {
        float y0 = sums[warp][r][2 * j], y1 = sums[warp][r][2 * j + 1];
#pragma unroll
        for (int i = 1; i < KW; ++i) {
            y0 += sums[warp + i][r][2 * j];
            y1 += sums[warp + i][r][2 * j + 1];
        }
        *reinterpret_cast<__half2*>(p.out + ((size_t)(b0 + r) * p.H + h) * D + d0 + 2 * j) = __floats2half2_rn(y0, y1);
    }
}

// ---------------------------------------------------------------- host
struct DecodeShape {
    int NH, groups, per;
    size_t parts, stats, total;   // offsets in the workspace; the absorbed queries come first
};
static DecodeShape decode_shape(int64_t batch, int H, int R) {
    DecodeShape s = {};
    s.NH = H <= 32 ? 32 : 64;
    s.groups = (H + s.NH - 1) / s.NH;
    s.per = std::min(H, s.NH);
    const size_t win = kMaxWin / s.groups + 1, rows = (size_t)s.groups * (batch + win) * s.per;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    s.parts = up((size_t)batch * H * (R + kRope) * 2 * (s.NH == 32 ? 2 : 1));
    s.stats = s.parts + rows * R * 4;
    s.total = s.stats + up(rows * 8);
    return s;
}

template <int D, int R, int NH>
static int decode_go(const AttnIn& a, bool chunk, const DecodeShape& sh, cudaStream_t s) {
    using C = Cfg<R, NH>;
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "latent attention: no device error record");
    static std::atomic<unsigned long long> done{0};
    QL_TRY_CUDA(allow_smem_once(mla_decode_kernel<R, NH>, C::SMEM, done));
    unsigned char* ws = static_cast<unsigned char*>(a.ws);
    int windows = std::min(num_sms(), kMaxWin) / sh.groups;
    if (windows < 1) windows = 1;
    AbsorbParams ap = {static_cast<const __half*>(a.q), static_cast<const __half*>(a.w), reinterpret_cast<__half*>(ws), (int)a.rows, a.H, C::HALVES, err};
    DecodeParams dp = {};
    const uint64_t row = (R + kRope) * 2;
    const uint64_t kd[4] = {64, 8, (uint64_t)C::CH, (uint64_t)a.num_blocks * 2}, kst[3] = {row, 128, 8 * row};
    const uint32_t kb[4] = {64, 8, (uint32_t)C::CH, 2};
    if (int rc = f16_tensor_map(a.pool, 4, kd, kst, kb, &dp.tk)) return rc;
    const uint64_t qd[5] = {64, (uint64_t)a.H, C::HALVES, (uint64_t)C::CH, (uint64_t)a.rows}, qst[4] = {row, a.H * row, 128, C::HALVES * a.H * row};
    const uint32_t qb[5] = {64, (uint32_t)NH, C::HALVES, (uint32_t)C::CH, 1};
    if (int rc = f16_tensor_map(ws, 5, qd, qst, qb, &dp.tq)) return rc;
    dp.tables = a.table;
    dp.lens = {chunk ? nullptr : a.lens, chunk ? a.lens : nullptr, (int)a.rows, (long long)a.maxb * kBlock};
    dp.parts = reinterpret_cast<float*>(ws + sh.parts);
    dp.stats = reinterpret_cast<float2*>(ws + sh.stats);
    dp.maxb = chunk ? 0 : a.maxb;
    dp.cap = (long long)a.maxb * kBlock;
    dp.num_blocks = a.num_blocks;
    dp.batch = (int)a.rows;
    dp.H = a.H;
    dp.windows = windows;
    dp.groups = sh.groups;
    dp.per = sh.per;
    dp.scale_log2 = a.scale * 1.44269504088896340736f;
    dp.err = err;
    dp.ns = 2000000000ull;
    JoinParams jp = {ap.w, dp.lens, dp.parts, dp.stats, static_cast<__half*>(a.out), dp.cap, (int)a.rows, a.H, windows, sh.per, kJoinRows};
    while (jp.rows > 1 && jp.rows / 2 >= a.rows) jp.rows /= 2;
    cudaError_t e = launch(mla_absorb_kernel<D, R>, dim3((unsigned)(a.H * (R / 64)), (unsigned)((a.rows + 63) / 64)), dim3(128), 0, s, true, ap);
    if (e == cudaSuccess) e = launch(mla_decode_kernel<R, NH>, dim3((unsigned)(windows * sh.groups)), dim3(C::THREADS), C::SMEM, s, true, dp);
    if (e == cudaSuccess)
        e = launch(mla_join_kernel<D, R, NH>, dim3((unsigned)(a.H * kJoinCtas), (unsigned)((a.rows + jp.rows - 1) / jp.rows)), dim3(kJoinThreads), 0, s,
                   true, jp);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "latent attention, absorbed form");
}

size_t absorbed_workspace(int64_t rows, int H, int R) { return decode_shape(rows, H, R).total; }

int absorbed_launch(const AttnIn& a, bool chunk, cudaStream_t s) {
    const DecodeShape sh = decode_shape(a.rows, a.H, a.R);
    const bool small = sh.NH == 32;
    if (a.D == 128) {
        if (a.R == 512) return small ? decode_go<128, 512, 32>(a, chunk, sh, s) : decode_go<128, 512, 64>(a, chunk, sh, s);
        return small ? decode_go<128, 256, 32>(a, chunk, sh, s) : decode_go<128, 256, 64>(a, chunk, sh, s);
    }
    if (a.R == 512) return small ? decode_go<64, 512, 32>(a, chunk, sh, s) : decode_go<64, 512, 64>(a, chunk, sh, s);
    return small ? decode_go<64, 256, 32>(a, chunk, sh, s) : decode_go<64, 256, 64>(a, chunk, sh, s);
}

}  // namespace mla
}  // namespace ql

extern "C" size_t ql_mla_decode_workspace_bytes(int64_t batch, int n_heads, int head_dim, int rank, int64_t max_blocks_per_seq) {
    if (!ql::mla::shape_ok(head_dim, rank) || batch < 1 || batch > 65535 || n_heads < 1 || n_heads > 1024 || batch * n_heads >= (1 << 22) ||
        max_blocks_per_seq < 1 || max_blocks_per_seq > (1 << 20) || batch * max_blocks_per_seq >= (1ll << 32))
        return 0;
    return ql::mla::absorbed_workspace(batch, n_heads, rank);
}

extern "C" int ql_mla_attn_decode(const void* d_q, const void* d_w_kv, const void* d_pool, const int32_t* d_block_tables,
                                  const int32_t* d_context_lens, int64_t batch, int n_heads, int head_dim, int rank, int rope_dim,
                                  int block_size, int64_t max_blocks_per_seq, int64_t num_blocks, float scale, void* d_out,
                                  void* d_workspace, size_t workspace_bytes, void* stream) {
    using namespace ql;
    using namespace ql::mla;
    const AttnIn a = {d_q, d_w_kv, d_pool, d_block_tables, d_context_lens, batch, batch, max_blocks_per_seq, num_blocks, n_heads, head_dim, rank,
                      rope_dim, block_size, scale, d_out, d_workspace, workspace_bytes};
    if (int rc = attn_check("ql_mla_attn_decode", a, ql_mla_decode_workspace_bytes(batch, n_heads, head_dim, rank, max_blocks_per_seq))) return rc;
    return absorbed_launch(a, false, static_cast<cudaStream_t>(stream));
}
