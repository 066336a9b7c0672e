// The next token of a row of logits: temperature, top-k, top-p, min-p and one uniform number.
//
// Every kept set is a prefix of one order (logit falling, index rising), so all filters together are
// one border (key, index); the token is then a position in the running sum over the kept tokens in
// index order. Weights w = 2^((l - max) log2(e) / T) are 40-bit fixed-point integers and sums 64-bit
// ones: exact, whatever the order of additions, and the same in every pass.
//
// The border of top-k (a count) or top-p (a weight) is found by digits, the histogram of 128 bins
// naming the bin that the border falls into and the next round dividing that bin: 7 bits at a time of
// the distance from the largest logit on a 23-bit scale of 24 T, then of the logit's ordered bits, then
// of the index, until few enough candidates are left, which are ranked against one another. Two shorter
// ways, where the lists that they need are long enough: a top-k of up to 128 takes its threshold from the
// threads' largest logits (list_first), and top-p divides a list of the first histogram's border bin
// (nucleus), so that two passes over the tokens are all.
//
// A row is read once: a thread-block cluster holds it in shared memory, each CTA a run of tokens, and
// sums, histograms and candidates are exchanged through distributed shared memory, one cluster
// barrier each; every CTA then draws the same conclusions. A histogram has a column per lane, so that
// a warp's additions never meet; its weights are split into 20-bit halves that 32-bit sums hold.
//
// Measured (vocab 151936): one row with top-k 50 and top-p 0.95 9.4 us, of which the load is 1.3, the
// largest logit 1.1, the threshold 1.1, the list 2.6 and the draw 2.4: barriers and latency, not memory.
// Top-p 0.9 alone 21 us at T 0.6 - 1.2 (15.3 at T 0.3), 38 us for 32 rows; 32 rows with min-p 0.02 too 17 us, no filter 13 us. 256 rows of
// 50021 without a filter 27.5 us (1.9 TB/s): a pass at memory speed (8.7 us), a barrier, and one of 28
// instructions a token (8.5 us), on the SMs that hold two rows of the 1.7 there are to each.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "ql_internal.h"
#include "ql_sample.h"

namespace ql {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 128, kDigit = 7;
constexpr int kList = 128;                      // candidates that are ranked directly
constexpr int kFewRows = 4;                     // rows whose clusters may have 16 CTAs
constexpr int kMaxCluster = 16, kPortableCluster = 8;
constexpr uint32_t kQMax = (1u << 23) - 1;      // the distance scale's last value: all that is farther
constexpr uint32_t kKeyMin = 0x00800000u;       // the key after -inf's

// 2^(j / 64) in 30 bits after the point
__device__ const uint32_t kExp2[64] = {
    0x40000000u, 0x40b268fau, 0x4166c34cu, 0x421d1462u, 0x42d561b4u, 0x438fb0cbu, 0x444c0740u, 0x450a6abbu,
    0x45cae0f2u, 0x468d6faeu, 0x47521cc6u, 0x4818ee22u, 0x48e1e9bau, 0x49ad1598u, 0x4a7a77d4u, 0x4b4a169cu,
    0x4c1bf829u, 0x4cf022cau, 0x4dc69cddu, 0x4e9f6cd4u, 0x4f7a9930u, 0x50582888u, 0x51382182u, 0x521a8ad7u,
    0x52ff6b55u, 0x53e6c9dau, 0x54d0ad5au, 0x55bd1cdbu, 0x56ac1f75u, 0x579dbc57u, 0x5891fac1u, 0x5988e209u,
    0x5a82799au, 0x5b7ec8f2u, 0x5c7dd7a4u, 0x5d7fad59u, 0x5e8451d0u, 0x5f8bccdbu, 0x60962665u, 0x61a3666du,
    0x62b39509u, 0x63c6ba64u, 0x64dcdec3u, 0x65f60a7fu, 0x6712460bu, 0x683199edu, 0x69540ec9u, 0x6a79ad56u,
    0x6ba27e65u, 0x6cce8ae1u, 0x6dfddbccu, 0x6f307a41u, 0x70666f76u, 0x719fc4b9u, 0x72dc8374u, 0x741cb528u,
    0x75606374u, 0x76a7980fu, 0x77f25cceu, 0x7940bb9eu, 0x7a92be8bu, 0x7be86fbau, 0x7d41d96eu, 0x7e9f0606u,
};

typedef unsigned long long u64;

struct Params {
    const void* logits;
    long long stride;
    int vocab, per;               // tokens of a row, and of a CTA (a multiple of 8)
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* uniform;
    long long uniform_stride;
    const int32_t* positions;
    const int32_t* active;
    int32_t* tokens;
    float* probs;
    bool early;   // the next grid may start at once: this one leaves it half of the SMs (on shared ones its CTAs
                  // would come to lie unevenly: 256 rows after 256 rows 34.0 us against 27.5)
};

// ---- the cluster
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the address of this CTA's shared variable in the CTA of rank r
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t r) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    return a;
}
__device__ __forceinline__ u64 remote_u64(const void* p, uint32_t r) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, r)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t r) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, r)) : "memory");
    return v;
}

__device__ __forceinline__ float canonical(float l) {
    return fminf(fmaxf(l, -INFINITY), FLT_MAX) + 0.0f;   // NaN: -inf, never drawn; -0 and +0 tie
}

// Bits that order as the logits do.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// What turns a logit into a weight and into a distance, the same for the whole row.
struct RowScale {
    float ref, c_hi, c_lo, magic, low;   // (l - ref) (c_hi + c_lo): the exponent in 64ths
    float top, dist;                     // distance (top - l) dist
    __device__ __forceinline__ void set(float t, float temp) {
        constexpr float k_hi = 92.332482616893656754f, k_lo = (float)(92.332482616893656754 - (double)k_hi);   // 64 log2(e)
        c_hi = __fdiv_rn(k_hi, temp);
        c_lo = __fdiv_rn(fmaf(-c_hi, temp, k_hi) + k_lo, temp);
        top = t;
        // exponents of logits near the largest stay below 2^21 in magnitude, where the floor is exact
        ref = fabsf(t * c_hi) > 0x1p20f ? t : 0.f;
        const float x = t - ref;
        magic = 12582912.0f - floorf(__fmul_rd(x, c_hi));
        low = fmaxf(x - __fdiv_rn(2600.f, c_hi), -FLT_MAX);            // 2^-40.6 of the largest: weight 0 (see hot)
        dist = fminf(__fdiv_rn(8388608.f / 24.f, temp), FLT_MAX);     // finite: 0 dist is 0
    }
    // No finite logit is so far below the largest (T of 1.2e37 and more): weight() takes -inf for the least finite
    // one, which weighs something. Passes over such a row look at each token's key (a border that is not all()) or
    // compare its logit with the least one kept.
    __device__ __forceinline__ bool hot() const { return low == -FLT_MAX; }
};

// The weight of logit l: 2^(40 + e / 64), e = (l - ref) 64 log2(e) / T minus its floor at the largest
// logit. The floor and the fraction come from fused multiply-adds of l itself, each rounded once, so
// that the error of a large l does not enter; 2^(fraction / 64) - 1 is the series of exp to the fourth
// power (the next term is below 2^-40), the product with the table is an integer one.
// The clamp keeps e / 64 above -42 and takes a NaN and -inf to weight 0, in a row that is not hot().
// REF false: r.ref is 0.
template <bool REF = true>
__device__ __forceinline__ u64 weight(float l, const RowScale& r, const uint32_t* table) {
    const float x = fmaxf(REF ? l - r.ref : l, r.low);
    const float z = __fmaf_rd(x, r.c_hi, r.magic);
    float f = __fmaf_rn(x, r.c_hi, r.magic - z);
    f = __fmaf_rn(x, r.c_lo, f);
    const uint32_t bits = __float_as_uint(z);    // 0x4B400000 + e
    constexpr float y = 0.010830424696249145f;   // ln 2 / 64
    constexpr float s = 4294967296.0f;
    float q = fmaf(f, s * y * y * y * y / 24.f, s * y * y * y / 6.f);
    q = fmaf(f, q, s * y * y / 2.f);
    q = fmaf(f, q, s * y);
    const int t = (int)table[bits & 63];
    const uint32_t m = (uint32_t)(t + __mulhi(t, __float2int_rn(f * q)));   // 30 bits after the point
    // m 2^(40 - 30 + e / 64) = (m 2^32) >> (22 - e / 64), the shift at most 63
    return ((u64)m << 32) >> (22u + 0x4B400000u / 64 - (bits >> 6));
}

__device__ __forceinline__ uint32_t distance(float l, const RowScale& r) {
    return __float_as_uint(__fadd_rz(fminf((r.top - l) * r.dist, (float)kQMax), 8388608.f)) - 0x4B000000u;   // truncated
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// inclusive sum over the lanes up to this one
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// A token's place in the order: kept are the tokens up to and with the border's.
struct Border {
    uint32_t key;
    int idx;
    __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= idx); }
    __device__ __forceinline__ bool all() const { return key == kKeyMin && idx == 0x7FFFFFFF; }
    __device__ __forceinline__ void tighten(const Border& o) {
        if (o.key > key || (o.key == key && o.idx < idx)) *this = o;
    }
};

struct __align__(16) Entry {
    u64 w;
    uint32_t key;
    int idx;
};

struct Shared {
    uint32_t table[64];
    u64 mine[2][kBins];          // this CTA's sums of a histogram's bins; every second round in turn
    u64 all[kBins];              // the cluster's
    uint32_t keys[kBins];
    uint32_t top;                // the key of this CTA's largest logit
    uint32_t wtop[kWarps];
    u64 part[kWarps];
    u64 whole;
    uint32_t nlist, found, nlong;
    int first;
    u64 sum;                     // this CTA's weight of all tokens
    float least;
    Border border;
    u64 scan[kWarps], wsum[kWarps];
};

// A CTA's run of a row: token i at data[sh + i - base]; the places before and after hold -inf.
struct Run {
    const float4* data;
    int base;        // the token at data[0], negative where the first row starts inside its vector
    int v0, v1;      // this warp's vectors
};
template <typename F>
__device__ __forceinline__ void each(const Run& r, int lane, F f) {
    for (int v = r.v0 + lane; v < r.v1; v += 32) {
        const float4 x = r.data[v];
        const int i = r.base + 4 * v;
        f(x.x, i);
        f(x.y, i + 1);
        f(x.z, i + 2);
        f(x.w, i + 3);
    }
}

// The same run read from memory: token i at src[i - first], this warp's at from .. to - 1 of src, of which
// those from v0 on lie in nv aligned vectors.
template <typename T>
struct Stream {
    static constexpr int W = 16 / (int)sizeof(T);
    const T* src;
    int from, to, v0, nv;
    __device__ __forceinline__ Stream(const T* s, int n, int warp) : src(s) {
        const int off = (int)((reinterpret_cast<uintptr_t>(s) % 16) / sizeof(T));
        const int head = min(n, (W - off) % W), body = (n - head) / W;
        const int per = (body + kWarps - 1) / kWarps, a = min(body, warp * per);
        nv = min(body, a + per) - a;
        v0 = head + a * W;
        from = warp == 0 ? 0 : v0;
        to = warp == kWarps - 1 ? n : v0 + nv * W;
        if (nv == 0 && warp != kWarps - 1) to = warp == 0 ? head : from;
    }
};
template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
// the logits of a 16-byte load, canonical or as they are
template <typename T, bool RAW = false>
__device__ __forceinline__ void unpack(const uint4 x, float (&l)[16 / sizeof(T)]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            l[j] = RAW ? __uint_as_float(u[j]) : canonical(__uint_as_float(u[j]));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
            l[2 * j] = RAW ? f.x : canonical(f.x);
            l[2 * j + 1] = RAW ? f.y : canonical(f.y);
        }
    }
}
template <bool RAW, typename T, typename F>
__device__ __forceinline__ void each(const Stream<T>& s, int lane, F f) {
    const uint4* v = reinterpret_cast<const uint4*>(s.src + s.v0);
#pragma unroll 4
    for (int i = lane; i < s.nv; i += 32) {
        float l[Stream<T>::W];
        unpack<T, RAW>(__ldg(v + i), l);
#pragma unroll
        for (int j = 0; j < Stream<T>::W; ++j) f(l[j]);
    }
    auto one = [&](int i) {
        const float l = to_float(__ldg(s.src + i));
        f(RAW ? l : canonical(l));
    };
    for (int i = s.from + lane; i < s.v0; i += 32) one(i);
    for (int i = s.v0 + s.nv * Stream<T>::W + lane; i < s.to; i += 32) one(i);
}

// What a search passes over: the CTA's run, or a list of its entries.
struct Tokens {
    static constexpr bool kAll = true;
    Run run;
    template <typename F>
    __device__ __forceinline__ void pass(F f) const {
        each(run, threadIdx.x & 31, f);
    }
};
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
struct Listed {
    static constexpr bool kAll = false;
    const Entry* e;
    int n;
    template <typename F>
    __device__ __forceinline__ void pass(F f) const {
        for (int j = threadIdx.x; j < n; j += kThreads) f(logit_of(e[j].key), e[j].idx);
    }
};

// What a search looks for: the border of the first `target` tokens of the order; that of the shortest
// prefix, within `in`, with at least the share `share` of the weight within `in`; or the first `target`
// tokens themselves (at most kList), which then lie in `ranked`, sh.found of them with a few more.
enum { kCount = 0, kMass = 1, kFirst = 2 };

// The interval that the border lies in, by what is open: distances qa .. qb, of one distance keys ka .. kb, of
// one key indices ia .. ib; what of the target lies before it.
struct Search {
    uint32_t qa, qb, ka, kb, ia, ib;
    u64 base, target;
    bool all;        // in: every token above -inf
    __device__ __forceinline__ Search(const RowScale& row, int vocab, const Border& in, u64 t)
        : qa(0), qb(kQMax), ka(kKeyMin), kb(key_of(row.top)), ia(0), ib((uint32_t)vocab - 1), base(0), target(t), all(in.all()) {}
    __device__ __forceinline__ int level() const { return qa < qb ? 0 : ka < kb ? 1 : 2; }
    // the digit's value of a token, above the interval's span where it is not one of those left. Tokens of -inf
    // are left in until the keys are divided: they weigh nothing, and come last in a count.
    __device__ __forceinline__ uint32_t digit(int lv, float l, int i, const RowScale& row, const Border& in) const {
        const uint32_t q = distance(l, row), k = key_of(l);
        if (lv == 0) return all || in.keeps(k, i) ? q - qa : ~0u;
        const bool ok = q == qa && k <= kb && k >= ka && (all || in.keeps(k, i));
        if (lv == 1) return ok ? kb - k : ~0u;
        return ok ? (uint32_t)i - ia : ~0u;
    }
};

// One round: the highest 7 bits of the first interval still open are divided; false where the target is not
// reached. COLS: the histogram's columns, one per lane where all tokens are passed over.
template <int KIND, int COLS, typename S>
__device__ bool divide(const S& src, Search& f, const RowScale& row, const Border& in, float share, bool first, uint32_t* hist,
                       Shared& sh, uint32_t ranks, int& turn, u64& in_bin) {
    constexpr bool MASS = KIND == kMass;
    const int tid = threadIdx.x, lane = tid & 31;
    const int level = f.level();
    const uint32_t a = level == 0 ? f.qa : level == 1 ? f.ka : f.ia, b = level == 0 ? f.qb : level == 1 ? f.kb : f.ib;
    const uint32_t span = b - a;
    const int bits = 32 - __clz((int)span);
    const int shift = bits > kDigit ? bits - kDigit : 0;
    for (int i = tid; i < kBins * COLS * (MASS ? 2 : 1) / 4; i += kThreads)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) sh.nlist = 0;
    __syncthreads();
    if (KIND != kMass && first && f.all) {   // every token counts
        src.pass([&](float l, int) { atomicAdd(hist + (distance(l, row) >> shift) * COLS + lane % COLS, 1u); });
    } else if (MASS && S::kAll && first && f.all) {
        if constexpr (S::kAll) {   // four tokens at a time and no branches: their chains overlap (a weight of 0 adds nothing)
            for (int v = src.run.v0 + lane; v < src.run.v1; v += 32) {
                const float4 x = src.run.data[v];
                const float l[4] = {x.x, x.y, x.z, x.w};
                u64 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = weight(l[j], row, sh.table);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t* h = hist + (distance(l[j], row) >> shift) * COLS + lane % COLS;
                    atomicAdd(h, (uint32_t)w[j] & 0xfffffu);
                    atomicAdd(h + kBins * COLS, (uint32_t)(w[j] >> 20));
                }
            }
        }
    } else src.pass([&](float l, int i) {
        const uint32_t v = f.digit(level, l, i, row, in);
        if (v > span) return;
        uint32_t* h = hist + (v >> shift) * COLS + lane % COLS;
        if (MASS) {
            const u64 w = weight(l, row, sh.table);
            if (w != 0) {
                atomicAdd(h, (uint32_t)w & 0xfffffu);
                atomicAdd(h + kBins * COLS, (uint32_t)(w >> 20));
            }
        } else {
            atomicAdd(h, 1u);
        }
    });
    __syncthreads();
    {   // four threads a bin, a quarter of the columns each, taken so that a warp's reads are on different banks
        const int bin = tid >> 2, c0 = (tid & 3) * (COLS / 4);
        u64 v = 0;
#pragma unroll
        for (int j = 0; j < COLS / 4; ++j) {   // a column holds at most 2^11 tokens of 2^20 each: below 2^32
            const int c = c0 + ((j + bin) & (COLS / 4 - 1));
            v += hist[bin * COLS + c];
            if (MASS) v += (u64)hist[(kBins + bin) * COLS + c] << 20;
        }
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((tid & 3) == 0) sh.mine[turn][bin] = v;
    }
    cluster_sync();
    if (tid < kBins) {
        u64 v = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) v += r < ranks ? remote_u64(&sh.mine[turn][tid], r) : 0;
        sh.all[tid] = v;
    }
    turn ^= 1;
    __syncthreads();
    // every warp: the bin in which the running sum reaches the target
    u64 v[kBins / 32], mine = 0;
#pragma unroll
    for (int j = 0; j < kBins / 32; ++j) {
        v[j] = sh.all[lane * (kBins / 32) + j];
        mine += v[j];
    }
    const u64 upto = warp_scan(mine, lane);
    if (MASS && first) {   // ceil(share * sum), exactly; 1 at least
        const u64 sum = __shfl_sync(0xffffffffu, upto, 31);
        const u64 s64 = share > 0.f ? __float2ull_rz(share * 0x1p64f) : 0;
        f.target = __umul64hi(s64, sum) + (s64 * sum != 0 ? 1 : 0);
        f.target = f.target == 0 ? 1 : f.target;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, f.base + upto >= f.target);
    if (!reach && KIND != kFirst) return false;   // fewer tokens
    const int l = reach ? __ffs(reach) - 1 : 31;
    u64 c = f.base + upto - mine;
    int bin = lane * (kBins / 32);
#pragma unroll
    for (int j = 0; j < kBins / 32 - 1; ++j) {
        if (bin == lane * (kBins / 32) + j && c + v[j] < f.target) {
            c += v[j];
            ++bin;
        }
    }
    bin = __shfl_sync(0xffffffffu, bin, l);
    f.base = __shfl_sync(0xffffffffu, c, l);
    in_bin = sh.all[bin];
    const uint32_t lo = (uint32_t)bin << shift, hi = lo + ((1u << shift) - 1);
    if (level == 1) {   // keys: bins fall from the largest
        const uint32_t last = f.kb;
        f.kb = last - lo;
        f.ka = hi < last - f.ka ? last - hi : f.ka;
    } else if (level == 0) {
        f.qb = hi < f.qb - f.qa ? f.qa + hi : f.qb;
        f.qa += lo;
    } else {
        f.ib = hi < f.ib - f.ia ? f.ia + hi : f.ib;
        f.ia += lo;
    }
    return true;
}

// The border, from the interval that f has come to (`rounds` of them done); `in` where there are fewer tokens.
// few: what is left fits the lists already.
template <int KIND, int COLS, typename S>
__device__ Border find_border(const S& src, Search f, const RowScale& row, int vocab, const Border in, float share, int rounds,
                              uint32_t* hist, Shared& sh, uint32_t ranks, int& turn, bool few = false) {
    constexpr bool MASS = KIND == kMass;
    const int tid = threadIdx.x, lane = tid & 31;
    Entry *list = reinterpret_cast<Entry*>(hist), *ranked = list + kList;   // once a histogram has been read
    static_assert(kBins * COLS * 4 * (MASS ? 2 : 1) >= 2 * kList * (int)sizeof(Entry), "");
    for (int round = rounds;; ++round) {
        if (!few) {
            u64 in_bin;
            if (!divide<KIND, COLS>(src, f, row, in, share, round == 0, hist, sh, ranks, turn, in_bin)) return in;
            if (!MASS) {
                if ((KIND == kFirst ? f.base : 0) + in_bin > kList) continue;
            } else if (round == 0 && vocab > 16 * kList) {   // rarely few enough after one digit
                continue;
            }
        }
        few = false;
        // the candidates: this CTA's, then everybody's
        const int at = f.level();
        const uint32_t rest = at == 0 ? f.qb - f.qa : at == 1 ? f.kb - f.ka : f.ib - f.ia;
        __syncthreads();   // the histogram has been read
        src.pass([&](float l2, int i) {
            if (KIND == kFirst) {   // all up to the interval's last: f.base and in_bin, kList at most
                const uint32_t k = key_of(l2), q = distance(l2, row);
                // (while keys are divided f.ka may be lower than any of this distance, and tokens of the next one lie above it)
                if (at == 0 ? q > f.qb : at == 1 ? q > f.qa || (q == f.qa && k < f.ka) : !(Border{f.ka, (int)f.ib}.keeps(k, i))) return;
            } else if (f.digit(at, l2, i, row, in) > rest) {
                return;
            }
            const u64 w = KIND == kCount ? 1 : weight(l2, row, sh.table);
            if (KIND != kCount && (w == 0 || l2 == -INFINITY)) return;
            const uint32_t n = atomicAdd(&sh.nlist, 1u);
            if (n < kList) list[n] = Entry{w, key_of(l2), i};
        });
        cluster_sync();
        // thread t takes the t-th of all candidates: the CTA in whose list it is, and its place there
        const uint32_t len = lane < (int)ranks ? remote_u32(&sh.nlist, (uint32_t)lane) : 0;
        const uint32_t ends = (uint32_t)warp_scan(len, lane);
        const uint32_t total = __shfl_sync(0xffffffffu, ends, 31);
        if (total <= kList) {
            uint32_t r = 0, start = 0;
#pragma unroll
            for (uint32_t k = 0; k < kMaxCluster; ++k) {
                const uint32_t end = __shfl_sync(0xffffffffu, ends, k);
                if ((uint32_t)tid >= end) {
                    r = k + 1;
                    start = end;
                }
            }
            if ((uint32_t)tid < total) {
                const Entry* e = &list[tid - start];
                const u64 w = remote_u64(&e->w, r), ki = remote_u64(&e->key, r);
                ranked[tid] = Entry{w, (uint32_t)ki, (int)(ki >> 32)};
            }
        }
        if (tid == 0) sh.border = in;
        cluster_sync();   // the lists may be written again
        if (KIND == kFirst) {
            if (tid == 0) sh.found = min(total, (uint32_t)kList);
            __syncthreads();
            return in;
        }
        if (total > kList) continue;
        static_assert(4 * kList == kThreads, "four threads a candidate");
        const Entry e = (uint32_t)tid / 4 < total ? ranked[tid / 4] : Entry{0, 0, 0};
        u64 cum = 0;
#pragma unroll 4
        for (uint32_t j = tid & 3; j < total; j += 4) {
            const Entry o = ranked[j];
            if (o.key > e.key || (o.key == e.key && o.idx <= e.idx)) cum += o.w;
        }
        cum += __shfl_xor_sync(0xffffffffu, cum, 1);
        cum += __shfl_xor_sync(0xffffffffu, cum, 2);
        cum += f.base;
        if ((uint32_t)tid / 4 < total && (tid & 3) == 0 && cum >= f.target && cum - e.w < f.target) sh.border = Border{e.key, e.idx};
        __syncthreads();
        const Border found = sh.border;
        __syncthreads();
        return found;
    }
}

// Top-p by two passes over the tokens: a histogram of weights, then this warp's sum of what lies before the bin
// that the border falls into and a list of the bin's tokens, which the rest is done with. sh.part: the warps'
// kept weights, of tokens with keys from `least` on. False (nothing done) where a list would be too long.
constexpr int kLong = 1024;
__device__ bool nucleus(const Run& run, const RowScale& row, int vocab, const Border in, uint32_t least, float share, uint32_t* hist,
                        Shared& sh, uint32_t ranks, int& turn, int vectors, Border& border) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Search f(row, vocab, in, 0);
    u64 in_bin;
    if (tid == 0) sh.nlong = 0;
    divide<kMass, 32>(Tokens{run}, f, row, in, share, true, hist, sh, ranks, turn, in_bin);
    Entry* list = reinterpret_cast<Entry*>(hist);
    u64 w = 0;
    for (int v = run.v0 + lane; v < run.v1; v += 32) {
        const float4 x = run.data[v];
        if (distance(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), row) > f.qb) continue;
        const float l[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t q = distance(l[j], row), k = key_of(l[j]);
            const int i = run.base + 4 * v + j;
            if (q > f.qb || !(f.all || in.keeps(k, i))) continue;
            const u64 x1 = weight(l[j], row, sh.table);
            if (q < f.qa) {
                if (k >= least) w += x1;
            } else if (x1 != 0) {
                const uint32_t n = atomicAdd(&sh.nlong, 1u);
                if (n < kLong) list[n] = Entry{x1, k, i};
            }
        }
    }
    w = warp_sum(w);
    if (lane == 0) sh.part[warp] = w;
    cluster_sync();
    const uint32_t len = lane < (int)ranks ? remote_u32(&sh.nlong, (uint32_t)lane) : 0u;
    if (__reduce_max_sync(0xffffffffu, len) > kLong) return false;
    const bool few = __reduce_add_sync(0xffffffffu, len) <= kList;
    const int n = (int)sh.nlong;
    border = find_border<kMass, 8>(Listed{list, n}, f, row, vocab, in, share, 1, reinterpret_cast<uint32_t*>(list + kLong), sh, ranks, turn,
                                    few);
    for (int j = tid; j < n; j += kThreads) {
        const Entry e = list[j];
        if (border.keeps(e.key, e.idx) && e.key >= least) atomicAdd(&sh.part[(e.idx - run.base) / 4 / vectors], e.w);
    }
    __syncthreads();
    if (warp == 0) {
        w = warp_sum(lane < kWarps ? sh.part[lane] : 0);
        if (lane == 0) sh.whole = w;
    }
    cluster_sync();
    return true;
}

// The first topk (<= kList) tokens of the order and a few more, sh.nlist of them, to `list` of rank 0; false
// where the few would be too many. At least topk tokens lie as near as topk threads'
// largest logits (mine) do, so that the threshold comes from a histogram of one value a thread.
__device__ bool list_first(const Run& run, const RowScale& row, float mine, int topk, uint32_t* hist, Shared& sh,
                           uint32_t ranks) {
    constexpr int kShift = 23 - kDigit;
    const int tid = threadIdx.x, lane = tid & 31;
    Entry* list = reinterpret_cast<Entry*>(hist);
    uint32_t* bins = reinterpret_cast<uint32_t*>(list + kList);
    const uint32_t count = remote(&sh.nlist, 0), entries = remote(list, 0);
    if (tid < kBins) bins[tid] = 0;
    if (tid == 0) sh.nlist = 0;
    __syncthreads();
    if (mine > -INFINITY) atomicAdd(bins + (distance(mine, row) >> kShift), 1u);
    __syncthreads();
    if (tid < kBins) sh.mine[0][tid] = bins[tid];
    cluster_sync();
    if (tid < kBins) {
        u64 v = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) v += r < ranks ? remote_u64(&sh.mine[0][tid], r) : 0;
        sh.all[tid] = v;
    }
    __syncthreads();
    uint32_t v[kBins / 32], sum = 0;
#pragma unroll
    for (int j = 0; j < kBins / 32; ++j) {
        v[j] = (uint32_t)sh.all[lane * (kBins / 32) + j];
        sum += v[j];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, upto >= (uint32_t)topk);
    uint32_t far = kQMax;
    if (reach) {
        uint32_t c = upto - sum;
        int bin = lane * (kBins / 32);
#pragma unroll
        for (int j = 0; j < kBins / 32 - 1; ++j) {
            if (bin == lane * (kBins / 32) + j && c + v[j] < (uint32_t)topk) {
                c += v[j];
                ++bin;
            }
        }
        bin = __shfl_sync(0xffffffffu, bin, __ffs(reach) - 1);
        far = ((uint32_t)(bin + 1) << kShift) - 1;
    }
    for (int i = run.v0 + lane; i < run.v1; i += 32) {
        const float4 x = run.data[i];
        if (distance(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), row) > far) continue;
        const float l[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (distance(l[j], row) > far) continue;
            const u64 w = weight(l[j], row, sh.table);
            if (w == 0 || l[j] == -INFINITY) continue;
            uint32_t n;
            asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(count) : "memory");
            if (n < kList)
                asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(entries + n * 16), "r"((uint32_t)w),
                             "r"((uint32_t)(w >> 32)), "r"(key_of(l[j])), "r"(run.base + 4 * i + j) : "memory");
        }
    }
    cluster_sync();
    return remote_u32(&sh.nlist, 0) <= kList;
}

// The draw among the n <= kList entries of the first top_k tokens and a few after them, by one CTA, four threads an
// entry. What is kept is a prefix of the order, so the entry at its end knows the kept weight.
__device__ void draw_small(const Entry* e, int n, int topk, float topp, uint32_t least, float u, int32_t* token, float* prob,
                           Shared& sh) {
    const int tid = threadIdx.x, at = tid >> 2, part = tid & 3;
    static_assert(4 * kList == kThreads && kList <= kBins, "four threads an entry");
    const Entry me = at < n ? e[at] : Entry{0, 0, 0x7FFFFFFF};
    auto quad = [](u64 v) {
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        return v + __shfl_xor_sync(0xffffffffu, v, 2);
    };
    u64 before = 0;
    uint32_t place = 0;
#pragma unroll 4
    for (int j = part; j < n; j += 4) {
        const Entry o = e[j];
        if (o.key > me.key || (o.key == me.key && o.idx < me.idx)) {
            before += o.w;
            ++place;
        }
    }
    before = quad(before);
    place += __shfl_xor_sync(0xffffffffu, place, 1);
    place += __shfl_xor_sync(0xffffffffu, place, 2);
    const int m = min(n, topk);
    if (part == 0 && at < n) {   // sums and keys in the order's places
        sh.all[place] = before + me.w;
        sh.keys[place] = me.key;
    }
    __syncthreads();
    u64 within = ~0ull;   // top-p: kept while less than this lies before
    if (topp < 1.f) {
        const u64 whole = sh.all[m - 1];
        const u64 s64 = topp > 0.f ? __float2ull_rz(topp * 0x1p64f) : 0;
        within = __umul64hi(s64, whole) + (s64 * whole != 0 ? 1 : 0);
        within = within == 0 ? 1 : within;
    }
    auto kept = [&](int q, u64 b, uint32_t key) { return q < m && b < within && key >= least; };
    const bool keep = at < n && kept((int)place, before, me.key);
    const u64 upto = before + me.w;
    if (part == 0) {
        sh.mine[0][at] = keep ? me.w : 0;
        if (keep && !((int)place + 1 < m && kept((int)place + 1, upto, sh.keys[place + 1]))) sh.whole = upto;
    }
    __syncthreads();
    const u64 total = sh.whole;
    const u64 target = __umul64hi(__float2ull_rz(u * 0x1p64f), total) + 1;
    u64 c = 0;
#pragma unroll 4
    for (int j = part; j < n; j += 4)
        if (e[j].idx <= me.idx) c += sh.mine[0][j];
    c = quad(c);
    if (keep && part == 0 && c >= target && c - me.w < target) {
        *token = me.idx;
        if (prob) *prob = (float)((double)me.w / (double)total);
    }
}

// The CTA's run of the row into shared memory, sh places further on so that 16-byte loads are aligned at
// both ends; returns this thread's largest logit.
template <typename T>
__device__ __forceinline__ float load_run(const T* src, int n, int off, float* data, int nvec) {
    constexpr int W = 16 / (int)sizeof(T);   // tokens of a 16-byte load
    float mx = -INFINITY;
    auto put = [&](int at, float l) {
        l = canonical(l);
        data[at] = l;
        mx = fmaxf(mx, l);
    };
    const int head = min(n, (W - off) % W);            // tokens before the first whole vector
    const int body = (n - head) / W;
    const uint4* v = reinterpret_cast<const uint4*>(src + head);
    float4* to = reinterpret_cast<float4*>(data + off + head);
#pragma unroll 4
    for (int i = threadIdx.x; i < body; i += kThreads) {
        float l[W];
        unpack<T>(__ldg(v + i), l);
#pragma unroll
        for (int j = 0; j < W; ++j) mx = fmaxf(mx, l[j]);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) to[i * (W / 4) + j] = make_float4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
    }
    const int tail = head + body * W;
    for (int i = threadIdx.x; i < head; i += kThreads) put(off + i, to_float(src[i]));
    for (int i = tail + threadIdx.x; i < n; i += kThreads) put(off + i, to_float(src[i]));
    for (int i = threadIdx.x; i < off; i += kThreads) data[i] = -INFINITY;
    for (int i = off + n + threadIdx.x; i < 4 * nvec; i += kThreads) data[i] = -INFINITY;
    return mx;
}

// A row's arguments. Every decision that follows from them is the same in all CTAs of the cluster.
struct RowArgs {
    float temp, topp, minp, u;
    int topk;
};
// Their loads, not waited for before row_args looks at them; false for an inactive row.
__device__ __forceinline__ bool row_loads(const Params& p, long long b, RowArgs& a) {
    const bool active = !p.active || p.active[b] != 0;
    a.temp = p.temperature ? p.temperature[b] : 1.0f;
    a.topp = p.top_p ? p.top_p[b] : 1.0f;
    a.minp = p.min_p ? p.min_p[b] : 0.0f;
    a.topk = p.top_k ? p.top_k[b] : 0;
    // a decode loop's numbers, one per position (a negative position has been recorded by the step)
    const long long at = p.uniform_stride <= 1 ? b : b * p.uniform_stride + max(p.positions[b], 0) % p.uniform_stride;
    a.u = p.uniform[at];
    return active;
}
// False where the arguments are out of range (recorded).
__device__ __forceinline__ bool row_args(const Params& p, long long b, uint32_t rank, const RowArgs& a, DevError* err) {
    if (a.temp >= 0.f && a.temp < INFINITY && a.topp == a.topp && a.minp == a.minp && a.u >= 0.f && a.u < 1.f) return true;
    if (threadIdx.x == 0 && rank == 0) {
        record_device_error(err, kErrSampleArg, b, 0);
        p.tokens[b] = -1;
        if (p.probs) p.probs[b] = 0.f;
    }
    return false;
}

// The row's largest logit from every thread's. False where the row has no token, which is written.
__device__ __forceinline__ bool row_top(const Params& p, long long b, uint32_t rank, uint32_t ranks, float& top, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t key = __reduce_max_sync(0xffffffffu, key_of(top));
    if (lane == 0) sh.wtop[warp] = key;
    __syncthreads();
    if (warp == 0) {
        key = __reduce_max_sync(0xffffffffu, sh.wtop[lane & (kWarps - 1)]);
        if (lane == 0) sh.top = key;
    }
    cluster_sync();
    key = __reduce_max_sync(0xffffffffu, lane < (int)ranks ? remote_u32(&sh.top, (uint32_t)lane) : 0u);
    top = logit_of(key);
    if (top != -INFINITY) return true;
    cluster_sync();   // nobody leaves while its shared memory may be read
    if (tid == 0 && rank == 0) {
        p.tokens[b] = -1;
        if (p.probs) p.probs[b] = 0.f;
    }
    return false;
}

// The arg max: the lowest of the threads' indices of the largest logit.
__device__ __forceinline__ void row_first(const Params& p, long long b, uint32_t rank, uint32_t ranks, int idx, Shared& sh) {
    const int tid = threadIdx.x;
    idx = __reduce_min_sync(0xffffffffu, idx);
    if (tid == 0) sh.first = 0x7FFFFFFF;
    __syncthreads();
    if ((tid & 31) == 0) atomicMin(&sh.first, idx);
    cluster_sync();
    if (tid == 0 && rank == 0) {
        int best = 0x7FFFFFFF;
        for (uint32_t r = 0; r < ranks; ++r) best = min(best, (int)remote_u32(&sh.first, r));
        p.tokens[b] = best;
        if (p.probs) p.probs[b] = 1.f;
    }
    cluster_sync();
}

// The least f32 at or above top + T ln(min_p), by thread 0 (a barrier must follow); its key.
__device__ __forceinline__ float min_p_least(const RowArgs& a, float top) {
    return (a.minp >= 1.f ? top : __double2float_ru((double)top + (double)a.temp * log((double)a.minp))) + 0.0f;
}

// The warps' sums w (and s) to sh.part (and sh.scan), the CTA's to sh.whole (and sh.sum), for all CTAs to read.
__device__ __forceinline__ void share_sums(u64 w, u64 s, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    w = warp_sum(w);
    s = warp_sum(s);
    if (lane == 0) {
        sh.part[warp] = w;
        sh.scan[warp] = s;
    }
    __syncthreads();
    if (warp == 0) {
        w = warp_sum(lane < kWarps ? sh.part[lane] : 0);
        s = warp_sum(lane < kWarps ? sh.scan[lane] : 0);
        if (lane == 0) {
            sh.whole = w;
            sh.sum = s;
        }
    }
    cluster_sync();
}

// The draw from the shared sums: the CTA, then the warp, then the thread in whose tokens the running sum
// reaches the target. tokens(warp, from, to): a warp's places; kept(place): its kept weight; index(place).
template <typename R, typename K, typename I>
__device__ __forceinline__ void draw(const Params& p, long long b, uint32_t rank, uint32_t ranks, float u, Shared& sh, R tokens,
                                     K kept, I index) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const u64 t = lane < (int)ranks ? remote_u64(&sh.whole, (uint32_t)lane) : 0;
    cluster_arrive();   // what this CTA reads of the others is read
    const u64 upto = warp_scan(t, lane);
    const u64 total = __shfl_sync(0xffffffffu, upto, 31), before = __shfl_sync(0xffffffffu, upto - t, (int)rank);
    // the first token at which the running sum exceeds u total: reaches floor(u total) + 1, exactly
    const u64 target = __umul64hi(__float2ull_rz(u * 0x1p64f), total) + 1;
    if (target > before && target <= before + sh.whole) {   // in this CTA
        const u64 mine = lane < kWarps ? sh.part[lane] : 0;
        const u64 ends = before + warp_scan(mine, lane);
        const int ow = __ffs(__ballot_sync(0xffffffffu, lane < kWarps && ends >= target)) - 1;
        u64 c = __shfl_sync(0xffffffffu, ends - mine, ow);
        // that warp's tokens over all threads, a few consecutive ones each
        int from, to;
        tokens(ow, from, to);
        const int n = (to - from + kThreads - 1) / kThreads;
        const int a = min(to, from + tid * n), e = min(to, a + n);
        u64 s = 0;
#pragma unroll 4
        for (int j = a; j < e; ++j) s += kept(j);
        const u64 incl = warp_scan(s, lane);
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        for (int k = 0; k < warp; ++k) c += sh.wsum[k];
        c += incl - s;
        if (c < target && c + s >= target) {
            for (int j = a; j < e; ++j) {
                const u64 x = kept(j);
                c += x;
                if (x != 0 && c >= target) {
                    p.tokens[b] = index(j);
                    if (p.probs) p.probs[b] = (float)((double)x / (double)total);
                    break;
                }
            }
        }
    }
    cluster_wait();   // nobody leaves while its shared memory may be read
}

// No top-k or top-p: two passes over the row, the second from L2, so that shared memory does not bound the
// CTAs of an SM.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) sample_plain_kernel(Params p, DevError* err) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const long long b = blockIdx.x / ranks;
    pdl_wait();
    if (p.early) pdl_trigger();
    RowArgs a;
    if (!row_loads(p, b, a)) return;
    const int first = (int)rank * p.per;
    const int n = max(0, min(p.vocab - first, p.per));
    const T* src = static_cast<const T*>(p.logits) + b * p.stride + first;
    const Stream<T> run(src, n, warp);
    if (tid < 64) sh.table[tid] = kExp2[tid];
    float top = -INFINITY;
    each<true>(run, lane, [&](float l) { top = fmaxf(top, l); });   // passes over NaN
    if (!row_args(p, b, rank, a, err)) return;
    if (!row_top(p, b, rank, ranks, top, sh)) return;
    const bool infinite = top == INFINITY;
    top = canonical(top);
    auto at = [&](int j) { return canonical(to_float(__ldg(src + j))); };
    if (a.temp < kMinTemperature) {
        int idx = 0x7FFFFFFF;
        for (int j = run.from + lane; j < run.to; j += 32)
            if (at(j) == top) idx = min(idx, first + j);
        row_first(p, b, rank, ranks, idx, sh);
        return;
    }
    RowScale row;
    row.set(top, a.temp);
    float least = row.hot() ? -FLT_MAX : -INFINITY;   // -inf weighs nothing
    if (a.minp > 0.f) {
        if (tid == 0) sh.least = min_p_least(a, top);
        __syncthreads();
        least = fmaxf(least, sh.least);
    }
    u64 w = 0;
    if (row.ref != 0.f || infinite) {
        each<false>(run, lane, [&](float l) { w += weight(l, row, sh.table) & -(u64)(l >= least); });
    } else if (least == -INFINITY) {
        each<true>(run, lane, [&](float l) { w += weight<false>(l, row, sh.table); });
    } else {
        each<true>(run, lane, [&](float l) { w += weight<false>(l, row, sh.table) & -(u64)(l >= least); });
    }
    share_sums(w, 0, sh);
    draw(p, b, rank, ranks, a.u, sh,
         [&](int ow, int& from, int& to) {
             const Stream<T> r(src, n, ow);
             from = r.from;
             to = r.to;
         },
         [&](int j) {
             const float l = at(j);
             return weight(l, row, sh.table) & -(u64)(l >= least);
         },
         [&](int j) { return first + j; });
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(Params p, DevError* err) {
    extern __shared__ __align__(16) float dyn[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const long long b = blockIdx.x / ranks;
    pdl_wait();
    if (p.early) pdl_trigger();
    RowArgs a;
    if (!row_loads(p, b, a)) return;
    const int first = (int)rank * p.per;
    const int n = max(0, min(p.vocab - first, p.per));
    const T* src = static_cast<const T*>(p.logits) + b * p.stride + first;
    const int off = (int)((reinterpret_cast<uintptr_t>(src) % 16) / sizeof(T));
    const int nvec = (off + n + 3) / 4;
    uint32_t* hist = reinterpret_cast<uint32_t*>(dyn + p.per + 8);
    if (tid < 64) sh.table[tid] = kExp2[tid];
    const float mine = load_run(src, n, off, dyn, nvec);
    float top = mine;
    if (!row_args(p, b, rank, a, err)) return;
    if (!row_top(p, b, rank, ranks, top, sh)) return;
    Run run;
    run.data = reinterpret_cast<const float4*>(dyn);
    run.base = first - off;
    const int vpw = (nvec + kWarps - 1) / kWarps;
    run.v0 = warp * vpw;
    run.v1 = min(nvec, run.v0 + vpw);
    int turn = 0;
    if (a.temp < kMinTemperature) {
        int idx = 0x7FFFFFFF;
        each(run, lane, [&](float l, int i) { idx = l == top && i < idx ? i : idx; });
        row_first(p, b, rank, ranks, idx, sh);
        return;
    }
    RowScale row;
    row.set(top, a.temp);
    // all that is above -inf; in a count -inf comes last and does no harm
    const Border any = {kKeyMin, 0x7FFFFFFF}, every = {kKeyMin, row.hot() ? 0x7FFFFFFE : 0x7FFFFFFF};
    Border border = every, prefix = every;
    if (a.minp > 0.f) {
        if (tid == 0) sh.least = min_p_least(a, top);
        __syncthreads();
        border.key = max(kKeyMin, key_of(sh.least));
    }
    if (a.topk > 0 && a.topk <= kList && a.topk < p.vocab) {
        const Entry* e = reinterpret_cast<const Entry*>(hist);
        const bool listed = list_first(run, row, mine, a.topk, hist, sh, ranks);
        cluster_arrive();   // this CTA has read rank 0's count
        if (!listed) {
            cluster_wait();
            find_border<kFirst, 32>(Tokens{run}, Search(row, p.vocab, any, (u64)a.topk), row, p.vocab, any, 0.f, 0, hist, sh, ranks, turn);
            e += kList;
        }
        if (rank == 0)
            draw_small(e, (int)(listed ? sh.nlist : sh.found), a.topk, a.topp, border.key, a.u, p.tokens + b,
                       p.probs ? p.probs + b : nullptr, sh);
        if (listed) cluster_wait();
        return;   // no CTA reads another's shared memory any more
    }
    if (a.topk > 0 && a.topk < p.vocab) {
        prefix.tighten(find_border<kCount, 32>(Tokens{run}, Search(row, p.vocab, any, (u64)a.topk), row, p.vocab, any, 0.f, 0, hist, sh, ranks, turn));
        border.tighten(prefix);
    }
    bool ready = false;   // the kept sums are there
    if (a.topp < 1.f && a.minp > 0.f && prefix.all()) {
        // where min-p keeps less weight than top-p asks for, it is the border
        const float least = sh.least;
        u64 w = 0, s = 0;
        each(run, lane, [&](float l, int) {
            const u64 x = weight(l, row, sh.table);
            s += x;
            if (l >= least) w += x;
        });
        share_sums(w, s, sh);
        const u64 kept = warp_sum(lane < (int)ranks ? remote_u64(&sh.whole, (uint32_t)lane) : 0);
        const u64 all = warp_sum(lane < (int)ranks ? remote_u64(&sh.sum, (uint32_t)lane) : 0);
        const u64 s64 = a.topp > 0.f ? __float2ull_rz(a.topp * 0x1p64f) : 0;
        ready = kept < __umul64hi(s64, all) + (s64 * all != 0 ? 1 : 0);
    }
    if (!ready && a.topp < 1.f) {
        Border mass = prefix;
        ready = nucleus(run, row, p.vocab, prefix, border.key, a.topp, hist, sh, ranks, turn, vpw, mass);
        if (!ready)
            mass = find_border<kMass, 32>(Tokens{run}, Search(row, p.vocab, prefix, 0), row, p.vocab, prefix, a.topp, 0, hist, sh, ranks,
                                          turn);
        border.tighten(mass);
    }
    if (!ready) {
        u64 w = 0;
        if (border.all()) {
            each(run, lane, [&](float l, int) { w += weight(l, row, sh.table); });   // -inf weighs nothing
        } else {
            each(run, lane, [&](float l, int i) { w += weight(l, row, sh.table) & -(u64)border.keeps(key_of(l), i); });
        }
        share_sums(w, 0, sh);
    }
    draw(p, b, rank, ranks, a.u, sh,
         [&](int ow, int& from, int& to) {
             from = 4 * min(nvec, ow * vpw);
             to = 4 * min(nvec, (ow + 1) * vpw);
         },
         [&](int j) {
             const float l = dyn[j];
             return weight(l, row, sh.table) & -(u64)border.keeps(key_of(l), run.base + j);
         },
         [&](int j) { return run.base + j; });
}

// CTAs of a row. Staged in shared memory (top-k, top-p): enough that two runs fit an SM beside their
// histograms. Otherwise one, as long as a batch has enough rows. More while the batch leaves SMs idle; 16 for a few
// long rows (top-p over 151936: 4 rows 30.3 us with 8 CTAs each, 24.7 with 16; 8 rows 30.6 and 31.3; over 32000 one row
// with top-k 50 7.9 and 8.5).
int cluster_for(int64_t batch, int64_t vocab, bool staged) {
    int c = 1;
    const int sms = num_sms();
    while (c < kPortableCluster && ((staged && vocab > 20000ll * c) || (batch * c * 2 <= 3 * sms && vocab > 2048ll * c))) c *= 2;
    if (batch <= kFewRows && vocab > 4096ll * kMaxCluster) c = kMaxCluster;
    return c;
}

template <typename T>
cudaError_t sample_go(bool staged, const cudaLaunchConfig_t& cfg, const Params& p, DevError* err) {
    static std::atomic<unsigned long long> done{0}, large[2] = {};
    if (cfg.attrs[0].val.clusterDim.x > kPortableCluster) {
        const void* k = staged ? reinterpret_cast<const void*>(sample_kernel<T>) : reinterpret_cast<const void*>(sample_plain_kernel<T>);
        const cudaError_t e = allow_once(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, large[staged]);
        if (e != cudaSuccess) return e;
    }
    if (!staged) return cudaLaunchKernelEx(&cfg, sample_plain_kernel<T>, p, err);
    const size_t most = (size_t)(kMaxSampleVocab / kPortableCluster + 8) * 4 + (size_t)kBins * 32 * 8;   // of any call
    const cudaError_t e = allow_smem_once(sample_kernel<T>, most, done);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, sample_kernel<T>, p, err) : e;
}

}  // namespace

int sample_launch(const SampleArgs& a, cudaStream_t s, bool pdl) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "sampling: no device error record");
    const bool staged = a.top_k || a.top_p;
    const int c = cluster_for(a.batch, a.vocab, staged);
    if (a.batch * c >= (1ll << 31)) return set_error(QL_EINVAL, "sampling: batch out of range");
    Params p = {};
    p.logits = a.logits;
    p.stride = a.row_stride;
    p.vocab = (int)a.vocab;
    p.per = (int)(((a.vocab + c - 1) / c + 7) / 8 * 8);
    p.temperature = a.temperature;
    p.top_k = a.top_k;
    p.top_p = a.top_p;
    p.min_p = a.min_p;
    p.uniform = a.uniform;
    p.uniform_stride = a.uniform_stride;
    p.positions = a.positions;
    p.active = a.active;
    p.tokens = a.tokens;
    p.probs = a.probs;
    p.early = a.batch * c * 2 <= num_sms();
    const size_t smem = staged ? (size_t)(p.per + 8) * 4 + (size_t)kBins * 32 * (a.top_p ? 8 : 4) : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.batch * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    const cudaError_t e = a.dtype == QL_DTYPE_F32 ? sample_go<float>(staged, cfg, p, err) : sample_go<__half>(staged, cfg, p, err);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "sampling launch");
}

}  // namespace ql

extern "C" int ql_sample(const void* d_logits, int dtype, int64_t row_stride, int64_t batch, int64_t vocab,
                         const float* d_temperature, const int32_t* d_top_k, const float* d_top_p,
                         const float* d_min_p, const float* d_uniform, const int32_t* d_active, int32_t* d_tokens,
                         float* d_probs, void* stream) {
    using namespace ql;
    QL_REQUIRE(d_logits && d_uniform && d_tokens, "ql_sample: null pointer");
    QL_REQUIRE(dtype == QL_DTYPE_F32 || dtype == QL_DTYPE_F16, "ql_sample: dtype must be f32 or f16");
    QL_REQUIRE(batch >= 1 && batch < (1ll << 31), "ql_sample: batch out of range");
    QL_REQUIRE(vocab >= 1 && vocab <= kMaxSampleVocab, "ql_sample: vocab must be in [1, 360448]");
    QL_REQUIRE(batch == 1 || row_stride >= vocab, "ql_sample: row_stride must be at least vocab");
    const uintptr_t size = dtype == QL_DTYPE_F32 ? 4 : 2;
    QL_REQUIRE(reinterpret_cast<uintptr_t>(d_logits) % size == 0, "ql_sample: misaligned logits");
    auto a4 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3) == 0; };
    QL_REQUIRE(a4(d_temperature) && a4(d_top_k) && a4(d_top_p) && a4(d_min_p) && a4(d_uniform) && a4(d_active) &&
                   a4(d_tokens) && a4(d_probs),
               "ql_sample: misaligned array");
    // The CTAs of a row read its arguments on their own and have to find the same ones: an output in their place would
    // send them different ways.
    const uintptr_t rows = (uintptr_t)batch * 4;
    auto apart = [](const void* p, uintptr_t np, const void* q, uintptr_t nq) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
        return !p || !q || a + np <= b || b + nq <= a;
    };
    const uintptr_t all = ((uintptr_t)(batch - 1) * (uintptr_t)(batch > 1 ? row_stride : 0) + (uintptr_t)vocab) * size;
    for (const void* out : {static_cast<const void*>(d_tokens), static_cast<const void*>(d_probs)}) {
        bool ok = apart(out, rows, d_logits, all);
        for (const void* in : {static_cast<const void*>(d_temperature), static_cast<const void*>(d_top_k),
                               static_cast<const void*>(d_top_p), static_cast<const void*>(d_min_p),
                               static_cast<const void*>(d_uniform), static_cast<const void*>(d_active)})
            ok = ok && apart(out, rows, in, rows);
        QL_REQUIRE(ok, "ql_sample: the outputs must not overlap the inputs");
    }
    QL_REQUIRE(apart(d_tokens, rows, d_probs, rows), "ql_sample: the outputs must not overlap");
    SampleArgs a = {};
    a.logits = d_logits;
    a.dtype = dtype;
    a.row_stride = row_stride;
    a.batch = batch;
    a.vocab = vocab;
    a.temperature = d_temperature;
    a.top_k = d_top_k;
    a.top_p = d_top_p;
    a.min_p = d_min_p;
    a.uniform = d_uniform;
    a.uniform_stride = 1;
    a.active = d_active;
    a.tokens = d_tokens;
    a.probs = d_probs;
    return sample_launch(a, static_cast<cudaStream_t>(stream), true);
}
