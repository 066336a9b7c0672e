// The next token of a row of logits: temperature, top-k, top-p, min-p and one uniform number.
//
// Every kept set is a prefix of one order (logit falling, index rising), so all filters together are
// one border (key, index); the token is then a position in the running sum over the kept tokens in
// index order. Weights w = 2^((l - max) log2(e) / T) are 40-bit fixed-point integers and sums 64-bit
// ones: exact, whatever the order of additions, and the same in every pass.
//
// The border of top-k (a count) or top-p (a weight) is found by digits, the histogram of 256 bins
// naming the bin that the border falls into and the next round dividing that bin: first 8 bits at a
// time of the distance from the largest logit on a 24-bit scale of 24 T, then of the logit's ordered
// bits, then of the index, until 32 candidates or fewer are left, which one warp ranks.
//
// One CTA per row, the row read from L2 in every pass.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "ql_internal.h"
#include "ql_sample.h"

namespace ql {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 256, kList = 32;
constexpr int kScale = 40;                      // fixed-point bits of a weight of 1
constexpr uint32_t kQMax = (1u << 24) - 1;      // the distance scale's last value: all that is farther

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
    int vocab;
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
};

__device__ __forceinline__ float canonical(float l) {
    l = l == l ? l : -INFINITY;          // NaN: never drawn
    return fminf(l, FLT_MAX) + 0.0f;     // -0 and +0 tie
}
__device__ __forceinline__ float load(const float* p, long long i) { return canonical(__ldg(p + i)); }
__device__ __forceinline__ float load(const __half* p, long long i) { return canonical(__half2float(__ldg(p + i))); }

// Bits that order as the logits do.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// What turns a logit into a weight and into a distance, the same for the whole row.
struct RowScale {
    float ref, c_hi, c_lo, magic, low;   // (l - ref) (c_hi + c_lo): the exponent in 64ths
    float top, dist;                     // distance (top - l) dist
};

// The weight of logit l: 2^(40 + e / 64), e = (l - ref) 64 log2(e) / T minus its floor at the largest
// logit. The floor and the fraction come from fused multiply-adds of l itself, each rounded once, so
// that the error of a large l does not enter; 2^(fraction / 64) - 1 is the series of exp to the fourth
// power (the next term is below 2^-40), the product with the table is an integer one.
__device__ __forceinline__ u64 weight(float l, const RowScale& r, const uint32_t* table) {
    const float x = fmaxf(l - r.ref, r.low);
    const float z = __fmaf_rd(x, r.c_hi, r.magic);
    float f = __fmaf_rn(x, r.c_hi, r.magic - z);
    f = __fmaf_rn(x, r.c_lo, f);
    const int k = __float_as_int(z) - 0x4B400000;
    constexpr float y = 0.010830424696249145f;   // ln 2 / 64
    constexpr float s = 4294967296.0f;
    float q = fmaf(f, s * y * y * y * y / 24.f, s * y * y * y / 6.f);
    q = fmaf(f, q, s * y * y / 2.f);
    q = fmaf(f, q, s * y);
    const int t = (int)table[k & 63];
    const uint32_t m = (uint32_t)(t + __mulhi(t, __float2int_rn(f * q)));
    const int sh = min(-(k >> 6), 63);
    return ((u64)m << (kScale - 30)) >> sh;
}

__device__ __forceinline__ uint32_t distance(float l, const RowScale& r) {
    return (uint32_t)fminf((r.top - l) * r.dist, (float)kQMax);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Shared {
    uint32_t table[64];
    u64 mass[kBins];
    uint32_t count[kBins];
    u64 part[kWarps];
    uint32_t wkey[kWarps];
    int widx[kWarps];
    uint32_t lkey[kList];
    int lidx[kList];
    u64 lw[kList];
    uint32_t nlist;
    RowScale row;
    uint32_t bkey;
    int bidx;
    int bin;
    uint32_t bin_count;
    u64 base, total;
    int token;
};

// The border of the shortest prefix of the order with at least `target` tokens (mass false) or weight
// (mass true): its last token's key and index, in sh.bkey and sh.bidx.
template <typename T>
__device__ void find_border(const T* lg, int vocab, bool mass, u64 target, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const RowScale row = sh.row;
    uint32_t qa = 0, qb = kQMax, ka = 0, kb = 0xFFFFFFFFu, ia = 0, ib = (uint32_t)vocab - 1;
    u64 base = 0;
    for (;;) {
        // the digit that this round divides: 8 bits of the widest interval still open
        const int level = qa < qb ? 0 : ka < kb ? 1 : 2;
        const uint32_t a = level == 0 ? qa : level == 1 ? ka : ia, b = level == 0 ? qb : level == 1 ? kb : ib;
        const int bits = 32 - __clz((int)(b - a));
        const int shift = bits > 8 ? bits - 8 : 0;
        for (int i = tid; i < kBins; i += kThreads) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
        for (int i = tid; i < vocab; i += kThreads) {
            const float l = load(lg, i);
            const uint32_t q = distance(l, row), k = key_of(l);
            if (q < qa || q > qb || k < ka || k > kb || (uint32_t)i < ia || (uint32_t)i > ib) continue;
            const uint32_t v = level == 0 ? q - a : level == 1 ? b - k : (uint32_t)i - a;
            atomicAdd(&sh.count[v >> shift], 1u);
            if (mass) atomicAdd(&sh.mass[v >> shift], weight(l, row, sh.table));
        }
        __syncthreads();
        if (tid == 0) {
            u64 c = base;
            int bin = kBins - 1;
            for (int i = 0; i < kBins; ++i) {
                const u64 v = mass ? sh.mass[i] : sh.count[i];
                if (c + v >= target) {
                    bin = i;
                    break;
                }
                c += v;
            }
            sh.bin = bin;
            sh.bin_count = sh.count[bin];
            sh.base = c;
            sh.nlist = 0;
        }
        __syncthreads();
        base = sh.base;
        const uint32_t lo = (uint32_t)sh.bin << shift, hi = lo + ((1u << shift) - 1);
        if (level == 1) {   // keys: bins fall from the largest
            const uint32_t top = kb;
            kb = top - lo;
            ka = hi < top - ka ? top - hi : ka;
        } else if (level == 0) {
            qb = hi < qb - qa ? qa + hi : qb;
            qa += lo;
        } else {
            ib = hi < ib - ia ? ia + hi : ib;
            ia += lo;
        }
        const uint32_t left = sh.bin_count;
        __syncthreads();
        if (left > kList) continue;
        for (int i = tid; i < vocab; i += kThreads) {
            const float l = load(lg, i);
            const uint32_t q = distance(l, row), k = key_of(l);
            if (q < qa || q > qb || k < ka || k > kb || (uint32_t)i < ia || (uint32_t)i > ib) continue;
            const uint32_t n = atomicAdd(&sh.nlist, 1u);
            sh.lkey[n] = k;
            sh.lidx[n] = i;
            sh.lw[n] = mass ? weight(l, row, sh.table) : 1;
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t n = sh.nlist;
            const uint32_t k = lane < n ? sh.lkey[lane] : 0;
            const int idx = lane < n ? sh.lidx[lane] : 0x7FFFFFFF;
            u64 cum = 0;
            for (uint32_t j = 0; j < n; ++j) {
                const uint32_t kj = sh.lkey[j];
                if (kj > k || (kj == k && sh.lidx[j] <= idx)) cum += sh.lw[j];
            }
            // the border: the first of the order whose running sum reaches the target, else the last
            const bool reach = lane < n && base + cum >= target;
            bool best = lane < n;
            for (uint32_t j = 0; j < n; ++j) {
                const bool rj = __shfl_sync(0xffffffffu, (int)reach, j);
                const uint32_t kj = sh.lkey[j];
                const bool before = kj > k || (kj == k && sh.lidx[j] < idx);
                if (rj && (!reach || before)) best = false;
                if (!rj && !reach && (kj < k || (kj == k && sh.lidx[j] > idx))) best = false;
            }
            if (best) {
                sh.bkey = k;
                sh.bidx = idx;
            }
        }
        __syncthreads();
        return;
    }
}

// The weight of the kept tokens of [lo, hi), all threads; the sum goes to sh.total.
template <typename T>
__device__ u64 kept_weight(const T* lg, int i, uint32_t bkey, int bidx, const RowScale& row, const uint32_t* table) {
    const float l = load(lg, i);
    const uint32_t k = key_of(l);
    return (k > bkey || (k == bkey && i <= bidx)) ? weight(l, row, table) : 0;
}

template <typename T>
__device__ void sum_kept(const T* lg, int vocab, uint32_t bkey, int bidx, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const RowScale row = sh.row;
    const int per = (vocab + kWarps - 1) / kWarps;
    u64 w = 0;
    const int end = min(vocab, (warp + 1) * per);
    for (int i = warp * per + lane; i < end; i += 32) w += kept_weight(lg, i, bkey, bidx, row, sh.table);
    w = warp_sum(w);
    if (lane == 0) sh.part[warp] = w;
    __syncthreads();
    if (tid == 0) {
        u64 t = 0;
        for (int i = 0; i < kWarps; ++i) t += sh.part[i];
        sh.total = t;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(Params p, DevError* err) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long b = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (p.active && p.active[b] == 0) return;
    const T* lg = static_cast<const T*>(p.logits) + b * p.stride;
    const float temp = p.temperature ? p.temperature[b] : 1.0f;
    const float topp = p.top_p ? p.top_p[b] : 1.0f;
    const float minp = p.min_p ? p.min_p[b] : 0.0f;
    const int topk = p.top_k ? p.top_k[b] : 0;
    // a decode loop's numbers, one per position (a negative position has been recorded by the step)
    const long long at = p.uniform_stride <= 1 ? b : b * p.uniform_stride + max(p.positions[b], 0) % p.uniform_stride;
    const float u = p.uniform[at];
    const bool ok = temp >= 0.f && temp < INFINITY && topp == topp && minp == minp && u >= 0.f && u < 1.f;
    if (!ok) {
        if (tid == 0) {
            record_device_error(err, kErrSampleArg, b, 0);
            p.tokens[b] = -1;
            if (p.probs) p.probs[b] = 0.f;
        }
        return;
    }
    if (tid < 64) sh.table[tid] = kExp2[tid];
    // the largest logit, at its lowest index
    uint32_t bk = 0;
    int bi = 0x7FFFFFFF;
    for (int i = tid; i < p.vocab; i += kThreads) {
        const uint32_t k = key_of(load(lg, i));
        if (k > bk) {
            bk = k;
            bi = i;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const uint32_t k = __shfl_xor_sync(0xffffffffu, bk, o);
        const int i = __shfl_xor_sync(0xffffffffu, bi, o);
        if (k > bk || (k == bk && i < bi)) {
            bk = k;
            bi = i;
        }
    }
    if (lane == 0) {
        sh.wkey[warp] = bk;
        sh.widx[warp] = bi;
    }
    __syncthreads();
    bk = sh.wkey[0];
    bi = sh.widx[0];
    for (int w = 1; w < kWarps; ++w) {
        if (sh.wkey[w] > bk || (sh.wkey[w] == bk && sh.widx[w] < bi)) {
            bk = sh.wkey[w];
            bi = sh.widx[w];
        }
    }
    const bool none = bk <= 0x007FFFFFu;   // the key of -inf
    if (none || temp < kMinTemperature) {
        if (tid == 0) {
            p.tokens[b] = none ? -1 : bi;
            if (p.probs) p.probs[b] = none ? 0.f : 1.f;
        }
        return;
    }
    const float top = __uint_as_float(bk & 0x80000000u ? bk ^ 0x80000000u : ~bk);
    if (tid == 0) {
        const double c = 64.0 * 1.4426950408889634 / (double)temp;
        RowScale r;
        // exponents of logits near the largest stay below 2^21 in magnitude, where the floor is exact
        r.ref = fabs((double)top * c) > 0x1p20 ? top : 0.f;
        r.c_hi = (float)c;
        r.c_lo = (float)(c - (double)r.c_hi);
        const float x = top - r.ref;
        r.magic = 12582912.0f - floorf(__fmul_rd(x, r.c_hi));
        r.low = fmaxf(x - (float)(3200.0 / c), -FLT_MAX);       // 2^-50 of the largest: weight 0
        r.top = top;
        r.dist = (float)fmin(16777216.0 / (24.0 * (double)temp), (double)FLT_MAX);   // finite: 0 r.dist is 0
        sh.row = r;
    }
    __syncthreads();
    uint32_t bkey = 0x00800000u;   // above -inf
    int bidx = 0x7FFFFFFF;
    if (minp > 0.f) {
        // the least f32 at or above top + T ln(min_p)
        const float thr = minp >= 1.f ? top : __double2float_ru((double)top + (double)temp * log((double)minp));
        const uint32_t k = key_of(thr + 0.0f);
        bkey = k > bkey ? k : bkey;
    }
    auto tighten = [&]() {
        if (sh.bkey > bkey || (sh.bkey == bkey && sh.bidx < bidx)) {
            bkey = sh.bkey;
            bidx = sh.bidx;
        }
    };
    uint32_t kkey = 0x00800000u;
    int kidx = 0x7FFFFFFF;
    if (topk > 0 && topk < p.vocab) {
        find_border(lg, p.vocab, false, (u64)topk, sh);
        kkey = sh.bkey;
        kidx = sh.bidx;
        tighten();
        __syncthreads();
    }
    if (topp < 1.f) {
        sum_kept(lg, p.vocab, kkey, kidx, sh);
        const double want = ceil((double)topp * (double)sh.total);
        find_border(lg, p.vocab, true, want < 1.0 ? 1ull : (u64)want, sh);
        tighten();
        __syncthreads();
    }
    // the draw: the warp whose range the running sum passes the target in, then that warp's tokens
    sum_kept(lg, p.vocab, bkey, bidx, sh);
    if (warp == 0) {
        const RowScale row = sh.row;
        const double target = (double)u * (double)sh.total;
        u64 c = 0;
        int w = 0;
        while (w < kWarps - 1 && (double)(c + sh.part[w]) <= target) c += sh.part[w++];
        const int per = (p.vocab + kWarps - 1) / kWarps;
        const int end = min(p.vocab, (w + 1) * per);
        int token = bi;
        u64 tw = 0;
        for (int i0 = w * per; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            const u64 wt = i < end ? kept_weight(lg, i, bkey, bidx, row, sh.table) : 0;
            u64 s = wt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            const unsigned pass = __ballot_sync(0xffffffffu, wt > 0 && (double)(c + s) > target);
            if (pass) {
                const int n = __ffs(pass) - 1;
                token = i0 + n;
                tw = __shfl_sync(0xffffffffu, wt, n);
                break;
            }
            c += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) {
            p.tokens[b] = token;
            if (p.probs) p.probs[b] = (float)((double)tw / (double)sh.total);
        }
    }
}

}  // namespace

int sample_launch(const SampleArgs& a, cudaStream_t s, bool pdl) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "sampling: no device error record");
    Params p = {};
    p.logits = a.logits;
    p.stride = a.row_stride;
    p.vocab = (int)a.vocab;
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
    const dim3 grid((unsigned)a.batch);
    const cudaError_t e = a.dtype == QL_DTYPE_F32
                              ? launch(sample_kernel<float>, grid, dim3(kThreads), 0, s, pdl, p, err)
                              : launch(sample_kernel<__half>, grid, dim3(kThreads), 0, s, pdl, p, err);
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
    return sample_launch(a, static_cast<cudaStream_t>(stream), false);
}
