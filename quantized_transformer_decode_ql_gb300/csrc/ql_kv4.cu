// Rows of K and V quantised into the 4-bit pool as they are written, and read back.
//
// A row of one kv head is 2 HD values in (or out) and 1.25 HD bytes out (or in). HD / 8 neighbouring lanes
// share the (row, kv head): 8 key values and 8 value values a lane, loaded before anything else, so that a
// full SM has 64 KB (f32) in flight. A CTA stays with one kv head (no division by the heads); its rows'
// pieces are at least 128 bytes each.
//
// Measured: 16000 rows of 8 x 64 f16 written in 15 us and read back in 8 (23 us together, 3.3 TB/s), 40960
// rows of 8 x 128 read back as f16 in 38 us (5.8 TB/s; a copy reaches 6.8). Reading is bound by memory;
// writing by its 370 instructions a lane (67% of the issue slots): each code's border is decided exactly.
#include "ql_internal.h"
#include "ql_kv4_rec.cuh"

namespace ql {
namespace {

constexpr int kKv4Threads = 128;   // with 256 a prompt written and read back takes 25.4 us instead of 24.5, a long context read 41.6 instead of 39.3

template <typename T>
__device__ __forceinline__ void load2(const T* p, float& a, float& b);
template <>
__device__ __forceinline__ void load2<float>(const float* p, float& a, float& b) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    a = v.x;
    b = v.y;
}
template <>
__device__ __forceinline__ void load2<__half>(const __half* p, float& a, float& b) {
    const float2 v = __half22float2(__ldg(reinterpret_cast<const __half2*>(p)));
    a = v.x;
    b = v.y;
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, float* x);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* x) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__half>(const __half* p, float* x) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

template <int HD, typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_write_kernel(const T* __restrict__ k, const T* __restrict__ v,
                                                                long long ks, long long vs,
                                                                const long long* __restrict__ slots, long long n,
                                                                uint8_t* __restrict__ pool, long long num_blocks,
                                                                DevError* err) {
    using R = Kv4<HD>;
    const long long i = ((long long)blockIdx.x * kKv4Threads + threadIdx.x) / R::LANES;
    const int l = threadIdx.x % R::LANES, b = l >> 2, j = l & 3, g = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    const bool in = i < n;   // the last warp's spare lanes still take part in its shuffles
    float xk[8] = {}, xv[8] = {};
    long long slot = -1;
    if (in) {
        slot = __ldg(slots + i);
        const T* kr = k + i * ks + (size_t)g * HD + 32 * b;
        const T* vr = v + i * vs + (size_t)g * HD + 32 * b;
        load4(kr + 4 * j, xk);
        load4(kr + 16 + 4 * j, xk + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) load2(vr + 2 * j + 8 * q, xv[q], xv[4 + q]);
    }
    const long long blk = slot >> 4;
    const bool live = slot >= 0 && blk < num_blocks;
    if (in && !live && slot != -1 && g == 0 && l == 0) record_device_error(err, kErrKvSlot, i, slot);
    uint8_t* rec = pool + ((size_t)(live ? blk : 0) * gridDim.y + g) * R::BYTES;
    const int fault = kv4_put_rows<HD>(xk, xv, rec, (int)(slot & 15), b, j, live);
    if (live && fault) record_device_error(err, fault == 2 ? kErrKvNonFinite : kErrKvOverflow, i, g);
}

// 8 consecutive values d c + m, each rounded once, from their codes in the bytes of c[0], c[1]. f16: one
// fused multiply-add of exact f16 codes (1024 + c has the code in its low byte); f32: d c is exact, and so
// the fused multiply-add rounds once.
__device__ __forceinline__ void put8(__half* o, const uint32_t (&c)[2], __half d, __half m) {
    const __half2 dd = __half2half2(d), mm = __half2half2(m), k1024 = __float2half2_rn(1024.f);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = __byte_perm(c[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140);
        const __half2 y = __hfma2(__hsub2(*reinterpret_cast<const __half2*>(&h), k1024), dd, mm);
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* o, const uint32_t (&c)[2], __half d, __half m) {
    const float df = __half2float(d), mf = __half2float(m);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)   // 2^23 + c, minus 2^23
        y[i] = fmaf(df, __uint_as_float(__byte_perm(c[i >> 2], 0x4B000000u, 0x7650 + (i & 3))) - 8388608.f, mf);
    reinterpret_cast<float4*>(o)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(y[4], y[5], y[6], y[7]);
}

// Whether one of those values overflows f16, d and m being finite: the largest code would have to first.
__device__ __forceinline__ bool overflows8(const uint32_t (&c)[2], __half d, __half m) {
    const float df = __half2float(d), mf = __half2float(m);
    if (!(fabsf(df) < INFINITY && fabsf(mf) < INFINITY && fabsf(fmaf(df, 15.f, mf)) >= 65520.f)) return false;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= fabsf(fmaf(df, (float)((c[i >> 2] >> (8 * (i & 3))) & 15u), mf)) >= 65520.f;
    return any;
}

// A lane writes elements 8 w .. 8 w + 7 of block b of the key row and of the value row. The value codes of
// those 8 elements lie in 8 units: each lane loads one word (a unit's two blocks), and the 8 lanes of a
// pair of blocks transpose their 8 words of 8 codes by three exchanges (halves, bytes, nibbles). A warp's
// life is two round trips (slots, records), so a thread takes two rows at once.
// BLOCKS: row i goes to slot i % 16 of block i / 16 of a pool [blocks][n_kv][16][HD] instead, and a finite value that
// is none as f16 is recorded (the format holds values up to 1e6, the attention that reads this pool does not).
constexpr int kReadRows = 2;
template <int HD, typename T, bool BLOCKS>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const uint8_t* __restrict__ pool,
                                                               const long long* __restrict__ slots, long long n,
                                                               long long num_blocks, T* __restrict__ k,
                                                               T* __restrict__ v, long long ks, long long vs,
                                                               DevError* err) {
    using R = Kv4<HD>;
    constexpr int P = R::NB / 2;                        // pairs of blocks
    constexpr int ROWS = kKv4Threads / R::LANES;        // rows of a CTA at a time
    const int l = threadIdx.x % R::LANES, pair = l % P, u = l / P, g = blockIdx.y;
    const int b = 2 * pair + (u >> 2), w = u & 3;
    const long long i0 = (long long)blockIdx.x * (kReadRows * ROWS) + threadIdx.x / R::LANES;
    long long slot[kReadRows];
    bool live[kReadRows];                               // the others still take part in the exchanges
    uint32_t k0[kReadRows], k1[kReadRows], x[kReadRows];
    __half dk[kReadRows], mk[kReadRows], dv[kReadRows], mv[kReadRows];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) slot[r] = i0 + r * ROWS < n ? __ldg(slots + i0 + r * ROWS) : -1;
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
        const long long blk = slot[r] >> 4;
        live[r] = slot[r] >= 0 && blk < num_blocks;
        if (!live[r] && slot[r] != -1 && g == 0 && l == 0) record_device_error(err, kErrKvSlot, i0 + r * ROWS, slot[r]);
        const int s = (int)(slot[r] & 15);
        const uint8_t* rec = pool + ((size_t)(live[r] ? blk : 0) * gridDim.y + g) * R::BYTES;
        const uint8_t* krow = rec + R::KC + s * (HD / 2) + 4 * (R::NB * 2 * (w & 1) + b);
        k0[r] = __ldg(reinterpret_cast<const uint32_t*>(krow));
        k1[r] = __ldg(reinterpret_cast<const uint32_t*>(krow + 4 * R::NB));
        x[r] = __ldg(reinterpret_cast<const uint32_t*>(rec + R::VC + s * (HD / 2) + R::vunit(s, u) + 4 * pair));
        dk[r] = reinterpret_cast<const __half*>(rec + R::KD)[s * R::NB + b];
        mk[r] = reinterpret_cast<const __half*>(rec + R::KM)[s * R::NB + b];
        dv[r] = reinterpret_cast<const __half*>(rec + R::VD)[R::vscale(s, b)];
        mv[r] = reinterpret_cast<const __half*>(rec + R::VM)[R::vscale(s, b)];
    }
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
        uint32_t y = __shfl_xor_sync(0xffffffffu, x[r], 4 * P);
        uint32_t z = __byte_perm(x[r], y, u & 4 ? 0x3276 : 0x5410);
        y = __shfl_xor_sync(0xffffffffu, z, 2 * P);
        z = __byte_perm(z, y, u & 2 ? 0x3715 : 0x6240);
        y = __shfl_xor_sync(0xffffffffu, z, P);
        z = u & 1 ? ((y >> 4) & 0x0f0f0f0fu) | (z & 0xf0f0f0f0u) : (z & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
        if (!live[r]) continue;
        const int sh = 4 * (w >> 1);
        const uint32_t ck[2] = {(k0[r] >> sh) & 0x0f0f0f0fu, (k1[r] >> sh) & 0x0f0f0f0fu};
        const uint32_t even = z & 0x0f0f0f0fu, odd = (z >> 4) & 0x0f0f0f0fu;
        const uint32_t cv[2] = {__byte_perm(even, odd, 0x5140), __byte_perm(even, odd, 0x7362)};
        const long long i = i0 + r * ROWS;
        const long long at = 32 * b + 8 * w + (BLOCKS ? ((i >> 4) * gridDim.y + g) * (16ll * HD) + (i & 15) * HD : (long long)g * HD);
        put8(k + (BLOCKS ? 0 : i * ks) + at, ck, dk[r], mk[r]);
        put8(v + (BLOCKS ? 0 : i * vs) + at, cv, dv[r], mv[r]);
        if (BLOCKS && (overflows8(ck, dk[r], mk[r]) || overflows8(cv, dv[r], mv[r]))) record_device_error(err, kErrKvOverflow, i, g);
    }
}

// The decode step's q and new K / V rows: per-head RMSNorm and NeoX rotation (pairs i, i + HD / 2) of the f32
// q | k | v projection, q to f16, the key row and the value row of a kv head quantised into the pool at the
// position's slot. As in the writer, HD / 8 lanes share a head, a lane holding 8 elements; it loads their
// rotation partners too, which are another lane's.
struct Kv4RopeParams {
    const float* qkv;
    const float* q_norm;
    const float* k_norm;
    const float* cos_t;
    const float* sin_t;
    const int32_t* positions;
    const int32_t* active;
    const int32_t* block_tables;
    float eps;
    int n_heads, n_kv;
    long long items, maxb, num_blocks, max_position;
    __half* q_out;
    uint8_t* pool;
};
template <int HD>
__global__ void __launch_bounds__(kKv4Threads) kv4_norm_rope_kernel(Kv4RopeParams p, DevError* err) {
    using R = Kv4<HD>;
    constexpr int H2 = HD / 2;
    const long long item = ((long long)blockIdx.x * kKv4Threads + threadIdx.x) / R::LANES;
    const int l = threadIdx.x % R::LANES, b = l >> 2, j = l & 3;
    pdl_wait();
    pdl_trigger();
    const int heads = p.n_heads + p.n_kv;
    const bool in = item < p.items;   // all lanes take part in the shuffles
    const long long t = in ? item / heads : 0;
    const int h = in ? (int)(item - t * heads) : 0;
    const bool act = in && (p.active == nullptr || p.active[t] != 0);
    const int pos = act ? p.positions[t] : 0;
    const bool ok = act && pos >= 0 && pos < p.max_position;
    if (act && !ok && h == 0 && l == 0) record_device_error(err, kErrRopePosition, t, pos);
    const bool is_q = h < p.n_heads;
    const float* src = p.qkv + (t * (p.n_heads + 2 * p.n_kv) + h) * HD;
    const float* w = is_q ? p.q_norm : p.k_norm;
    const float* c = p.cos_t + (size_t)(ok ? pos : 0) * H2;
    const float* s = p.sin_t + (size_t)(ok ? pos : 0) * H2;
    // elements e, e + 1, ... of this lane's two quads and their partners
    const int e0 = 32 * b + 4 * j;
    const bool low = e0 < H2;
    float x[8], y[8];
    float ss = 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = e0 + 16 * q, o = low ? e + H2 : e - H2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * q + i] = ok ? __ldcg(src + e + i) : 0.f;
            y[4 * q + i] = ok ? __ldcg(src + o + i) : 0.f;
            ss = fmaf(x[4 * q + i], x[4 * q + i], ss);
        }
    }
#pragma unroll
    for (int o = R::LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, 1.0f / (float)HD, p.eps));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = e0 + 16 * q, o = low ? e + H2 : e - H2, a = low ? e : o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float xn = x[4 * q + i] * r * __ldg(w + e + i), yn = y[4 * q + i] * r * __ldg(w + o + i);
            const float cc = __ldg(c + a + i), sn = __ldg(s + a + i);
            x[4 * q + i] = low ? xn * cc - yn * sn : yn * sn + xn * cc;
        }
    }
    if (ok && is_q) {
        __half* qo = p.q_out + (t * p.n_heads + h) * HD;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const __half2 a = __floats2half2_rn(x[4 * q], x[4 * q + 1]), d = __floats2half2_rn(x[4 * q + 2], x[4 * q + 3]);
            *reinterpret_cast<uint2*>(qo + e0 + 16 * q) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&d));
        }
    }
    const int g = h - p.n_heads;
    const long long lb = pos >> 4;
    const int phys = ok && !is_q ? p.block_tables[t * p.maxb + lb] : -1;   // max_position is 16 maxb at most
    const bool live = phys >= 0 && phys < p.num_blocks;
    if (ok && !is_q && !live && l == 0) record_device_error(err, kErrRopeBlock, t * p.maxb + lb, phys);
    float v[8] = {};
    if (live) {
        const float* vs = src + (size_t)p.n_kv * HD + 32 * b + 2 * j;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = __ldcg(vs + 8 * q);
            v[4 + q] = __ldcg(vs + 8 * q + 1);
        }
    }
    uint8_t* rec = p.pool + ((size_t)(live ? phys : 0) * p.n_kv + (live ? g : 0)) * R::BYTES;
    const int fault = kv4_put_rows<HD>(x, v, rec, pos & 15, b, j, live);
    if (live && fault) record_device_error(err, fault == 2 ? kErrKvNonFinite : kErrKvOverflow, t, g);
}

// The checks that the writer and the reader share; `grid` for n > 0, each CTA `times` as many rows as its threads hold.
int kv4_rows_check(const char* name, const void* k, const void* v, int dtype, int64_t ks, int64_t vs,
                   const int64_t* slots, int64_t n, int n_kv, int hd, const void* pool, int64_t num_blocks,
                   int times, unsigned* grid) {
    const std::string nm(name);
    if (dtype != QL_DTYPE_F32 && dtype != QL_DTYPE_F16) return set_error(QL_EINVAL, nm + ": dtype must be f32 or f16");
    if (hd != 64 && hd != 128) return set_error(QL_EINVAL, nm + ": head_dim must be 64 or 128");
    if (n < 0 || n_kv <= 0 || num_blocks <= 0)
        return set_error(QL_EINVAL, nm + ": need n >= 0, n_kv_heads and num_blocks > 0");
    *grid = 0;
    if (n == 0) return QL_OK;
    if (!k || !v || !slots || !pool) return set_error(QL_EINVAL, nm + ": null pointer");
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    if (!a16(k) || !a16(v) || !a16(pool))
        return set_error(QL_EINVAL, nm + ": k, v and the pool must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(slots) & 7) != 0) return set_error(QL_EINVAL, nm + ": slots must be 8-byte aligned");
    const int64_t per = dtype == QL_DTYPE_F32 ? 4 : 8;
    if (n > 1 && (ks < (int64_t)n_kv * hd || vs < (int64_t)n_kv * hd || ks % per || vs % per))
        return set_error(QL_EINVAL, nm + ": row strides must be multiples of 16 bytes and at least n_kv_heads * head_dim");
    const int64_t rows = (int64_t)times * kKv4Threads / (hd / 8);   // of a CTA
    if (n > ((1ll << 31) - 1) * rows || n_kv > 65535) return set_error(QL_EINVAL, nm + ": too many rows or heads");
    *grid = (unsigned)((n + rows - 1) / rows);
    return QL_OK;
}

}  // namespace

int kv4_norm_rope_launch(const RopeArgs& a, uint8_t* pool, cudaStream_t s, bool pdl) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "4-bit norm_rope: no device error record");
    Kv4RopeParams p = {};
    p.qkv = a.qkv;
    p.q_norm = a.q_norm;
    p.k_norm = a.k_norm;
    p.cos_t = a.cos_t;
    p.sin_t = a.sin_t;
    p.positions = a.positions;
    p.active = a.active;
    p.block_tables = a.block_tables;
    p.eps = a.eps;
    p.n_heads = a.n_heads;
    p.n_kv = a.n_kv_heads;
    p.items = (long long)a.batch * (a.n_heads + a.n_kv_heads);
    p.maxb = a.max_blocks_per_seq;
    p.num_blocks = a.num_blocks;
    p.max_position = a.max_position;
    p.q_out = a.q_out;
    p.pool = pool;
    const long long grid = (p.items * (a.head_dim / 8) + kKv4Threads - 1) / kKv4Threads;
    const cudaError_t e = a.head_dim == 128
                              ? launch(kv4_norm_rope_kernel<128>, dim3((unsigned)grid), dim3(kKv4Threads), 0, s, pdl, p, err)
                              : launch(kv4_norm_rope_kernel<64>, dim3((unsigned)grid), dim3(kKv4Threads), 0, s, pdl, p, err);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "4-bit norm_rope launch");
}

int kv4_read_blocks_launch(const uint8_t* pool, const long long* slots, long long n, int n_kv, int head_dim, long long num_blocks,
                           __half* k, __half* v, cudaStream_t s) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "4-bit read: no device error record");
    const long long rows = kReadRows * kKv4Threads / (head_dim / 8);
    const dim3 grid((unsigned)((n + rows - 1) / rows), (unsigned)n_kv);
    auto go = [&](auto kernel) {
        return launch(kernel, grid, dim3(kKv4Threads), 0, s, false, pool, slots, n, num_blocks, k, v, 0ll, 0ll, err);
    };
    const cudaError_t e = head_dim == 128 ? go(kv4_read_kernel<128, __half, true>) : go(kv4_read_kernel<64, __half, true>);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "4-bit read launch");
}

}  // namespace ql

extern "C" int64_t ql_kv4_record_bytes(int head_dim) {
    return (head_dim == 64 || head_dim == 128) ? (int64_t)20 * head_dim : 0;
}

extern "C" int ql_kv4_write(const void* d_k, const void* d_v, int dtype, int64_t k_stride, int64_t v_stride,
                            const int64_t* d_slots, int64_t n, int n_kv_heads, int head_dim, void* d_pool,
                            int64_t num_blocks, void* stream) {
    using namespace ql;
    unsigned grid = 0;
    if (int rc = kv4_rows_check("ql_kv4_write", d_k, d_v, dtype, k_stride, v_stride, d_slots, n, n_kv_heads, head_dim,
                                d_pool, num_blocks, 1, &grid))
        return rc;
    if (grid == 0) return QL_OK;
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "ql_kv4_write: no device error record");
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        return launch(kernel, dim3(grid, (unsigned)n_kv_heads), dim3(kKv4Threads), 0, static_cast<cudaStream_t>(stream), true,
                      static_cast<const T*>(d_k), static_cast<const T*>(d_v), (long long)k_stride, (long long)v_stride,
                      reinterpret_cast<const long long*>(d_slots), (long long)n,
                      static_cast<uint8_t*>(d_pool), (long long)num_blocks, err);
    };
    const bool f32 = dtype == QL_DTYPE_F32;
    const cudaError_t e = head_dim == 128 ? (f32 ? go(kv4_write_kernel<128, float>, 0.f)
                                                 : go(kv4_write_kernel<128, __half>, __half()))
                                          : (f32 ? go(kv4_write_kernel<64, float>, 0.f)
                                                 : go(kv4_write_kernel<64, __half>, __half()));
    return e == cudaSuccess ? QL_OK : cuda_error(e, "ql_kv4_write");
}

extern "C" int ql_kv4_read(const void* d_pool, const int64_t* d_slots, int64_t n, int n_kv_heads, int head_dim,
                           int64_t num_blocks, void* d_k, void* d_v, int dtype, int64_t k_stride, int64_t v_stride,
                           void* stream) {
    using namespace ql;
    unsigned grid = 0;
    if (int rc = kv4_rows_check("ql_kv4_read", d_k, d_v, dtype, k_stride, v_stride, d_slots, n, n_kv_heads, head_dim,
                                d_pool, num_blocks, kReadRows, &grid))
        return rc;
    if (grid == 0) return QL_OK;
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "ql_kv4_read: no device error record");
    auto go = [&](auto kernel, auto zero) {
        using T = decltype(zero);
        return launch(kernel, dim3(grid, (unsigned)n_kv_heads), dim3(kKv4Threads), 0, static_cast<cudaStream_t>(stream), true,
                      static_cast<const uint8_t*>(d_pool), reinterpret_cast<const long long*>(d_slots),
                      (long long)n, (long long)num_blocks, static_cast<T*>(d_k),
                      static_cast<T*>(d_v), (long long)k_stride, (long long)v_stride, err);
    };
    const bool f32 = dtype == QL_DTYPE_F32;
    const cudaError_t e = head_dim == 128 ? (f32 ? go(kv4_read_kernel<128, float, false>, 0.f)
                                                 : go(kv4_read_kernel<128, __half, false>, __half()))
                                          : (f32 ? go(kv4_read_kernel<64, float, false>, 0.f)
                                                 : go(kv4_read_kernel<64, __half, false>, __half()));
    return e == cudaSuccess ? QL_OK : cuda_error(e, "ql_kv4_read");
}
