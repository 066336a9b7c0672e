// Latent attention, the rows: a token's latent vector normalised and its key part rotated into the paged cache, its query
// heads' last 64 values rotated.
//
//   row of the cache = f16( x[0:R] / sqrt(mean x[0:R]^2 + eps) * w | rot(x[R:R+64], p) )
//   query head       = f16( q[0:D] | rot(q[D:D+64], p) )
//
// rot turns the pairs (i, i + 32) by the tables' angle of position p. A warp takes one head of a row, or its latent vector.
#include "ql_mla.h"

namespace ql {
namespace {

using mla::kRope;

// N consecutive values (a multiple of 4) from a 16-byte (f32) or 8-byte (f16) boundary, in f32
template <int N>
__device__ __forceinline__ void load_row(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
    }
}
template <int N>
__device__ __forceinline__ void load_row(const __half* p, float* x) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 v = __half22float2(__ldg(reinterpret_cast<const __half2*>(p + i)));
        x[i] = v.x;
        x[i + 1] = v.y;
    }
}
__device__ __forceinline__ float load_one(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_one(const __half* p) { return __half2float(__ldg(p)); }

template <int N>
__device__ __forceinline__ void store_row(__half* p, const float* x) {
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<__half2*>(p + i) = __floats2half2_rn(x[i], x[i + 1]);
}

struct AppendParams {
    const void* q;
    const void* kv;
    long long q_stride, kv_stride;
    const float* norm;
    const float* cos_t;
    const float* sin_t;
    const int32_t* positions;
    const long long* slots;
    float eps;
    int n_heads;
    __half* q_out;
    __half* pool;
    long long num_blocks, max_position;
};

template <int D, int R, typename T>
__global__ void __launch_bounds__(256) mla_append_kernel(AppendParams p, DevError* err) {
    const long long i = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);   // 0: the latent vector, 1 + h: head h
    pdl_wait();
    pdl_trigger();
    if (item > (p.q != nullptr ? p.n_heads : 0)) return;
    const long long slot = __ldg(p.slots + i);
    const int pos = __ldg(p.positions + i);
    const bool head = item > 0;
    const T* src = head ? static_cast<const T*>(p.q) + i * p.q_stride + (long long)(item - 1) * (D + kRope)
                        : static_cast<const T*>(p.kv) + i * p.kv_stride;
    if (slot < 0 || slot >= 16 * p.num_blocks || pos < 0 || pos >= p.max_position) {
        if (!head && lane == 0 && slot != -1) {
            const bool bad_slot = slot < 0 || slot >= 16 * p.num_blocks;
            record_device_error(err, bad_slot ? kErrKvSlot : kErrRopePosition, i, bad_slot ? slot : pos);
        }
        return;
    }
    const float c = __ldg(p.cos_t + (long long)pos * (kRope / 2) + lane), s = __ldg(p.sin_t + (long long)pos * (kRope / 2) + lane);
    const T* tail = src + (head ? D : R);
    const float a = load_one(tail + lane), b = load_one(tail + kRope / 2 + lane);
    const float ra = a * c - b * s, rb = b * c + a * s;
    if (head) {
        float x[D / 32];
        load_row<D / 32>(src + lane * (D / 32), x);
        __half* o = p.q_out + (i * p.n_heads + item - 1) * (D + kRope);
        store_row<D / 32>(o + lane * (D / 32), x);
        o[D + lane] = __float2half_rn(ra);
        o[D + kRope / 2 + lane] = __float2half_rn(rb);
        return;
    }
    constexpr int V = R / 32;
    float x[V], w[V], ss = 0.f;
    load_row<V>(src + lane * V, x);
    load_row<V>(p.norm + lane * V, w);
#pragma unroll
    for (int k = 0; k < V; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, 1.0f / (float)R, p.eps));
    __half* o = p.pool + slot * (R + kRope);
    float most = fmaxf(fabsf(ra), fabsf(rb));
    bool nan = !(most <= INFINITY) || ra != ra || rb != rb;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        x[k] *= r * w[k];
        nan |= x[k] != x[k];
        most = fmaxf(most, fabsf(x[k]));
    }
    store_row<V>(o + lane * V, x);
    o[R + lane] = __float2half_rn(ra);
    o[R + kRope / 2 + lane] = __float2half_rn(rb);
    if (nan || most >= 65520.f) record_device_error(err, kErrLatentValue, i, 0);
}

// ---------------------------------------------------------------- attention, one warp a token
// scratch: q' f32 [rows][H][R + 64], o f32 [rows][H][R]
template <int D, int R>
__global__ void __launch_bounds__(256) mla_absorb_kernel(const __half* q, const __half* w, float* qc, int H, DevError* err) {
    __shared__ float qs[D];
    const long long row = (long long)blockIdx.x;
    const int h = blockIdx.y;
    const __half* src = q + (row * H + h) * (D + kRope);
    for (int d = threadIdx.x; d < D; d += 256) qs[d] = __half2float(src[d]);
    __syncthreads();
    float* dst = qc + (row * H + h) * (R + kRope);
    for (int r = threadIdx.x; r < R; r += 256) {
        float a = 0.f;
        for (int d = 0; d < D; ++d) a = fmaf(qs[d], __half2float(w[((long long)h * 2 * D + d) * R + r]), a);
        dst[r] = a;
        if (!(fabsf(a) < 65520.f)) record_device_error(err, kErrLatentValue, row, h);
    }
    for (int r = threadIdx.x; r < kRope; r += 256) dst[R + r] = __half2float(src[D + r]);
}

template <int R>
__global__ void __launch_bounds__(256) mla_simple_kernel(const float* qc, const __half* pool, const int32_t* tables, const int32_t* lens,
                                                         const int32_t* position, long long maxb, long long num_blocks, float scale,
                                                         float* o, int H, DevError* err) {
    constexpr int W = R + kRope, V = W / 32, VR = R / 32;
    __shared__ float sm[8], sl[8], sa[8][R];
    const long long row = blockIdx.x;
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t* table = tables + (position ? 0 : row * maxb);
    const long long len = position ? (long long)*position + row + 1 : lens[row];
    const bool bad = position ? *position < 0 || *position + (long long)gridDim.x > maxb * 16 : len <= 0 || len > maxb * 16;
    if (bad) {
        if (len != 0 && threadIdx.x == 0 && h == 0) record_device_error(err, kErrAttnLength, row, len);
        return;
    }
    float x[V], acc[VR], m = -INFINITY, l = 0.f;
    for (int k = 0; k < V; ++k) x[k] = qc[(row * H + h) * W + k * 32 + lane] * scale;
    for (int k = 0; k < VR; ++k) acc[k] = 0.f;
    for (long long t = warp; t < len; t += 8) {
        const int blk = table[t >> 4];
        if (blk < 0 || blk >= num_blocks) {
            if (lane == 0) record_device_error(err, kErrAttnBlock, row * maxb + (t >> 4), blk);
            continue;
        }
        const __half* src = pool + ((long long)blk * 16 + (t & 15)) * W;
        float c[V], d = 0.f;
        for (int k = 0; k < V; ++k) {
            c[k] = __half2float(src[k * 32 + lane]);
            d = fmaf(c[k], x[k], d);
        }
        for (int s = 16; s; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
        const float mn = fmaxf(m, d), f = m == -INFINITY ? 0.f : __expf(m - mn), e = __expf(d - mn);
        m = mn;
        l = l * f + e;
        for (int k = 0; k < VR; ++k) acc[k] = acc[k] * f + e * c[k];
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int k = 0; k < VR; ++k) sa[warp][k * 32 + lane] = acc[k];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, f[8];
    for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < 8; ++w) {
        f[w] = sm[w] == -INFINITY ? 0.f : __expf(sm[w] - mm);
        ll += sl[w] * f[w];
    }
    for (int r = threadIdx.x; r < R; r += 256) {
        float a = 0.f;
        for (int w = 0; w < 8; ++w) a += sa[w][r] * f[w];
        o[(row * H + h) * R + r] = ll > 0.f ? a / ll : 0.f;
    }
}

template <int D, int R>
__global__ void __launch_bounds__(128) mla_out_kernel(const float* o, const __half* w, const int32_t* lens, const int32_t* position, long long cap, __half* out, int H) {
    __shared__ float os[R];
    const long long row = blockIdx.x;
    const int h = blockIdx.y;
    if (lens ? lens[row] <= 0 || lens[row] > cap : *position < 0 || *position + (long long)gridDim.x > cap) return;
    for (int r = threadIdx.x; r < R; r += 128) os[r] = o[(row * H + h) * R + r];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 128) {
        float a = 0.f;
        for (int r = 0; r < R; ++r) a = fmaf(os[r], __half2float(w[((long long)h * 2 * D + D + d) * R + r]), a);
        out[(row * H + h) * D + d] = __float2half_rn(a);
    }
}

template <int D, int R>
int simple(const __half* q, const __half* w, const __half* pool, const int32_t* tables, const int32_t* lens, const int32_t* position,
           long long rows, int H, long long maxb, long long num_blocks, float scale, __half* out, void* ws, cudaStream_t s) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "latent attention: no device error record");
    float* qc = static_cast<float*>(ws);
    float* o = qc + rows * H * (R + kRope);
    const dim3 grid((unsigned)rows, (unsigned)H);
    mla_absorb_kernel<D, R><<<grid, 256, 0, s>>>(q, w, qc, H, err);
    mla_simple_kernel<R><<<grid, 256, 0, s>>>(qc, pool, tables, lens, position, maxb, num_blocks, scale, o, H, err);
    mla_out_kernel<D, R><<<grid, 128, 0, s>>>(o, w, lens, position, maxb * 16, out, H);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? QL_OK : cuda_error(e, "latent attention");
}

}  // namespace

int mla::attn_check(const char* name, const void* q, const void* w, const void* pool, const void* table, const void* lens, int head_dim,
                    int rank, int rope_dim, int block_size, int64_t num_blocks, const void* out, const void* ws, size_t ws_bytes, size_t need) {
    const std::string nm(name);
    if (!q || !w || !pool || !table || !lens || !out || !ws) return set_error(QL_EINVAL, nm + ": null pointer");
    if (!mla::shape_ok(head_dim, rank) || rope_dim != kRope || block_size != mla::kBlock)
        return set_error(QL_EINVAL, nm + ": head_dim must be 64 or 128, rank 256 or 512, rope_dim 64, block_size 16");
    if (need == 0 || num_blocks < 1 || num_blocks >= (1ll << 27))
        return set_error(QL_EINVAL, nm + ": sizes out of range");
    auto aligned = [](const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (!aligned(q, 16) || !aligned(w, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(ws, 128))
        return set_error(QL_EINVAL, nm + ": q, the weights, the pool and the output must be 16-byte, the workspace 128-byte aligned");
    if (!aligned(table, 4) || !aligned(lens, 4)) return set_error(QL_EINVAL, nm + ": the table and the lengths must be 4-byte aligned");
    if (ws_bytes < need) return set_error(QL_EINVAL, nm + ": the workspace is too small");
    return QL_OK;
}

}  // namespace ql

extern "C" int ql_mla_append(const void* d_q, const void* d_kv, int dtype, int64_t q_stride, int64_t kv_stride, const float* d_norm_w,
                             const float* d_cos, const float* d_sin, const int32_t* d_positions, const int64_t* d_slots, float eps,
                             int64_t n, int n_heads, int head_dim, int rank, int rope_dim, void* d_q_out, void* d_pool,
                             int64_t num_blocks, int64_t max_position, void* stream) {
    using namespace ql;
    QL_REQUIRE(dtype == QL_DTYPE_F32 || dtype == QL_DTYPE_F16, "ql_mla_append: dtype must be f32 or f16");
    QL_REQUIRE(mla::shape_ok(head_dim, rank) && rope_dim == kRope,
               "ql_mla_append: head_dim must be 64 or 128, rank 256 or 512, rope_dim 64");
    QL_REQUIRE(n >= 0 && n < (1ll << 31) && n_heads >= 1 && n_heads <= 1024 && num_blocks >= 1 && num_blocks < (1ll << 27) &&
                   max_position >= 1,
               "ql_mla_append: need 0 <= n < 2^31, 1 <= n_heads <= 1024, 1 <= num_blocks < 2^27, max_position >= 1");
    if (n == 0) return QL_OK;
    QL_REQUIRE(d_kv && d_norm_w && d_cos && d_sin && d_positions && d_slots && d_pool && (d_q == nullptr) == (d_q_out == nullptr),
               "ql_mla_append: null pointer");
    auto aligned = [](const void* p, int k) { return (reinterpret_cast<uintptr_t>(p) & (k - 1)) == 0; };
    QL_REQUIRE(aligned(d_q, 16) && aligned(d_kv, 16) && aligned(d_norm_w, 16) && aligned(d_q_out, 16) && aligned(d_pool, 16),
               "ql_mla_append: rows, norm weights, the queries' output and the pool must be 16-byte aligned");
    QL_REQUIRE(aligned(d_cos, 4) && aligned(d_sin, 4) && aligned(d_positions, 4) && aligned(d_slots, 8),
               "ql_mla_append: tables and positions must be 4-byte, slots 8-byte aligned");
    const int64_t per = dtype == QL_DTYPE_F32 ? 4 : 8, q_row = (int64_t)n_heads * (head_dim + kRope);
    QL_REQUIRE(n == 1 || (kv_stride >= rank + kRope && kv_stride % per == 0 && kv_stride < (1ll << 31) &&
                          (!d_q || (q_stride >= q_row && q_stride % per == 0 && q_stride < (1ll << 31)))),
               "ql_mla_append: row strides must be multiples of 16 bytes, at least a row and below 2^31");
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "ql_mla_append: no device error record");
    AppendParams p = {d_q, d_kv, q_stride, kv_stride, d_norm_w, d_cos, d_sin, d_positions,
                      reinterpret_cast<const long long*>(d_slots), eps, n_heads, static_cast<__half*>(d_q_out),
                      static_cast<__half*>(d_pool), (long long)num_blocks, (long long)max_position};
    const int items = d_q ? n_heads + 1 : 1, gy = (items + 7) / 8, warps = (items + gy - 1) / gy;
    const dim3 grid((unsigned)n, (unsigned)gy), block((unsigned)(32 * warps));
    auto go = [&](auto kernel) { return launch(kernel, grid, block, 0, static_cast<cudaStream_t>(stream), true, p, err); };
    const bool f32 = dtype == QL_DTYPE_F32;
    cudaError_t e;
    if (head_dim == 128)
        e = rank == 512 ? (f32 ? go(mla_append_kernel<128, 512, float>) : go(mla_append_kernel<128, 512, __half>))
                        : (f32 ? go(mla_append_kernel<128, 256, float>) : go(mla_append_kernel<128, 256, __half>));
    else
        e = rank == 512 ? (f32 ? go(mla_append_kernel<64, 512, float>) : go(mla_append_kernel<64, 512, __half>))
                        : (f32 ? go(mla_append_kernel<64, 256, float>) : go(mla_append_kernel<64, 256, __half>));
    return e == cudaSuccess ? QL_OK : cuda_error(e, "ql_mla_append");
}

extern "C" size_t ql_mla_chunk_workspace_bytes(int64_t n_tokens, int n_heads, int head_dim, int rank, int64_t max_blocks_per_seq) {
    if (!ql::mla::shape_ok(head_dim, rank) || n_tokens < 1 || n_tokens > 65535 || n_heads < 1 || n_heads > 1024 || max_blocks_per_seq < 1 ||
        max_blocks_per_seq > (1 << 16))
        return 0;
    return (size_t)n_tokens * n_heads * (2 * rank + ql::mla::kRope) * 4;
}

namespace ql {
namespace {
template <typename... A>
int simple_of(int D, int R, A... a) {
    return D == 128 ? (R == 512 ? simple<128, 512>(a...) : simple<128, 256>(a...))
                    : (R == 512 ? simple<64, 512>(a...) : simple<64, 256>(a...));
}
}  // namespace
}  // namespace ql

extern "C" int ql_mla_attn_chunk(const void* d_q, const void* d_w_kv, const void* d_pool, const int32_t* d_block_table,
                                 const int32_t* d_position, int64_t n_tokens, int n_heads, int head_dim, int rank, int rope_dim,
                                 int block_size, int64_t max_blocks_per_seq, int64_t num_blocks, float scale, void* d_out,
                                 void* d_workspace, size_t workspace_bytes, void* stream) {
    using namespace ql;
    if (int rc = mla::attn_check("ql_mla_attn_chunk", d_q, d_w_kv, d_pool, d_block_table, d_position, head_dim, rank, rope_dim, block_size, num_blocks, d_out, d_workspace, workspace_bytes,
                            ql_mla_chunk_workspace_bytes(n_tokens, n_heads, head_dim, rank, max_blocks_per_seq)))
        return rc;
    return simple_of(head_dim, rank, static_cast<const __half*>(d_q), static_cast<const __half*>(d_w_kv),
                     static_cast<const __half*>(d_pool), d_block_table, (const int32_t*)nullptr, d_position, (long long)n_tokens, n_heads,
                     (long long)max_blocks_per_seq, (long long)num_blocks, scale, static_cast<__half*>(d_out), d_workspace,
                     static_cast<cudaStream_t>(stream));
}
