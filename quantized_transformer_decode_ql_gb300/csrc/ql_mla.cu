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

}  // namespace

int mla::attn_check(const char* name, const void* q, const void* w, const void* pool, const void* table, const void* lens, int head_dim,
                    int rank, int rope_dim, int block_size, int64_t num_blocks, float scale, const void* out, const void* ws, size_t ws_bytes, size_t need) {
    const std::string nm(name);
    if (!q || !w || !pool || !table || !lens || !out || !ws) return set_error(QL_EINVAL, nm + ": null pointer");
    if (!mla::shape_ok(head_dim, rank) || rope_dim != kRope || block_size != mla::kBlock)
        return set_error(QL_EINVAL, nm + ": head_dim must be 64 or 128, rank 256 or 512, rope_dim 64, block_size 16");
    if (need == 0 || num_blocks < 1 || num_blocks >= (1ll << 27))
        return set_error(QL_EINVAL, nm + ": sizes out of range");
    if (!(scale > 0.f && scale < INFINITY)) return set_error(QL_EINVAL, nm + ": the scale must be positive and finite");
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
