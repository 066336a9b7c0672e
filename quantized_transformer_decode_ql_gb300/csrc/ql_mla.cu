// Latent attention, the rows: a token's latent vector normalised and its key part rotated into the paged cache, its query
// heads' last 64 values rotated.
//
//   row of the cache = f16( x[0:R] / sqrt(mean x[0:R]^2 + eps) * w | rot(x[R:R+64], p) )
//   query head       = f16( q[0:D] | rot(q[D:D+64], p) )
//
// rot turns the pairs (i, i + 32) by the tables' angle of position p. A warp takes four heads of a row, all of their
// loads in flight together (16 bytes a lane and more), or the row's latent vector. Means and products are f32, the stored
// values f16, as the cache and the attention's operands are. Bound by HBM for a prompt: 8000 f32 rows of 32 heads of 128 and rank 512 take
// 48 us, 6.7 TB/s of what is read and written (a head a warp, narrower loads: 97 us); a step's rows take 1.6 us.
#include "ql_mla.h"

#include <algorithm>

namespace ql {
namespace {

using mla::kRope;

// N consecutive values in f32, the address a multiple of N * sizeof(T) up to 16 bytes
template <int N>
__device__ __forceinline__ void load_row(const float* p, float* x) {
    if constexpr (N == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p));
        x[0] = v.x;
        x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
            x[i] = v.x;
            x[i + 1] = v.y;
            x[i + 2] = v.z;
            x[i + 3] = v.w;
        }
    }
}
template <int N>
__device__ __forceinline__ void load_row(const __half* p, float* x) {
    uint32_t u[N / 2];
    if constexpr (N == 2) u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    else if constexpr (N == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        u[0] = v.x;
        u[1] = v.y;
    } else {
        static_assert(N == 8, "");
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        u[0] = v.x;
        u[1] = v.y;
        u[2] = v.z;
        u[3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i / 2]));
        x[i] = f.x;
        x[i + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t two(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The larger magnitude of each half, NaN where there is one; whether both are numbers.
__device__ __forceinline__ __half2 larger(__half2 a, uint32_t b) { return __hmax2_nan(a, __habs2(*reinterpret_cast<const __half2*>(&b))); }
__device__ __forceinline__ bool held(__half2 a) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&a);
    return (u & 0x7c00u) != 0x7c00u && (u & 0x7c000000u) != 0x7c000000u;
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

constexpr int kHeads = 4;   // of a warp

template <int D, int R, typename T>
__global__ void __launch_bounds__(512) mla_append_kernel(AppendParams p, DevError* err) {
    const long long i = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);   // 0: the latent vector, 1 + k: heads 4 k ..
    const int heads = p.q != nullptr ? p.n_heads : 0, h0 = (item - 1) * kHeads;
    pdl_wait();
    pdl_trigger();
    if (item > 0 && h0 >= heads) return;
    const long long slot = __ldg(p.slots + i);
    const int pos = __ldg(p.positions + i);
    if (slot < 0 || slot >= 16 * p.num_blocks || pos < 0 || pos >= p.max_position) {
        if (item == 0 && lane == 0 && slot != -1) {
            const bool bad_slot = slot < 0 || slot >= 16 * p.num_blocks;
            record_device_error(err, bad_slot ? kErrKvSlot : kErrRopePosition, i, bad_slot ? slot : pos);
        }
        return;
    }
    // lanes 0-15 and 16-31 turn the pairs j, j + 1 of two heads
    const int j = 2 * (lane & 15), sub = lane >> 4;
    const float2 c = __ldg(reinterpret_cast<const float2*>(p.cos_t + (long long)pos * (kRope / 2) + j));
    const float2 s = __ldg(reinterpret_cast<const float2*>(p.sin_t + (long long)pos * (kRope / 2) + j));
    if (item > 0) {
        constexpr int LANES = D / 8, AT = 32 / LANES;   // lanes of a head's first D values, heads of the warp at a time
        const T* q = static_cast<const T*>(p.q) + i * p.q_stride + (long long)h0 * (D + kRope);
        __half* o = p.q_out + (i * p.n_heads + h0) * (D + kRope);
        float x[kHeads / AT][8], a[kHeads / 2][2], b[kHeads / 2][2];
#pragma unroll
        for (int k = 0; k < kHeads / AT; ++k) {
            const int h = k * AT + lane / LANES;
            if (h0 + h < heads) load_row<8>(q + h * (D + kRope) + lane % LANES * 8, x[k]);
        }
#pragma unroll
        for (int k = 0; k < kHeads / 2; ++k) {
            const int h = 2 * k + sub;
            if (h0 + h < heads) {
                load_row<2>(q + h * (D + kRope) + D + j, a[k]);
                load_row<2>(q + h * (D + kRope) + D + kRope / 2 + j, b[k]);
            }
        }
        __half2 most = __floats2half2_rn(0.f, 0.f);   // the lane's largest magnitudes, NaN where there is one
#pragma unroll
        for (int k = 0; k < kHeads / AT; ++k) {
            const int h = k * AT + lane / LANES;
            if (h0 + h < heads) {
                const uint4 u = make_uint4(two(x[k][0], x[k][1]), two(x[k][2], x[k][3]), two(x[k][4], x[k][5]), two(x[k][6], x[k][7]));
                *reinterpret_cast<uint4*>(o + h * (D + kRope) + lane % LANES * 8) = u;
                most = larger(larger(larger(larger(most, u.x), u.y), u.z), u.w);
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads / 2; ++k) {
            const int h = 2 * k + sub;
            if (h0 + h < heads) {
                uint32_t* t = reinterpret_cast<uint32_t*>(o + h * (D + kRope) + D + j);
                t[0] = two(a[k][0] * c.x - b[k][0] * s.x, a[k][1] * c.y - b[k][1] * s.y);
                t[kRope / 4] = two(b[k][0] * c.x + a[k][0] * s.x, b[k][1] * c.y + a[k][1] * s.y);
                most = larger(larger(most, t[0]), t[kRope / 4]);
            }
        }
        if (!held(most)) {   // (rare) whose it is: the lane's values read back
            for (int h = 0; h < kHeads && h0 + h < heads; ++h) {
                const uint32_t* r = reinterpret_cast<const uint32_t*>(o + h * (D + kRope));
                __half2 m = __floats2half2_rn(0.f, 0.f);
                if (h % AT == lane / LANES)
                    for (int e = 0; e < 4; ++e) m = larger(m, r[lane % LANES * 4 + e]);
                if (h % 2 == sub) m = larger(larger(m, r[(D + j) / 2]), r[(D + j) / 2 + kRope / 4]);
                if (!held(m)) record_device_error(err, kErrLatentValue, i, 1 + h0 + h);
            }
        }
        return;
    }
    constexpr int V = R / 32;
    const T* src = static_cast<const T*>(p.kv) + i * p.kv_stride;
    float x[V], w[V], a[2], b[2], ss = 0.f;
#pragma unroll
    for (int k = 0; k < V; k += 4) load_row<4>(src + 32 * k + 4 * lane, x + k);
    load_row<2>(src + R + j, a);
    load_row<2>(src + R + kRope / 2 + j, b);
#pragma unroll
    for (int k = 0; k < V; k += 4) load_row<4>(p.norm + 32 * k + 4 * lane, w + k);
#pragma unroll
    for (int k = 0; k < V; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, 1.0f / (float)R, p.eps));
    __half* o = p.pool + slot * (R + kRope);
    const float t[4] = {a[0] * c.x - b[0] * s.x, a[1] * c.y - b[1] * s.y, b[0] * c.x + a[0] * s.x, b[1] * c.y + a[1] * s.y};
    bool whole = ss < INFINITY;   // by f16, and the squares' sum by f32
#pragma unroll
    for (int k = 0; k < 4; ++k) whole &= fabsf(t[k]) < 65520.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        x[k] *= r * w[k];
        whole &= fabsf(x[k]) < 65520.f;
    }
#pragma unroll
    for (int k = 0; k < V; k += 4) *reinterpret_cast<uint2*>(o + 32 * k + 4 * lane) = make_uint2(two(x[k], x[k + 1]), two(x[k + 2], x[k + 3]));
    if (sub == 0) {
        uint32_t* u = reinterpret_cast<uint32_t*>(o + R + j);
        u[0] = two(t[0], t[1]);
        u[kRope / 4] = two(t[2], t[3]);
    }
    if (!whole) record_device_error(err, kErrLatentValue, i, 0);
}

}  // namespace

// Whether [a, a + an) and [b, b + bn) share a byte.
static bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an && bn && x < y + bn && y < x + an;
}
static bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int mla::attn_check(const char* name, const AttnIn& a, size_t need) {
    const std::string nm(name);
    if (!a.q || !a.w || !a.pool || !a.table || !a.lens || !a.out || !a.ws) return set_error(QL_EINVAL, nm + ": null pointer");
    if (!shape_ok(a.D, a.R) || a.rope != kRope || a.block != kBlock)
        return set_error(QL_EINVAL, nm + ": head_dim must be 64 or 128, rank 256 or 512, rope_dim 64, block_size 16");
    if (need == 0 || a.num_blocks < 1 || a.num_blocks >= (1ll << 27)) return set_error(QL_EINVAL, nm + ": sizes out of range");
    if (!(a.scale > 0.f && a.scale < INFINITY)) return set_error(QL_EINVAL, nm + ": the scale must be positive and finite");
    if (!aligned(a.q, 16) || !aligned(a.w, 16) || !aligned(a.pool, 16) || !aligned(a.out, 16) || !aligned(a.ws, 128))
        return set_error(QL_EINVAL, nm + ": q, the weights, the pool and the output must be 16-byte, the workspace 128-byte aligned");
    if (!aligned(a.table, 4) || !aligned(a.lens, 4)) return set_error(QL_EINVAL, nm + ": misaligned table or lengths");
    if (a.ws_bytes < need) return set_error(QL_EINVAL, nm + ": the workspace is too small");
    const size_t row = (size_t)a.rows * a.H;
    const struct {
        const void* p;
        size_t n;
    } in[] = {{a.q, row * (a.D + kRope) * 2}, {a.w, (size_t)a.H * 2 * a.D * a.R * 2}, {a.pool, (size_t)a.num_blocks * kBlock * (a.R + kRope) * 2},
              {a.table, (size_t)a.tables * a.maxb * 4}, {a.lens, (size_t)a.tables * 4}};
    for (const auto& i : in)
        if (overlap(a.out, row * a.D * 2, i.p, i.n) || overlap(a.ws, need, i.p, i.n))
            return set_error(QL_EINVAL, nm + ": the output or the workspace overlaps an input");
    if (overlap(a.out, row * a.D * 2, a.ws, need)) return set_error(QL_EINVAL, nm + ": the output overlaps the workspace");
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
    QL_REQUIRE(aligned(d_q, 16) && aligned(d_kv, 16) && aligned(d_norm_w, 16) && aligned(d_q_out, 16) && aligned(d_pool, 16),
               "ql_mla_append: rows, norm weights, the queries' output and the pool must be 16-byte aligned");
    QL_REQUIRE(aligned(d_cos, 8) && aligned(d_sin, 8) && aligned(d_positions, 4) && aligned(d_slots, 8),
               "ql_mla_append: the tables and the slots must be 8-byte, positions 4-byte aligned");
    const int64_t per = dtype == QL_DTYPE_F32 ? 4 : 8, q_row = (int64_t)n_heads * (head_dim + kRope);
    QL_REQUIRE(n == 1 || (kv_stride >= rank + kRope && kv_stride % per == 0 && kv_stride < (1ll << 31) &&
                          (!d_q || (q_stride >= q_row && q_stride % per == 0 && q_stride < (1ll << 31)))),
               "ql_mla_append: row strides must be multiples of 16 bytes, at least a row and below 2^31");
    const size_t size = dtype == QL_DTYPE_F32 ? 4 : 2, q_bytes = d_q ? ((n - 1) * (n > 1 ? q_stride : 0) + q_row) * size : 0;
    const size_t kv_bytes = ((n - 1) * (n > 1 ? kv_stride : 0) + rank + kRope) * size, out_bytes = d_q ? (size_t)n * q_row * 2 : 0;
    const size_t pool_bytes = (size_t)num_blocks * mla::kBlock * (rank + kRope) * 2;
    // (rows of the tables that an int32 position reaches)
    const size_t turns = (size_t)std::min<int64_t>(max_position, 1ll << 31) * (kRope / 2) * 4;
    const struct {
        const void* p;
        size_t n;
    } in[] = {{d_q, q_bytes}, {d_kv, kv_bytes}, {d_norm_w, (size_t)rank * 4}, {d_cos, turns}, {d_sin, turns}, {d_positions, (size_t)n * 4}, {d_slots, (size_t)n * 8}};
    bool apart = !overlap(d_q_out, out_bytes, d_pool, pool_bytes);
    for (const auto& i : in) apart = apart && !overlap(d_q_out, out_bytes, i.p, i.n) && !overlap(d_pool, pool_bytes, i.p, i.n);
    QL_REQUIRE(apart, "ql_mla_append: the queries' output and the pool overlap each other or an input");
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "ql_mla_append: no device error record");
    AppendParams p = {d_q, d_kv, q_stride, kv_stride, d_norm_w, d_cos, d_sin, d_positions,
                      reinterpret_cast<const long long*>(d_slots), eps, n_heads, static_cast<__half*>(d_q_out),
                      static_cast<__half*>(d_pool), (long long)num_blocks, (long long)max_position};
    const int items = d_q ? (n_heads + kHeads - 1) / kHeads + 1 : 1, gy = (items + 15) / 16, warps = (items + gy - 1) / gy;
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
