// Paged decode attention over the 4-bit pool: out = softmax(q . K scale) V for one query token per
// sequence, each kv head shared by a group of query heads.
//
// One CTA of 4 warps per (sequence, kv head, up to 8 query heads of its group); a warp takes every
// fourth key, a lane element 32 b + lane of each block b of a row, with a running maximum and sum
// per head in f32; the warps' sums are joined in shared memory.
#include <cuda_fp16.h>
#include <math.h>

#include "ql_internal.h"
#include "ql_kv4_attn.h"
#include "ql_kv4_rec.cuh"

namespace ql {
namespace {

constexpr int kHeads = 8;    // query heads per CTA
constexpr int kWarps = 4;

struct Params {
    const __half* q;
    const uint8_t* pool;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* positions;
    const int32_t* active;
    int n_heads, n_kv, group, chunks;
    long long maxb, num_blocks;
    float scale_log2;
    __half* out;
};

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) kv4_attn_kernel(Params p, DevError* err) {
    using R = Kv4<HD>;
    constexpr int NB = R::NB;
    __shared__ float sm[kWarps][kHeads], sl[kWarps][kHeads], so[kWarps][kHeads][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.x / p.chunks, c = blockIdx.x % p.chunks, b = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    if (p.active && p.active[b] == 0) return;
    const long long len = p.context_lens ? (long long)p.context_lens[b] : (long long)p.positions[b] + 1;
    if (len < 0 || len > p.maxb * 16) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_device_error(err, kErrAttnLength, b, len);
        return;
    }
    if (len == 0) return;
    const int h0 = g * p.group + c * kHeads;
    const int nh = min(kHeads, p.group - c * kHeads);
    float q[kHeads][NB], o[kHeads][NB], m[kHeads], l[kHeads];
    for (int h = 0; h < kHeads; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        for (int k = 0; k < NB; ++k) {
            q[h][k] = h < nh ? __half2float(p.q[((size_t)b * p.n_heads + h0 + h) * HD + 32 * k + lane]) : 0.f;
            o[h][k] = 0.f;
        }
    }
    for (long long t = warp; t < len; t += kWarps) {
        const long long blk = p.block_tables[(size_t)b * p.maxb + (t >> 4)];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) record_device_error(err, kErrAttnBlock, (long long)b * p.maxb + (t >> 4), blk);
            continue;
        }
        const int s = (int)(t & 15);
        const uint8_t* rec = p.pool + ((size_t)blk * p.n_kv + g) * R::BYTES;
        float kx[NB], vx[NB];
        for (int k = 0; k < NB; ++k) {
            const int j = (lane & 15) >> 2, i = lane & 3;
            const int kc = rec[R::KC + s * (HD / 2) + 4 * (NB * j + k) + i] >> (4 * (lane >> 4)) & 15;
            const int vc = rec[R::VC + s * (HD / 2) + R::vunit(s, lane & 7) + 2 * k + (lane >> 4)] >> (4 * ((lane >> 3) & 1)) & 15;
            kx[k] = fmaf(__half2float(reinterpret_cast<const __half*>(rec + R::KD)[s * NB + k]), (float)kc,
                         __half2float(reinterpret_cast<const __half*>(rec + R::KM)[s * NB + k]));
            vx[k] = fmaf(__half2float(reinterpret_cast<const __half*>(rec + R::VD)[R::vscale(s, k)]), (float)vc,
                         __half2float(reinterpret_cast<const __half*>(rec + R::VM)[R::vscale(s, k)]));
        }
        for (int h = 0; h < kHeads; ++h) {
            float x = 0.f;
            for (int k = 0; k < NB; ++k) x = fmaf(q[h][k], kx[k], x);
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            x *= p.scale_log2;
            const float mn = fmaxf(m[h], x), a = exp2f(m[h] - mn), w = exp2f(x - mn);
            m[h] = mn;
            l[h] = l[h] * a + w;
            for (int k = 0; k < NB; ++k) o[h][k] = fmaf(w, vx[k], o[h][k] * a);
        }
    }
    for (int h = 0; h < kHeads; ++h) {
        if (lane == 0) {
            sm[warp][h] = m[h];
            sl[warp][h] = l[h];
        }
        for (int k = 0; k < NB; ++k) so[warp][h][32 * k + lane] = o[h][k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * HD; i += kWarps * 32) {
        const int h = i / HD, e = i % HD;
        float mx = -INFINITY, ls = 0.f, os = 0.f;
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm[w][h] == -INFINITY ? 0.f : exp2f(sm[w][h] - mx);
            ls += sl[w][h] * f;
            os += so[w][h][e] * f;
        }
        p.out[((size_t)b * p.n_heads + h0 + h) * HD + e] = __float2half_rn(ls > 0.f ? os / ls : 0.f);
    }
}

}  // namespace

size_t kv4_attn_workspace_bytes(int64_t batch, int n_heads, int n_kv, int head_dim, int64_t maxb) {
    (void)batch, (void)n_heads, (void)n_kv, (void)head_dim, (void)maxb;
    return 16;
}

int kv4_attn_launch(const Kv4AttnArgs& a, cudaStream_t s, bool pdl) {
    DevError* err = device_error_record();
    if (!err) return set_error(QL_ECUDA, "4-bit attention: no device error record");
    Params p = {};
    p.q = a.q;
    p.pool = a.pool;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.positions = a.positions;
    p.active = a.active;
    p.n_heads = a.n_heads;
    p.n_kv = a.n_kv_heads;
    p.group = a.n_heads / a.n_kv_heads;
    p.chunks = (p.group + kHeads - 1) / kHeads;
    p.maxb = a.max_blocks_per_seq;
    p.num_blocks = a.num_blocks;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.out = a.out;
    const dim3 grid((unsigned)(a.n_kv_heads * p.chunks), (unsigned)a.batch);
    const cudaError_t e = a.head_dim == 128 ? launch(kv4_attn_kernel<128>, grid, dim3(kWarps * 32), 0, s, pdl, p, err)
                                            : launch(kv4_attn_kernel<64>, grid, dim3(kWarps * 32), 0, s, pdl, p, err);
    return e == cudaSuccess ? QL_OK : cuda_error(e, "4-bit attention launch");
}

}  // namespace ql

extern "C" size_t ql_paged_attn_kv4_workspace_bytes(int64_t batch, int n_heads, int n_kv_heads, int head_dim,
                                                    int64_t max_blocks_per_seq) {
    if (batch < 1 || n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || (head_dim != 64 && head_dim != 128) ||
        max_blocks_per_seq < 1)
        return 0;
    return ql::kv4_attn_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq);
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
    QL_REQUIRE(n_heads > 0 && n_kv_heads > 0 && n_heads % n_kv_heads == 0,
               std::string(nm) + ": n_heads must be a multiple of n_kv_heads");
    QL_REQUIRE(batch >= 1 && batch <= 65535 && batch * n_heads < (1ll << 31) / 128, std::string(nm) + ": batch out of range");
    QL_REQUIRE(max_blocks_per_seq >= 1 && max_blocks_per_seq < (1ll << 27) && num_blocks >= 1 && num_blocks < (1ll << 31),
               std::string(nm) + ": bad table or pool size");
    QL_REQUIRE((reinterpret_cast<uintptr_t>(d_pool) & 15) == 0 && (reinterpret_cast<uintptr_t>(d_workspace) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(d_q) & 3) == 0 && (reinterpret_cast<uintptr_t>(d_out) & 3) == 0,
               std::string(nm) + ": the pool and the workspace must be 16-byte aligned, q and the output 4-byte aligned");
    QL_REQUIRE(workspace_bytes >= kv4_attn_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq),
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
    return kv4_attn_launch(a, static_cast<cudaStream_t>(stream), false);
}
