// Building blocks of the latent attention's tensor-core kernels: bounded barrier waits, bulk tensor copies, tcgen05
// products, tensor memory loads and stores.
#pragma once

#include <cuda.h>

#include "ql_mla.h"
#include "ql_persist.cuh"

namespace ql {
namespace mla {

__device__ __forceinline__ uint32_t su32(const void* q) { return static_cast<uint32_t>(__cvta_generic_to_shared(q)); }

__device__ __forceinline__ void bar_init(uint32_t mb, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mb), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t mb) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mb) : "memory"); }
__device__ __forceinline__ void bar_expect(uint32_t mb, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
}
// expected bytes whose copy is not going to be issued
__device__ __forceinline__ void bar_forgo(uint32_t mb, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
}
// What a bounded wait needs: an expiry records an error (index = CTA, value = where), raises the CTA's abort flag, which ends the
// other roles' waits, and returns false.
struct Waits {
    DevError* err;
    int* abort_flag;
    unsigned long long ns;
};
// In a pair of CTAs it raises the other's flag, too, so that both know once they have met.
struct PairWaits : Waits {};
template <bool PAIR>
static __device__ __noinline__ bool wait_slow(uint32_t mb, uint32_t parity, Waits w, int where) {
    const unsigned long long t0 = persist::global_ns();
    for (unsigned int spin = 1;; ++spin) {
        if (persist::mbar_test(mb, parity)) return true;
        if ((spin & 63u) == 0) {
            if (w.abort_flag != nullptr && *reinterpret_cast<volatile int*>(w.abort_flag)) return false;
            if (persist::global_ns() - t0 > w.ns) break;
        }
    }
    if constexpr (PAIR) {
        uint32_t other;
        asm volatile("{\n .reg .u32 r;\n mov.u32 r, %%cluster_ctarank;\n xor.b32 r, r, 1;\n mapa.shared::cluster.u32 %0, %1, r;\n"
                     " st.shared::cluster.u32 [%0], %2;\n}" : "=&r"(other) : "r"(su32(w.abort_flag)), "r"(1) : "memory");
    }
    if (w.abort_flag == nullptr || atomicExch(w.abort_flag, 1) == 0) record_device_error(w.err, kErrLatentStage, blockIdx.x, where);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t mb, uint32_t parity, const Waits& w, int where) {
    if (persist::mbar_test(mb, parity) || persist::mbar_test(mb, parity)) return true;
    return wait_slow<false>(mb, parity, w, where);
}
__device__ __forceinline__ bool bar_wait(uint32_t mb, uint32_t parity, const PairWaits& w, int where) {
    if (persist::mbar_test(mb, parity) || persist::mbar_test(mb, parity)) return true;
    return wait_slow<true>(mb, parity, w, where);
}
// by every lane, one answer for the warp
template <typename W>
__device__ __forceinline__ bool warp_wait(uint32_t mb, uint32_t parity, const W& w, int where) {
    return __all_sync(0xffffffffu, bar_wait(mb, parity, w, where));
}

__device__ __forceinline__ void copy_box4(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int u, uint32_t mb) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(mb) : "memory");
}
// from shared memory; the issuing thread's copies so far have been read, or have arrived
__device__ __forceinline__ void store_box2(const CUtensorMap* m, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(x),
                 "r"(y), "r"(src) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void copy_box5(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int u, int v, uint32_t mb) {
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(mb) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Shared-memory operand descriptor: start address, leading and stride byte offsets, swizzle (2: 128 bytes, 4: 64 bytes).
// K-major: stride = bytes between groups of 8 rows (leading unused). MN-major: leading = bytes between swizzle-wide runs of the
// rows' dimension, stride = bytes between groups of 8 along K.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading, uint32_t stride, uint32_t swizzle) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) |
           ((uint64_t)swizzle << 61);
}
// Instruction descriptor: D f32, A and B f16; MN-major operands by their flags.
__host__ __device__ constexpr uint32_t instr(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Products and commits are issued by a whole warp that runs converged, `one` true in its elected lane: descriptors that the
// compiler knows to be the same in all lanes cost an addition each (computed in a branch of one lane, 65 cycles a product).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(one));
    return one;
}
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n .reg .pred pa, pe;\n setp.ne.u32 pa, %4, 0;\n setp.ne.u32 pe, %5, 0;\n"
                 " @pe tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pa;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one) : "memory");
}
// The MMAs issued so far arrive on the barrier as they complete.
__device__ __forceinline__ void mma_commit(uint32_t one, uint32_t mb) {
    asm volatile("{\n .reg .pred pe;\n setp.ne.u32 pe, %1, 0;\n"
                 " @pe tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(mb), "r"(one) : "memory");
}
// ---- pairs of CTAs (clusters of two): one product of 256 rows, 128 of them in each CTA, as is each half of B's rows and of the result
template <uint32_t COLS>
__device__ __forceinline__ void tmem_alloc2(uint32_t* at) {   // by one whole warp of both CTAs
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(at)), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_free2(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(COLS) : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n .reg .pred pa, pe;\n setp.ne.u32 pa, %4, 0;\n setp.ne.u32 pe, %5, 0;\n"
                 " @pe tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, pa;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one) : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {   // A in tensor memory
    asm volatile("{\n .reg .pred pa, pe;\n setp.ne.u32 pa, %4, 0;\n setp.ne.u32 pe, %5, 0;\n"
                 " @pe tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, pa;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one) : "memory");
}
// arrives on the barrier of this address in both CTAs
__device__ __forceinline__ void mma2_commit(uint32_t one, uint32_t mb) {
    asm volatile("{\n .reg .pred pe;\n .reg .b16 m;\n setp.ne.u32 pe, %1, 0;\n mov.b16 m, 3;\n"
                 " @pe tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(mb), "r"(one) : "memory");
}
// a copy into this CTA that reports to a barrier of the pair
__device__ __forceinline__ void copy2_box2(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t mb) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(mb) : "memory");
}
__device__ __forceinline__ void copy2_box3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t mb) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(mb) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// mb: an address in the cluster. What the arrival reports lies in tensor memory, ordered by the tcgen05 fences around it: a release
// of the whole cluster's memory is not needed (and takes 1500 cycles).
__device__ __forceinline__ void bar_arrive_cluster(uint32_t mb) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mb) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int load_cluster(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// After an abort, by one thread of rank 0, behind a barrier of the pair: no copy is issued any more. Every copy into a ring of n stages, of
// which each CTA brings `bytes`, reports to rank 0's barriers at mb, and each CTA has noted at `issued` how many it has asked for (rank 0 has
// armed the barrier for its own). Each waited for its stage first, so that they are a ring apart at most and the phase before is complete.
// What only one of them has asked for is armed, or given up, for the other, and the copies in flight are waited for.
__device__ __forceinline__ void settle_ring(uint32_t mb, int n, uint32_t issued, uint32_t bytes, const Waits& alone, int where) {
    const int mine = load_cluster(in_cta(issued, 0)), other = load_cluster(in_cta(issued, 1)), all = max(mine, other);
    for (int i = min(mine, other); i < all; ++i) {
        if (i >= mine) bar_expect(mb + i % n * 8, bytes);
        else bar_forgo(mb + i % n * 8, bytes);
    }
    for (int i = max(0, all - n); i < all; ++i) bar_wait(mb + i % n * 8, (uint32_t)(i / n) & 1u, alone, where);
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// generic-proxy writes to shared memory made visible to copies and MMAs
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 (16) consecutive columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t a, float* f) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
                 "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]), "=f"(f[9]),
                   "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15]), "=f"(f[16]), "=f"(f[17]), "=f"(f[18]),
                   "=f"(f[19]), "=f"(f[20]), "=f"(f[21]), "=f"(f[22]), "=f"(f[23]), "=f"(f[24]), "=f"(f[25]), "=f"(f[26]), "=f"(f[27]),
                   "=f"(f[28]), "=f"(f[29]), "=f"(f[30]), "=f"(f[31])
                 : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, float* f) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]), "=f"(f[9]),
                   "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15])
                 : "r"(a) : "memory");
}
// Between the wait for a load and the first use of what it brought: the uses stay behind the wait.
__device__ __forceinline__ void tie16(float* f) {
    asm volatile("" : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]), "+f"(f[8]), "+f"(f[9]),
                 "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15]));
}
__device__ __forceinline__ void tie32(float* f) {
    tie16(f);
    tie16(f + 16);
}
template <int N>
__device__ __forceinline__ void tmem_raw(uint32_t a, float* f) {
    static_assert(N == 16 || N == 32, "");
    if constexpr (N == 32) tmem_ld32(a, f);
    else tmem_ld16(a, f);
}
template <int N>
__device__ __forceinline__ void tie(float* f) {
#pragma unroll
    for (int i = 0; i < N; i += 16) tie16(f + i);
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t a, float* f) {   // and wait
    tmem_raw<N>(a, f);
    wait_ld();
    tie<N>(f);
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
                 "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
                 "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
                 "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
                 "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t* at) {   // by one whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(at)), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_free(uint32_t base) {   // by the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(COLS) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two f32 at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n"
        " mov.b64 {%0, %1}, d;\n}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace mla
}  // namespace ql
