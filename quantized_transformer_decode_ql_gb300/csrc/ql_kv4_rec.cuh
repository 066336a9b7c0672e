// The 4-bit KV pool: where a record keeps its fields, and the row quantiser.
//
// A row of HD values is cut into 32-element blocks with m = f16(min x), d = f16((max x - min x) / 15)
// and codes c = clamp(rint((x - m) / d), 0, 15); its values are d c + m. One record per (physical
// block of 16 tokens, kv head), 20 HD bytes (160 B per token at HD 128, against 512 for f16), every
// field 16-byte aligned, in the order in which the attention's matrix instructions take them:
//   KC  u8  [16][HD / 2]  key codes: a lane of the score product reads its 8 elements of every
//                         block as one word each, the words of one lane in a row
//   VC  u8  [16][HD / 2]  value codes: 16-bit words of 4 elements 8 apart, the blocks' words of one
//                         lane of the value product in a row; at HD 128 the lanes' units of two of
//                         every four slots are swapped in halves, which keeps the shared-memory
//                         reads of the four slots of a lane group on different banks
//   KD, KM  f16 [16][HD / 32]             key scales and minima
//   VD, VM  f16 [4][2][HD / 32][2]        value scales and minima of slot q + 4 e + 8 h at
//                                         [q][h][block][e]: the pairs that a lane multiplies
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ql_internal.h"

namespace ql {

template <int HD>
struct Kv4 {
    static constexpr int NB = HD / 32;   // 32-element blocks per row
    static constexpr int KC = 0, VC = 8 * HD, KD = 16 * HD, KM = 17 * HD, VD = 18 * HD, VM = 19 * HD;
    static constexpr int BYTES = 20 * HD;
    static constexpr int LANES = 4 * NB;   // lanes per row of the writer and the reader
    // byte of a row's value unit w (the 4 NB-bit words of elements w, w + 8, w + 16, w + 24 of every block)
    __host__ __device__ static constexpr int vunit(int slot, int w) {
        return 2 * NB * (HD == 128 ? (w ^ (((slot >> 1) & 1) << 2)) : w);
    }
    // f16 index of (slot, block) in VD and VM
    __host__ __device__ static constexpr int vscale(int slot, int b) {
        return 4 * NB * (slot & 3) + 2 * NB * (slot >> 3) + 2 * b + ((slot >> 2) & 1);
    }
};

#ifdef __CUDACC__
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest and the smallest of a block of 32 elements, 8 in each of 4 neighbouring lanes.
__device__ __forceinline__ void kv4_range(const float (&x)[8], float& mn, float& mx) {
    mn = x[0];
    mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn = fminf(mn, x[i]);
        mx = max_nan(mx, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
}

// The stored scale and minimum of a block, each its exact value rounded once: d from the difference with its
// rounding error, compared with the border between its f16 neighbours. id: 1 / (15 d), 0 where d is.
// A block with a value that is not finite decodes to NaN. Returns 0, 1 if the minimum or the scale
// overflows f16, 2 if a value is not finite.
__device__ __forceinline__ int kv4_scale(float mn, float mx, __half& dh, __half& mh, float& id) {
    mh = __hadd(__float2half_rn(mn), __float2half_rn(0.f));   // a zero minimum is stored as +0
    // mx - mn = s + e exactly
    const float s = __fsub_rn(mx, mn);
    const float t = __fsub_rn(s, mx);
    const float e = __fadd_rn(__fsub_rn(mx, __fsub_rn(s, t)), __fsub_rn(-mn, t));
    const __half lo = __float2half_rd(__fmul_rn(s, 1.0f / 15.0f));
    const uint16_t lob = __half_as_ushort(lo);
    const float lof = __half2float(lo);
    // the next f16 after lo (65536 stands in for the one after the largest: the border is 65520)
    const float hif = lob >= 0x7BFFu ? 65536.f : __half2float(__ushort_as_half((uint16_t)(lob + 1)));
    const float border = 0.5f * (lof + hif);
    const float over = __fadd_rn(__fsub_rn(s, 15.0f * border), e);   // 15 border has 16 bits: exact
    const bool up = over > 0.f || (over == 0.f && (lob & 1));
    dh = __ushort_as_half((uint16_t)(lob + (up && lob < 0x7C00u ? 1 : 0)));
    const float d = __half2float(dh);
    asm("rcp.approx.f32 %0, %1;" : "=f"(id) : "f"(d));
    id = d > 0.f ? __fmul_rn(id, 1.0f / 15.0f) : 0.f;
    return !(s < INFINITY) ? 2 : __hisinf(dh) || __hisinf(mh) ? 1 : 0;
}

// The codes of this lane's 8 elements, code[i] = kCodeOne + the code of x[i], its exact value rounded once: from
// g = (x - m) / (15 d) clamped to [0, 1] in f32, 15 g + 1.5 2^23 leaving the nearest integer in the low bits.
// Every step's error is relative: 15 g is off by at most 6 2^-24 of itself (a difference, a reciprocal good to
// 2^-23, three products). Where 15 g (1 - 2^-20) and 15 g (1 + 2^-20) do not round alike, the exact difference
// is compared with the border.
constexpr uint32_t kCodeOne = 0x4B400000u;   // the constant part of a code
__device__ __forceinline__ void kv4_codes(const float (&x)[8], __half dh, __half mh, float id, uint32_t (&code)[8]) {
    const float m = __half2float(mh);
    float g[8];
    uint32_t apart = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] = __saturatef(__fmul_rn(__fsub_rn(x[i], m), id));
        code[i] = __float_as_uint(__fmaf_rn(g[i], 15.0f * (1.0f + 0x1p-20f), 12582912.0f));
        apart |= code[i] ^ __float_as_uint(__fmaf_rn(g[i], 15.0f * (1.0f - 0x1p-20f), 12582912.0f));
    }
    if (apart != 0) {
        const float d = __half2float(dh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // x - m = y + ye exactly, against the border (k + 1/2) d, which has 16 bits
            const float k = floorf(15.0f * g[i]);
            const float y = __fsub_rn(x[i], m), z = __fsub_rn(y, x[i]);
            const float ye = __fadd_rn(__fsub_rn(x[i], __fsub_rn(y, z)), __fsub_rn(-m, z));
            const float v = __fadd_rn(__fsub_rn(y, __fmul_rn(k + 0.5f, d)), ye);
            const bool odd = ((int)k & 1) != 0;
            if (fabsf(__fmaf_rn(g[i], 15.0f, -k) - 0.5f) < 0x1p-15f)
                code[i] = kCodeOne + (uint32_t)k + (v > 0.f || (v == 0.f && odd) ? 1u : 0u);
        }
    }
}

// Quantise a key row and a value row into slot `slot` of a record, by LANES neighbouring lanes: this
// lane is word j (0..3) of block b. xk: elements 4 j + {0..3} and 16 + 4 j + {0..3} of the block of
// the key row; xv: elements 2 j + 8 q and 2 j + 1 + 8 q (q = 0..3) of the value row, at q and 4 + q.
// Of the 4 lanes of a block two work out the key block's scale, two the value block's.
// Stores only where `live`; all 32 lanes of the warp take part. Returns what kv4_scale does, the larger.
template <int HD>
__device__ __forceinline__ int kv4_put_rows(const float (&xk)[8], const float (&xv)[8], uint8_t* rec, int slot, int b,
                                             int j, bool live) {
    using R = Kv4<HD>;
    float nk, tk, nv, tv, id;
    kv4_range(xk, nk, tk);
    kv4_range(xv, nv, tv);
    const bool val = j & 1;
    __half d, m;
    const int fault = kv4_scale(val ? nv : nk, val ? tv : tk, d, m, id);
    // the other block's, from the neighbour
    const __half2 dm = __halves2half2(d, m);
    const uint32_t own = *reinterpret_cast<const uint32_t*>(&dm), their = __shfl_xor_sync(0xffffffffu, own, 1);
    const float id2 = __shfl_xor_sync(0xffffffffu, id, 1);
    const uint32_t wk = val ? their : own, wv = val ? own : their;
    const __half2 k2 = *reinterpret_cast<const __half2*>(&wk), v2 = *reinterpret_cast<const __half2*>(&wv);
    uint32_t ck[8], cv[8];
    kv4_codes(xk, __low2half(k2), __high2half(k2), val ? id2 : id, ck);
    kv4_codes(xv, __low2half(v2), __high2half(v2), val ? id : id2, cv);
    if (live) {
        // the codes' constant parts add up to a constant each
        uint32_t w = 0u - kCodeOne * 0x11111111u;
#pragma unroll
        for (int i = 0; i < 4; ++i) w += ck[i] * (1u << (8 * i)) + ck[4 + i] * (16u << (8 * i));
        *reinterpret_cast<uint32_t*>(rec + R::KC + slot * (HD / 2) + 4 * (R::NB * j + b)) = w;
        uint8_t* vrow = rec + R::VC + slot * (HD / 2) + 2 * b;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint16_t*>(vrow + R::vunit(slot, 2 * j + u)) =
                (uint16_t)(cv[4 * u] + cv[4 * u + 1] * 16u + cv[4 * u + 2] * 256u + cv[4 * u + 3] * 4096u - kCodeOne * 0x1111u);
        // lane 0 the key scale, 1 the value scale, 2 the key minimum, 3 the value minimum
        const int at = val ? R::VD + 2 * R::vscale(slot, b) : R::KD + 2 * (slot * R::NB + b);
        *reinterpret_cast<uint16_t*>(rec + at + (j & 2 ? R::KM - R::KD : 0)) = (uint16_t)(j & 2 ? own >> 16 : own);
    }
    return fault;
}
#endif

}  // namespace ql
