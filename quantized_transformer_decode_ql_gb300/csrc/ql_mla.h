// Latent attention: what its translation units share (not part of the ABI).
#pragma once

#include "ql_internal.h"

namespace ql {
namespace mla {

constexpr int kRope = 64;    // rotated values of a cache row and of a query head
constexpr int kBlock = 16;   // tokens of a pool block
// The weights of the softmax are f16 numbers relative to a running reference, log2 of which lies kLift below the largest score when it is
// set: half a step of f16's subnormals is then 2^-31 of the largest weight, so that many keys far below it still count (2^20 keys, each
// 2^-25.2 of the largest, weigh 2.6% together; with the reference at the largest they were 0). It is moved when a score lies kLag above it.
constexpr float kLift = 6.f, kLag = 15.f;   // f16 holds 2^15

inline bool shape_ok(int head_dim, int rank) { return (head_dim == 64 || head_dim == 128) && (rank == 256 || rank == 512); }

// The arguments that the attention entry points share.
struct AttnIn {
    const void *q, *w, *pool;
    const int32_t *table, *lens;      // lens: the lengths, or a chunk's position
    int64_t rows, tables, maxb, num_blocks;   // rows of q and the output, rows of the table
    int H, D, R, rope, block;
    float scale;
    void *out, *ws;
    size_t ws_bytes;
};
// The absorbed form of a's rows: sequences with a length each, or (chunk) one sequence's queries from the position on (ql_mla_decode.cu).
int absorbed_launch(const AttnIn& a, bool chunk, cudaStream_t s);
size_t absorbed_workspace(int64_t rows, int H, int R);
// Their checks; `need`: the workspace's bytes, 0 where the sizes are out of range.
int attn_check(const char* name, const AttnIn& a, size_t need);

}  // namespace mla
}  // namespace ql
