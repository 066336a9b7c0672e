// Latent attention: what its translation units share (not part of the ABI).
#pragma once

#include "ql_internal.h"

namespace ql {
namespace mla {

constexpr int kRope = 64;    // rotated values of a cache row and of a query head
constexpr int kBlock = 16;   // tokens of a pool block
constexpr float kLag = 14.f; // log2 of how far a weight may lie above its reference: f16 holds 2^15, and O is scaled rarely

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
