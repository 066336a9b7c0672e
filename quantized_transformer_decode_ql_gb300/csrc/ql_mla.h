// Latent attention: what its translation units share (not part of the ABI).
#pragma once

#include "ql_internal.h"

namespace ql {
namespace mla {

constexpr int kRope = 64;    // rotated values of a cache row and of a query head
constexpr int kBlock = 16;   // tokens of a pool block
constexpr float kLag = 14.f; // log2 of how far a weight may lie above its reference: f16 holds 2^15, and O is scaled rarely

inline bool shape_ok(int head_dim, int rank) { return (head_dim == 64 || head_dim == 128) && (rank == 256 || rank == 512); }

// The checks that the attention entry points share; `need`: the workspace's bytes, 0 where the sizes are out of range.
int attn_check(const char* name, const void* q, const void* w, const void* pool, const void* table, const void* lens, int head_dim, int rank,
               int rope_dim, int block_size, int64_t num_blocks, float scale, const void* out, const void* ws, size_t ws_bytes, size_t need);

}  // namespace mla
}  // namespace ql
