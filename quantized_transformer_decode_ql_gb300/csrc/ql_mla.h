// Latent attention: what its translation units share (not part of the ABI).
#pragma once

#include "ql_internal.h"

namespace ql {
namespace mla {

constexpr int kRope = 64;    // rotated values of a cache row and of a query head
constexpr int kBlock = 16;   // tokens of a pool block

inline bool shape_ok(int head_dim, int rank) { return (head_dim == 64 || head_dim == 128) && (rank == 256 || rank == 512); }

}  // namespace mla
}  // namespace ql
