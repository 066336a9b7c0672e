// Decode attention over the 4-bit KV pool (ql_kv4_attn.cu): the internal launch interface.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ql {

struct Kv4AttnArgs {
    const __half* q;              // [batch][n_heads][head_dim]
    const uint8_t* pool;          // one layer: [num_blocks][n_kv_heads][20 head_dim]
    const int32_t* block_tables;  // [batch][max_blocks_per_seq]
    const int32_t* context_lens;  // [batch]; null: positions[b] + 1 (decode step form)
    const int32_t* positions;
    const int32_t* active;        // [batch] or null: rows with 0 are left out
    int batch, n_heads, n_kv_heads, head_dim;
    int64_t max_blocks_per_seq, num_blocks;
    float scale;
    bool early;                   // only q and the rows in a sequence's last block may come from the preceding kernel:
                                  // lengths, tables and the other blocks are read before it has ended (decode step)
    __half* out;                  // [batch][n_heads * head_dim]
    void* workspace;              // kv4_attn_workspace_bytes, zero-filled once
    size_t workspace_bytes;
};

constexpr int64_t kKv4MaxBlocks = 1ll << 25;   // of a table row: the tiles of 32 sequences fit 31 bits

size_t kv4_attn_workspace_bytes();   // of any shape, on the current device
int kv4_attn_launch(const Kv4AttnArgs& a, cudaStream_t s, bool pdl);

}  // namespace ql
