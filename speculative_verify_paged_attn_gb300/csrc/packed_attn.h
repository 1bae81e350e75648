// packed_attn.h -- arguments and launches of the packed-query attention
// kernel (packed_attn_tc.cu): prompt attention over pages and verification
// attention behind a shared prefix.
#pragma once

#include "svpa_internal.h"

namespace svpa {

// Query rows of one 128-row MMA tile: tpt tokens x G heads of one kv head.
struct PackedArgs {
    const int32_t *block_table;    // [B, max_blocks]
    const int32_t *cu;             // [B + 1] packed query offsets (prompt)
    const int32_t *lens;           // [B] kv lengths (prompt) or committed histories (verify)
    const int32_t *prefix_blocks;  // [prefix_pages] (verify)
    const int32_t *order;          // [B] sequences, longest first, or null (verify)
    __nv_bfloat16 *out;            // [T, Hq, D]
    float *lse;                    // [T, Hq] or null
    // partials, one row for each (slot, kv head, 128-row query tile, row of the
    // tile): unnormalised outputs, 32 rows at a time as [D / 4][32 rows][4]
    // (a warp that holds one row a lane then reads and writes 512 bytes in one
    // piece), and (reference maximum in log2 units, sum)
    float *part_o;
    float2 *part_ml;
    int32_t *member;               // [B] the sequence's table begins with the prefix (split verify only)
    int32_t *sched;                // [3]: next unit, CTAs finished, warps that wrote a prefix unit; zero between calls
    int32_t *err;
    int32_t verify;                // 0 = prompt, 1 = verification behind a shared prefix
    int32_t B, T, Hq, Hkv, G, n_q, tpt, tiles;  // tiles: ceil(T / tpt)
    int32_t max_blocks, num_blocks, prefix_pages;
    int32_t pairs;                 // prompt: unit slots per kv head; verify: tile pairs of the prefix units
    int32_t p_units, total_units;  // prefix units come first
    int32_t p_splits, s_splits;    // KV splits of the prefix units and of the others
    float scale_log2;
    unsigned long long anc[kMaxNq];
};

struct PackedMaps {
    CUtensorMap k, v;       // one (page, kv head) tile per copy
    CUtensorMap qt[2];      // 64-column slabs of tpt tokens x G heads
    CUtensorMap qs[2];      // the same of n_q tokens (verify: one sequence)
};

cudaError_t launch_packed_attn(const PackedMaps &m, const PackedArgs &a, int head_dim, int grid, cudaStream_t stream);
// Merges the partial rows when units were split (s_splits > 1).
cudaError_t launch_packed_combine(const PackedArgs &a, int head_dim, cudaStream_t stream);

}  // namespace svpa
