// fp4_attn.h -- arguments and launch of the verification attention over 4-bit pages.
#pragma once

#include "svpa_internal.h"

namespace svpa {

struct Fp4AttnArgs {
    const float *k_factor;  // [Hkv] or null
    const float *v_factor;
    const int32_t *block_table;
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *err;
    int32_t *tickets;  // [B * Hkv]: parts written of a pair cut between CTAs
    float *part_ml;    // [2 * grid, M, 2] (reference maximum in log2 units, sum), two parts a CTA
    float *part_acc;   // [2 * grid, M, D]
    int32_t B, n_q, Hq, Hkv, G, M, max_blocks, num_blocks;
    float scale_log2;  // sm_scale * log2(e)
    // bit c of slots[i]: query row c (query c / G, head c % G) sees speculative slot i
    unsigned long long slots[kMaxNq][2];
};

struct Fp4AttnMaps {
    CUtensorMap kc, vc;  // codes: [(page, kv head)][16 rows][D / 2 bytes]
    CUtensorMap ks, vs;  // scales: [(page, kv head)][16 * D / 16 bytes]
    CUtensorMap q[2];    // 64-column slabs of one (sequence, kv head)'s queries
};

// CTAs of a launch; each has two part slots.
int fp4_attn_grid();
cudaError_t launch_paged_verify_attn_fp4(const Fp4AttnMaps &maps, const Fp4AttnArgs &a, int D, cudaStream_t stream);

}  // namespace svpa
