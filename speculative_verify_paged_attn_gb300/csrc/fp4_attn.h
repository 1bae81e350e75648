// fp4_attn.h -- arguments and launch of the verification attention over 4-bit pages.
#pragma once

#include "svpa_internal.h"

namespace svpa {

// A pair whose parts are to be joined: the first part's slot and their number (0: none).
struct Fp4Join {
    int32_t b, h, slot, parts;
};

struct Fp4AttnArgs {
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const float *k_factor;  // [Hkv] or null
    const float *v_factor;
    const int32_t *block_table;
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *err;
    Fp4Join *joins;    // [grid]: the pair that begins in a CTA's share and goes on behind it
    float *part_ml;    // [2 * grid, M, 2] (reference maximum in log2 units, sum), two parts a CTA
    float *part_acc;   // [2 * grid, M, D]
    int32_t B, n_q, Hq, Hkv, G, M, max_blocks, num_blocks;
    float scale_log2;  // sm_scale * log2(e)
    // bit c of slots[i]: query row c (query c / G, head c % G) sees speculative slot i
    unsigned long long slots[kMaxNq][2];
};

// CTAs of a launch; each has two part slots.
int fp4_attn_grid();
// mq: the maps of the two 64-column slabs of one (sequence, kv head)'s queries (D 64: one).
cudaError_t launch_paged_verify_attn_fp4(const CUtensorMap *mq, const Fp4AttnArgs &a, int D, cudaStream_t stream);

}  // namespace svpa
