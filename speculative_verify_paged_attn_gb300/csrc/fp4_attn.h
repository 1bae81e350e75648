// fp4_attn.h -- arguments and launch of the verification attention over 4-bit pages.
#pragma once

#include "svpa_internal.h"

namespace svpa {

struct Fp4AttnArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const float *k_factor;
    const float *v_factor;
    const int32_t *block_table;
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *err;
    int32_t B, n_q, Hq, Hkv, G, M, max_blocks, num_blocks;
    float scale_log2;  // sm_scale * log2(e)
    unsigned long long anc[kMaxNq];
};
cudaError_t launch_paged_verify_attn_fp4(const Fp4AttnArgs &a, int D, cudaStream_t stream);

}  // namespace svpa
