// admit.h -- arguments and launches of the kernels that admit requests and
// feed the samplers: block tables and slot maps, the K/V scatter, and the
// logits processing.
#pragma once

#include "svpa_internal.h"

namespace svpa {

constexpr int kMaxBuildBatch = 8192;  // two prefix sums of the batch in shared memory

struct BuildArgs {
    const int32_t *seq_lens;
    const int32_t *prefix_blocks;
    int32_t *block_table;
    int32_t *cu_seqlens;
    int32_t *slot_map;
    int32_t *refcount;
    const int32_t *free_stack;
    int32_t *free_top;
    int32_t *ticket;  // CTAs finished, zero between calls
    int32_t *err;
    int32_t B, max_blocks, num_blocks, prefix_pages, slots;
};
cudaError_t launch_block_table_build(const BuildArgs &a, cudaStream_t stream);

struct WriteArgs {
    const uint16_t *k;  // bf16 bits, rows of Hkv * D, k_stride elements apart
    const uint16_t *v;
    const int32_t *slot_map;
    uint8_t *k_pool;
    uint8_t *v_pool;
    float *k_scale;
    float *v_scale;
    int32_t *err;
    long long k_stride, v_stride;
    int32_t T, Hkv, D, num_blocks, fp8;
};
cudaError_t launch_kv_write(const WriteArgs &a, cudaStream_t stream);

struct ProcessArgs {
    const void *in;  // fp32 or bf16 [B, rows, V]
    float *out;      // fp32 [B, rows, V]
    const int32_t *history;
    const int32_t *prompt_lens;
    const int32_t *hist_lens;
    const int32_t *drafts;
    const float *repetition;
    const float *presence;
    const float *frequency;
    const int32_t *bias_offsets;
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *mask;
    int32_t *err;
    int32_t B, rows, V, max_hist, draft_stride, bf16;
    int32_t split_rows;  // one row a CTA (set by the launch)
    unsigned long long path[kMaxNq];  // bit i of row j: draft entry i counts for row j
    unsigned long long used;          // the entries that count for any row
};
cudaError_t launch_logits_process(const ProcessArgs &a, cudaStream_t stream);

}  // namespace svpa
