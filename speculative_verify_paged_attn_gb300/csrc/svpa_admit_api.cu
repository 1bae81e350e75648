// svpa_admit_api.cu -- the C ABI of the block-table build, the K/V scatter and
// the logits processing: host-side validation and the launches.  No function
// here allocates device memory.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/svpa.h"
#include "admit.h"

using namespace svpa;

namespace {

constexpr size_t kAlign = 256;
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
svpa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SVPA_OK : SVPA_ERR_CUDA; }

}  // namespace

extern "C" {

svpa_status svpa_block_table_build_workspace_size(int32_t batch, size_t *bytes) {
    if (!bytes || batch < 0) return SVPA_ERR_INVALID_ARG;
    if (batch > kMaxBuildBatch) return SVPA_ERR_UNSUPPORTED;
    *bytes = kAlign;
    return SVPA_OK;
}

svpa_status svpa_block_table_build(int32_t batch, int32_t block_size, int32_t max_blocks_per_seq, int32_t num_blocks,
                                   int32_t num_slots, const int32_t *seq_lens, const int32_t *prefix_blocks,
                                   int32_t prefix_len, int32_t *block_table, int32_t *cu_seqlens, int32_t *slot_map,
                                   int32_t *refcount, const int32_t *free_stack, int32_t *free_top, void *workspace,
                                   size_t workspace_bytes, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_block_table_build");
    if (batch < 0 || block_size != kBlockSize || max_blocks_per_seq < 1 || num_blocks < 1 || num_slots < 0 ||
        prefix_len < 0 || prefix_len % kBlockSize != 0 || prefix_len / kBlockSize > max_blocks_per_seq)
        return SVPA_ERR_INVALID_ARG;
    // slots are int32, table entries counted in 31 bits per row
    if (batch > kMaxBuildBatch || num_blocks > 0x7fffffff / kBlockSize ||
        max_blocks_per_seq > 0x7fffffff / kBlockSize - 1 || num_slots > (1 << 30))
        return SVPA_ERR_UNSUPPORTED;
    if (batch == 0) return SVPA_OK;
    if (!seq_lens || !block_table || !cu_seqlens || (num_slots > 0 && !slot_map) || !refcount || !free_stack ||
        !free_top || !error_flag || (prefix_len > 0 && !prefix_blocks))
        return SVPA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kAlign || !aligned(workspace, 16)) return SVPA_ERR_WORKSPACE;
    BuildArgs a;
    a.seq_lens = seq_lens;
    a.prefix_blocks = prefix_blocks;
    a.block_table = block_table;
    a.cu_seqlens = cu_seqlens;
    a.slot_map = slot_map;
    a.refcount = refcount;
    a.free_stack = free_stack;
    a.free_top = free_top;
    a.ticket = static_cast<int32_t *>(workspace);
    a.err = error_flag;
    a.B = batch;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.prefix_pages = prefix_len / kBlockSize;
    a.slots = num_slots;
    return from_cuda(launch_block_table_build(a, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_kv_write(int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          int32_t num_blocks, int32_t kv_dtype, int32_t scale_tile, const void *new_k,
                          const void *new_v, int64_t k_stride, int64_t v_stride, const int32_t *slot_map,
                          void *k_pool, void *v_pool, float *k_scale, float *v_scale, int32_t *error_flag,
                          void *stream) {
    svpa::NvtxRange nvtx_range("svpa_kv_write");
    if (num_tokens < 0 || num_kv_heads < 1 || num_kv_heads > 4096 || head_dim < 8 || head_dim % 8 != 0 ||
        head_dim > 1024 || block_size != kBlockSize || num_blocks < 1 ||
        (kv_dtype != SVPA_KV_BF16 && kv_dtype != SVPA_KV_FP8_E4M3))
        return SVPA_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == SVPA_KV_FP8_E4M3;
    if (scale_tile != 0 && (scale_tile != 64 || !fp8)) return SVPA_ERR_INVALID_ARG;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return SVPA_ERR_INVALID_ARG;
    // one scale per page needs the page's other rows: svpa_kv_append
    if (fp8 && (scale_tile == 0 || head_dim % 64 != 0)) return SVPA_ERR_UNSUPPORTED;
    // 16-byte words of all rows, a warp taking at most 128 of them
    if (num_tokens > (1 << 28) || (row / 8 / 128 + 1) * num_tokens > (1LL << 31)) return SVPA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SVPA_OK;
    if (!new_k || !new_v || !slot_map || !k_pool || !v_pool || !error_flag || (fp8 && (!k_scale || !v_scale)))
        return SVPA_ERR_INVALID_ARG;
    if (!aligned(new_k, 16) || !aligned(new_v, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
        return SVPA_ERR_INVALID_ARG;
    WriteArgs a;
    a.k = static_cast<const uint16_t *>(new_k);
    a.v = static_cast<const uint16_t *>(new_v);
    a.slot_map = slot_map;
    a.k_pool = static_cast<uint8_t *>(k_pool);
    a.v_pool = static_cast<uint8_t *>(v_pool);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.err = error_flag;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.T = num_tokens;
    a.Hkv = num_kv_heads;
    a.D = head_dim;
    a.num_blocks = num_blocks;
    a.fp8 = fp8;
    return from_cuda(launch_kv_write(a, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_logits_process(const svpa_logits_params *p, const void *logits, const int32_t *history,
                                const int32_t *prompt_lens, const int32_t *hist_lens, const int32_t *draft_tokens,
                                const int32_t *parent, const float *repetition, const float *presence,
                                const float *frequency, const int32_t *bias_offsets, const int32_t *bias_tokens,
                                const float *bias_values, const uint32_t *mask, float *out, int32_t *error_flag,
                                void *stream) {
    svpa::NvtxRange nvtx_range("svpa_logits_process");
    if (!p || p->batch < 0 || p->rows < 1 || p->rows > kMaxNq || p->vocab < 1 || p->max_history < 0 ||
        (p->logits_dtype != SVPA_LOGITS_FP32 && p->logits_dtype != SVPA_LOGITS_BF16))
        return SVPA_ERR_INVALID_ARG;
    // a token's count has 29 bits, and the history's index runs a CTA's step past its end
    if (p->vocab > (1 << 24) || p->batch > 65535 || p->max_history > (1 << 28)) return SVPA_ERR_UNSUPPORTED;
    ProcessArgs a;
    memset(&a, 0, sizeof a);
    for (int j = 0; j < p->rows; ++j) {
        if (!parent) {  // row j follows the drafts 0 .. j - 1
            a.path[j] = j == 0 ? 0ull : (~0ull >> (64 - j));
            continue;
        }
        if (j == 0 ? parent[0] != -1 : (parent[j] < 0 || parent[j] >= j)) return SVPA_ERR_INVALID_ARG;
        a.path[j] = j == 0 ? 0ull : (a.path[parent[j]] | 1ull << j);
    }
    for (int j = 0; j < p->rows; ++j) a.used |= a.path[j];
    if (p->batch == 0) return SVPA_OK;
    if (!logits || !out || !error_flag) return SVPA_ERR_INVALID_ARG;
    const bool bf16 = p->logits_dtype == SVPA_LOGITS_BF16;
    if (!aligned(logits, bf16 ? 2 : 4) || !aligned(out, 4)) return SVPA_ERR_INVALID_ARG;
    if (bf16 && logits == out) return SVPA_ERR_INVALID_ARG;  // in place needs one element size
    if (history && (!hist_lens || p->max_history < 1)) return SVPA_ERR_INVALID_ARG;
    if (bias_tokens && (!bias_offsets || !bias_values)) return SVPA_ERR_INVALID_ARG;
    a.in = logits;
    a.out = out;
    a.history = history;
    a.prompt_lens = prompt_lens;
    a.hist_lens = hist_lens;
    a.draft_stride = parent ? p->rows : p->rows - 1;
    a.drafts = a.draft_stride > 0 ? draft_tokens : nullptr;
    a.repetition = repetition;
    a.presence = presence;
    a.frequency = frequency;
    a.bias_offsets = bias_offsets;
    a.bias_tokens = bias_tokens;
    a.bias_values = bias_values;
    a.mask = mask;
    a.err = error_flag;
    a.B = p->batch;
    a.rows = p->rows;
    a.V = p->vocab;
    a.max_hist = p->max_history;
    a.bf16 = bf16;
    return from_cuda(launch_logits_process(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
