// svpa_fp4_api.cu -- the C ABI of the norms and rotation, of the pages they
// write and the reads back, and of the append and the verification attention
// on 4-bit pages: host-side validation and the launches.  No function here
// allocates device memory.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <cmath>

#include "../../include/svpa.h"
#include "fp4_attn.h"
#include "rope_kv.h"

using namespace svpa;

namespace {

constexpr int kMaxPoolBlocks = 0x7fffffff / kBlockSize;  // slots are int32

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
svpa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SVPA_OK : SVPA_ERR_CUDA; }

// The page kind of (kv_dtype, scale_tile) for rows of head_dim elements.
svpa_status page_kind(int32_t kv_dtype, int32_t scale_tile, int32_t head_dim, Pages *out) {
    if (kv_dtype != SVPA_KV_BF16 && kv_dtype != SVPA_KV_FP8_E4M3 && kv_dtype != SVPA_KV_FP4_E2M1)
        return SVPA_ERR_INVALID_ARG;
    if (scale_tile != 0 && (scale_tile != 64 || kv_dtype != SVPA_KV_FP8_E4M3)) return SVPA_ERR_INVALID_ARG;
    // (one scale per page needs the page's other rows: svpa_kv_append)
    if (kv_dtype == SVPA_KV_FP8_E4M3 && (scale_tile == 0 || head_dim % 64 != 0)) return SVPA_ERR_UNSUPPORTED;
    if (kv_dtype == SVPA_KV_FP4_E2M1 && head_dim % 16 != 0) return SVPA_ERR_INVALID_ARG;
    *out = kv_dtype == SVPA_KV_BF16 ? Pages::kBf16 : kv_dtype == SVPA_KV_FP8_E4M3 ? Pages::kFp8 : Pages::kFp4;
    return SVPA_OK;
}

svpa_status check_rope(const svpa_rope_params *p, bool pages) {
    if (!p || p->num_tokens < 0 || p->num_q_heads < 0 || p->num_q_heads > 4096 || p->num_kv_heads < 1 ||
        p->num_kv_heads > 4096 || p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 2 != 0 ||
        p->max_position < 1 || !(p->eps >= 0.f) || !std::isfinite(p->eps) ||
        (p->interleaved != 0 && p->interleaved != 1))
        return SVPA_ERR_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return SVPA_ERR_UNSUPPORTED;
    if (p->rotary_dim % 16 != 0 || p->num_tokens > (1 << 28)) return SVPA_ERR_UNSUPPORTED;
    const int64_t qrow = (int64_t)p->num_q_heads * p->head_dim, krow = (int64_t)p->num_kv_heads * p->head_dim;
    const int64_t strides[5] = {p->q_stride, p->q_out_stride, p->k_stride, pages ? p->v_stride : krow,
                                pages ? krow : p->k_out_stride};
    for (int i = 0; i < 5; ++i) {
        if (i < 2 && p->num_q_heads == 0) continue;
        if (strides[i] < (i < 2 ? qrow : krow) || strides[i] % 8 != 0) return SVPA_ERR_INVALID_ARG;
    }
    // a warp takes at least 4 heads of a token, a CTA 8 warps
    if ((int64_t)p->num_tokens * ((p->num_q_heads + 3) / 4 + 2 * ((p->num_kv_heads + 3) / 4)) > (1LL << 33))
        return SVPA_ERR_UNSUPPORTED;
    return SVPA_OK;
}

// What both calls pass on, and the checks of the pointers they share.
svpa_status fill_rope(const svpa_rope_params *p, const void *q, const void *k, const int32_t *positions,
                      const float *cos_sin, const void *q_weight, const void *k_weight, void *q_out,
                      int32_t *error_flag, RopeArgs &a) {
    memset(&a, 0, sizeof a);
    if (!k || !error_flag || (p->num_q_heads > 0 && (!q || !q_out)) ||
        (p->rotary_dim > 0 && (!positions || !cos_sin)))
        return SVPA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(cos_sin, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(q_out, 16))
        return SVPA_ERR_INVALID_ARG;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.q_weight = static_cast<const uint16_t *>(q_weight);
    a.k_weight = static_cast<const uint16_t *>(k_weight);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.err = error_flag;
    a.q_stride = p->q_stride;
    a.k_stride = p->k_stride;
    a.v_stride = p->v_stride;
    a.q_out_stride = p->q_out_stride;
    a.k_out_stride = p->k_out_stride;
    a.T = p->num_tokens;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.R = p->rotary_dim;
    a.interleaved = p->interleaved;
    a.max_position = p->max_position;
    a.eps = p->eps;
    return SVPA_OK;
}

svpa_status check_attn(const svpa_attn_params *p) {
    if (!p || p->batch < 0 || p->n_q < 1 || p->n_q > kMaxNq || p->num_q_heads < 1 || p->num_kv_heads < 1 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->block_size != kBlockSize || p->max_blocks_per_seq < 1 ||
        p->num_blocks < 1 || !(p->sm_scale > 0.f) || !std::isfinite(p->sm_scale) || p->split_pages < 0 ||
        p->kv_dtype != SVPA_KV_FP4_E2M1 || p->variant != 0 || p->scale_tile != 0)
        return SVPA_ERR_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return SVPA_ERR_UNSUPPORTED;
    if ((long long)p->num_q_heads / p->num_kv_heads * p->n_q > kMaxRows || p->batch > 65535 ||
        p->num_kv_heads > 65535 || (long long)p->num_blocks * p->num_kv_heads > 0x7fffffffLL ||
        p->max_blocks_per_seq > kMaxPoolBlocks - 8)  // (positions rounded up to 128 stay int32)
        return SVPA_ERR_UNSUPPORTED;
    return SVPA_OK;
}

// The attention's workspace: [other calls' counters and tickets, not touched][pairs
// to join][parts' (max, sum)][parts' accumulators].
struct AttnSpace {
    size_t off_joins, off_ml, off_acc, bytes;
};
svpa_status attn_space(const svpa_attn_params *p, AttnSpace *sp) {
    const svpa_status s = check_attn(p);
    if (s != SVPA_OK) return s;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)2 * fp4_attn_grid() * (p->num_q_heads / p->num_kv_heads) * p->n_q;
    sp->off_joins = kWorkspaceCounterBytes + kTicketBytes;
    sp->off_ml = sp->off_joins + up(fp4_attn_grid() * sizeof(Fp4Join));
    sp->off_acc = sp->off_ml + up(rows * 2 * sizeof(float));
    sp->bytes = sp->off_acc + up(rows * p->head_dim * sizeof(float));
    return SVPA_OK;
}

}  // namespace

extern "C" {

svpa_status svpa_qk_norm_rope(const svpa_rope_params *p, const void *q, const void *k, const int32_t *positions,
                              const float *cos_sin, const void *q_weight, const void *k_weight, void *q_out,
                              void *k_out, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_qk_norm_rope");
    svpa_status s = check_rope(p, false);
    if (s != SVPA_OK) return s;
    if (p->num_tokens == 0) return SVPA_OK;
    RopeArgs a;
    s = fill_rope(p, q, k, positions, cos_sin, q_weight, k_weight, q_out, error_flag, a);
    if (s != SVPA_OK) return s;
    if (!k_out || !aligned(k_out, 16)) return SVPA_ERR_INVALID_ARG;
    // in place a row's new values go where its old ones were
    if ((q == q_out && p->num_q_heads > 0 && p->q_stride != p->q_out_stride) ||
        (k == k_out && p->k_stride != p->k_out_stride))
        return SVPA_ERR_INVALID_ARG;
    a.k_out = static_cast<uint16_t *>(k_out);
    return from_cuda(launch_rope(a, p->head_dim, Pages::kRows, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_rope_kv_write(const svpa_rope_params *p, const void *q, const void *k, const void *v,
                               const int32_t *positions, const int32_t *slot_map, const float *cos_sin,
                               const void *q_weight, const void *k_weight, void *q_out, void *k_pool, void *v_pool,
                               float *k_scale, float *v_scale, const float *k_factor, const float *v_factor,
                               int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_rope_kv_write");
    svpa_status s = check_rope(p, true);
    if (s != SVPA_OK) return s;
    if (p->block_size != kBlockSize || p->num_blocks < 1) return SVPA_ERR_INVALID_ARG;
    Pages kind;
    s = page_kind(p->kv_dtype, p->scale_tile, p->head_dim, &kind);
    if (s != SVPA_OK) return s;
    if (p->num_blocks > kMaxPoolBlocks) return SVPA_ERR_UNSUPPORTED;
    if (p->num_tokens == 0) return SVPA_OK;
    RopeArgs a;
    s = fill_rope(p, q, k, positions, cos_sin, q_weight, k_weight, q_out, error_flag, a);
    if (s != SVPA_OK) return s;
    if (!v || !slot_map || !k_pool || !v_pool || (kind == Pages::kFp8 && (!k_scale || !v_scale)))
        return SVPA_ERR_INVALID_ARG;
    if (!aligned(v, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16)) return SVPA_ERR_INVALID_ARG;
    if (q == q_out && p->num_q_heads > 0 && p->q_stride != p->q_out_stride) return SVPA_ERR_INVALID_ARG;
    a.v = static_cast<const uint16_t *>(v);
    a.slot_map = slot_map;
    a.k_pool = static_cast<uint8_t *>(k_pool);
    a.v_pool = static_cast<uint8_t *>(v_pool);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_factor = k_factor;
    a.v_factor = v_factor;
    a.num_blocks = p->num_blocks;
    return from_cuda(launch_rope(a, p->head_dim, kind, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_kv_read(int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         int32_t num_blocks, int32_t kv_dtype, int32_t scale_tile, const int32_t *slot_map,
                         const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale,
                         const float *k_factor, const float *v_factor, void *k_out, void *v_out, int64_t k_stride,
                         int64_t v_stride, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_kv_read");
    if (num_tokens < 0 || num_kv_heads < 1 || num_kv_heads > 4096 || head_dim < 8 || head_dim % 8 != 0 ||
        head_dim > 1024 || block_size != kBlockSize || num_blocks < 1)
        return SVPA_ERR_INVALID_ARG;
    Pages kind;
    const svpa_status s = page_kind(kv_dtype, scale_tile, head_dim, &kind);
    if (s != SVPA_OK) return s;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return SVPA_ERR_INVALID_ARG;
    if (num_tokens > (1 << 28) || (row / 8 / 128 + 1) * num_tokens > (1LL << 31) || num_blocks > kMaxPoolBlocks)
        return SVPA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return SVPA_OK;
    if (!slot_map || !k_pool || !v_pool || !k_out || !v_out || !error_flag ||
        (kind == Pages::kFp8 && (!k_scale || !v_scale)))
        return SVPA_ERR_INVALID_ARG;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return SVPA_ERR_INVALID_ARG;
    ReadArgs a;
    a.slot_map = slot_map;
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_factor = k_factor;
    a.v_factor = v_factor;
    a.k = static_cast<uint16_t *>(k_out);
    a.v = static_cast<uint16_t *>(v_out);
    a.err = error_flag;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.T = num_tokens;
    a.Hkv = num_kv_heads;
    a.D = head_dim;
    a.num_blocks = num_blocks;
    return from_cuda(launch_kv_read(a, kind, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_kv_append_fp4(int32_t batch, int32_t n_new, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t max_blocks_per_seq, int32_t num_blocks, const void *new_k,
                               const void *new_v, int32_t *block_table, const int32_t *context_lens,
                               int32_t *refcount, int32_t *free_stack, int32_t *free_top, void *k_pool, void *v_pool,
                               const float *k_factor, const float *v_factor, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_kv_append_fp4");
    if (batch < 0 || n_new < 1 || n_new > kMaxAppendRows || num_kv_heads < 1 || num_kv_heads > 4096 ||
        head_dim < 16 || head_dim % 16 != 0 || head_dim > 1024 || block_size != kBlockSize ||
        max_blocks_per_seq < 1 || num_blocks < 1)
        return SVPA_ERR_INVALID_ARG;
    if (batch == 0) return SVPA_OK;
    if (!new_k || !new_v || !block_table || !context_lens || !refcount || !free_stack || !free_top || !k_pool ||
        !v_pool || !error_flag)
        return SVPA_ERR_INVALID_ARG;
    if (!aligned(new_k, 16) || !aligned(new_v, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
        return SVPA_ERR_INVALID_ARG;
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.new_k = static_cast<const uint16_t *>(new_k);
    a.new_v = static_cast<const uint16_t *>(new_v);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.refcount = refcount;
    a.free_stack = free_stack;
    a.free_top = free_top;
    a.k_pool = static_cast<uint8_t *>(k_pool);
    a.v_pool = static_cast<uint8_t *>(v_pool);
    a.k_factor = k_factor;
    a.v_factor = v_factor;
    a.err = error_flag;
    a.page_bytes = (size_t)num_kv_heads * 9 * head_dim;
    a.B = batch;
    a.n_new = n_new;
    a.Hkv = num_kv_heads;
    a.D = head_dim;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.fp4 = 1;
    // w / (D / 8) as a product's high word: exact for w (D / 8) < 2^32
    a.magic = (uint32_t)(((1ull << 32) + head_dim / 8 - 1) / (head_dim / 8));
    return from_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

svpa_status svpa_paged_verify_attn_fp4_workspace_size(const svpa_attn_params *p, size_t *bytes) {
    AttnSpace sp;
    const svpa_status s = attn_space(p, &sp);
    if (s != SVPA_OK) return s;
    if (!bytes) return SVPA_ERR_INVALID_ARG;
    *bytes = sp.bytes;
    return SVPA_OK;
}

svpa_status svpa_paged_verify_attn_fp4(const svpa_attn_params *p, const void *q, const void *k_pool,
                                       const void *v_pool, const float *k_factor, const float *v_factor,
                                       const int32_t *block_table, const int32_t *context_lens,
                                       const uint64_t *ancestor_mask, void *out, float *lse, void *workspace,
                                       size_t workspace_bytes, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_paged_verify_attn_fp4");
    AttnSpace sp;
    svpa_status s = attn_space(p, &sp);
    if (s != SVPA_OK) return s;
    if (p->batch == 0) return SVPA_OK;
    s = check_attn_call(p, q, k_pool, v_pool, nullptr, nullptr, block_table, context_lens, ancestor_mask, out,
                        error_flag);
    if (s != SVPA_OK) return s;
    if (!workspace || workspace_bytes < sp.bytes || !aligned(workspace, 16)) return SVPA_ERR_WORKSPACE;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return SVPA_ERR_CUDA;

    const int D = p->head_dim, G = p->num_q_heads / p->num_kv_heads;
    CUtensorMap mq[2];
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    // queries [B, n_q, Hq, D]: (64 columns, G heads, n_q queries) of a sequence at a time
    const cuuint64_t qd[4] = {64, (cuuint64_t)p->num_q_heads, (cuuint64_t)p->n_q, (cuuint64_t)p->batch};
    const cuuint64_t qs[3] = {(cuuint64_t)D * 2, (cuuint64_t)p->num_q_heads * D * 2,
                              (cuuint64_t)p->n_q * p->num_q_heads * D * 2};
    const cuuint32_t qb[4] = {64, (cuuint32_t)G, (cuuint32_t)p->n_q, 1};
    for (int i = 0; i < 2; ++i) {
        uint8_t *base = static_cast<uint8_t *>(const_cast<void *>(q)) + (D == 128 ? 128 * i : 0);
        if (enc(&mq[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, qd, qs, qb, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SVPA_ERR_CUDA;
    }

    Fp4AttnArgs a;
    memset(&a, 0, sizeof a);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.k_factor = k_factor;
    a.v_factor = v_factor;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.err = error_flag;
    a.joins = reinterpret_cast<Fp4Join *>(ws + sp.off_joins);
    a.part_ml = reinterpret_cast<float *>(ws + sp.off_ml);
    a.part_acc = reinterpret_cast<float *>(ws + sp.off_acc);
    a.B = p->batch;
    a.n_q = p->n_q;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.G = G;
    a.M = G * p->n_q;
    a.max_blocks = p->max_blocks_per_seq;
    a.num_blocks = p->num_blocks;
    a.scale_log2 = p->sm_scale * 1.4426950408889634f;
    for (int j = 0; j < p->n_q; ++j) {
        const uint64_t sees = ancestor_mask ? ancestor_mask[j] : ~0ull >> (63 - j);
        for (int i = 0; i <= j; ++i) {
            if (!(sees >> i & 1)) continue;
            for (int c = j * G; c < (j + 1) * G; ++c) a.slots[i][c >> 6] |= 1ull << (c & 63);
        }
    }
    return from_cuda(launch_paged_verify_attn_fp4(mq, a, D, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
