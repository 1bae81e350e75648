// svpa_prompt_api.cu -- the C ABI of the packed-query attention calls: prompt
// attention over pages and verification behind a shared prefix.  Host-side
// validation, split choice, workspace layout, tensor maps and the launches;
// no function here allocates device memory.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "../../include/svpa.h"
#include "packed_attn.h"

using namespace svpa;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxSplits = 32;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
svpa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SVPA_OK : SVPA_ERR_CUDA; }

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

bool encode_bf16(EncodeTiledFn enc, CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims,
                 const cuuint64_t *strides, const cuuint32_t *box) {
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One (page, kv head) tile per copy, landing as [row half][64-column slab][8 rows][128 B].
bool encode_pages(EncodeTiledFn enc, CUtensorMap *m, const void *pool, int D, long long tiles) {
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)(D / 64), 2, (cuuint64_t)tiles};
    const cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)8 * D * 2, (cuuint64_t)16 * D * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)(D / 64), 2, 1};
    return encode_bf16(enc, m, pool, 5, dims, strides, box);
}

// Query slabs of 64 columns: boxes of `tokens` tokens x G heads.
bool encode_queries(EncodeTiledFn enc, CUtensorMap m[2], const void *q, int D, int Hq, int G, long long T,
                    long long stride, int tokens) {
    const cuuint64_t dims[3] = {64, (cuuint64_t)Hq, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
    for (int s = 0; s < 2; ++s) {
        const char *base = static_cast<const char *>(q) + (s < D / 64 ? s : 0) * 128;
        if (!encode_bf16(enc, &m[s], base, 3, dims, strides, box)) return false;
    }
    return true;
}

struct Plan {
    int tpt, tiles, pairs, p_units, p_splits, s_splits, total_units;
    bool shared, ordered;
    size_t off_member, off_ml, off_o, bytes;
};

// Workspace: [counters][tickets of the verification kernels, never written here]
// [member or order][partial (max, sum)][partial outputs], one partial slot for
// each KV split of the prefix units and, when split, of the others.
svpa_status layout(Plan *pl, long long units, long long T, int Hkv, int D, int members) {
    // the kernels' counter runs up to a CTA count past the last unit
    if (units > 0x7fffffff - 65536) return SVPA_ERR_UNSUPPORTED;
    pl->total_units = (int)units;
    const size_t slots = (size_t)pl->p_splits + (pl->s_splits > 1 ? pl->s_splits : 0);
    pl->tiles = (int)ceil_div(T, pl->tpt);
    const size_t rows = (size_t)Hkv * pl->tiles * kMaxRows;
    pl->off_member = kWorkspaceCounterBytes + kTicketBytes;
    pl->off_ml = pl->off_member + align_up((size_t)members * sizeof(int32_t));
    pl->off_o = pl->off_ml + align_up(slots * rows * sizeof(float2));
    pl->bytes = pl->off_o + align_up(slots * rows * D * sizeof(float));
    return SVPA_OK;
}

svpa_status plan_prompt(const svpa_prompt_params *p, Plan *pl) {
    if (!p || p->batch < 0 || p->total_q < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1 ||
        p->num_q_heads % p->num_kv_heads != 0 || p->block_size != kBlockSize || p->max_blocks_per_seq < 1 ||
        p->num_blocks < 1 || !(p->sm_scale > 0.f) || !std::isfinite(p->sm_scale) ||
        (p->kv_dtype != SVPA_KV_BF16 && p->kv_dtype != SVPA_KV_FP8_E4M3))
        return SVPA_ERR_INVALID_ARG;
    if (p->q_stride != 0 &&
        (p->q_stride % 8 != 0 || p->q_stride < (long long)p->num_q_heads * p->head_dim))
        return SVPA_ERR_INVALID_ARG;
    const int G = p->num_q_heads / p->num_kv_heads;
    if ((p->head_dim != 64 && p->head_dim != 128) || p->kv_dtype != SVPA_KV_BF16 || G > kMaxRows ||
        p->max_blocks_per_seq > (0x7fffffff - 4096) / kBlockSize ||
        (long long)p->num_blocks * p->num_kv_heads > 0x7fffffff || p->num_kv_heads > 65535 ||
        p->batch > (1 << 20) || p->total_q > (1 << 28))
        return SVPA_ERR_UNSUPPORTED;
    pl->tpt = kMaxRows / G;
    pl->pairs = p->total_q / (2 * pl->tpt) + p->batch;
    pl->p_units = 0;
    pl->p_splits = 0;
    const long long units = (long long)pl->pairs * p->num_kv_heads;
    const int blocks = (int)ceil_div(p->max_blocks_per_seq, 8);
    // few tiles against long histories (a chunk or single tokens behind a long
    // cache): split the kv range until every SM has a unit
    pl->s_splits = 1;
    if (units > 0 && units < sm_count())
        pl->s_splits = std::max(1, std::min({(int)(sm_count() / units), blocks / 8, kMaxSplits}));
    return layout(pl, units * pl->s_splits, p->total_q, p->num_kv_heads, p->head_dim, 0);
}

svpa_status plan_prefix(const svpa_attn_params *p, int32_t prefix_len, Plan *pl) {
    size_t alone_bytes;
    const svpa_status s = svpa_attn_workspace_size(p, &alone_bytes);
    if (s != SVPA_OK) return s;
    if (prefix_len < 0 || prefix_len % kBlockSize != 0 || prefix_len / kBlockSize > p->num_blocks)
        return SVPA_ERR_INVALID_ARG;
    if (p->kv_dtype != SVPA_KV_BF16 || p->variant == 1 || p->batch > 65535 || p->num_kv_heads > 65535 ||
        (long long)p->num_blocks * p->num_kv_heads > 0x7fffffff ||
        p->max_blocks_per_seq > (0x7fffffff - 4096) / kBlockSize)
        return SVPA_ERR_UNSUPPORTED;
    const int G = p->num_q_heads / p->num_kv_heads;
    const long long T = (long long)p->batch * p->n_q;
    pl->tpt = kMaxRows / G;
    pl->pairs = (int)ceil_div(T, 2 * pl->tpt);
    const int slots = sm_count();
    const long long own = (long long)p->batch * p->num_kv_heads;
    const int pb = (int)ceil_div(prefix_len, 8 * kBlockSize);
    const int sb = std::max(1, (int)ceil_div(p->max_blocks_per_seq, 8) - pb);  // own blocks at most
    const long long tiles = (long long)pl->pairs * p->num_kv_heads;
    // Sharing pays when reading the prefix for each sequence costs more than
    // reading it for 256 query rows at a time and joining the two parts.  Per
    // sequence and kv head, in thousands of cycles (traces of small and large
    // cases): 1.75 a block alone, against its share of a prefix unit (3 a block
    // and 8 besides) and 2 for joining.  Against svpa_paged_verify_attn, 64
    // sequences of up to 400 tokens more, 32/8 heads: 1 token behind 64: 23.4 us
    // alone, 33.7 shared; behind 1024: 66.9 and 40.8; 6 drafts behind 256: 34.5
    // and 36.6; behind 512: 44.5 and 40.4; trees of 29 nodes, 116 rows of a
    // 128-row tile as they are, behind 800: 61.6 and 64.6; behind 2048: 112 and
    // 90.  Over 138 such cases the rule is 4% behind the better side on average
    // and 1.65 times at worst (8 x 1 tokens of 64/8 heads behind 128: 22.6 us
    // alone, 13.7 shared).  The batch has no part in it: for one sequence sharing
    // splits the prefix over SMs (32/8 heads, 1 token behind 1024: 27.3 us alone,
    // 15.6 shared; 32/32 heads: 15.4 and 17.9).
    const double rows = (double)p->n_q * G;
    pl->shared = rows / 256. * (3. * pb + 8.) + 2. < 1.75 * pb;
    if (!pl->shared) {
        pl->bytes = alone_bytes;
        return SVPA_OK;
    }
    // Splits of the prefix: rounds of units over the SMs times a unit's length
    // (3 a block for a pair of tiles, 1.5 for one; 8 besides), and one more for
    // each split that an own unit joins.
    const double block = T > pl->tpt ? 3.0 : 1.5;
    double best = 0.;
    pl->p_splits = 0;
    for (int sp = 1; sp <= std::min(kMaxSplits, std::max(1, pb / 2)); ++sp) {
        const double cost = (double)ceil_div(tiles * sp, slots) * ((double)ceil_div(pb, sp) * block + 8.) +
                            (double)ceil_div(own, slots) * sp;
        if (pl->p_splits == 0 || cost < best) {
            best = cost;
            pl->p_splits = sp;
        }
    }
    if (tiles * pl->p_splits > 0x7fffffff) return SVPA_ERR_UNSUPPORTED;
    pl->p_units = (int)(tiles * pl->p_splits);
    // the sequences' own parts: split when they alone leave SMs idle
    pl->s_splits = 1;
    if (own > 0 && own < slots)
        pl->s_splits = (int)std::max<long long>(1, std::min<long long>({slots / own, sb / 8, (long long)kMaxSplits}));
    // units of different lengths on every SM: longest first
    pl->ordered = pl->s_splits == 1 && p->batch > 1 && p->batch <= kMaxOrderedSeqs && own > slots;
    return layout(pl, pl->p_units + own * pl->s_splits, T, p->num_kv_heads, p->head_dim, p->batch);
}

void fill(PackedArgs &a, const Plan &pl, void *workspace) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.sched = reinterpret_cast<int32_t *>(ws);
    a.member = pl.s_splits > 1 ? reinterpret_cast<int32_t *>(ws + pl.off_member) : nullptr;
    a.part_ml = reinterpret_cast<float2 *>(ws + pl.off_ml);
    a.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    a.tpt = pl.tpt;
    a.tiles = pl.tiles;
    a.pairs = pl.pairs;
    a.p_units = pl.p_units;
    a.p_splits = pl.p_splits;
    a.s_splits = pl.s_splits;
    a.total_units = pl.total_units;
}

svpa_status launch(const PackedMaps &maps, const PackedArgs &a, int D, cudaStream_t st) {
    cudaError_t e = launch_packed_attn(maps, a, D, std::min(sm_count(), a.total_units), st);
    if (e == cudaSuccess && a.s_splits > 1) e = launch_packed_combine(a, D, st);
    return from_cuda(e);
}

}  // namespace

extern "C" {

svpa_status svpa_paged_prompt_attn_workspace_size(const svpa_prompt_params *p, size_t *bytes) {
    if (!bytes) return SVPA_ERR_INVALID_ARG;
    Plan pl;
    const svpa_status s = plan_prompt(p, &pl);
    if (s == SVPA_OK) *bytes = pl.bytes;
    return s;
}

svpa_status svpa_paged_prompt_attn(const svpa_prompt_params *p, const void *q, const void *k_pool,
                                   const void *v_pool, const int32_t *block_table, const int32_t *cu_seqlens,
                                   const int32_t *kv_lens, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_paged_prompt_attn");
    Plan pl;
    const svpa_status s = plan_prompt(p, &pl);
    if (s != SVPA_OK) return s;
    if (p->batch == 0 || p->total_q == 0) return SVPA_OK;
    if (!q || !k_pool || !v_pool || !block_table || !cu_seqlens || !kv_lens || !out || !error_flag)
        return SVPA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return SVPA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SVPA_ERR_WORKSPACE;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return SVPA_ERR_CUDA;
    const int G = p->num_q_heads / p->num_kv_heads, D = p->head_dim;
    const long long tiles = (long long)p->num_blocks * p->num_kv_heads;
    const long long stride = p->q_stride ? p->q_stride : (long long)p->num_q_heads * D;
    PackedMaps maps;
    if (!encode_pages(enc, &maps.k, k_pool, D, tiles) || !encode_pages(enc, &maps.v, v_pool, D, tiles) ||
        !encode_queries(enc, maps.qt, q, D, p->num_q_heads, G, p->total_q, stride, pl.tpt))
        return SVPA_ERR_CUDA;
    maps.qs[0] = maps.qt[0];
    maps.qs[1] = maps.qt[1];
    PackedArgs a;
    memset(&a, 0, sizeof a);
    fill(a, pl, workspace);
    a.block_table = block_table;
    a.cu = cu_seqlens;
    a.lens = kv_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.err = error_flag;
    a.B = p->batch;
    a.T = p->total_q;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.G = G;
    a.max_blocks = p->max_blocks_per_seq;
    a.num_blocks = p->num_blocks;
    a.scale_log2 = p->sm_scale * 1.4426950408889634f;
    return launch(maps, a, D, static_cast<cudaStream_t>(stream));
}

svpa_status svpa_prefix_verify_attn_workspace_size(const svpa_attn_params *p, int32_t prefix_len, size_t *bytes) {
    if (!bytes) return SVPA_ERR_INVALID_ARG;
    Plan pl;
    const svpa_status s = plan_prefix(p, prefix_len, &pl);
    if (s == SVPA_OK) *bytes = pl.bytes;
    return s;
}

svpa_status svpa_prefix_verify_attn(const svpa_attn_params *p, const void *q, const void *k_pool, const void *v_pool,
                                    const int32_t *prefix_blocks, int32_t prefix_len, const int32_t *block_table,
                                    const int32_t *context_lens, const uint64_t *ancestor_mask, void *out, float *lse,
                                    void *workspace, size_t workspace_bytes, int32_t *error_flag, void *stream) {
    svpa::NvtxRange nvtx_range("svpa_prefix_verify_attn");
    Plan pl;
    svpa_status s = plan_prefix(p, prefix_len, &pl);
    if (s != SVPA_OK) return s;
    if (p->batch == 0) return SVPA_OK;
    s = check_attn_call(p, q, k_pool, v_pool, nullptr, nullptr, block_table, context_lens, ancestor_mask, out,
                        error_flag);
    if (s != SVPA_OK) return s;
    if (prefix_len > 0 && !prefix_blocks) return SVPA_ERR_INVALID_ARG;
    if (!pl.shared)  // not worth sharing: every sequence reads its whole history itself
        return svpa_paged_verify_attn(p, q, k_pool, v_pool, nullptr, nullptr, block_table, context_lens, ancestor_mask,
                                      out, lse, workspace, workspace_bytes, error_flag, stream);
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SVPA_ERR_WORKSPACE;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return SVPA_ERR_CUDA;
    const int G = p->num_q_heads / p->num_kv_heads, D = p->head_dim;
    const long long tiles = (long long)p->num_blocks * p->num_kv_heads;
    const long long T = (long long)p->batch * p->n_q, stride = (long long)p->num_q_heads * D;
    PackedMaps maps;
    if (!encode_pages(enc, &maps.k, k_pool, D, tiles) || !encode_pages(enc, &maps.v, v_pool, D, tiles) ||
        !encode_queries(enc, maps.qt, q, D, p->num_q_heads, G, T, stride, pl.tpt) ||
        !encode_queries(enc, maps.qs, q, D, p->num_q_heads, G, T, stride, p->n_q))
        return SVPA_ERR_CUDA;
    PackedArgs a;
    memset(&a, 0, sizeof a);
    fill(a, pl, workspace);
    a.block_table = block_table;
    a.lens = context_lens;
    a.prefix_blocks = prefix_blocks;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.err = error_flag;
    a.verify = 1;
    a.B = p->batch;
    a.T = (int)T;
    a.Hq = p->num_q_heads;
    a.Hkv = p->num_kv_heads;
    a.G = G;
    a.n_q = p->n_q;
    a.max_blocks = p->max_blocks_per_seq;
    a.num_blocks = p->num_blocks;
    a.prefix_pages = prefix_len / kBlockSize;
    a.scale_log2 = p->sm_scale * 1.4426950408889634f;
    for (int j = 0; j < p->n_q; ++j)
        a.anc[j] = ancestor_mask ? ancestor_mask[j] : ((j == 63) ? ~0ull : ((1ull << (j + 1)) - 1ull));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.ordered) {
        int32_t *order = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + pl.off_member);
        const cudaError_t e = launch_seq_order(context_lens, p->batch, order, st);
        if (e != cudaSuccess) return from_cuda(e);
        a.order = order;
    }
    return launch(maps, a, D, st);
}

}  // extern "C"
