// rope_kv.h -- arguments and launches of the norm and rotation of queries and
// keys, their write into pages, and the read of pages.
#pragma once

#include "svpa_internal.h"

namespace svpa {

// where keys (and values) go
enum class Pages { kRows, kBf16, kFp8, kFp4 };

struct RopeArgs {
    const uint16_t *q;  // bf16 bits
    const uint16_t *k;
    const uint16_t *v;          // pages only
    const int32_t *positions;
    const int32_t *slot_map;    // pages only
    const float *cos_sin;       // [max_position, R]
    const uint16_t *q_weight;   // [D] or null
    const uint16_t *k_weight;
    uint16_t *q_out;
    uint16_t *k_out;            // rows only
    uint8_t *k_pool;
    uint8_t *v_pool;
    float *k_scale;
    float *v_scale;
    const float *k_factor;
    const float *v_factor;
    int32_t *err;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    int32_t T, Hq, Hkv, R, interleaved, max_position, num_blocks;
    float eps;
    int32_t split_log;  // log2 of the warps a token (set by the launch)
};
cudaError_t launch_rope(const RopeArgs &a, int D, Pages pages, cudaStream_t stream);

struct ReadArgs {
    const int32_t *slot_map;
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const float *k_scale;
    const float *v_scale;
    const float *k_factor;
    const float *v_factor;
    uint16_t *k;
    uint16_t *v;
    int32_t *err;
    long long k_stride, v_stride;
    int32_t T, Hkv, D, num_blocks;
    int32_t split_log;  // as above
    uint32_t magic;     // ceil(2^32 / (D / 16)) (set by the launch)
};
cudaError_t launch_kv_read(const ReadArgs &a, Pages pages, cudaStream_t stream);

}  // namespace svpa
