// rope_kv.cu -- norms of queries and keys for each head and the position
// rotation in one pass, into rows or on the way into the pages; and pages read
// back into rows.
//
//   n = x / sqrt(mean(x^2) + eps) * w              (with a weight, over a head)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)   for the pairs (i, i + R/2)
//   or (2i, 2i + 1) of the first R elements, t = the angle of (position, i)
// All of it in fp32, one rounding to bf16; FP8 and 4-bit pages encode that bf16
// value, so that a row has the same codes whether it is rotated on the way into
// the pages or before.  Each operation on a key is rounded by itself and its sum
// of squares has one order (ordered_squares): a value next to the border of two
// codes moves by up to half of itself when its last fp32 bit does, so a key's
// codes are made reproducible by plain fp32 operations.  (This file is compiled
// without fused multiply-adds.)
//
// Bytes only: each row is read once and written once.  A lane holds eight
// elements (16 bytes), a head is D / 8 lanes, and a warp takes four words a
// lane of one token's queries, keys or values, all in flight together; a pair's
// other half comes by a shuffle.  The token's cosines and sines are read once
// for the warp's heads.
#include "fp4.cuh"
#include "rope_kv.h"

namespace svpa {

namespace {

constexpr int kThreads = 256;
constexpr int kWords = 4;  // 16-byte words a lane takes

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
    f[0] = bf16_lo(x.x), f[1] = bf16_hi(x.x), f[2] = bf16_lo(x.y), f[3] = bf16_hi(x.y);
    f[4] = bf16_lo(x.z), f[5] = bf16_hi(x.z), f[6] = bf16_lo(x.w), f[7] = bf16_hi(x.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// The sum of a head's squares in one fixed order: 32 partial sums, of the
// elements i, i + 32, i + 64, ... in turn, added in pairs of neighbours.
template <int D>
__device__ __forceinline__ float ordered_squares(const float (&f)[8], int lane) {
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float sq = f[j] * f[j];
        s[j] = sq;
        // (complete in a head's first four lanes)
#pragma unroll
        for (int m = 1; m < D / 32; ++m) s[j] += __shfl_down_sync(0xffffffffu, sq, 4 * m);
    }
    float sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    return __shfl_sync(0xffffffffu, sum, lane & ~(D / 8 - 1));
}

// One lane's eight bf16 values of head h, chunk c, into slot `slot` of the pages.
template <Pages P, int D>
__device__ __forceinline__ void store_row(const uint4 &x, bool live, int h, int c, int Hkv, long long tile, int at,
                                          uint8_t *pool, float *scales, const float *factor, int32_t *err) {
    if constexpr (P == Pages::kBf16) {
        if (live) reinterpret_cast<uint4 *>(pool)[((tile + h) * 16 + at) * (D / 8) + c] = x;
    } else if constexpr (P == Pages::kFp8) {
        // a scale for each 64 elements: eight consecutive lanes (as svpa_kv_write)
        float f[8], amax = 0.f;
        unpack8(x, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (!live) return;
        const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        uint16_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(code[i])
                : "f"(__fdiv_rn(f[2 * i + 1], sc)), "f"(__fdiv_rn(f[2 * i], sc)));
        const long long row = (tile + h) * 16 + at;
        reinterpret_cast<uint2 *>(pool)[row * (D / 8) + c] =
            make_uint2(code[0] | (uint32_t)code[1] << 16, code[2] | (uint32_t)code[3] << 16);
        if ((c & 7) == 0) scales[row * (D / 64) + c / 8] = sc;
    } else {
        // a scale for each 16 elements: a pair of lanes
        uint32_t amax = bf16_amax8(x);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (!live) return;
        if (amax > 0x7f7fu) raise_error(err, SVPA_DEVERR_BAD_VALUE);
        uint32_t scale;
        const uint32_t codes = fp4_encode8(x, amax, fp4_factor(factor, h, err), scale);
        uint8_t *page = pool + (tile + h) * fp4_tile_bytes(D);
        reinterpret_cast<uint32_t *>(page + at * (D / 2))[c] = codes;
        if ((c & 1) == 0) page[fp4_code_bytes(D) + at * (D / 16) + c / 2] = (uint8_t)scale;
    }
}

template <Pages P, int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kLanes = D / 8;              // of a head
    constexpr int kHeads = 32 / kLanes;        // a warp holds at a time
    constexpr int kChunk = kHeads * kWords;    // heads a warp takes
    const int lane = threadIdx.x & 31;
    const int qc = (a.Hq + kChunk - 1) / kChunk, kc = (a.Hkv + kChunk - 1) / kChunk;
    const int items = qc + (P == Pages::kRows ? 1 : 2) * kc;
    const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= (long long)a.T * items) return;
    const int t = (int)(item / items);
    int part = (int)(item - (long long)t * items);
    // queries, keys or values
    const int kind = part < qc ? 0 : part < qc + kc ? 1 : 2;
    part -= kind == 0 ? 0 : kind == 1 ? qc : qc + kc;
    const int heads = kind == 0 ? a.Hq : a.Hkv, h0 = part * kChunk + lane / kLanes, c = lane % kLanes;
    const uint16_t *src = kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
    uint4 x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int h = h0 + i * kHeads;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < heads) x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + (long long)h * D) + c);
    }
    int slot = 0;
    if constexpr (P != Pages::kRows) {
        slot = __ldg(a.slot_map + t);
        if (slot < 0) return;  // a padding row
        if (slot / kBlockSize >= a.num_blocks) {
            if (kind == 1 && part == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
            return;
        }
    }
    const bool turns = kind < 2 && 8 * c < a.R;
    float cs[8], sn[8];  // of this lane's elements (interleaved: of its four pairs)
    if (kind < 2 && a.R > 0) {
        const int pos = __ldg(a.positions + t);
        if (pos < 0 || pos >= a.max_position) {
            if (part == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            return;
        }
        if (turns) {
            const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (long long)pos * a.R);
            const int half = a.R / 8;  // float4 of the cosines
            const int at = a.interleaved ? c : 2 * (c < a.R / 16 ? c : c - a.R / 16);
            const float4 u = __ldg(row + at), w = __ldg(row + half + at);
            cs[0] = u.x, cs[1] = u.y, cs[2] = u.z, cs[3] = u.w;
            sn[0] = w.x, sn[1] = w.y, sn[2] = w.z, sn[3] = w.w;
            if (!a.interleaved) {
                const float4 u2 = __ldg(row + at + 1), w2 = __ldg(row + half + at + 1);
                cs[4] = u2.x, cs[5] = u2.y, cs[6] = u2.z, cs[7] = u2.w;
                sn[4] = w2.x, sn[5] = w2.y, sn[6] = w2.z, sn[7] = w2.w;
            }
        }
    }
    const uint16_t *weight = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    float wt[8];
    if (weight) unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + c), wt);
    // the lane that holds the other half of this one's pairs
    const int low = c < a.R / 16;
    const int mate = turns && !a.interleaved ? lane + (low ? a.R / 16 : -(a.R / 16)) : lane;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int h = h0 + i * kHeads;
        const bool live = h < heads;
        if (part * kChunk + i * kHeads >= heads) break;  // the same for the whole warp
        if (kind < 2) {
            float f[8];
            unpack8(x[i], f);
            if (weight) {
                float sum = 0.f;
                if (kind == 1) {
                    sum = ordered_squares<D>(f, lane);
                } else {  // any order: queries are rounded to bf16 alone
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                }
                const float r = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = f[j] * r * wt[j];
            }
            if (a.interleaved) {
                if (turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float u = f[2 * j], w = f[2 * j + 1];
                        f[2 * j] = u * cs[j] - w * sn[j];
                        f[2 * j + 1] = w * cs[j] + u * sn[j];
                    }
                }
            } else if (a.R > 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float o = __shfl_sync(0xffffffffu, f[j], mate);
                    if (turns) f[j] = low ? f[j] * cs[j] - o * sn[j] : f[j] * cs[j] + o * sn[j];
                }
            }
            x[i] = pack8(f);
        }
        if (kind == 0) {
            if (live) reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + (long long)h * D)[c] = x[i];
        } else if constexpr (P == Pages::kRows) {
            if (live) reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + (long long)h * D)[c] = x[i];
        } else {
            store_row<P, D>(x[i], live, h, c, a.Hkv, (long long)(slot / kBlockSize) * a.Hkv, slot % kBlockSize,
                            kind == 1 ? a.k_pool : a.v_pool, kind == 1 ? a.k_scale : a.v_scale,
                            kind == 1 ? a.k_factor : a.v_factor, a.err);
        }
    }
}

// Row t of the pages, slot_map[t], as bf16: each value rounded once.
template <Pages P>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    const int lane = threadIdx.x & 31;
    const int wph = a.D / 8, wpr = a.Hkv * wph;  // 16-byte words of a head and of a row
    const int chunks = (wpr + 32 * kWords - 1) / (32 * kWords);
    const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= 2LL * a.T * chunks) return;
    const int t = (int)(item / (2 * chunks)), rest = (int)(item - (long long)t * 2 * chunks);
    const int kv = rest / chunks, c0 = (rest - kv * chunks) * 32 * kWords;
    const int slot = __ldg(a.slot_map + t);
    if (slot < 0) return;  // a padding row
    const int blk = slot / kBlockSize, at = slot % kBlockSize;
    if (blk >= a.num_blocks) {
        if (rest == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
        return;
    }
    const uint8_t *pool = kv ? a.v_pool : a.k_pool;
    uint4 *dst = reinterpret_cast<uint4 *>(kv ? a.v + t * a.v_stride : a.k + t * a.k_stride);
    uint4 raw[kWords];
    float scale[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int w = c0 + lane + 32 * i, h = w / wph, c = w - h * wph;
        if (w >= wpr) break;
        const long long tile = (long long)blk * a.Hkv + h, row = tile * kBlockSize + at;
        if constexpr (P == Pages::kBf16) {
            raw[i] = __ldg(reinterpret_cast<const uint4 *>(pool) + row * wph + c);
        } else if constexpr (P == Pages::kFp8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(pool) + row * wph + c);
            raw[i].x = u.x, raw[i].y = u.y;
            scale[i] = __ldg((kv ? a.v_scale : a.k_scale) + row * (wph / 8) + c / 8);
        } else {
            const uint8_t *page = pool + tile * fp4_tile_bytes(a.D);
            raw[i].x = __ldg(reinterpret_cast<const uint32_t *>(page + at * (a.D / 2)) + c);
            raw[i].y = __ldg(page + fp4_code_bytes(a.D) + at * (a.D / 16) + c / 2);
            scale[i] = fp4_factor(kv ? a.v_factor : a.k_factor, h, a.err);
        }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int w = c0 + lane + 32 * i;
        if (w >= wpr) break;
        if constexpr (P != Pages::kBf16) {
            uint32_t p[4];
            float f[8];
            if constexpr (P == Pages::kFp8) {
                p[0] = e4m3x2_to_f16x2(raw[i].x & 0xffffu), p[1] = e4m3x2_to_f16x2(raw[i].x >> 16);
                p[2] = e4m3x2_to_f16x2(raw[i].y & 0xffffu), p[3] = e4m3x2_to_f16x2(raw[i].y >> 16);
            } else {
                // code times scale is exact in f16, then one product with the factor
                e2m1x8_to_f16(raw[i].x, p);
                const uint32_t s = e4m3x2_to_f16x2(raw[i].y * 0x101u);
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = mul_f16x2(p[j], s);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = f16x2_to_float2(p[j]);
                f[2 * j] = v.x * scale[i], f[2 * j + 1] = v.y * scale[i];
            }
            raw[i] = pack8(f);
        }
        dst[w] = raw[i];
    }
}

template <Pages P, int D>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
    constexpr int kChunk = 32 / (D / 8) * kWords;
    const int qc = (a.Hq + kChunk - 1) / kChunk, kc = (a.Hkv + kChunk - 1) / kChunk;
    const long long items = (long long)a.T * (qc + (P == Pages::kRows ? 1 : 2) * kc);
    const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
    rope_kernel<P, D><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <Pages P>
cudaError_t launch_d(const RopeArgs &a, int D, cudaStream_t stream) {
    return D == 64 ? launch<P, 64>(a, stream) : D == 128 ? launch<P, 128>(a, stream) : launch<P, 256>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int D, Pages pages, cudaStream_t stream) {
    switch (pages) {
        case Pages::kRows: return launch_d<Pages::kRows>(a, D, stream);
        case Pages::kBf16: return launch_d<Pages::kBf16>(a, D, stream);
        case Pages::kFp8: return launch_d<Pages::kFp8>(a, D, stream);
        default: return launch_d<Pages::kFp4>(a, D, stream);
    }
}

cudaError_t launch_kv_read(const ReadArgs &a, Pages pages, cudaStream_t stream) {
    const long long wpr = (long long)a.Hkv * (a.D / 8);
    const long long items = 2LL * a.T * ((wpr + 32 * kWords - 1) / (32 * kWords));
    const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
    if (pages == Pages::kBf16) read_kernel<Pages::kBf16><<<grid, kThreads, 0, stream>>>(a);
    else if (pages == Pages::kFp8) read_kernel<Pages::kFp8><<<grid, kThreads, 0, stream>>>(a);
    else read_kernel<Pages::kFp4><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace svpa
