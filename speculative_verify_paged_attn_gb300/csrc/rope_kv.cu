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
// Each row is read once and written once.  A lane holds eight elements (16
// bytes), a head is D / 8 lanes, and a warp takes up to four words a lane of one
// token's queries, keys or values, all in flight together; a pair's other half
// comes by a shuffle.  The token's cosines and sines are read once for the
// warp's heads.  8192 tokens of 64 + 8 heads of 128: 55.6 us, 81% of the copy rate.
// No unit is saturated (issue slots 68%, ALU 49%, a third of the warps resident):
// an issue waits as long for memory as for shuffles.
#include "fp4.cuh"
#include "rope_kv.h"

namespace svpa {

namespace {

constexpr int kThreads = 256;
constexpr int kWords = 4;  // 16-byte words a lane takes (few tokens: 1 or 2)

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

// One word (eight elements) of a query: x' = r (x wc + o ws), with o the other
// halves of its pairs and the weights and the sines' signs in wc and ws.
template <int D>
__device__ __forceinline__ uint4 turn_query(const uint4 &x, const float (&wc)[8], const float (&ws)[8], bool norm,
                                            float eps, int mate, bool turns, bool interleaved) {
    float f[8], o[8];
    unpack8(x, f);
    float r = 1.f;
    if (norm) {  // the sum in any order: queries are rounded to bf16 alone
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
#pragma unroll
        for (int k = 1; k < D / 8; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        r = rsqrtf(sum * (1.f / D) + eps);
    }
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = f[j ^ 1];
    } else {
        uint4 y;
        y.x = __shfl_sync(0xffffffffu, x.x, mate), y.y = __shfl_sync(0xffffffffu, x.y, mate);
        y.z = __shfl_sync(0xffffffffu, x.z, mate), y.w = __shfl_sync(0xffffffffu, x.w, mate);
        unpack8(y, o);
    }
    if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = r * fmaf(o[j], ws[j], f[j] * wc[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = r * (f[j] * wc[j]);
    }
    return pack8(f);
}

// ... of a key, each operation rounded by itself: x r w, then the turn.
template <int D>
__device__ __forceinline__ uint4 turn_key(const uint4 &x, const float (&wt)[8], const float (&cs)[8],
                                          const float (&sn)[8], bool norm, float eps, int mate, bool turns, bool low,
                                          bool interleaved, int lane) {
    float f[8], o[8];
    unpack8(x, f);
    if (norm) {
        const float r = rsqrtf(ordered_squares<D>(f, lane) * (1.f / D) + eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * r * wt[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = interleaved ? f[j ^ 1] : __shfl_sync(0xffffffffu, f[j], mate);
    if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // the first of a pair less, the second more
            f[j] = (interleaved ? (j & 1) == 0 : low) ? f[j] * cs[j] - o[j] * sn[j] : f[j] * cs[j] + o[j] * sn[j];
        }
    }
    return pack8(f);
}

// A token's queries, keys and values are parts of kChunk heads; 1 << split_log
// warps of each of gridDim.y CTAs share them.
template <Pages P, int D, int W>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kLanes = D / 8;              // of a head
    constexpr int kHeads = 32 / kLanes;        // a warp holds at a time
    constexpr int kChunk = kHeads * W;    // heads a warp takes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long token = (long long)blockIdx.x * ((kThreads / 32) >> a.split_log) + (warp >> a.split_log);
    if (token >= a.T) return;
    const int t = (int)token, c = lane % kLanes;
    int slot = 0, pos = 0;
    if constexpr (P != Pages::kRows) slot = __ldg(a.slot_map + t);
    if (a.R > 0) pos = __ldg(a.positions + t);
    const int qc = (a.Hq + kChunk - 1) / kChunk, kc = (a.Hkv + kChunk - 1) / kChunk;
    const int parts = qc + (P == Pages::kRows ? 1 : 2) * kc;
    const int stride = (int)gridDim.y << a.split_log;
    int part = (warp & ((1 << a.split_log) - 1)) + ((int)blockIdx.y << a.split_log);
    auto fetch = [&](int at, uint4 (&x)[W]) {
        const int kind = at < qc ? 0 : at < qc + kc ? 1 : 2;
        const int heads = kind == 0 ? a.Hq : a.Hkv, begin = kind == 0 ? 0 : kind == 1 ? qc : qc + kc;
        const int h0 = (at - begin) * kChunk + lane / kLanes;
        const uint16_t *row = kind == 0   ? a.q + t * a.q_stride
                              : kind == 1 ? a.k + t * a.k_stride
                                          : a.v + t * a.v_stride;
        const uint16_t *src = row + h0 * D + c * 8;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h0 + i * kHeads < heads) x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + i * kHeads * D));
        }
    };
    uint4 x[W];
    if (part < parts) fetch(part, x);
    if constexpr (P != Pages::kRows) {
        if (slot < 0) return;  // a padding row
        if (slot / kBlockSize >= a.num_blocks) {
            if (part == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
            return;
        }
    }
    if (a.R > 0 && (pos < 0 || pos >= a.max_position)) {
        if (part == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        return;
    }
    // the angles of this lane's elements, and the lane that holds the other half of
    // its pairs
    const bool turns = 8 * c < a.R, low = c < a.R / 16, interleaved = a.interleaved;
    const int mate = turns && !interleaved ? lane + (low ? a.R / 16 : -(a.R / 16)) : lane;
    // (loaded for the queries and again for the keys: registers)
    auto angles = [&](float (&cs)[8], float (&sn)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cs[j] = 1.f, sn[j] = 0.f;
        if (!turns) return;
        const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (long long)pos * a.R);
        const int half = a.R / 8;  // float4 of the cosines
        const int at = interleaved ? c : 2 * (low ? c : c - a.R / 16);
        const float4 u = __ldg(row + at), w = __ldg(row + half + at);
        if (interleaved) {
            cs[0] = cs[1] = u.x, cs[2] = cs[3] = u.y, cs[4] = cs[5] = u.z, cs[6] = cs[7] = u.w;
            sn[0] = sn[1] = w.x, sn[2] = sn[3] = w.y, sn[4] = sn[5] = w.z, sn[6] = sn[7] = w.w;
        } else {
            const float4 u2 = __ldg(row + at + 1), w2 = __ldg(row + half + at + 1);
            cs[0] = u.x, cs[1] = u.y, cs[2] = u.z, cs[3] = u.w, cs[4] = u2.x, cs[5] = u2.y, cs[6] = u2.z, cs[7] = u2.w;
            sn[0] = w.x, sn[1] = w.y, sn[2] = w.z, sn[3] = w.w, sn[4] = w2.x, sn[5] = w2.y, sn[6] = w2.z, sn[7] = w2.w;
        }
    };
    if (part < qc) {
        // queries: the weights go into the angles
        float wc[8], ws[8];
        angles(wc, ws);
        const uint4 *wq = reinterpret_cast<const uint4 *>(a.q_weight);
        float wt[8], wo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wt[j] = wo[j] = 1.f;
        if (wq) {
            unpack8(__ldg(wq + c), wt);
            unpack8(__ldg(wq + mate % kLanes), wo);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            wc[j] *= wt[j];
            const float s = (interleaved ? wt[j ^ 1] : wo[j]) * ws[j];
            ws[j] = (interleaved ? (j & 1) == 0 : low) ? -s : s;
        }
#pragma unroll 1
        for (; part < qc; part += stride) {
            const int h0 = part * kChunk + lane / kLanes;
            uint16_t *dst = a.q_out + t * a.q_out_stride + h0 * D + c * 8;
            uint4 ahead[W];
            if (part + stride < parts) fetch(part + stride, ahead);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (part * kChunk + i * kHeads >= a.Hq) break;  // the same for the whole warp
                const uint4 y = turn_query<D>(x[i], wc, ws, wq != nullptr, a.eps, mate, turns, interleaved);
                if (h0 + i * kHeads < a.Hq) *reinterpret_cast<uint4 *>(dst + i * kHeads * D) = y;
            }
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = ahead[i];
        }
    }
    const long long tile = (long long)(slot / kBlockSize) * a.Hkv;
    if (part < qc + kc) {
        float wt[8], cs[8], sn[8];
        angles(cs, sn);
        if (a.k_weight) unpack8(__ldg(reinterpret_cast<const uint4 *>(a.k_weight) + c), wt);
#pragma unroll 1
        for (; part < qc + kc; part += stride) {
            const int h0 = (part - qc) * kChunk + lane / kLanes;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if ((part - qc) * kChunk + i * kHeads >= a.Hkv) break;
                const int h = h0 + i * kHeads;
                const uint4 y = turn_key<D>(x[i], wt, cs, sn, a.k_weight != nullptr, a.eps, mate, turns, low,
                                            interleaved, lane);
                if constexpr (P == Pages::kRows) {
                    if (h < a.Hkv) reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride + (long long)h * D)[c] = y;
                } else {
                    store_row<P, D>(y, h < a.Hkv, h, c, a.Hkv, tile, slot % kBlockSize, a.k_pool, a.k_scale, a.k_factor,
                                    a.err);
                }
            }
            if (part + stride < parts) fetch(part + stride, x);
        }
    }
    if constexpr (P != Pages::kRows) {
#pragma unroll 1
        for (; part < parts; part += stride) {
            const int h0 = (part - qc - kc) * kChunk + lane / kLanes;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if ((part - qc - kc) * kChunk + i * kHeads >= a.Hkv) break;
                const int h = h0 + i * kHeads;
                store_row<P, D>(x[i], h < a.Hkv, h, c, a.Hkv, tile, slot % kBlockSize, a.v_pool, a.v_scale, a.v_factor,
                                a.err);
            }
            if (part + stride < parts) fetch(part + stride, x);
        }
    }
}

// Row t of the pages, slot_map[t], as bf16: one fp32 product with the scale or the
// factor, then one rounding.  A lane takes W groups at a time.
template <Pages P, int W>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long token = (long long)blockIdx.x * ((kThreads / 32) >> a.split_log) + (warp >> a.split_log);
    if (token >= a.T) return;
    const int t = (int)token;
    const int slot = __ldg(a.slot_map + t);
    if (slot < 0) return;  // a padding row
    const int blk = slot / kBlockSize, at = slot % kBlockSize;
    int part = warp & ((1 << a.split_log) - 1);
    if (blk >= a.num_blocks) {
        if (part == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
        return;
    }
    const long long tile0 = (long long)blk * a.Hkv;
    if constexpr (P == Pages::kFp4) {
        // a lane takes groups of 16 elements, K's and V's: eight bytes of codes, a
        // scale, 32 bytes out
        const int gph = a.D / 16, gpr = a.Hkv * gph;
#pragma unroll 1
        for (; part * 32 * W < 2 * gpr; part += 1 << a.split_log) {
            const int c0 = part * 32 * W + lane;
            uint2 codes[W];
            uint32_t sc[W];
            float f[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int u = c0 + 32 * i, kv = u >= gpr, w = kv ? u - gpr : u;
                if (u >= 2 * gpr) break;
                const int h = gph == 1 ? w : (int)__umulhi((unsigned)w, a.magic), g = w - h * gph;
                const uint8_t *page = (kv ? a.v_pool : a.k_pool) + (tile0 + h) * fp4_tile_bytes(a.D);
                codes[i] = __ldg(reinterpret_cast<const uint2 *>(page + at * (a.D / 2)) + g);
                sc[i] = __ldg(page + fp4_code_bytes(a.D) + at * (a.D / 16) + g);
                f[i] = fp4_factor(kv ? a.v_factor : a.k_factor, h, a.err);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int u = c0 + 32 * i, kv = u >= gpr, w = kv ? u - gpr : u;
                if (u >= 2 * gpr) break;
                uint32_t p[8], out[8];
                uint32_t half[4];
                const uint32_t s = e4m3x2_to_f16x2(sc[i] * 0x101u);
                e2m1x8_to_f16(codes[i].x, half);
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = mul_f16x2(half[j], s);
                e2m1x8_to_f16(codes[i].y, half);
#pragma unroll
                for (int j = 0; j < 4; ++j) p[4 + j] = mul_f16x2(half[j], s);
                // code times scale is exact in f16, then one product with the factor
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = f16x2_to_float2(p[j]);
                    out[j] = pack_bf16x2(v.x * f[i], v.y * f[i]);
                }
                uint8_t *to = reinterpret_cast<uint8_t *>(kv ? a.v + t * a.v_stride : a.k + t * a.k_stride) + 32LL * w;
                if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(out[0]),
                                 "r"(out[1]), "r"(out[2]), "r"(out[3]), "r"(out[4]), "r"(out[5]), "r"(out[6]),
                                 "r"(out[7])
                                 : "memory");
                } else {
                    reinterpret_cast<uint4 *>(to)[0] = make_uint4(out[0], out[1], out[2], out[3]);
                    reinterpret_cast<uint4 *>(to)[1] = make_uint4(out[4], out[5], out[6], out[7]);
                }
            }
        }
    } else {
        const int wph = a.D / 8, wpr = a.Hkv * wph;  // 16-byte words of a head and of a row
        const int chunks = (wpr + 32 * W - 1) / (32 * W);
#pragma unroll 1
        for (; part < 2 * chunks; part += 1 << a.split_log) {
            const int kv = part >= chunks, c0 = (part - kv * chunks) * 32 * W + lane;
            const uint8_t *pool = kv ? a.v_pool : a.k_pool;
            uint4 *dst = reinterpret_cast<uint4 *>(kv ? a.v + t * a.v_stride : a.k + t * a.k_stride);
            uint4 raw[W];
            float scale[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int w = c0 + 32 * i, h = (int)((unsigned)w / (unsigned)wph), c = w - h * wph;
                if (w >= wpr) break;
                const long long row = (tile0 + h) * kBlockSize + at;
                if constexpr (P == Pages::kBf16) {
                    raw[i] = __ldg(reinterpret_cast<const uint4 *>(pool) + row * wph + c);
                } else {
                    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(pool) + row * wph + c);
                    raw[i].x = u.x, raw[i].y = u.y;
                    scale[i] = __ldg((kv ? a.v_scale : a.k_scale) + row * (wph / 8) + c / 8);
                }
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int w = c0 + 32 * i;
                if (w >= wpr) break;
                if constexpr (P == Pages::kFp8) {
                    const uint32_t p[4] = {e4m3x2_to_f16x2(raw[i].x & 0xffffu), e4m3x2_to_f16x2(raw[i].x >> 16),
                                           e4m3x2_to_f16x2(raw[i].y & 0xffffu), e4m3x2_to_f16x2(raw[i].y >> 16)};
                    float f[8];
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
    }
}

// Warps a token (log2): few enough that a warp's angles serve several parts, and
// enough warps for the GPU.  Queries and keys of 64 + 8 heads of 128, by 1, 2, 4
// and 8 warps a token: 8192 tokens 58.2, 55.4, 65.7 and 91.0 us (floor 45.2); 24
// tokens 12.6, 8.2, 6.0 and 4.7.  Into 4-bit pages, 16384 tokens: 136, 133, 177
// and 245 us (floor 93).
int split_log(long long tokens, int parts) {
    const long long want = 32LL * sm_count();
    int s = 0;
    while (s < 3 && (1 << s) < parts && (s == 0 || (tokens << s) < want)) ++s;
    return s;
}

unsigned grid_of(long long tokens, int split) {
    const long long per = (kThreads / 32) >> split;  // tokens of a CTA
    return (unsigned)((tokens + per - 1) / per);
}

// (the parts of a token, of W words a lane)
template <Pages P, int D, int W>
int parts_of(const RopeArgs &a) {
    constexpr int kChunk = 32 / (D / 8) * W;
    return (a.Hq + kChunk - 1) / kChunk + (P == Pages::kRows ? 1 : 2) * ((a.Hkv + kChunk - 1) / kChunk);
}

template <Pages P, int D, int W>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    const int parts = parts_of<P, D, W>(a);
    a.split_log = split_log(a.T, parts);
    // few tokens: more CTAs for each (up to 64 warps)
    const bool few = a.split_log == 3 && (long long)a.T * 8 < 32LL * sm_count();
    const unsigned more = few ? (unsigned)min((parts + 7) / 8, 8) : 1u;
    rope_kernel<P, D, W><<<dim3(grid_of(a.T, a.split_log), more), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// Words a lane: all of a token's loads at once, one or two words a lane, while the
// GPU has the warps for it.  64 + 8 heads of 128 by 1, 2 and 4: 24 tokens 2.5, 2.7
// and 3.2 us (4.7 in one CTA a token); 100 tokens 4.3, 3.3 and 3.9; 600 tokens 13.0,
// 9.8 and 8.7.  Into 4-bit pages: 57 tokens 3.4, 3.9 and 5.2 us (6.7 in one CTA a
// token), 200 tokens 6.8, 6.1 and 6.4, 1200 tokens 29.5, 21.5 and 22.6.
template <Pages P, int D>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
    if ((long long)a.T * parts_of<P, D, 1>(a) <= 16LL * sm_count()) return launch<P, D, 1>(a, stream);
    if ((long long)a.T * parts_of<P, D, 2>(a) <= 24LL * sm_count()) return launch<P, D, 2>(a, stream);
    return launch<P, D, kWords>(a, stream);
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

namespace {

template <Pages P, int W>
cudaError_t launch_read(ReadArgs a, cudaStream_t stream) {
    const int wpr = a.Hkv * (a.D / 8), chunks = (wpr + 32 * W - 1) / (32 * W);
    const int parts = P == Pages::kFp4 ? chunks : 2 * chunks;  // (of 32 and of 16 bytes out a lane)
    a.split_log = parts > 4 ? 3 : parts > 2 ? 2 : parts > 1 ? 1 : 0;
    // w / (D / 16) as a product's high word: exact for w (D / 16) < 2^32
    a.magic = a.D >= 32 ? (unsigned)(((1ull << 32) + a.D / 16 - 1) / (a.D / 16)) : 0u;
    read_kernel<P, W><<<grid_of(a.T, a.split_log), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs &a, Pages pages, cudaStream_t stream) {
    if (pages == Pages::kBf16) return launch_read<Pages::kBf16, kWords>(a, stream);
    if (pages == Pages::kFp8) return launch_read<Pages::kFp8, kWords>(a, stream);
    // A group a lane while all warps run at once, four then, and eight of long rows
    // of many tokens.  By 1, 4 and 8: 700 tokens of 8 heads of 128 2.4, 3.0 and 3.1
    // us; 65536 of them 80.4, 58.1 and 58.7 (floor 50.8); 16000 of 32 heads 65.1, 58.0
    // and 54.2 (floor 49.6), 600 of them 3.6, 3.9 and 4.7.
    const int wpr = a.Hkv * (a.D / 8);  // groups of a token's K and V
    const long long warps = (long long)a.T * ((wpr + 31) / 32);
    if (warps <= 64LL * sm_count()) return launch_read<Pages::kFp4, 1>(a, stream);
    if (wpr >= 256 && warps > 512LL * sm_count()) return launch_read<Pages::kFp4, 8>(a, stream);
    return launch_read<Pages::kFp4, kWords>(a, stream);
}

}  // namespace svpa
