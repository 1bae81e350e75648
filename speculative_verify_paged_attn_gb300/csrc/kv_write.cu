// kv_write.cu -- packed K/V rows scattered into their pages through a slot map.
//
// "The Sub-Millisecond Speculative Decoding Meltdown", "Custom FP8 Quantized
// Memory Block Layout" and its implementation checklist (E4M3 pages, scales
// for each 64-element tile).  Row t of K and of V (Hkv x D values) goes to slot
// s = slot_map[t]: page s / 16, row s % 16 of every kv head's tile.
//
// Bytes only: each row is read once and written once.  A warp takes 128
// 16-byte words of one row, four per lane, so that its loads are in flight
// together; consecutive rows fill consecutive rows of a page.  FP8: eight lanes
// hold a 64-value tile, its scale is amax / 448 (1 for a tile of zeros) and its
// codes the values over the scale, each rounded once.  32768 rows of 8 x 128:
// bf16 42 us, 95% of the measured copy rate; FP8 55 us against a floor of 31,
// bound by the instructions of the quotients and conversions (75% of the issue
// slots taken, the ALU pipe 62% busy, DRAM 34%).
#include "admit.h"
#include "svpa_device.cuh"

namespace svpa {

namespace {

constexpr int kThreads = 256;
constexpr int kWords = 128;  // 16-byte words of a row one warp takes

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four fp32 values to E4M3 (nearest even, saturating at +-448).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// v / sc, correctly rounded, from inv = 1 / sc correctly rounded (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): the remainder of v * inv comes from one fused multiply-add, and adding
// its share rounds once.  Of the 128 x 128 pairs of significands (v, and the
// scale of a maximum), the remainder is rounded itself in 35, and the result is
// the correctly rounded quotient in all (enumerated in rationals).  Holds for a
// scale whose significand is not all ones and remainders that do not underflow;
// a quotient too small for the latter (below 2^-10 for sc >= 2^-89) has the code
// 0 either way.  Three instructions
// for the IEEE division's dozen: eight of those per 16 bytes made the kernel
// bound by instructions.
__device__ __forceinline__ float over_scale(float v, float sc, float inv) {
    const float q = __fmul_rn(v, inv);
    return __fmaf_rn(__fmaf_rn(-q, sc, v), inv, q);
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteArgs a) {
    const int lane = threadIdx.x & 31;
    const int wpr = a.Hkv * (a.D / 8);  // words per row
    const int chunks = (wpr + kWords - 1) / kWords;
    const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= 2LL * a.T * chunks) return;
    const int t = (int)(item / (2 * chunks)), rest = (int)(item - (long long)t * 2 * chunks);
    const int kv = rest / chunks, c0 = (rest - kv * chunks) * kWords;
    const uint4 *src = reinterpret_cast<const uint4 *>(kv ? a.v + t * a.v_stride : a.k + t * a.k_stride);
    const int slot = __ldg(a.slot_map + t);
    uint4 x[kWords / 32];
#pragma unroll
    for (int i = 0; i < kWords / 32; ++i) {
        const int w = c0 + lane + 32 * i;
        x[i] = w < wpr ? __ldcs(src + w) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (slot < 0) return;  // a padding row
    const int blk = slot / kBlockSize, at = slot % kBlockSize;
    if (blk >= a.num_blocks) {
        if (rest == 0 && lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
        return;
    }
    const int wph = a.D / 8;  // words per head
    uint8_t *pool = kv ? a.v_pool : a.k_pool;
#pragma unroll
    for (int i = 0; i < kWords / 32; ++i) {
        const int w = c0 + lane + 32 * i;
        const int h = w / wph, c = w - h * wph;
        const size_t row = ((size_t)blk * a.Hkv + h) * kBlockSize + at;
        if (!FP8) {
            if (w < wpr) reinterpret_cast<uint4 *>(pool)[row * wph + c] = x[i];
            continue;
        }
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(lo_f32(u[j])), fabsf(hi_f32(u[j]))));
        // a tile is eight consecutive lanes (wpr and wph are multiples of 8)
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (w >= wpr) continue;
        const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        const float inv = __frcp_rn(sc);
        float f[8];
        const bool plain = sc >= 0x1p-89f && sc < 0x1p127f && (__float_as_uint(sc) & 0x7fffffu) != 0x7fffffu;
        if (plain) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = over_scale(lo_f32(u[j]), sc, inv);
                f[2 * j + 1] = over_scale(hi_f32(u[j]), sc, inv);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __fdiv_rn(lo_f32(u[j]), sc);
                f[2 * j + 1] = __fdiv_rn(hi_f32(u[j]), sc);
            }
        }
        uint2 codes;
        codes.x = to_e4m3x4(f[0], f[1], f[2], f[3]);
        codes.y = to_e4m3x4(f[4], f[5], f[6], f[7]);
        reinterpret_cast<uint2 *>(pool)[row * wph + c] = codes;
        if ((c & 7) == 0) (kv ? a.v_scale : a.k_scale)[row * (a.D / 64) + c / 8] = sc;
    }
}

}  // namespace

cudaError_t launch_kv_write(const WriteArgs &a, cudaStream_t stream) {
    const int wpr = a.Hkv * (a.D / 8);
    const long long items = 2LL * a.T * ((wpr + kWords - 1) / kWords);
    const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
    if (a.fp8) write_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else write_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace svpa
