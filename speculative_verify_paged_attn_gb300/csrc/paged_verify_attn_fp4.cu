// paged_verify_attn_fp4.cu -- paged verification attention over 4-bit pages.
//
// One CTA per (sequence, kv head): the pages in turn decoded into shared
// memory, scores and the running maximum and sum of each query row in fp32,
// the output in registers.
#include <math_constants.h>

#include "fp4.cuh"
#include "fp4_attn.h"

namespace svpa {

namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) fp4_attn_kernel(const __grid_constant__ Fp4AttnArgs a) {
    extern __shared__ float sm[];
    const int M = a.M, tid = threadIdx.x, b = blockIdx.y, h = blockIdx.x;
    float *sq = sm, *sk = sq + M * (D + 1), *sv = sk + 16 * (D + 1), *sp = sv + 16 * (D + 1);
    float *mx = sp + M * 17, *sum = mx + M, *alpha = sum + M;
    const int L = a.context_lens[b];
    const long long end = (long long)L + a.n_q;
    const int pages = (int)((end + 15) / 16);
    if (L < 0 || pages > a.max_blocks) {
        if (tid == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        return;
    }
    for (int i = tid; i < M * D; i += kThreads) {
        const int r = i / D, d = i % D;
        const float x =
            __bfloat162float(a.q[(((size_t)b * a.n_q + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G) * D + d]);
        if (!(fabsf(x) <= 3.4e38f)) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        sq[r * (D + 1) + d] = x;
    }
    for (int r = tid; r < M; r += kThreads) mx[r] = -CUDART_INF_F, sum[r] = 0.f;
    const float fk = fp4_factor(a.k_factor, h, a.err), fv = fp4_factor(a.v_factor, h, a.err);
    constexpr int kAcc = 128 * D / kThreads;
    float acc[kAcc];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = 0.f;
    for (int p = 0; p < pages; ++p) {
        int blk = a.block_table[(size_t)b * a.max_blocks + p];
        if (blk < 0 || blk >= a.num_blocks) {
            if (tid == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
            blk = 0;
        }
        __syncthreads();
        const size_t tile = ((size_t)blk * a.Hkv + h) * fp4_tile_bytes(D);
        for (int i = tid; i < 2 * 16 * D / 8; i += kThreads) {
            const int kv = i / (16 * D / 8), w = i % (16 * D / 8), s = w / (D / 8), c = w % (D / 8);
            const uint8_t *page = (kv ? a.v_pool : a.k_pool) + tile;
            uint32_t e[4];
            e2m1x8_to_f16(reinterpret_cast<const uint32_t *>(page + s * (D / 2))[c], e);
            const float sc = e4m3_value(page[fp4_code_bytes(D) + s * (D / 16) + c / 2]);
            float *dst = (kv ? sv : sk) + s * (D + 1) + 8 * c;
            const bool in = p * 16 + s < end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = f16x2_to_float2(e[j]);
                dst[2 * j] = in ? f.x * sc : 0.f;
                dst[2 * j + 1] = in ? f.y * sc : 0.f;
            }
        }
        __syncthreads();
        for (int i = tid; i < M * 16; i += kThreads) {
            const int r = i / 16, s = i % 16, at = p * 16 + s - L;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(sq[r * (D + 1) + d], sk[s * (D + 1) + d], dot);
            const bool seen = at < 0 || (at < a.n_q && (a.anc[r / a.G] >> at & 1));
            sp[r * 17 + s] = seen ? dot * (a.scale_log2 * fk) : -CUDART_INF_F;
        }
        __syncthreads();
        for (int r = tid; r < M; r += kThreads) {
            float top = mx[r];
            for (int s = 0; s < 16; ++s) top = fmaxf(top, sp[r * 17 + s]);
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            alpha[r] = ex2_approx(mx[r] - ref);
            float l = sum[r] * alpha[r];
            for (int s = 0; s < 16; ++s) {
                const float e = ex2_approx(sp[r * 17 + s] - ref);
                sp[r * 17 + s] = e;
                l += e;
            }
            mx[r] = top;
            sum[r] = l;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int r = (tid + i * kThreads) / D, d = tid % D;
            if (r >= M) break;
            float v = acc[i] * alpha[r];
            for (int s = 0; s < 16; ++s) v = fmaf(sp[r * 17 + s], sv[s * (D + 1) + d], v);
            acc[i] = v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAcc; ++i) {
        const int r = (tid + i * kThreads) / D, d = tid % D;
        if (r >= M) break;
        const size_t o = ((size_t)b * a.n_q + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G;
        a.out[o * D + d] = __float2bfloat16_rn(acc[i] * fv / sum[r]);
        if (d == 0 && a.lse) a.lse[o] = (mx[r] + __log2f(sum[r])) * 0.69314718055994530942f;
    }
}

template <int D>
cudaError_t launch(const Fp4AttnArgs &a, cudaStream_t st) {
    const int smem = (a.M * (D + 1) + 32 * (D + 1) + a.M * 20) * 4;
    const cudaError_t e =
        cudaFuncSetAttribute(fp4_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 << 10);
    if (e != cudaSuccess) return e;
    fp4_attn_kernel<D><<<dim3(a.Hkv, a.B), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_verify_attn_fp4(const Fp4AttnArgs &a, int D, cudaStream_t st) {
    return D == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace svpa
