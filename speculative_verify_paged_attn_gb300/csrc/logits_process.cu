// logits_process.cu -- penalties for repeated tokens, biases and grammar masks
// on the target's logits, before the samplers.
//
// Row i of sequence b, token v, with n(v) the times v was generated before row
// i (the history behind the prompt and the drafts on row i's path):
//   x = logit;  x = x > 0 ? x / r : x * r   if v is in the prompt or n(v) > 0
//   x -= f * n(v);  x -= p if n(v) > 0;  x += bias(v);  x = -inf if not allowed
// in this order, each step rounded to fp32.
//
// Bytes only: the logits read once, the results written once.  A CTA takes a
// slab of 4096 tokens of one sequence and all its rows.  It forms n(v) of the
// slab in shared memory from the sequence's history (read by every slab of the
// sequence, from L2) and marks biased tokens and drafts there, so the pass over
// the rows needs one word of shared memory per token, kept in registers for
// all rows; drafts, whose count differs from row to row, and biases take a slow
// path for the few tokens that are marked.
#include "admit.h"
#include "svpa_device.cuh"

namespace svpa {

namespace {

constexpr int kThreads = 256;
constexpr int kSlab = 4096;
constexpr int kMaxDrafts = kMaxNq;

// a token's word: times generated << 3 | biased << 2 | drafted << 1 | in the prompt
constexpr unsigned kInPrompt = 1, kDrafted = 2, kBiased = 4, kOnce = 8;

struct Shared {
    unsigned word[kSlab];
    int bias[kSlab];  // last entry of the bias list for the token
    int drafts[kMaxDrafts];
};

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) process_kernel(const __grid_constant__ ProcessArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sm = *reinterpret_cast<Shared *>(raw);
    const int b = blockIdx.y, v0 = blockIdx.x * kSlab, n = min(kSlab, a.V - v0);
    const bool marks = a.history || a.drafts || a.bias_tokens;
    if (marks) {
        for (int i = threadIdx.x; i < kSlab; i += kThreads) sm.word[i] = 0u;
        if (a.bias_tokens)
            for (int i = threadIdx.x; i < kSlab; i += kThreads) sm.bias[i] = -1;
        __syncthreads();
        if (a.history) {
            int hn = a.hist_lens[b], pn = a.prompt_lens ? a.prompt_lens[b] : 0;
            if (hn < 0 || hn > a.max_hist || pn < 0 || pn > hn) {
                if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                hn = min(max(hn, 0), a.max_hist);
                pn = min(max(pn, 0), hn);
            }
            const int32_t *h = a.history + (size_t)b * a.max_hist;
            for (int i = threadIdx.x; i < hn; i += kThreads) {
                const int v = h[i];
                const unsigned x = (unsigned)(v - v0);
                if (x < (unsigned)n) {
                    if (i < pn) atomicOr(&sm.word[x], kInPrompt);
                    else atomicAdd(&sm.word[x], kOnce);
                } else if (blockIdx.x == 0 && (v < 0 || v >= a.V)) {
                    raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                }
            }
        }
        if (a.drafts)
            for (int i = threadIdx.x; i < a.draft_stride; i += kThreads) {
                const int v = a.drafts[(size_t)b * a.draft_stride + i];
                bool used = false;  // an entry no row counts (a tree's root) may hold anything
                for (int j = 0; j < a.rows; ++j) used = used || ((a.path[j] >> i) & 1ull);
                sm.drafts[i] = v;
                const unsigned x = (unsigned)(v - v0);
                if (used && x < (unsigned)n) atomicOr(&sm.word[x], kDrafted);
                else if (used && blockIdx.x == 0 && (v < 0 || v >= a.V)) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            }
        if (a.bias_tokens) {
            const int lo = a.bias_offsets[b], hi = a.bias_offsets[b + 1];
            if (lo < 0 || hi < lo) {
                if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            } else {
                for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
                    const int v = a.bias_tokens[i];
                    const unsigned x = (unsigned)(v - v0);
                    if (x < (unsigned)n) {
                        atomicOr(&sm.word[x], kBiased);
                        atomicMax(&sm.bias[x], i);
                    } else if (blockIdx.x == 0 && (v < 0 || v >= a.V)) {
                        raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                    }
                }
            }
        }
        __syncthreads();
    }
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const bool penal = a.repetition || a.presence || a.frequency;
    const int words = (a.V + 31) / 32;

    auto process = [&](float x, unsigned w, int i, int j) -> float {
        if (w == 0u) return x;
        unsigned count = w / kOnce;
        if (w & kDrafted) {
            for (unsigned long long m = a.path[j]; m; m &= m - 1)
                count += sm.drafts[__ffsll((long long)m) - 1] == v0 + i;
        }
        if (penal) {
            if ((w & kInPrompt) || count) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
            if (count) x = __fadd_rn(__fadd_rn(x, -__fmul_rn(freq, (float)count)), -pres);
        }
        if (w & kBiased) x = __fadd_rn(x, a.bias_values[sm.bias[i]]);
        return x;
    };

    const T *in = static_cast<const T *>(a.in) + ((size_t)b * a.rows) * a.V + v0;
    float *out = a.out + ((size_t)b * a.rows) * a.V + v0;
    const uint32_t *mask = a.mask ? a.mask + (size_t)b * a.rows * words + v0 / 32 : nullptr;
    if (VEC) {
        for (int i = threadIdx.x * 4; i < n; i += kThreads * 4) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (marks) w = *reinterpret_cast<const uint4 *>(&sm.word[i]);
            const bool any = (w.x | w.y | w.z | w.w) != 0u;
            for (int j0 = 0; j0 < a.rows; j0 += 4) {
                float4 x[4];
                uint32_t ok[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (j0 + k >= a.rows) break;
                    x[k] = load4(in + (size_t)(j0 + k) * a.V + i);
                    ok[k] = mask ? mask[(size_t)(j0 + k) * words + i / 32] >> (i & 31) : 15u;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (j0 + k >= a.rows) break;
                    if (any) {
                        x[k].x = process(x[k].x, w.x, i, j0 + k);
                        x[k].y = process(x[k].y, w.y, i + 1, j0 + k);
                        x[k].z = process(x[k].z, w.z, i + 2, j0 + k);
                        x[k].w = process(x[k].w, w.w, i + 3, j0 + k);
                    }
                    const float ninf = __int_as_float(0xff800000);
                    if (!(ok[k] & 1u)) x[k].x = ninf;
                    if (!(ok[k] & 2u)) x[k].y = ninf;
                    if (!(ok[k] & 4u)) x[k].z = ninf;
                    if (!(ok[k] & 8u)) x[k].w = ninf;
                    *reinterpret_cast<float4 *>(out + (size_t)(j0 + k) * a.V + i) = x[k];
                }
            }
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const unsigned w = marks ? sm.word[i] : 0u;
            for (int j = 0; j < a.rows; ++j) {
                float x = process(load1(in + (size_t)j * a.V + i), w, i, j);
                if (mask && !((mask[(size_t)j * words + i / 32] >> (i & 31)) & 1u)) x = __int_as_float(0xff800000);
                out[(size_t)j * a.V + i] = x;
            }
        }
    }
}

template <typename T>
cudaError_t launch_t(const ProcessArgs &a, cudaStream_t st) {
    const bool vec = a.V % 4 == 0 && (reinterpret_cast<uintptr_t>(a.in) & (4 * sizeof(T) - 1)) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
    const dim3 grid((a.V + kSlab - 1) / kSlab, a.B);
    if (vec) process_kernel<T, true><<<grid, kThreads, sizeof(Shared), st>>>(a);
    else process_kernel<T, false><<<grid, kThreads, sizeof(Shared), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits_process(const ProcessArgs &a, cudaStream_t st) {
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace svpa
