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
// slab of tokens of one sequence and its rows (or one of them, where there are
// few CTAs).  It forms n(v) of the slab in shared memory, one word a token,
// from the sequence's history (read by every slab of the sequence, from L2),
// marks drafts and biased tokens there and lists the tokens that are marked at
// all.  The rows are then streamed through with the mask alone, and the listed
// tokens put right in the output, one a lane, while their lines are in L2: with
// the rules applied on the way, a warp took the long path for the one token in
// fifty that needs it (64 x 6 rows of 128256 bf16 logits, histories of 8192:
// 119 us, against 84; applying them on the way in slabs with many marks alone
// gained 1.5 us there and cost 0.4 to 6 elsewhere).  Listing the marked tokens in
// order gained 5 us there and cost 0.6 to 3.5 on short histories and odd rows,
// and 19 on long ones of fp32 rows.  84 us is 54% of the bytes'
// floor: without histories the same rows take 59 us.
#include "admit.h"
#include "svpa_device.cuh"

namespace svpa {

namespace {

constexpr int kMaxDrafts = kMaxNq;
constexpr int kBiasList = 256;  // biased tokens of a slab kept in shared memory

// a token's word: times generated << 3 | biased << 2 | drafted << 1 | in the prompt
constexpr unsigned kInPrompt = 1, kDrafted = 2, kBiased = 4, kOnce = 8;

template <int SLAB>
struct Shared {
    unsigned word[SLAB];
    union {
        uint16_t marked[SLAB];  // tokens with a word, in no order
        int last[SLAB / 2];     // many biased tokens: 1 + the last list entry of each of half the tokens
    };
    int bias_at[kBiasList];     // token of the slab
    int bias_entry[kBiasList];  // its place in the list
    int bias_n, marked_n;
    int drafts[kMaxDrafts];
};
static_assert(sizeof(Shared<4096>) <= 36 * 1024, "six CTAs per SM");

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 u = __ldcs(reinterpret_cast<const float4 *>(p)), v = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float load1(const float *p) { return __ldcs(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
    return __uint_as_float((unsigned)__ldcs(reinterpret_cast<const unsigned short *>(p)) << 16);
}

// VEC: eight consecutive tokens a thread, from the row's first one on a 16-byte
// boundary on (a row of an odd vocabulary starts anywhere; its first few tokens
// are taken by themselves); else, for arrays off that boundary, four that lie
// 32 apart.
template <typename T, bool VEC, int SLAB, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) process_kernel(const __grid_constant__ ProcessArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared<SLAB> &sm = *reinterpret_cast<Shared<SLAB> *>(raw);
    // (slabs of the same tokens first: the common ones, with the most marks, start together)
    const int b = blockIdx.x, v0 = blockIdx.y * SLAB, n = min(SLAB, a.V - v0);
    const int r0 = a.split_rows ? blockIdx.z : 0, r1 = a.split_rows ? r0 + 1 : a.rows;
    const bool marks = a.history || a.drafts || a.bias_tokens;
    const bool report = blockIdx.y == 0 && blockIdx.z == 0;
    if (marks) {
        int hn = 0, pn = 0, lo = 0, hi = 0;
        if (a.history) {
            hn = a.hist_lens[b];
            pn = a.prompt_lens ? a.prompt_lens[b] : 0;
        }
        if (a.bias_tokens) {
            lo = a.bias_offsets[b];
            hi = a.bias_offsets[b + 1];
        }
        if (hn < 0 || hn > a.max_hist || pn < 0 || pn > hn || lo < 0 || hi < lo) {
            if (report && threadIdx.x == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            hn = min(max(hn, 0), a.max_hist);
            pn = min(max(pn, 0), hn);
            if (lo < 0 || hi < lo) lo = hi = 0;
        }
        for (int i = threadIdx.x; i < SLAB / 4; i += THREADS)
            reinterpret_cast<uint4 *>(sm.word)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (threadIdx.x == 0) sm.bias_n = sm.marked_n = 0;
        __syncthreads();
        // the first mark of a token lists it; the lanes that list one here share an add
        auto listed = [&](unsigned before, unsigned x) {
            if (before != 0u) return;
            const unsigned here = __activemask(), lane = threadIdx.x & 31;
            int at = 0;
            if (lane == __ffs(here) - 1) at = atomicAdd(&sm.marked_n, __popc(here));
            at = __shfl_sync(here, at, __ffs(here) - 1) + __popc(here & ((1u << lane) - 1u));
            sm.marked[at] = (uint16_t)x;
        };
        auto mark = [&](int i, int v) {
            const unsigned x = (unsigned)(v - v0);
            if (x < (unsigned)n)
                listed(i < pn ? atomicOr(&sm.word[x], kInPrompt) : atomicAdd(&sm.word[x], kOnce), x);
        };
        const int32_t *h = a.history + (size_t)b * a.max_hist;
        // sixteen tokens a thread in flight; few are the slab's
        const bool quads = ((reinterpret_cast<uintptr_t>(h)) & 15) == 0;
        int i0 = 0;
        if (quads) {
            constexpr int kAhead = 4;
            for (; i0 + 4 * kAhead * THREADS <= hn; i0 += 4 * kAhead * THREADS) {
                int4 v[kAhead];
                const int i1 = i0 + threadIdx.x * 4;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) v[k] = __ldg(reinterpret_cast<const int4 *>(h + i1 + k * 4 * THREADS));
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int i = i1 + k * 4 * THREADS;
                    const bool mine = min(min((unsigned)(v[k].x - v0), (unsigned)(v[k].y - v0)),
                                          min((unsigned)(v[k].z - v0), (unsigned)(v[k].w - v0))) < (unsigned)n;
                    if (!mine) continue;
                    mark(i, v[k].x);
                    mark(i + 1, v[k].y);
                    mark(i + 2, v[k].z);
                    mark(i + 3, v[k].w);
                }
            }
        }
        for (; i0 < hn; i0 += 4 * THREADS) {
            int v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + threadIdx.x + k * THREADS;
                v[k] = i < hn ? __ldg(h + i) : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) mark(i0 + threadIdx.x + k * THREADS, v[k]);
        }
        if (report) {
            bool bad = false;
            for (int i = threadIdx.x; i < hn; i += THREADS) bad = bad || (unsigned)__ldg(h + i) >= (unsigned)a.V;
            if (bad) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        }
        if (a.drafts)
            for (int i = threadIdx.x; i < a.draft_stride; i += THREADS) {
                const int v = a.drafts[(size_t)b * a.draft_stride + i];
                sm.drafts[i] = v;
                if (!((a.used >> i) & 1ull)) continue;  // an entry no row counts (a tree's root) may hold anything
                const unsigned x = (unsigned)(v - v0);
                if (x < (unsigned)n) listed(atomicOr(&sm.word[x], kDrafted), x);
                else if (report && (v < 0 || v >= a.V)) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            }
        for (int i = lo + threadIdx.x; i < hi; i += THREADS) {
            const int v = a.bias_tokens[i];
            const unsigned x = (unsigned)(v - v0);
            if (x < (unsigned)n) {
                listed(atomicOr(&sm.word[x], kBiased), x);
                const int at = atomicAdd(&sm.bias_n, 1);
                if (at < kBiasList) {
                    sm.bias_at[at] = (int)x;
                    sm.bias_entry[at] = i;
                }
            } else if (report && (v < 0 || v >= a.V)) {
                raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
            }
        }
    }

    // ---- every token: the mask
    const int words = (a.V + 31) / 32;
    const float ninf = __int_as_float(0xff800000);
    const T *in = static_cast<const T *>(a.in) + ((size_t)b * a.rows + r0) * a.V + v0;
    float *const out = a.out + ((size_t)b * a.rows + r0) * a.V + v0;
    const uint32_t *mask = a.mask ? a.mask + ((size_t)b * a.rows + r0) * words + v0 / 32 : nullptr;
    if constexpr (VEC) {
        // elements past a multiple of eight of row r0's slab, and of each row after the one before
        const int off0 = (int)((((size_t)b * a.rows + r0) * a.V + v0) & 7), step = a.V & 7;
        auto head_of = [&](int j) -> int { return (8 - ((off0 + (j - r0) * step) & 7)) & 7; };
        auto one = [&](int j, int i) {  // a token by itself
            const uint32_t bit = mask ? __ldg(mask + (size_t)(j - r0) * words + i / 32) >> (i & 31) : 1u;
            const size_t at = (size_t)(j - r0) * a.V + i;
            const float x = load1(in + at);
            out[at] = bit & 1u ? x : ninf;
        };
        if ((off0 | step) != 0)
            for (int z = threadIdx.x; z < 8 * (r1 - r0); z += THREADS)
                if ((z & 7) < min(head_of(r0 + z / 8), n)) one(r0 + z / 8, z & 7);
        for (int c8 = threadIdx.x * 8; c8 < n; c8 += THREADS * 8) {
#pragma unroll 2
            for (int j = r0; j < r1; ++j) {
                const int i = head_of(j) + c8;
                const size_t at = (size_t)(j - r0) * a.V + i;
                if (i + 8 > n) {
                    for (int k = i; k < n; ++k) one(j, k);
                    continue;
                }
                float x[8];
                uint32_t ok = 0xffu;
                load8(in + at, x);
                if (mask) {
                    const uint32_t *bits = mask + (size_t)(j - r0) * words + i / 32;
                    ok = __ldg(bits) >> (i & 31);
                    if ((i & 31) > 24) ok |= __ldg(bits + 1) << (32 - (i & 31));  // i + 7 < n lies there
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!((ok >> e) & 1u)) x[e] = ninf;
                float4 *dst = reinterpret_cast<float4 *>(out + at);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    } else {
        for (int i = (threadIdx.x >> 5) * 128 + (threadIdx.x & 31); i < n; i += THREADS * 4) {
            for (int j = r0; j < r1; ++j) {
                const uint32_t *bits = mask ? mask + (size_t)(j - r0) * words + i / 32 : nullptr;
                const size_t at = (size_t)(j - r0) * a.V + i;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (i + e * 32 >= n) continue;
                    const float x = load1(in + at + e * 32);
                    out[at + e * 32] = !mask || (__ldg(bits + e) >> (i & 31)) & 1u ? x : ninf;
                }
            }
        }
    }
    if (!marks) return;
    __syncthreads();

    // ---- the marked tokens: their logits are in the output, -inf where masked
    // (or given so: it stays)
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    // Where the slab has more biased tokens than the list holds, the sequence's
    // biases are read twice more, each time keeping the last entry of half the
    // slab's tokens where the marked ones were listed.  64 x 6 rows of 128256
    // fp32 logits: 76 us without biases, 97 with lists of up to 300 among the
    // first 4096 tokens, 112 with up to 4096, 490 with up to 128256 of the whole
    // vocabulary.  One loop for both: with a copy of the rules for each, the rows
    // above took 97 us without any biases (and 114 for 95 with histories of 8192).
    const int m = sm.marked_n, c = sm.bias_n;
    const bool many = c > kBiasList;
#pragma unroll 1
    for (int x0 = 0; x0 < (many ? n : 1); x0 += SLAB / 2) {
        const int end = many ? min(SLAB / 2, n - x0) : m;
        if (many) {
            __syncthreads();
            for (int i = threadIdx.x; i < SLAB / 2; i += THREADS) sm.last[i] = 0;
            __syncthreads();
            const int hi = a.bias_offsets[b + 1];
#pragma unroll 4
            for (int i = a.bias_offsets[b] + threadIdx.x; i < hi; i += THREADS) {
                const unsigned x = (unsigned)a.bias_tokens[i] - (unsigned)(v0 + x0);
                if (x < (unsigned)end) atomicMax(&sm.last[x], i + 1);
            }
            __syncthreads();
        }
        for (int z = threadIdx.x; z < end; z += THREADS) {
            const int i = many ? x0 + z : sm.marked[z];
            const unsigned w = sm.word[i];
            if (many && w == 0u) continue;
            float bias = 0.f;
            if (w & kBiased) {  // the last entry of the list that names the token
                int entry = -1;
                if (many) entry = sm.last[z] - 1;
                else
                    for (int k = 0; k < c; ++k)
                        if (sm.bias_at[k] == i) entry = max(entry, sm.bias_entry[k]);
                bias = a.bias_values[entry];
            }
            float *dst = out + i;
#pragma unroll 4
            for (int j = r0; j < r1; ++j, dst += a.V) {
                float x = *dst;
                unsigned count = w / kOnce;
                if (w & kDrafted)
                    for (unsigned long long path = a.path[j]; path; path &= path - 1)
                        count += sm.drafts[__ffsll((long long)path) - 1] == v0 + i;
                if ((w & kInPrompt) || count) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
                if (count) x = __fadd_rn(__fadd_rn(x, -__fmul_rn(freq, (float)count)), -pres);
                if (w & kBiased) x = __fadd_rn(x, bias);
                if (*dst != ninf) *dst = x;
            }
        }
    }
}

template <typename T, int SLAB, int THREADS>
cudaError_t launch_s(const ProcessArgs &a, cudaStream_t st) {
    const bool vec = (reinterpret_cast<uintptr_t>(a.in) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
    const dim3 grid(a.B, (a.V + SLAB - 1) / SLAB, a.split_rows ? a.rows : 1);
    static DeviceMemo<int> attr_set;  // the shared-memory opt-in, once per device
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [](int *v) {
        *v = 1;
        const int bytes = (int)sizeof(Shared<SLAB>);
        cudaError_t r = cudaFuncSetAttribute(process_kernel<T, true, SLAB, THREADS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(process_kernel<T, false, SLAB, THREADS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        return r;
    });
    if (e != cudaSuccess) return e;
    if (vec) process_kernel<T, true, SLAB, THREADS><<<grid, THREADS, sizeof(Shared<SLAB>), st>>>(a);
    else process_kernel<T, false, SLAB, THREADS><<<grid, THREADS, sizeof(Shared<SLAB>), st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(ProcessArgs a, cudaStream_t st) {
    // the largest slab that still leaves every SM a few CTAs; below that, a
    // row a CTA
    const long long tokens = (long long)a.V * a.B;
    if (tokens >= 4096LL * 152 * 6) return launch_s<T, 4096, 256>(a, st);
    if (tokens >= 2048LL * 152 * 4) return launch_s<T, 2048, 256>(a, st);
    a.split_rows = 1;
    return launch_s<T, 1024, 128>(a, st);
}

}  // namespace

cudaError_t launch_logits_process(const ProcessArgs &a, cudaStream_t st) {
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace svpa
