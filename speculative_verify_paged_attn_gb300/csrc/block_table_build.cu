// block_table_build.cu -- block tables and slot maps of admitted requests,
// from their lengths, in one launch.
//
// "Speculative Decoding & KV-Cache PagedAttention in Enterprise LLM Serving",
// PagedKVCacheManager.AllocateSessionBlocks (a request takes ceil(n / 16)
// blocks; the blocks of a shared prefix are referenced, not copied).
//
// With pages_b = ceil(n_b / 16), P prefix pages and own_b = pages_b - P for a
// live request (n_b > 0), request b's i-th own page is the free stack's entry
//   free_stack[free_top - 1 - (own_0 + .. + own_{b-1} + i)]
// and its new tokens take the packed rows from sum of the earlier requests'
// new tokens on.  Both are prefix sums over the batch: every CTA forms them
// for itself in shared memory (a few kilobytes read from L2; no CTA waits for
// another), checks the whole call the same way, then writes its share of the
// table and the slot map.  The last CTA to finish lowers *free_top.
#include "admit.h"
#include "svpa_device.cuh"

namespace svpa {

namespace {

// Small admissions are one CTA of 1024 threads, whose warps take 128 entries
// at a time (nothing to wait for at the end); others CTAs of 256, 256 entries a
// warp.  With a 4-byte copy before each call (0.9 us alone): 8 requests of some
// hundred tokens 7.9 us, bound by the launch and dependent loads (lengths,
// counts, stack); 256 requests of up to 32768 tokens, 4 million slots, 15.1 us,
// the rest of it instructions (searches and index arithmetic: 59% of the issue
// slots; stalls an issue: fixed latencies 2.9, loads 2.4, barriers 2.3).
constexpr int kOneCta = 32768;     // entries and slots
constexpr int kMaxCtas = 152 * 5;  // resident at once for batches of up to about 5500

// Exclusive sums of two values per thread over the CTA; totals returned too.
template <int kThreads>
__device__ __forceinline__ void scan2(int &x, int &y, int &tx, int &ty, int2 *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int px = __shfl_up_sync(0xffffffffu, ix, o), py = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += px;
            iy += py;
        }
    }
    if (lane == 31) warp_sums[warp] = make_int2(ix, iy);
    __syncthreads();
    int bx = 0, by = 0;
    tx = ty = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int2 s = warp_sums[w];
        if (w < warp) {
            bx += s.x;
            by += s.y;
        }
        tx += s.x;
        ty += s.y;
    }
    x = bx + ix - x;
    y = by + iy - y;
}

template <int kThreads, int kChunk>
__global__ void __launch_bounds__(kThreads) build_kernel(const __grid_constant__ BuildArgs a) {
    extern __shared__ int32_t sh[];
    int32_t *first = sh;               // [B + 1] own pages of the requests before
    int32_t *cu = sh + a.B + 1;        // [B + 1] new tokens of the requests before
    __shared__ int2 warp_sums[kThreads / 32];
    __shared__ long long warp_pages[kThreads / 32], warp_tokens[kThreads / 32];
    __shared__ int warp_live[kThreads / 32], warp_bad[kThreads / 32];
    const int P = a.prefix_pages, prefix_len = P * kBlockSize;
    const int top = *a.free_top;
    // lengths: each thread takes a run of requests
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    int bad = 0, live = 0;
    long long lp = 0, lt = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = a.seq_lens[b];
        if (n < 0 || n > (long long)a.max_blocks * kBlockSize || (n > 0 && n < prefix_len)) {
            bad |= SVPA_DEVERR_BAD_VALUE;
        } else if (n > 0) {
            ++live;
            lp += (n + kBlockSize - 1) / kBlockSize - P;
            lt += n - prefix_len;
        }
    }
    for (int i = threadIdx.x; i < P; i += kThreads) {
        const int id = a.prefix_blocks[i];
        if (id < 0 || id >= a.num_blocks) bad |= SVPA_DEVERR_BAD_BLOCK;
        else if (*(volatile int32_t *)(a.refcount + id) < 1) bad |= SVPA_DEVERR_BAD_VALUE;
    }
    {
        // totals over the CTA, in 64 bits (a batch of bad lengths may exceed 32)
        long long sp = lp, st = lt;
        int sl = live, sb = bad;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sp += __shfl_xor_sync(0xffffffffu, sp, o);
            st += __shfl_xor_sync(0xffffffffu, st, o);
            sl += __shfl_xor_sync(0xffffffffu, sl, o);
            sb |= __shfl_xor_sync(0xffffffffu, sb, o);
        }
        if ((threadIdx.x & 31) == 0) {
            warp_pages[threadIdx.x >> 5] = sp;
            warp_tokens[threadIdx.x >> 5] = st;
            warp_live[threadIdx.x >> 5] = sl;
            warp_bad[threadIdx.x >> 5] = sb;
        }
    }
    __syncthreads();
    long long s_pages = 0, s_tokens = 0;
    int s_live = 0;
    bad = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        s_pages += warp_pages[w];
        s_tokens += warp_tokens[w];
        s_live += warp_live[w];
        bad |= warp_bad[w];
    }
    if (top < 0 || top > a.num_blocks || s_tokens > a.slots) bad |= SVPA_DEVERR_BAD_VALUE;
    else if (s_pages > top) bad |= SVPA_DEVERR_FREE_OVERFLOW;
    if (bad) {
        // every CTA sees the same and leaves everything as it was
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, bad);
        return;
    }
    // the sums fit: at most num_blocks pages and `slots` tokens
    int x = (int)lp, y = (int)lt, tp, tt;
    scan2<kThreads>(x, y, tp, tt, warp_sums);
    for (int b = b0; b < b1; ++b) {
        first[b] = x;
        cu[b] = y;
        const int n = a.seq_lens[b];
        if (n > 0) {
            x += (n + kBlockSize - 1) / kBlockSize - P;
            y += n - prefix_len;
        }
    }
    if (threadIdx.x == 0) {
        first[a.B] = tp;
        cu[a.B] = tt;
    }
    __syncthreads();

    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= a.B; b += kThreads) a.cu_seqlens[b] = cu[b];
        if (s_live)
            for (int i = threadIdx.x; i < P; i += kThreads) atomicAdd(&a.refcount[a.prefix_blocks[i]], s_live);
    }
    // the block of request b's page i, with its own pages popped in order
    auto block_of = [&](int b, int i) -> int {
        return __ldg(i < P ? a.prefix_blocks + i : a.free_stack + (top - 1 - (first[b] + i - P)));
    };
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    const long long w0 = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long entries = (long long)a.B * a.max_blocks;
    const long long table_chunks = (entries + kChunk - 1) / kChunk;
    const long long all_chunks = table_chunks + (a.slots + kChunk - 1) / kChunk;
    // the table's chunks, then the slot map's, over all warps
    long long c = w0;
    for (; c < table_chunks; c += warps) {
        const long long e0 = c * kChunk;
        const int row0 = (int)(e0 / a.max_blocks);
        const unsigned col0 = (unsigned)(e0 - (long long)row0 * a.max_blocks);
#pragma unroll 8
        for (int k = lane; k < kChunk; k += 32) {
            if (e0 + k >= entries) continue;
            const unsigned q = (col0 + k) / (unsigned)a.max_blocks;
            const int b = row0 + (int)q, i = (int)(col0 + k - q * a.max_blocks);
            const int own = first[b + 1] - first[b];
            int id = -1;
            // (a request without pages of its own has new tokens in none, and
            // holds the prefix only if its length says so)
            if (i < P + own && (own > 0 || __ldg(a.seq_lens + b) > 0)) {
                id = block_of(b, i);
                if (i >= P) {
                    if (id < 0 || id >= a.num_blocks) {
                        raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
                        id = -1;
                    } else {
                        a.refcount[id] = 1;
                    }
                }
            }
            a.block_table[e0 + k] = id;
        }
    }
    const int total = cu[a.B];
    const bool vec = (reinterpret_cast<uintptr_t>(a.slot_map) & 15) == 0;
    for (; c < all_chunks; c += warps) {
        const int s0 = (int)((c - table_chunks) * kChunk), s1 = min(s0 + kChunk, a.slots);
        // the requests of the chunk's first and last rows
        auto request_of = [&](int t, int lo, int hi) -> int {  // in [lo, hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            return lo;
        };
        const int lo = s0 < total ? request_of(s0, 0, a.B) : 0;
        const int hi = s0 < total ? request_of(min(s1, total) - 1, lo, a.B) + 1 : 1;
#pragma unroll
        for (int k = 0; k < kChunk / 128; ++k) {
            const int t0 = s0 + k * 128 + lane * 4;
            if (t0 >= s1) break;
            int b = t0 < total ? request_of(t0, lo, hi) : 0;
            int slot[4];
            if (t0 < total && t0 + 3 < cu[b + 1]) {
                // four rows of one request: of one page, or of two that follow
                const int pos = prefix_len + t0 - cu[b], page = pos / kBlockSize, last = (pos + 3) / kBlockSize;
                const int id0 = block_of(b, page), id1 = last == page ? id0 : block_of(b, last);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int id = (pos + z) / kBlockSize == page ? id0 : id1;
                    // (one outside the pool is raised with the table)
                    slot[z] = (unsigned)id < (unsigned)a.num_blocks ? id * kBlockSize + (pos + z) % kBlockSize : -1;
                }
            } else {
                int page = -1, row = -1, id = -1;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int t = t0 + z;
                    slot[z] = -1;
                    if (t < total) {
                        while (cu[b + 1] <= t) ++b;
                        const int pos = prefix_len + t - cu[b];
                        if (b != row || pos / kBlockSize != page) {
                            row = b;
                            page = pos / kBlockSize;
                            id = block_of(b, page);
                            if (id < 0 || id >= a.num_blocks) id = -1;  // raised with the table
                        }
                        if (id >= 0) slot[z] = id * kBlockSize + pos % kBlockSize;
                    }
                }
            }
            if (vec && t0 + 4 <= a.slots) {
                *reinterpret_cast<int4 *>(a.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            } else {
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (t0 + z < a.slots) a.slot_map[t0 + z] = slot[z];
            }
        }
    }
    // *free_top is lowered once every CTA has read it
    __syncthreads();
    if (threadIdx.x == 0) {
        if (gridDim.x == 1) {
            *a.free_top = top - tp;
            return;
        }
        __threadfence();
        if (atomicAdd(a.ticket, 1) == (int)gridDim.x - 1) {
            *a.ticket = 0;
            *a.free_top = top - tp;
        }
    }
}

}  // namespace

namespace {

template <int kThreads, int kChunk>
cudaError_t launch_t(const BuildArgs &a, int grid, cudaStream_t stream) {
    const size_t smem = (size_t)2 * (a.B + 1) * sizeof(int32_t);
    if (smem > 40 * 1024) {  // (a few hundred bytes are static)
        static DeviceMemo<int> attr_set;
        int done = 0;
        const cudaError_t e = attr_set.get(&done, [](int *v) {
            *v = 1;
            return cudaFuncSetAttribute(build_kernel<kThreads, kChunk>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)(2 * (kMaxBuildBatch + 1) * sizeof(int32_t)));
        });
        if (e != cudaSuccess) return e;
    }
    build_kernel<kThreads, kChunk><<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_table_build(const BuildArgs &a, cudaStream_t stream) {
    const long long entries = (long long)a.B * a.max_blocks + a.slots;
    if (entries <= kOneCta) return launch_t<1024, 128>(a, 1, stream);
    const long long ctas = (entries + 256 * 8 - 1) / (256 * 8);
    return launch_t<256, 256>(a, (int)(ctas > kMaxCtas ? kMaxCtas : ctas), stream);
}

}  // namespace svpa
