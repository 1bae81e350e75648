// packed_attn_tc.cu -- attention of many query tokens over paged K/V on the
// 5th-generation tensor cores (tcgen05 + TMEM), sm_103a.
//
//   out[t][h] = sum_p softmax_p( q[t][h] . K[p] * scale ) V[p],  p visible to t
//
// Two entry points share it.  Prompt attention: token t of a sequence sees
// the positions up to its own.  Verification behind a shared prefix: with the
// visible set split as prefix + own part,
//   m = max(m_p, m_o),  l = l_p 2^(m_p - m) + l_o 2^(m_o - m),
//   out = (O_p 2^(m_p - m) + O_o 2^(m_o - m)) / l
// so the prefix part (O_p, m_p, l_p) of ALL sequences' queries is formed by
// units that read the prefix pages once per 256 query rows instead of once
// per sequence, and joined with each sequence's own part.
//
// A query tile is 128 rows: 128 / G tokens x the G query heads of one kv head
// (all heads of a group share the K/V tile).  A unit of work is
//   pair: two query tiles A, B over the same K/V blocks (128 tokens each), or
//   alt:  one query tile whose even blocks go to A and odd blocks to B
//         (tiles too small to pair: one sequence's drafts, short prompts);
// either way two softmax groups work on two score tiles in turn, so that the
// tensor cores compute one while the exponentials of the other are taken.
// Persistent CTAs, one per SM (TMEM 512 columns, 224 KB of shared memory),
// take units from an atomic counter.  Warps:
//   0      producer: streams K and V blocks (8 pages per block, one TMA copy per
//          page and kv head) through one ring, and the query tiles;
//   1, 2   MMA issuers of tile A and tile B (warp 1 owns the TMEM):
//          O_t += P_t V with P_t read from TMEM over S_t's own columns, then
//          S_t = Q_t K^T of the next block;
//   3      scheduler: decodes units ahead of the producer and reports prefix
//          units whose partials are written;
//   4-7    softmax of tile A, one thread per query row: mask, lazy running
//   8-11   maximum (O_t rescaled only when it grows by more than 2^8), fp32
//          row sum, P as bf16 (the MMA's input type; the sum is taken before
//          that rounding); then the unit's epilogue.
// 8192 tokens, 64/8 heads, D 128: 693 us, 1.59 PFLOP/s, in a burst at 2070 MHz;
// 746 us, 1.47 PFLOP/s, sustained at the power limit (1927 MHz).  Bound by one
// tile's chain from scores to the next scores: a pair's block takes about 3000 cycles,
// 2048 of them MMAs (the exponentials of both tiles about 1000, the rest waits
// and fences of some 100 to 250 each).  40 x 6 queries behind 8192 shared
// tokens: 84 to 91 us by process (247 with every sequence reading the prefix).
//
// A commit on S_t's barrier covers the PV_t issued before it, so a softmax
// warp that sees S_t may rescale O_t at once.  All waits are bounded.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "packed_attn.h"
#include "svpa_device.cuh"

namespace svpa {

namespace {

constexpr int kThreads = 384;
// registers are launched evenly (168 a thread, 64512 in all) and moved to the
// softmax warps: 128 * 80 + 256 * 208 = 63488
constexpr int kRegsFew = 80, kRegsMany = 208;
constexpr int kPagesPerBlock = 8;
constexpr int kNB = kPagesPerBlock * kBlockSize;  // kv tokens per block
constexpr int kRing = 5;                          // K and V tiles in flight
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kTmemCols = 512, kTmemO = 0, kTmemS = 256;
constexpr float kLn2 = 0.69314718055994530942f;

enum { kEnd = 0, kPair = 1, kAlt = 2 };

struct Unit {
    int32_t kind;        // kEnd, kPair, kAlt
    int32_t h;           // kv head
    int32_t tok0, tok1;  // query tokens [tok0, tok1) of the unit
    int32_t nA, nB;      // blocks of tile A and tile B
    int32_t base;        // ring index of the unit's first K tile
    int32_t pos0;        // kv position of its first block
    int32_t kv_end;      // positions from here on hold no token
    int32_t lim0;        // token tok0 sees positions below lim0 ...
    int32_t causal;      // ... and each later token one more, or
    int32_t use_anc;     // the draft slots of its ancestors
    int32_t slot;        // partial slot, or -1: final
    int32_t merge;       // join the prefix partials
    int32_t prefix;      // a prefix unit: count it when written
};

// A unit with what its copies need: its table, pages and blocks, and the tokens
// of one query tile's copy.
struct Job {
    Unit w;
    const int32_t *bt;
    int32_t page0, npages, nblk, n_tok_load;
    int32_t once;  // its K/V is read by this unit alone
};

template <int D>
struct Smem {
    static constexpr int kTile = kNB * D * 2;
    static constexpr int kQTile = 128 * D * 2;
    uint8_t q[2][kQTile];  // 1024-aligned: [64-column slab][128 rows][128 B]
    uint8_t kv[kRing][kTile];
    uint64_t full[kRing], empty[kRing];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t both;  // the two softmax groups meet
    uint64_t drain[2];
    uint64_t turn[2];  // a pair's tiles issue their MMAs in turn
    uint64_t job_full, job_want;  // a decoded unit, scheduler -> producer
    uint64_t prefix_done;         // every prefix unit's partials are written
    Job job;
    int32_t job_ids[32];
    Unit unit;
    int32_t written[2];  // each group's warps that wrote a prefix unit's partials
    float2 stat[2][128];
    uint32_t tmem_base;
};
static_assert(sizeof(Smem<128>) <= 232448, "packed attention shared memory");

__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Packed fp32 pairs: each half rounded as the scalar operation.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void st_32bytes(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Sixteen values of a row as bf16 to `dst` (32 bytes: in one store where they may be).
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16 *dst, const float *f, float scale, bool wide) {
    uint32_t v[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = pack_bf16x2(f[2 * x] * scale, f[2 * x + 1] * scale);
    if (wide) {
        st_32bytes(dst, v);
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Bounded wait on a barrier that is usually about to complete: the clock is
// read only after a while (a read costs more than many probes).
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, int32_t *err) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, err);
}

__device__ __forceinline__ bool mbar_wait_all(uint64_t *bar, uint32_t phase, int32_t *err) {
    return __all_sync(0xffffffffu, bar_wait(bar, phase & 1u, err));
}

template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ int ld_acquire(const int32_t *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_"
        "hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// The pool's (page, kv head) tile of the unit's page i; one past the pool (it
// reads as zeros) behind its last page.
__device__ __forceinline__ int page_tile(const PackedArgs &a, const Job &d, int i) {
    if (i >= d.npages) return a.num_blocks * a.Hkv;
    int blk = __ldg(d.bt + d.page0 + i);
    if (blk < 0 || blk >= a.num_blocks) {
        raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
        blk = 0;
    }
    return blk * a.Hkv + d.w.h;
}

// Largest b with cu[b] / step + b <= slot (cu[0] = 0), by the whole warp:
// 32 candidates a round.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int step, int slot, int lane) {
    int lo = 0, n = B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int stride = (n + 31) / 32;
        const int b = lo + lane * stride;
        const bool le = lane * stride < n && __ldg(cu + b) / step + b <= slot;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz((int)m) : 0;
        lo += k * stride;
        n = min(stride, n - k * stride);
    }
    return lo;
}

// The partial row of (slot, kv head h, token, head gi of the group).
__device__ __forceinline__ size_t part_row(const PackedArgs &a, int slot, int h, int tok, int gi) {
    const int tile = tok / a.tpt;
    return (((size_t)slot * a.Hkv + h) * a.tiles + tile) * 128 + (size_t)((tok - tile * a.tpt) * a.G + gi);
}
// Its four columns 4 g .. 4 g + 3 are at g * 32 of this.
template <int D>
__device__ __forceinline__ float4 *part_cols(const PackedArgs &a, size_t row) {
    return reinterpret_cast<float4 *>(a.part_o) + (row & ~(size_t)31) * (D / 4) + (row & 31);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mqt0, const __grid_constant__ CUtensorMap mqt1,
                       const __grid_constant__ CUtensorMap mqs0, const __grid_constant__ CUtensorMap mqs1,
                       const __grid_constant__ PackedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    using SM = Smem<D>;
    // all of the opt-in shared memory is used, with no room to move the base:
    // the only shared memory of this kernel, it starts on its 1 KB alignment
    SM &sm = *reinterpret_cast<SM *>(smem_raw);
    if (smem_u32(smem_raw) & 1023u) {
        if (threadIdx.x == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        return;
    }
    constexpr int kSlabs = D / 64;
    constexpr int kQSlab = 128 * 128;
    constexpr int kPageBytes = kBlockSize * D * 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // A prompt's first units go by CTA.  Units of a verification are all taken
    // from the counter, so that every prefix unit is a running CTA's before any
    // unit that waits for it is taken (the first, while the CTA sets itself up).
    int next = -1;
    if (threadIdx.x == 96) next = a.verify ? atomicAdd(&a.sched[0], 1) : (int)blockIdx.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 2);  // the two MMA issuers
        }
        mbar_init(&sm.both, 8);
        sm.written[0] = sm.written[1] = 0;
        mbar_init(&sm.job_full, 1);
        mbar_init(&sm.job_want, 1);
        mbar_init(&sm.prefix_done, 1);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 10);  // the MMA issuers and the eight softmax warps
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t], 4);
            mbar_init(&sm.o_full[t], 1);
            mbar_init(&sm.drain[t], 1);
            mbar_init(&sm.turn[t], 1);
        }
        fence_mbar_init();
    }
    // (rows of a query tile past its tokens are never written by the copies and
    // hold anything: a row of S, P and O comes from its own row of Q alone, and
    // theirs are not stored)
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp < 4) {
        regs_dec<kRegsFew>();
        if (warp == 0) {
        // ================================================= producer
        const uint64_t keep = policy_evict_normal(), stream_once = policy_evict_first();
        if (lane == 0) {
            prefetch_tensormap(&mk);
            prefetch_tensormap(&mv);
            prefetch_tensormap(&mqt0);
            prefetch_tensormap(&mqt1);
        }
        int tile = 0, units = 0;  // ring tiles issued, units started
        bool ok = true;
        auto issue_q = [&](const Job &d) -> bool {
            if (units >= 1) {
                int good = 1;
                if (lane == 0) good = mbar_wait(&sm.q_empty, (uint32_t)((units - 1) & 1), a.err);
                if (!__shfl_sync(0xffffffffu, good, 0)) return false;
            }
            if (lane == 0) {
                sm.unit = d.w;
                const bool two = d.w.kind == kPair;
                const uint32_t bytes = d.nblk == 0 ? 0u : (uint32_t)(d.n_tok_load * a.G * D * 2) * (two ? 2u : 1u);
                mbar_arrive_expect_tx(&sm.q_full, bytes);
                if (bytes) {
                    const uint64_t pol = d.once ? stream_once : keep;
#pragma unroll
                    for (int s = 0; s < kSlabs; ++s) {
                        const CUtensorMap *m = d.w.use_anc ? (s ? &mqs1 : &mqs0) : (s ? &mqt1 : &mqt0);
                        tma_load_3d(&sm.q[0][s * kQSlab], m, 0, d.w.h * a.G, d.w.tok0, &sm.q_full, pol);
                        if (two)
                            tma_load_3d(&sm.q[1][s * kQSlab], m, 0, d.w.h * a.G, d.w.tok0 + a.tpt, &sm.q_full, pol);
                    }
                }
            }
            __syncwarp();
            return true;
        };
        // K and V tiles in the order the MMA issuers take them
        auto issue_tile = [&](const CUtensorMap *map, int id, uint64_t pol) -> bool {
            const int s = tile % kRing;
            if (tile >= kRing) {
                int good = 1;
                if (lane == 0) good = mbar_wait(&sm.empty[s], (uint32_t)(((tile / kRing) & 1) ^ 1), a.err);
                if (!__shfl_sync(0xffffffffu, good, 0)) return false;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)SM::kTile);
            __syncwarp();
            if (lane < kPagesPerBlock)
                tma_load_5d(&sm.kv[s][lane * kPageBytes], map, 0, 0, 0, 0, id, &sm.full[s], pol);
            ++tile;
            return true;
        };
        for (; ok; ++units) {
            ok = mbar_wait_all(&sm.job_full, (uint32_t)units, a.err);
            if (!ok) break;
            Job job = sm.job;
            int ids = sm.job_ids[lane], ids_next = 0;
            __syncwarp();
            // the next unit is asked for a few blocks before this one's end: taken
            // earlier, the last units would wait behind a busy CTA
            const int ask = max(0, job.nblk - 4);
            if (job.w.kind == kEnd) break;
            job.w.base = tile;
            const uint64_t pol = job.once ? stream_once : keep;
            bool q_out = false;
            for (int j = 0; j < job.nblk && ok; ++j) {
                if ((j & 3) == 0) {
                    if (j > 0) ids = ids_next;
                    if (j + 4 < job.nblk) ids_next = page_tile(a, job, (j + 4) * kPagesPerBlock + lane);
                }
                if (j == ask && lane == 0) mbar_arrive(&sm.job_want);
                const int id = __shfl_sync(0xffffffffu, ids, ((j & 3) * kPagesPerBlock + (lane & 7)) & 31);
                ok = issue_tile(&mk, id, pol);
                if (ok) ok = issue_tile(&mv, id, pol);
                // the first block of the next unit is on its way before the
                // query buffers are free
                if (ok && !q_out) {
                    ok = issue_q(job);
                    q_out = true;
                }
            }
            if (ok && !q_out) ok = issue_q(job);
            if (job.nblk == 0 && lane == 0) mbar_arrive(&sm.job_want);
        }
        if (lane == 0) {
            if (ok && units >= 1) ok = mbar_wait(&sm.q_empty, (uint32_t)((units - 1) & 1), a.err);
            if (ok) {
                sm.unit.kind = kEnd;
                mbar_arrive(&sm.q_full);
            }
            // copies still in flight land before the CTA ends
            for (int i = tile >= kRing ? tile - kRing : 0; i < tile; ++i)
                if (!mbar_wait(&sm.full[i % kRing], (uint32_t)((i / kRing) & 1), a.err)) break;
        }
        __syncwarp();
        } else if (warp < 3) {
            // ================================================= MMA issuers
            // The whole warp runs the loop with warp-uniform values and one
            // elected lane issues: an MMA's operands then go straight through
            // uniform registers (issued from a branch that one lane takes, an
            // MMA cost 80 to 145 cycles of issue; it runs 64).  Each wait costs
            // about 100 cycles even when the barrier is complete, more than the
            // MMAs queued behind the one running can cover: hence one issuer
            // per tile, V waited for before P, and K behind P V's issue.
            const int t = __shfl_sync(0xffffffffu, warp - 1, 0);
            constexpr uint32_t idS = umma_idesc_bf16(128, kNB, false);
            constexpr uint32_t idPV = umma_idesc_bf16(128, D, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t dS = tm + kTmemS + (uint32_t)t * kNB, dO = tm + kTmemO + (uint32_t)t * 128;
            // descriptors count 16-byte units; an address field never carries (below 2^14)
            const uint64_t q0 = umma_desc_sw128(smem_u32(&sm.q[0][0]), 16, 1024);
            const uint64_t k0 = umma_desc_sw128(smem_u32(&sm.kv[0][0]), 16, kSlabs * 1024);
            const uint64_t v0 = umma_desc_sw128(smem_u32(&sm.kv[0][0]), 1024, kSlabs * 1024);
            auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
                return __all_sync(0xffffffffu, bar_wait(bar, phase & 1u, a.err));
            };
            // A barrier tells two phases apart only, so each issuer waits for
            // every tile that lands, its own and those only the other reads
            // (alt units, the last blocks of a pair's tile B): a slot is filled
            // anew after one arrival of each, a commit or, for the latter, this.
            auto tile_wait = [&](int i) -> bool { return wait(&sm.full[i % kRing], (uint32_t)(i / kRing)); };
            auto pass_over = [&](int i) -> bool {
                if (!tile_wait(i)) return false;
                if (lane == 0) mbar_arrive(&sm.empty[i % kRing]);
                __syncwarp();
                return true;
            };
            uint32_t np = 0, nt = 0;  // phases of p_full, turn
            bool ok = true;
            for (int unit = 0; ok; ++unit) {
                if (!wait(&sm.q_full, (uint32_t)unit)) break;
                const int kind = __shfl_sync(0xffffffffu, sm.unit.kind, 0);
                const int n = __shfl_sync(0xffffffffu, t ? sm.unit.nB : sm.unit.nA, 0);
                const int other = __shfl_sync(0xffffffffu, t ? sm.unit.nA : sm.unit.nB, 0);
                const int base = __shfl_sync(0xffffffffu, sm.unit.base, 0);
                if (kind == kEnd) break;
                const bool pair = kind == kPair;
                const uint64_t qd = q0 + (pair && t ? SM::kQTile / 16 : 0);
                if (n == 0 && lane == 0) mbar_arrive(&sm.q_empty);
                // O_t += P_t V of block j - 1
                auto issue_pv = [&](int j, int sv) {
                    const uint64_t vd = v0 + (uint32_t)sv * (SM::kTile / 16);
#pragma unroll
                    for (int kt = 0; kt < kNB / 16; ++kt)
                        umma_bf16_tmem_a(dO, dS + kt * 8, vd + kt * (kPageBytes / 16), idPV,
                                         kt > 0 ? 1u : (uint32_t)(j - 1));
                    if (j == n) umma_commit(&sm.o_full[t]);
                };
                // A pair's tiles take turns: two queues of MMAs would be served
                // in alternation, and both tiles' next scores be late.  B's
                // step j follows A's step j, A's step j + 1 B's step j.
                auto my_turn = [&](int j) -> bool {
                    const bool waits = t ? j <= other : j > 1;
                    return !waits || wait(&sm.turn[t], nt++);
                };
                // S_t = Q_t K^T of block j, over the P_t that the MMA before has read
                auto issue_s = [&](int j, int sk) {
                    const uint64_t kd = k0 + (uint32_t)sk * (SM::kTile / 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(dS, qd + ((kk >> 2) * kQSlab + (kk & 3) * 32) / 16,
                                  kd + ((kk >> 2) * 1024 + (kk & 3) * 32) / 16, idS, kk > 0 ? 1u : 0u);
                    umma_commit(&sm.s_full[t]);
                    umma_commit(&sm.empty[sk]);
                    if (j == n - 1) umma_commit(&sm.q_empty);
                };
#pragma unroll 1
                for (int j = 0; j <= n && n > 0; ++j) {
                    const int ik = base + 2 * (pair ? j : 2 * j + t), sk = ik % kRing;
                    const int iv = ik + 1 - (pair ? 2 : 4), sv = iv % kRing;
                    if (pair) {
                        // K (from L2) has landed long before P is ready: wait
                        // for it first, and both MMAs go out together
                        ok = (j == n || tile_wait(ik)) &&
                             (j == 0 || (tile_wait(iv) && my_turn(j) && wait(&sm.p_full[t], np++)));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (j > 0) issue_pv(j, sv);
                            if (j < n) issue_s(j, sk);
                            if (j > 0) umma_commit(&sm.empty[sv]);
                            if (j > 0 && (t == 0 || j < other)) mbar_arrive(&sm.turn[1 - t]);
                        }
                        __syncwarp();
                        continue;
                    }
                    if (j > 0) {
                        ok = tile_wait(iv) && wait(&sm.p_full[t], np++);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(j, sv);
                            umma_commit(&sm.empty[sv]);
                        }
                        __syncwarp();
                        if (j - 1 < other) ok = pass_over(base + 2 * (2 * (j - 1) + 1 - t) + 1);
                        if (!ok) break;
                    }
                    if (j < n) {
                        ok = tile_wait(ik);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) issue_s(j, sk);
                        __syncwarp();
                        if (j < other) ok = pass_over(base + 2 * (2 * j + 1 - t));
                        if (!ok) break;
                    }
                }
                // blocks that only the other tile has
                for (int j = n; j < other && ok; ++j) {
                    const int i = base + 2 * (pair ? j : 2 * j + 1 - t);
                    ok = pass_over(i) && pass_over(i + 1);
                }
            }
            if (!ok) {  // a wait ran out: the MMAs issued so far end before the CTA does
                if (elect_one()) umma_commit(&sm.drain[t]);
                __syncwarp();
                wait(&sm.drain[t], 0);
            }
        } else {
            // ================================================= scheduler
            // Decodes the producer's next unit (chains of dependent loads), and makes
            // a prefix unit's partials visible to the other CTAs and counts it, where
            // the fence holds up no softmax warp.
            const int tpt2 = 2 * a.tpt;
        // The next unit that has work; false when there is none.
        auto decode = [&](Job &d) -> bool {
            while (true) {
                if (lane == 0 && next < 0) next = atomicAdd(&a.sched[0], 1) + (a.verify ? 0 : (int)gridDim.x);
                const int u = __shfl_sync(0xffffffffu, next, 0);
                if (u >= a.total_units) return false;
                next = -1;
                Unit &w = d.w;
                w.use_anc = w.merge = w.prefix = 0;
                w.causal = 0;
                w.slot = -1;
                d.once = false;
                if (u < a.p_units) {
                    const int h = u % a.Hkv, x = u / a.Hkv;
                    const int split = x % a.p_splits, pair = x / a.p_splits;
                    w.h = h;
                    w.tok0 = pair * tpt2;
                    w.tok1 = min(w.tok0 + tpt2, a.T);
                    d.bt = a.prefix_blocks;
                    const int nb = (a.prefix_pages + kPagesPerBlock - 1) / kPagesPerBlock;
                    const int b0 = (int)((long long)nb * split / a.p_splits);
                    const int b1 = (int)((long long)nb * (split + 1) / a.p_splits);
                    d.page0 = b0 * kPagesPerBlock;
                    d.npages = min(a.prefix_pages, b1 * kPagesPerBlock) - d.page0;
                    d.nblk = b1 - b0;
                    w.kv_end = w.lim0 = a.prefix_pages * kBlockSize;
                    w.kind = w.tok1 - w.tok0 > a.tpt ? kPair : kAlt;
                    w.slot = split;
                    w.prefix = 1;
                    d.n_tok_load = a.tpt;
                } else if (a.verify) {
                    const int x = u - a.p_units;
                    const int h = x % a.Hkv, y = x / a.Hkv;
                    const int split = y % a.s_splits;
                    const int b = a.order ? __ldg(a.order + y / a.s_splits) : y / a.s_splits;
                    const int L = __ldg(a.lens + b);
                    d.bt = a.block_table + (size_t)b * a.max_blocks;
                    const long long total = (long long)L + a.n_q;
                    if (L < 0 || total > (long long)a.max_blocks * kBlockSize) {
                        if (lane == 0 && split == 0 && h == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                        continue;
                    }
                    // a sequence whose table begins with the prefix joins it; any
                    // other attends its whole history itself
                    bool mine = L >= a.prefix_pages * kBlockSize;
                    for (int i0 = 0; i0 < a.prefix_pages && mine; i0 += 256) {
                        int p[8], q[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int i = i0 + 32 * k + lane;
                            const bool in = i < a.prefix_pages;
                            p[k] = in ? __ldg(d.bt + i) : 0;
                            q[k] = in ? __ldg(a.prefix_blocks + i) : 0;
                        }
                        bool same = true;
#pragma unroll
                        for (int k = 0; k < 8; ++k) same = same && p[k] == q[k];
                        mine = __all_sync(0xffffffffu, same);
                    }
                    if (a.member && lane == 0 && split == 0 && h == 0) a.member[b] = mine ? 1 : 0;
                    const int first = mine ? a.prefix_pages : 0;
                    const int pages = (int)((total + kBlockSize - 1) / kBlockSize) - first;
                    const int nb = (pages + kPagesPerBlock - 1) / kPagesPerBlock;
                    const int b0 = (int)((long long)nb * split / a.s_splits);
                    const int b1 = (int)((long long)nb * (split + 1) / a.s_splits);
                    d.page0 = first + b0 * kPagesPerBlock;
                    d.npages = min(pages, b1 * kPagesPerBlock) - b0 * kPagesPerBlock;
                    d.nblk = b1 - b0;
                    w.h = h;
                    w.tok0 = b * a.n_q;
                    w.tok1 = w.tok0 + a.n_q;
                    w.kv_end = (int)total;
                    w.lim0 = L;
                    w.use_anc = 1;
                    w.kind = kAlt;
                    w.merge = mine && a.s_splits == 1;
                    w.slot = a.s_splits == 1 ? -1 : a.p_splits + split;
                    d.n_tok_load = a.n_q;
                    d.once = true;
                } else {
                    // long tiles first: the last tiles of a sequence see the most
                    const int h = u % a.Hkv, y = u / a.Hkv;
                    const int split = y % a.s_splits, slot = a.pairs - 1 - y / a.s_splits;
                    int b, c0, c1, kv;
                    if (a.B <= 32) {  // the whole batch in one round of loads
                        const bool in = lane < a.B;
                        c0 = in ? __ldg(a.cu + lane) : 0;
                        c1 = in ? __ldg(a.cu + lane + 1) : 0;
                        kv = in ? __ldg(a.lens + lane) : 0;
                        const unsigned m = __ballot_sync(0xffffffffu, in && c0 / tpt2 + lane <= slot);
                        b = m ? 31 - __clz((int)m) : 0;
                        c0 = __shfl_sync(0xffffffffu, c0, b);
                        c1 = __shfl_sync(0xffffffffu, c1, b);
                        kv = __shfl_sync(0xffffffffu, kv, b);
                    } else {
                        b = find_sequence(a.cu, a.B, tpt2, slot, lane);
                        c0 = __ldg(a.cu + b);
                        c1 = __ldg(a.cu + b + 1);
                        kv = __ldg(a.lens + b);
                    }
                    if (c0 < 0 || c1 < c0 || c1 > a.T) {
                        if (lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                        continue;
                    }
                    const int t0 = c0 + (slot - (c0 / tpt2 + b)) * tpt2;
                    if (t0 >= c1) continue;  // no tile here
                    if (t0 < c0 || kv < c1 - c0 || kv > (long long)a.max_blocks * kBlockSize) {
                        if (lane == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                        continue;
                    }
                    w.h = h;
                    w.tok0 = t0;
                    w.tok1 = min(t0 + tpt2, c1);
                    w.lim0 = kv - (c1 - t0) + 1;
                    w.causal = 1;
                    w.kv_end = kv;
                    d.bt = a.block_table + (size_t)b * a.max_blocks;
                    const int seen = w.lim0 + (w.tok1 - 1 - t0);  // positions the unit's last token sees
                    const int pages = (seen + kBlockSize - 1) / kBlockSize;
                    const int nb = (seen + kNB - 1) / kNB;
                    const int b0 = (int)((long long)nb * split / a.s_splits);
                    const int b1 = (int)((long long)nb * (split + 1) / a.s_splits);
                    d.page0 = b0 * kPagesPerBlock;
                    d.npages = min(pages, b1 * kPagesPerBlock) - d.page0;
                    d.nblk = b1 - b0;
                    w.kind = w.tok1 - w.tok0 > a.tpt ? kPair : kAlt;
                    w.slot = a.s_splits == 1 ? -1 : split;
                    d.n_tok_load = a.tpt;
                }
                w.pos0 = d.page0 * kBlockSize;
                if (w.kind == kPair) {
                    w.nA = w.nB = d.nblk;
                    if (w.causal) {
                        // tile A's last token may end one block or more earlier
                        const int seenA = w.lim0 + a.tpt - 1;
                        w.nA = min(d.nblk, max(0, (seenA - w.pos0 + kNB - 1) / kNB));
                    }
                } else {
                    w.nA = (d.nblk + 1) / 2;
                    w.nB = d.nblk / 2;
                }
                return true;
            }
        };
            // A prompt's offsets, a share for each CTA: decoding sees a sequence only
            // in the slots that it finds, and one whose offsets fall may own none.
            auto check_offsets = [&]() {
                const int per = (a.B + (int)gridDim.x - 1) / (int)gridDim.x;
                const int b0 = (int)blockIdx.x * per, b1 = min(b0 + per, a.B);
                bool bad = blockIdx.x == 0 && __ldg(a.cu) != 0;
                for (int b = b0 + lane; b < b1; b += 32) {
                    const int end = __ldg(a.cu + b + 1);
                    bad = bad || end < __ldg(a.cu + b) || end > a.T;
                }
                if (bad) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
                __syncwarp();
            };
            int prefixes = 0, reported = 0;  // prefix units handed on, and counted
            auto report = [&]() {
                // A unit is written when both groups have written it, four warps
                // each.  Counted together, one group's next unit could stand for
                // the other's; a group's own warps cannot be a unit apart (each
                // block's P is all four's, and each prefix unit has a block).
                if (reported >= prefixes) return;
                const volatile int32_t *w = sm.written;
                const int n = min(w[0], w[1]);
                if (__shfl_sync(0xffffffffu, n, 0) < 4 * (reported + 1)) return;
                if (lane == 0) {
                    __threadfence();
                    atomicAdd(a.sched + 2, 1);
                }
                __syncwarp();
                ++reported;
            };
            // bounded, reporting meanwhile
            auto until = [&](auto done) -> bool {
                unsigned long long start = 0;
                while (!done()) {
                    report();
                    __nanosleep(100);
                    const unsigned long long now = global_ns();
                    if (start == 0) start = now;
                    if (__any_sync(0xffffffffu, now - start > kWaitLimitNs)) {
                        if (lane == 0) raise_error(a.err, SVPA_DEVERR_TIMEOUT);
                        return false;
                    }
                }
                return true;
            };
            bool told = false;  // that the prefix is complete
            for (int jobs = 0;; ++jobs) {
                Job d;
                const bool more = decode(d);
                if (!more) d.w.kind = kEnd;
                const int ids = more ? page_tile(a, d, lane) : 0;
                if (lane == 0) sm.job = d;
                sm.job_ids[lane] = ids;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.job_full);
                if (!more) break;
                prefixes += d.w.prefix;
                // the producer has this one and is near its end
                if (!until([&]() -> bool {
                        return __all_sync(0xffffffffu, mbar_test(&sm.job_want, (uint32_t)(jobs & 1)));
                    }))
                    break;
                // a CTA whose unit waits for the prefix takes no second one: the CTAs
                // that end their prefix units take the rest (2 x 1 tokens of 32 heads
                // behind 4096: 27 us; with up to three units queued behind the wait 42)
                if (d.w.merge && !told) {
                    // every prefix unit was taken by a running CTA before this unit
                    // was: they end without waiting for anything of this one
                    if (!until([&]() -> bool {
                            return __all_sync(0xffffffffu, ld_acquire(a.sched + 2) >= a.p_units);
                        }))
                        break;
                    told = true;
                    if (lane == 0) mbar_arrive(&sm.prefix_done);
                }
            }
            until([&]() -> bool { return reported >= prefixes; });
            // (beside the last unit's work; behind the first unit it cost a short call 0.4 us)
            if (!a.verify) check_offsets();
        }
    } else {
        // ================================================= softmax and epilogue
        regs_inc<kRegsMany>();
        const int t = warp >= 8;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // query row of the tile == TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + kTmemS + (uint32_t)t * kNB + lane_off;
        const uint32_t tO = tmem + kTmemO + lane_off;
        const int gtid = (warp & 3) * 32 + lane;  // thread of the group
        const int G = a.G, jq = r / G, gi = r - jq * G;
        const float sc = a.scale_log2;
        uint32_t ns = 0, no[2] = {0, 0};  // phases of s_full[t], o_full[0], o_full[1]
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        uint32_t nb2 = 0;                 // phases of both
        bool ok = true;
        // bounded waits of the whole warp: one outcome for all lanes
        auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
            return __all_sync(0xffffffffu, bar_wait(bar, phase & 1u, a.err));
        };
        auto meet = [&]() -> bool {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.both);
            const bool good = wait(&sm.both, nb2++);
            tc_fence_after();
            return good;
        };
        for (int unit = 0; ok; ++unit) {
            if (!wait(&sm.q_full, (uint32_t)unit)) break;
            const Unit w = sm.unit;
            __syncwarp();
            if (w.kind == kEnd) break;
            if (lane == 0) mbar_arrive(&sm.q_empty);
            const bool pair = w.kind == kPair;
            const int n = t ? w.nB : w.nA;
            const int tok = w.tok0 + (pair && t ? a.tpt : 0) + jq;
            const int lim = w.lim0 + (w.causal ? tok - w.tok0 : 0);
            const unsigned long long anc = w.use_anc && jq < a.n_q ? a.anc[jq] : 0ull;
            float m_ref = -CUDART_INF_F, l_run = 0.f;
            for (int i = 0; i < n; ++i) {
                ok = wait(&sm.s_full[t], ns);
                if (!ok) break;
                ++ns;
                tc_fence_after();
                const int blk = pair ? i : 2 * i + t;
                const int pos0 = w.pos0 + blk * kNB;
                // all four loads in flight, one wait
                uint32_t raw[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, raw[c]);
                tmem_ld_wait();
                float s[kNB];
#pragma unroll
                for (int x = 0; x < kNB; ++x) s[x] = __uint_as_float(raw[x >> 5][x & 31]);
                const int h0 = lim - pos0;  // tokens of the block below the limit
                if (h0 < kNB) {
#pragma unroll
                    for (int x = 0; x < kNB / 64; ++x) {
                        const int sh = h0 - 64 * x;
                        const int hw = min(max(sh, 0), 64);
                        unsigned long long vis = hw == 64 ? ~0ull : ((1ull << hw) - 1ull);
                        if (sh >= 0) {
                            if (sh < 64) vis |= anc << sh;
                        } else if (sh > -64) {
                            vis |= anc >> (-sh);
                        }
#pragma unroll
                        for (int y = 0; y < 64; ++y)
                            if (!((vis >> y) & 1ull)) s[64 * x + y] = -CUDART_INF_F;
                    }
                }
                float pm[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) pm[x] = fmaxf(s[x], s[x + 4]);
#pragma unroll
                for (int x = 8; x < kNB; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y) pm[y] = fmaxf(fmaxf(pm[y], s[x + y]), s[x + y + 4]);
                const float mraw = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
                const float mx = mraw == -CUDART_INF_F ? -CUDART_INF_F : mraw * sc;
                float alpha = 1.f;
                bool rescale = false;
                if (mx > m_ref + kRescaleLog2 || (m_ref == -CUDART_INF_F && mx != -CUDART_INF_F)) {
                    alpha = ex2_approx(m_ref - mx);  // 0 when m_ref is -inf
                    m_ref = mx;
                    rescale = i > 0;
                    l_run *= alpha;
                }
                const float neg_m = m_ref == -CUDART_INF_F ? 0.f : -m_ref;
                const uint64_t sc2 = pack2(sc, sc), neg2 = pack2(neg_m, neg_m);
                uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < kNB / 32; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = unpack2(fma2(pack2(s[c * 32 + 2 * e], s[c * 32 + 2 * e + 1]), sc2, neg2));
                        const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                        ls[e & 3] = add2(ls[e & 3], pack2(p0, p1));
                        p[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(tS + c * 16, p);
                }
                const float2 lsum = unpack2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])));
                l_run += lsum.x + lsum.y;
                // V rows behind the last token may hold anything; both groups
                // clear them before they give out P
                if (pos0 + kNB > w.kv_end) {
                    const int vi = w.base + 2 * blk + 1;
                    ok = wait(&sm.full[vi % kRing], (uint32_t)(vi / kRing));
                    if (!ok) break;
                    const int t0 = w.kv_end - pos0;
                    constexpr int kVecs = kSlabs * 8;  // 16-byte words of a row
                    uint8_t *sv = sm.kv[vi % kRing];
                    for (int z = gtid; z < (kNB - t0) * kVecs; z += 128) {
                        const int row = t0 + z / kVecs, c = z % kVecs;
                        *reinterpret_cast<uint4 *>(sv + (row >> 3) * (kSlabs * 1024) + (c >> 3) * 1024 +
                                                   (row & 7) * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (__any_sync(0xffffffffu, rescale)) {
                    const float f = rescale ? alpha : 1.f;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t raw[32];
                        tmem_ld32(tO + t * 128 + c * 32, raw);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 32; ++x) raw[x] = __float_as_uint(__uint_as_float(raw[x]) * f);
                        tmem_st32(tO + t * 128 + c * 32, raw);
                    }
                }
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[t]);
            }
            if (!ok) break;

            // ---- epilogue
            const bool live = r < a.tpt * G && tok < w.tok1;
            const size_t row = (size_t)tok * a.Hq + (size_t)w.h * G + gi;
            const size_t prow = live ? part_row(a, max(w.slot, 0), w.h, tok, gi) : 0;
            const size_t pslot = (size_t)a.Hkv * a.tiles * 128;  // partial rows of a slot
            float m = m_ref, l = l_run;
            if (pair) {
                if (n > 0) {
                    ok = wait(&sm.o_full[t], no[t]);
                    if (!ok) break;
                    tc_fence_after();
                }
                const float inv = l > 0.f ? 1.f / l : 0.f;
                if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t raw[32];
                        tmem_ld32(tO + t * 128 + c * 32, raw);
                        tmem_ld_wait();
                        if (!live) continue;
                        if (w.slot < 0) {
                            const float *f = reinterpret_cast<const float *>(raw);
                            store_bf16x16(a.out + row * D + c * 32, f, inv, wide);
                            store_bf16x16(a.out + row * D + c * 32 + 16, f + 16, inv, wide);
                        } else {
                            float4 *o = part_cols<D>(a, prow) + c * 8 * 32;
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                o[x * 32] =
                                    make_float4(__uint_as_float(raw[4 * x]), __uint_as_float(raw[4 * x + 1]),
                                                __uint_as_float(raw[4 * x + 2]), __uint_as_float(raw[4 * x + 3]));
                        }
                    }
                    tc_fence_before();
                }
                if (live) {
                    if (w.slot >= 0) a.part_ml[prow] = make_float2(m, l);
                    else if (a.lse) a.lse[row] = (m + __log2f(l)) * kLn2;
                }
            } else {
                sm.stat[t][r] = make_float2(m_ref, l_run);
                if (w.merge) ok = wait(&sm.prefix_done, 0);
                if (!ok) break;
                ok = meet();
                if (!ok) break;
                const float2 sA = sm.stat[0][r], sB = sm.stat[1][r];
                if (w.nA > 0) ok = wait(&sm.o_full[0], no[0]);
                if (ok && w.nB > 0) ok = wait(&sm.o_full[1], no[1]);
                if (!ok) break;
                tc_fence_after();
                const int np = live && w.merge ? a.p_splits : 0;
                m = fmaxf(sA.x, sB.x);
                float fA = sA.x == -CUDART_INF_F ? 0.f : ex2_approx(sA.x - m);
                float fB = sB.x == -CUDART_INF_F ? 0.f : ex2_approx(sB.x - m);
                l = sA.y * fA + sB.y * fB;
                if (np == 0 && w.slot < 0) {
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    fA *= inv;
                    fB *= inv;
                }
                // group t takes half of the columns of both accumulators
                constexpr int kHalf = D / 2, kC = D / 64;  // columns, pieces of 32
                float o[kHalf];
                {
                    uint32_t ra[kC][32];
                    if (w.nA > 0) {
#pragma unroll
                        for (int c = 0; c < kC; ++c) tmem_ld32(tO + (t * kC + c) * 32, ra[c]);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int x = 0; x < kHalf; ++x) o[x] = w.nA > 0 ? __uint_as_float(ra[x >> 5][x & 31]) * fA : 0.f;
                    if (w.nB > 0) {
#pragma unroll
                        for (int c = 0; c < kC; ++c) tmem_ld32(tO + 128 + (t * kC + c) * 32, ra[c]);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < kHalf; ++x) o[x] = fmaf(__uint_as_float(ra[x >> 5][x & 31]), fB, o[x]);
                    }
                }
                // O is read: the next unit's first P V may start while this one is joined and stored
                ok = meet();
                if (!ok) break;
                for (int p = 0; p < np; ++p) {
                    const float2 ml = __ldcg(&a.part_ml[p * pslot + prow]);
                    const float4 *src = part_cols<D>(a, p * pslot + prow) + t * (kHalf / 4) * 32;
                    float4 v[kHalf / 4];
#pragma unroll
                    for (int x = 0; x < kHalf / 4; ++x) v[x] = __ldcg(src + x * 32);
                    if (ml.y == 0.f) continue;  // nothing there: not even zeros (a NaN stays)
                    const float mn = fmaxf(m, ml.x);
                    const float fo = l > 0.f ? ex2_approx(m - mn) : 0.f, fp = ex2_approx(ml.x - mn);
                    l = l * fo + ml.y * fp;
                    m = mn;
#pragma unroll
                    for (int x = 0; x < kHalf / 4; ++x) {
                        o[4 * x] = fmaf(v[x].x, fp, o[4 * x] * fo);
                        o[4 * x + 1] = fmaf(v[x].y, fp, o[4 * x + 1] * fo);
                        o[4 * x + 2] = fmaf(v[x].z, fp, o[4 * x + 2] * fo);
                        o[4 * x + 3] = fmaf(v[x].w, fp, o[4 * x + 3] * fo);
                    }
                }
                if (np > 0) {
                    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
                    for (int x = 0; x < kHalf; ++x) o[x] *= inv;
                }
                if (live) {
                    if (w.slot < 0) {
#pragma unroll
                        for (int x = 0; x < kHalf / 16; ++x)
                            store_bf16x16(a.out + row * D + t * kHalf + x * 16, o + x * 16, 1.f, wide);
                        if (t == 0 && a.lse) a.lse[row] = (m + __log2f(l)) * kLn2;
                    } else {
                        float4 *d = part_cols<D>(a, prow) + t * (kHalf / 4) * 32;
                        if (w.nA + w.nB > 0)
#pragma unroll
                            for (int x = 0; x < kHalf / 4; ++x)
                                d[x * 32] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                        if (t == 0) a.part_ml[prow] = make_float2(m, l);
                    }
                }
            }
            no[0] += w.nA > 0;
            no[1] += w.nB > 0;
            if (w.prefix) {
                __syncwarp();
                if (lane == 0) {
                    __threadfence_block();
                    atomicAdd(&sm.written[t], 1);
                }
            }
        }
    }
    // the softmax warps have waited for the issuer's last operations
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&a.sched[1], 1) == (int)gridDim.x - 1) {
            a.sched[0] = 0;
            a.sched[1] = 0;
            a.sched[2] = 0;
        }
    }
}

// Joins the partials of 32 rows of a query tile with log-sum-exp weights: one
// row a lane, the columns over the CTA's warps.
template <int D>
__global__ void __launch_bounds__(256) packed_combine_kernel(const __grid_constant__ PackedArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = D / 32;  // groups of four columns a warp takes
    const int quarter = blockIdx.x & 3, tile = blockIdx.x >> 2, h = blockIdx.y;
    const int r = quarter * 32 + lane, jq = r / a.G, gi = r - jq * a.G;
    const int tok = tile * a.tpt + jq;
    bool live = jq < a.tpt && tok < a.T;
    int first = 0;
    const int slots = a.p_splits + a.s_splits;
    if (live && a.verify) {
        const int b = tok / a.n_q;
        const int L = a.lens[b];
        // a bad length was reported, not computed
        live = L >= 0 && (long long)L + a.n_q <= (long long)a.max_blocks * kBlockSize;
        if (live && !a.member[b]) first = a.p_splits;
    } else if (live) {
        live = tok < a.cu[a.B];  // rows behind the last sequence stay as they are
    }
    if (!live) return;
    const size_t pslot = (size_t)a.Hkv * a.tiles * 128;
    const size_t prow = ((size_t)h * a.tiles + tile) * 128 + r;
    float m = -CUDART_INF_F, l = 0.f;
    float4 o[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int s = first; s < slots; ++s) {
        const float2 ml = a.part_ml[s * pslot + prow];
        if (ml.y == 0.f) continue;  // nothing there (a NaN is, and stays)
        const float mn = fmaxf(m, ml.x);
        const float fo = ex2_approx(m - mn), fn = ex2_approx(ml.x - mn);
        const float4 *src = part_cols<D>(a, s * pslot + prow) + warp * kPer * 32;
        l = l * fo + ml.y * fn;
        m = mn;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const float4 v = src[x * 32];
            o[x].x = o[x].x * fo + v.x * fn;
            o[x].y = o[x].y * fo + v.y * fn;
            o[x].z = o[x].z * fo + v.z * fn;
            o[x].w = o[x].w * fo + v.w * fn;
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t row = (size_t)tok * a.Hq + (size_t)h * a.G + gi;
    uint2 *dst = reinterpret_cast<uint2 *>(a.out + row * D + warp * kPer * 4);
#pragma unroll
    for (int x = 0; x < kPer; ++x)
        dst[x] = make_uint2(pack_bf16x2(o[x].x * inv, o[x].y * inv), pack_bf16x2(o[x].z * inv, o[x].w * inv));
    if (warp == 0 && a.lse) a.lse[row] = (m + __log2f(l)) * kLn2;
}

template <int D>
cudaError_t launch_t(const PackedMaps &m, const PackedArgs &a, int grid, cudaStream_t st) {
    const size_t smem = sizeof(Smem<D>);
    static DeviceMemo<int> attr_set;  // the shared-memory opt-in, once per device
    int done = 0;
    cudaError_t e = attr_set.get(&done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(packed_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    packed_attn_kernel<D><<<grid, kThreads, smem, st>>>(m.k, m.v, m.qt[0], m.qt[1], m.qs[0], m.qs[1], a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_attn(const PackedMaps &m, const PackedArgs &a, int head_dim, int grid, cudaStream_t st) {
    return head_dim == 128 ? launch_t<128>(m, a, grid, st) : launch_t<64>(m, a, grid, st);
}

cudaError_t launch_packed_combine(const PackedArgs &a, int head_dim, cudaStream_t st) {
    const dim3 grid(4 * a.tiles, a.Hkv);
    if (head_dim == 128) packed_combine_kernel<128><<<grid, 256, 0, st>>>(a);
    else packed_combine_kernel<64><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace svpa
