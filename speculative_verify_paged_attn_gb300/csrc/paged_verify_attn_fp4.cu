// paged_verify_attn_fp4.cu -- paged verification attention over 4-bit pages, on
// the 5th-generation tensor cores (tcgen05 + TMEM) for sm_103a.
//
// out = softmax(Q K^T * scale + mask) V with K and V decoded on the way: a code
// times its scale is exact in f16, so both products are f16 MMAs whose only
// rounded operand is the softmax's weights; the heads' factors go into the
// scores' scale and the output's.
//
// Both products are formed transposed.  S^T = K Q^T: the 128 tokens of a block
// are the rows of the MMA and the query rows (heads of the group x queries) its
// columns, padded to 16, 32, 64 or 128; O^T += V^T P^T: the head dimensions are
// the rows.  A token's row of codes is what one thread decodes: for K into its
// TMEM lane, which the MMA reads as its A operand, for V into shared memory.  In
// the other orientation the query rows would be padded to 128 and both decoded
// tiles would pass through shared memory twice, whose bandwidth is what bounds
// this kernel.
//
// The softmax has a token a thread, so that a column's maximum lies across
// threads: it is taken in a group's first block of a unit, and after that only
// when some score exceeds it by 11 in log2 units (a vote a block).  The reference
// lies 5 below that maximum, so that the largest weights are 2^5 to 2^16 and f16
// holds the small ones: 11 bits down to 2^-19 of the row's largest weight, below
// that an error of at most 2^-30 of it.  (At the maximum itself, tokens of 2^-18
// behind one dominant token were off by up to a hundredth, and of 2^-25 lost, while
// the fp32 sums counted them.  Further below it more blocks are done twice: 64 x 6
// queries whose scores have a standard deviation of 1.3, 2.5, 3.8 and 5 took 514,
// 515, 529 and 561 us at the maximum, 518, 518, 568 and 651 at 5 below, 518, 557, 655
// and 778 at 8.)
//
// Work: the 128-token blocks of all (sequence, kv head) pairs, in that order,
// split evenly over one persistent CTA per SM; the parts of the pairs that are
// cut are joined by a second kernel.
// Warps, up to 64 columns: 0-3 decode K, 12-15 decode V; 4-7 and 8-11 are two
// softmax groups that take the blocks in turn, and the epilogue; 16 copies the
// queries and turns them to f16 with 19; 17 and 18 issue the MMAs of P V and of S.
// (128 columns: Cfg.)  A warp reads the TMEM lanes of quadrant warp % 4.  Every
// role walks the same list of blocks.
// A decoding warp copies the pages of its own tokens ahead of itself (cp.async),
// so that it waits for no other warp.  64 x 1 queries of 64 / 8 heads of 128
// behind 8K to 32K tokens: tiled bulk copies of each page's codes and scales, 32 a
// block at some 95 cycles each, 855 us; a copying warp each for K and V 624; this
// 532, and 414 with the later steps; whole pages by untiled bulk copies into padded
// places 488, whose rows then lie two to a bank.
//
// The same workload reads 1.57 GB: 232 us at 6.8 TB/s.  No unit is saturated at 414:
// DRAM 56%; shared memory 60% (112 KB a block of 1,500 cycles; with 6 queries, 519
// us, 979 wavefronts and 64 KB of operands in 1,950); with 6 queries the tensor pipe
// 26% and the issue slots 59%.  The busiest warps are V's, 1,300 of a block's 1,500
// cycles (850 decoding, 450 issuing copies).  Left out, by 1 and by 6 queries: all
// copies 402, 510; all decoding 344, 457; all but one column's softmax 411, 441; seven
// eighths of both products' MMAs 409, 490; all of that but the scores' MMAs at once
// 335, 352.  So two thirds of the time and more is the chain of handovers of a block
// between the roles (scores, vote, weights, product), which two blocks in flight do
// not cover; which links of it has not been measured.  29-node trees of 32/8 heads, 64 behind 1K to 8K
// tokens: 264 (79 for their products).
// All waits are bounded: a role whose wait ran out goes on without waiting.
#include <math_constants.h>

#include <algorithm>
#include <cstddef>

#include "fp4.cuh"
#include "fp4_attn.h"

namespace svpa {

namespace {

constexpr int kPB = 8;                        // pages per block
constexpr int kNB = kPB * kBlockSize;         // tokens per block
constexpr float kMaxWeight = 65504.f;  // f16's largest
constexpr float kTopWeight = 5.f;      // log2 of a maximum's weight where the reference is taken from it
constexpr uint32_t kTmemCols = 512, kTmemS = 0, kTmemO = 256, kTmemK = 384;
constexpr int kSlab = kNB * 128;              // 64 f16 columns of 128 rows
constexpr float kLn2 = 0.69314718055994530942f;
enum { kBarHalf0 = 1, kBarSoft = 3, kBarPrep = 4 };  // named barriers

// ---------------------------------------------------------------- the work list
struct Piece {
    int b, h, f, n, nb, L;  // sequence, kv head, first block, blocks, the pair's blocks, history
    long long x;            // the first block's place in the list
};

__device__ __forceinline__ int blocks_of(const Fp4AttnArgs &a, int L) {
    const long long pages = ((long long)L + a.n_q + kBlockSize - 1) / kBlockSize;
    return L < 0 || pages > a.max_blocks ? 0 : (int)((pages + kPB - 1) / kPB);
}

// CTAs that get a share of W blocks.  (Shares of at least 2 to 6 blocks, against the
// cost of writing and joining parts, are slower unless pairs happen to fill them.)
__device__ __forceinline__ int shares_of(long long W) { return (int)min((long long)gridDim.x, W); }

struct Walk {
    int b, h, f, nb, L;
    long long x, left;
    __device__ __forceinline__ bool next(const Fp4AttnArgs &a, Piece &p) {
        if (left <= 0) return false;
        while (nb == 0) {
            L = __ldg(a.context_lens + b);
            nb = blocks_of(a, L);
            if (nb == 0) ++b;  // (counts no blocks)
        }
        p.b = b, p.h = h, p.f = f, p.nb = nb, p.L = L, p.x = x;
        p.n = (int)min((long long)(nb - f), left);
        left -= p.n, x += p.n, f += p.n;
        if (f == nb) {
            f = 0;
            if (++h == a.Hkv) h = 0, ++b, nb = 0;
        }
        return true;
    }
};

// A warp's place in the list, its unit and the one after (worked out while the
// warp waits for its unit's first data anyway), kept in shared memory: the
// registers are for scores, sums and codes.
struct Cursor {
    Walk w;
    Piece p[2];
    int more, at;
    __device__ __forceinline__ void look(const Fp4AttnArgs &a, int to) {
        if ((threadIdx.x & 31) == 0) {
            Walk u = w;
            more = u.next(a, p[to]);
            w = u;
        }
        __syncwarp();
    }
    __device__ __forceinline__ void begin(const Fp4AttnArgs &a, const Walk &from) {
        if ((threadIdx.x & 31) == 0) w = from, at = 1;
        look(a, 0);
    }
    // Whether there is a next unit; it is unit() then.
    __device__ __forceinline__ bool next(const Fp4AttnArgs &a) {
        __syncwarp();
        const int have = more, to = at;
        __syncwarp();
        if (!have) return false;
        if ((threadIdx.x & 31) == 0) at = to ^ 1;
        look(a, to);
        return true;
    }
    __device__ __forceinline__ const Piece &unit() const { return p[at]; }
};

template <int D, int NP>
struct Cfg {
    // Up to 64 columns: the two softmax groups take the blocks in turn, each with
    // a reference, sums and an O of its own, so that one block's chain of waits
    // runs beside the other's.  128: each takes half of every block's columns (two
    // O do not fit TMEM), and warps 0-3 decode V too.
    static constexpr bool kAlt = NP < 128;
    static constexpr int kQueryWarp = kAlt ? 16 : 12;  // the queries' copies; then the MMAs: P V, S; one idle
    static constexpr int kPvWarp = kQueryWarp + 1, kScoreWarp = kQueryWarp + 2;
    static constexpr int kThreads = 32 * (kQueryWarp + 4);
    // registers a thread, from the 96 (128 with 16 warps) at launch: their sum
    // over the warps of a scheduler stays within 5 * 96 (4 * 128)
    static constexpr int kRegsDecode = kAlt ? 64 : 112, kRegsIssue = NP == 64 ? 48 : 64;
    static constexpr int kRegsSoftmax = NP == 64 ? 152 : kAlt ? 128 : 160;
    static_assert((kAlt ? 2 : 1) * kRegsDecode + kRegsIssue + 2 * kRegsSoftmax <= (kAlt ? 5 * 96 : 4 * 128),
                  "registers handed over");
    static constexpr int kNH = kAlt ? NP : 64;        // columns of a softmax thread
    static constexpr int kCH = kNH < 32 ? kNH : 32;   // ... taken at a time
    static constexpr int kEC = NP / 2;                // columns of a group in the epilogue
    static constexpr int kSBufs = kAlt ? 4 : 2, kVBufs = kAlt ? 3 : 2, kQBufs = kAlt ? 2 : 1;
    static constexpr int kQ = NP * D * 2, kP = kNB * NP * 2;
    static constexpr int kCodes = kNB * D / 2, kScales = kPB * 128;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kRest = 13312;  // what is behind the tiles, and their alignment
    static constexpr int kRoom = (232448 - kRest - kQBufs * kQ - 2 * kP - kVBufs * 2 * kSlab) / kStage;
    static constexpr int kStages = kRoom < 8 ? kRoom : 8;
};

template <int D, int NP>
struct Smem {
    using C = Cfg<D, NP>;
    uint8_t q[C::kQBufs][C::kQ];      // [slab][NP rows][128 B], 128-byte swizzle
    uint8_t v[C::kVBufs][2 * kSlab];  // decoded V: [slab][128 tokens][128 B] (D 64: one slab)
    uint8_t p[2][C::kP];              // weights: [token][NP columns]
    uint8_t kc[C::kStages][C::kCodes], vc[C::kStages][C::kCodes];
    uint8_t ks[C::kStages][C::kScales], vs[C::kStages][C::kScales];
    float negm[2][64];                 // a group's columns: minus the reference maxima (0: none yet)
    float fac[2][64];                  // what a raised maximum leaves of the sums
    float top[2][4][64];               // a column's maximum in each quadrant
    float m[2][2][64];                 // [unit parity][group]: the reference maxima
    float sums[2][2][4][64];           // ... and each quadrant's sums
    // score -> log2 units, of the units in flight: one is written once S of the unit
    // two before is there, whose buffer the softmax has read four blocks earlier
    float mult[8];
    int32_t row_off[128];              // query row -> row of out behind the unit's first
    uint64_t k_full[2], k_empty[2], v_full[C::kVBufs], v_empty[C::kVBufs];
    uint64_t q_full[2], q_ready[2], q_empty[2];
    uint64_t s_full[C::kSBufs], s_empty[C::kSBufs], p_full[2], pv_done[2];
    uint64_t o_full, o_empty;
    long long scan[32];
    long long work;                    // all blocks
    int32_t b0, h0, f0;                // this CTA's first
    uint32_t tmem_base;
    uint32_t qmax[2][2];
    Cursor cursor[16], ahead[8];  // the warps' places in the list: where they work, and where they copy
};

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// A bounded wait; a role whose earlier wait ran out passes over it.
__device__ __forceinline__ void wait(bool &ok, uint64_t *bar, int phase, int32_t *err) {
    if (!ok || mbar_try_wait(bar, (uint32_t)(phase & 1))) return;
    const unsigned long long t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, (uint32_t)(phase & 1))) {
        if (global_ns() - t0 > kWaitLimitNs) {
            raise_error(err, SVPA_DEVERR_TIMEOUT);
            ok = false;
            return;
        }
    }
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Whether `v` holds for any of the `threads` threads of a named barrier.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
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
// Both halves times a factor, 0 where that is 0 (in place: registers).
__device__ __forceinline__ void scale_sums(uint64_t &v, float x, float y) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .f32 a, b;\n\tmov.b64 {a, b}, %0;\n\t"
        "setp.gt.f32 p, %1, 0f00000000;\n\tsetp.gt.f32 q, %2, 0f00000000;\n\t"
        "mul.rn.f32 a, a, %1;\n\tmul.rn.f32 b, b, %2;\n\t"
        "selp.f32 a, a, 0f00000000, p;\n\tselp.f32 b, b, 0f00000000, q;\n\t"
        "mov.b64 %0, {a, b};\n\t}"
        : "+l"(v)
        : "f"(x), "f"(y)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// N consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) { tmem_ld32(at, r); }
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The sums over a warp's lanes of N columns: v[0] of lane l is column l % N's.
template <int N>
__device__ __forceinline__ void column_sums(float (&v)[N], int lane) {
#pragma unroll
    for (int h = N / 2; h >= 1; h /= 2) {
        const bool upper = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float send = upper ? v[i] : v[i + h], keep = upper ? v[i + h] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
        }
    }
#pragma unroll
    for (int h = N; h < 32; h *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], h);
}

// Byte of column chunk c (eight columns) of token t in the weights' tile, whose
// rows of NP columns (64 a slab) have the swizzle as wide as they are.
template <int NP>
__device__ __forceinline__ uint32_t p_at(int t, int c) {
    if constexpr (NP == 16) return (uint32_t)(t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
    else if constexpr (NP == 32) return (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
    else return (uint32_t)((c >> 3) * kSlab + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}
// Its descriptor (MN-major, the tokens are K), from its first byte.
template <int NP>
__device__ __forceinline__ uint64_t p_desc(uint32_t at) {
    constexpr uint32_t row = NP < 64 ? 2 * NP : 128;
    constexpr uint64_t layout = NP == 16 ? 6 : NP == 32 ? 4 : 2;
    return (umma_desc_sw128(at, kSlab, 8 * row) & ~(7ull << 61)) | layout << 61;
}

// A descriptor `bytes` further on (within the 14 bits of its address field).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) {
    uint64_t r;
    asm("{\n\t.reg .b32 lo, hi;\n\tmov.b64 {lo, hi}, %1;\n\tadd.u32 lo, lo, %2;\n\tmov.b64 %0, {lo, hi};\n\t}"
        : "=l"(r)
        : "l"(d), "r"(bytes >> 4));
    return r;
}

// f16 A and B, fp32 D, 128 rows; A and B as they lie (1: MN-major).
__host__ __device__ constexpr uint32_t idesc(int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// ---------------------------------------------------------------- decoding
// 32 codes and their two scales to 16 f16 pairs.
__device__ __forceinline__ void decode32(const uint4 &w, uint32_t two_scales, uint32_t *out) {
    const uint32_t s = e4m3x2_to_f16x2(two_scales & 0xffffu);
    const __half2 pair = *reinterpret_cast<const __half2 *>(&s);
    const __half2 first = __low2half2(pair), second = __high2half2(pair);
    const uint32_t lo = *reinterpret_cast<const uint32_t *>(&first);
    const uint32_t hi = *reinterpret_cast<const uint32_t *>(&second);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[4];
        e2m1x8_to_f16(in[i], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[4 * i + j] = mul_f16x2(h[j], i < 2 ? lo : hi);
    }
}

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ void st_shared(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A staged row of codes (32 of them at codes ^ 16 c) to its place as an MMA
// operand: K's into the TMEM lane at `to`, V's into shared memory (its 16-byte
// piece k of a slab at to ^ 16 k).  (Two quarters of a row of 128 at a time: one
// costs 4% more; all four gain 1% on long sequences and cost short ones 3 to 6%,
// whose roles' loops share an instruction cache.)
template <int D>
__device__ __forceinline__ void decode_row(uint32_t codes, uint2 scales, bool is_v, uint32_t to) {
#pragma unroll 1
    for (int c = 0; c < D / 32; c += 2) {
        const uint4 w0 = ld_shared(codes ^ (16 * c)), w1 = ld_shared(codes ^ (16 * c + 16));
        uint32_t r[16];
        decode32(w0, scales.x, r);
        if (is_v) {
#pragma unroll
            for (int k = 0; k < 4; ++k) st_shared(to ^ (16 * k), r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        } else {
            tmem_st(to, r);
        }
        decode32(w1, scales.x >> 16, r);
        if (is_v) {
#pragma unroll
            for (int k = 0; k < 4; ++k) st_shared(to ^ (16 * k + 64), r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
            to += kSlab;
        } else {
            tmem_st(to + 16, r);
            to += 32;
        }
        scales.x = scales.y;  // the next two
    }
}

// The unit's queries, bf16 as they landed, to f16 in place at one power of two
// that puts the largest of them in [2^14, 2^15); what falls below f16's smallest
// value there is less than 2^-39 of it.  Sets the scores' multiplier.
template <int D, int NP>
__device__ __forceinline__ void prepare_queries(Smem<D, NP> &sm, const Fp4AttnArgs &a, int slot, int unit, float kf,
                                                int tid) {  // by two warps
    constexpr int kRow = 8, kSlabs = D / 64;  // 16-byte chunks of a row of a slab
    uint4 *q = reinterpret_cast<uint4 *>(sm.q[slot]);
    const int per = a.M * kRow;
    uint32_t top = 0u;
#pragma unroll 1
    for (int s = 0; s < kSlabs; ++s)
#pragma unroll 2
        for (int i = tid; i < per; i += 64) top = max(top, bf16_amax8(q[s * NP * kRow + i]));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) sm.qmax[unit & 1][tid >> 5] = top;
    named_barrier_sync(kBarPrep, 64);
    top = max(sm.qmax[unit & 1][0], sm.qmax[unit & 1][1]);
    int e = 0;
    if (top > 0x7f7fu) {
        if (tid == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
    } else if (top != 0u) {
        e = min(max(141 - (int)(top >> 7), -126), 126);
    }
    const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 1
    for (int s = 0; s < kSlabs; ++s)
#pragma unroll 2
        for (int i = tid; i < per; i += 64) {
            const uint4 x = q[s * NP * kRow + i];
            uint4 y;
            y.x = pack_f16x2(bf16_lo(x.x) * scale, bf16_hi(x.x) * scale);
            y.y = pack_f16x2(bf16_lo(x.y) * scale, bf16_hi(x.y) * scale);
            y.z = pack_f16x2(bf16_lo(x.z) * scale, bf16_hi(x.z) * scale);
            y.w = pack_f16x2(bf16_lo(x.w) * scale, bf16_hi(x.w) * scale);
            q[s * NP * kRow + i] = y;
        }
    // (positive, so that a masked score stays -inf)
    if (tid == 0)
        sm.mult[unit & 7] = fmaxf(a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23) * kf, 1e-30f);
}

// A decoding warp: the pages of its own 32 tokens of every block, copied 16
// bytes a lane (cp.async) kStages - 1 blocks ahead, K's (kv 0), V's (1) or both.
template <int D, int NP>
__device__ __forceinline__ void decode_role(Smem<D, NP> &sm, const Fp4AttnArgs &a, const Walk &w, uint32_t tmem,
                                            int kv0, int kv1) {
    using C = Cfg<D, NP>;
    constexpr int kStages = C::kStages, kCodePage = kBlockSize * D / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp & 3, t = 32 * part + lane;
    const uint32_t k_at = tmem + ((uint32_t)(32 * part) << 16) + kTmemK;
    Cursor &cur = sm.cursor[warp], &ahead = sm.ahead[part + (warp & 4)];
    cur.begin(a, w);
    ahead.begin(a, w);
    // half a warp copies a page, 256 bytes of its codes at a time: where a lane's 16
    // go (in the swizzle that makes the rows' reads free of conflicts; 128
    // dimensions: ^ 32 in the odd quarters), and those of the scales
    constexpr int kRowChunks = D / 32, kScaleLanes = D / 16;
    const int half = lane >> 4, hl = lane & 15, page = 2 * part + half;
    const uint32_t code_dst = (uint32_t)(page * kCodePage + (hl / kRowChunks) * (D / 2) +
                                         (((hl % kRowChunks) ^ (hl >> 3)) << 4));
    const uint32_t scale_dst = (uint32_t)(page * 128 + hl * 16);
    // this thread's row of a stage (the swizzle is in the address already), its scales and its V row
    const uint32_t raw0 = smem_u32(kv0 ? sm.vc[0] : sm.kc[0]), raws0 = smem_u32(kv0 ? sm.vs[0] : sm.ks[0]);
    const uint32_t my_codes = (uint32_t)(t * (D / 2)) + ((D == 128 ? (t >> 1) & 3 : (t >> 2) & 1) << 4);
    const uint32_t my_scales = (uint32_t)((t >> 4) * 128 + (t & 15) * (D / 16));
    const uint32_t v_row = smem_u32(sm.v[0]) + t * 128 + ((t & 7) << 4);
    constexpr uint32_t kToV = sizeof(sm.kc), kToVs = sizeof(sm.ks);  // from K's stages to V's
    int ids = -1, ci = 0, cn = 0, cst = 0, ch = 0;  // copies: pages, block in the piece, its blocks, stage, kv head
    bool more = true;
    auto copy_block = [&]() {
        if (more && ci == cn) {
            more = ahead.next(a);
            ci = 0, cn = more ? ahead.unit().n : 0, ch = ahead.unit().h;
        }
        if (more) {
            if ((ci & 15) == 0) {  // the pages of 16 blocks, two a block
                const Piece &p = ahead.unit();
                const int at = (ci + lane / 2) * kPB + 2 * part + (lane & 1);
                const int pages = (p.L + a.n_q + kBlockSize - 1) / kBlockSize - p.f * kPB;
                ids = -1;
                if (at < pages && at < cn * kPB) {
                    ids = __ldg(a.block_table + (size_t)p.b * a.max_blocks + (size_t)p.f * kPB + at);
                    if (ids < 0 || ids >= a.num_blocks) {
                        if (kv0 == 0) raise_error(a.err, SVPA_DEVERR_BAD_BLOCK);
                        ids = -1;
                    }
                }
            }
            // (A page behind the sequence's last is not copied: its tokens are masked, their V
            // rows zeroed.  Nor is one whose id was refused: what the stage held goes into that
            // sequence's rows, and the call reports it.)
            const int id = __shfl_sync(0xffffffffu, ids, 2 * (ci & 15) + half);
            if (id >= 0) {
                // (num_blocks * Hkv is below 2^31)
                const size_t at = (size_t)(uint32_t)(id * a.Hkv + ch) * fp4_tile_bytes(D) + (uint32_t)(16 * hl);
#pragma unroll 1
                for (int kv = kv0; kv < kv1; ++kv) {
                    const uint8_t *src = (kv ? a.v_pool : a.k_pool) + at;
                    const bool next = kv != kv0;
                    const uint32_t dst = raw0 + (next ? kToV : 0u) + cst * C::kCodes + code_dst;
#pragma unroll
                    for (int k = 0; k < kCodePage / 256; ++k)
                        cp_async_16((D == 128 && (k & 1) ? dst ^ 32 : dst) + 256 * k, src + 256 * k);
                    if (hl < kScaleLanes)
                        cp_async_16(raws0 + (next ? kToVs : 0u) + cst * C::kScales + scale_dst, src + kCodePage);
                }
            }
            ++ci;
            cst = cst + 1 == kStages ? 0 : cst + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy_block();
    bool ok = true;
    int j = 0, st = 0, vb = 0, vphase = 0;
#pragma unroll 1
    while (cur.next(a)) {
        const Piece &p = cur.unit();
        const int n = p.n;
        int left = p.L + a.n_q - p.f * kNB - t;  // > 0: this thread's token is one of the sequence's
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++j, left -= kNB) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
#pragma unroll 1
            for (int kv = kv0; kv < kv1; ++kv) {
                const bool next = kv != kv0;
                const uint32_t sc_at = raws0 + (next ? kToVs : 0u) + st * C::kScales + my_scales;
                uint2 sc = make_uint2(0u, 0u);
                if (D == 128) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(sc.x), "=r"(sc.y) : "r"(sc_at));
                else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc.x) : "r"(sc_at));
                if (kv) {
                    if (left <= 0) sc = make_uint2(0u, 0u);  // (what such a slot holds is anything)
                    if (j >= C::kVBufs) wait(ok, &sm.v_empty[vb], vphase ^ 1, a.err);
                } else if (j >= 2) {
                    wait(ok, &sm.k_empty[j & 1], (j - 2) >> 1, a.err);
                    tc_fence_after();
                }
                decode_row<D>(raw0 + (next ? kToV : 0u) + st * C::kCodes + my_codes, sc, kv,
                              kv ? v_row + vb * (2 * kSlab) : k_at + 64 * (j & 1));
                if (kv) {
                    fence_proxy_async_smem();
                    warp_arrive(&sm.v_full[vb]);
                    if (++vb == C::kVBufs) vb = 0, vphase ^= 1;
                } else {
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(&sm.k_full[j & 1]);
                }
            }
            copy_block();  // (behind the arrivals: the products begin meanwhile)
            st = st + 1 == kStages ? 0 : st + 1;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- the softmax
template <int D, int NP>
__device__ __forceinline__ void softmax_role(Smem<D, NP> &sm, const Fp4AttnArgs &a, const Walk &w, uint32_t tmem) {
    using C = Cfg<D, NP>;
    constexpr bool kAlt = C::kAlt;
    constexpr int NH = C::kNH, CH = C::kCH, NCH = NH / CH, kStep = kAlt ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, g = (warp - 4) >> 2, t = 32 * quad + lane, c0 = kAlt ? 0 : g * NH;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t o_at = lanes + kTmemO + (kAlt ? g * NP : c0);  // this group's columns of O
    const int live = min(max(a.M - c0, 0), NH);  // columns with a query row
    Cursor &cur = sm.cursor[warp];
    cur.begin(a, w);
    bool ok = true;
    int j0 = 0, unit = 0, last = 0;  // the unit's first block; whether the last unit is cut at its end
    uint64_t sum[NH / 2];
#pragma unroll 1
    for (; cur.next(a); ++unit) {
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) sum[i] = 0ull;
        const Piece &p = cur.unit();
        const float fv = fp4_factor(a.v_factor, p.h, a.err);
        const int n = p.n, seen = p.L - p.f * kNB;  // blocks; history from the first block on
        float *m_unit = sm.m[unit & 1][g];
        float mult = 1.f;
#pragma unroll 1
        for (int i = kAlt ? (g - j0) & 1 : 0; i < n; i += kStep) {
            const int j = j0 + i, sb = j % C::kSBufs;
            const bool first = i < kStep;
            wait(ok, &sm.s_full[sb], j / C::kSBufs, a.err);
            tc_fence_after();
            if (first) mult = sm.mult[unit & 7];
            const uint64_t mult2 = pack2(mult, mult);
            const uint32_t sa = lanes + kTmemS + (uint32_t)(sb * NP + c0);
            // which columns see this thread's token
            const int at = i * kNB + t - seen;  // >= 0: a speculative slot
            const bool edge = (i + 1) * kNB > seen;
            unsigned long long vis = ~0ull;
            if (edge && at >= 0) vis = at >= a.n_q ? 0ull : a.slots[at][kAlt ? 0 : g];
            uint8_t *pt = sm.p[j & 1];
            uint32_t s[CH];
            auto load = [&](int ch) {
                tmem_ld(sa + (uint32_t)(ch * CH), s);
                tmem_ld_wait();
                if (edge) {
                    asm volatile("" ::: "memory");  // (a branch, no predicates)
                    const uint32_t v = (uint32_t)(vis >> (ch * CH));
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if (!(v >> c & 1u)) s[c] = 0xff800000u;
                }
            };
            // A weight may be up to f16's largest value.  Beyond that the block is taken
            // back, what cancels being below 2^-24 of the sums to come, and done again
            // under new references.
            bool raise = first;
            float sign = 1.f;
#pragma unroll 1
            while (true) {
                if (raise) {
                    // the columns' maxima over the block's tokens, and new references
#pragma unroll 1
                    for (int ch = 0; ch < NCH; ++ch) {
                        load(ch);
                        float mine = -CUDART_INF_F;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const float v = warp_max(__uint_as_float(s[c]));
                            if (lane == c) mine = v;
                        }
                        if (lane < CH) sm.top[g][quad][ch * CH + lane] = mine;
                    }
                    named_barrier_sync(kBarHalf0 + g, 128);
                    // (a column a thread)
                    const int c = threadIdx.x & 127;
                    float m_new = 0.f, fac = 0.f;
                    if (c < NH) {
                        const float top = fmaxf(fmaxf(sm.top[g][0][c], sm.top[g][1][c]),
                                                fmaxf(sm.top[g][2][c], sm.top[g][3][c])) *
                                              mult -
                                          kTopWeight;
                        const float old = first ? -CUDART_INF_F : m_unit[c];
                        m_new = fmaxf(old, top);
                        // (0 well before a weight under the old reference overflows, at 2^128: what
                        // that leaves in the sums is no number)
                        fac = old == m_new ? 1.f : m_new - old > 96.f ? 0.f : ex2_approx(old - m_new);
                        m_unit[c] = m_new;
                        sm.negm[g][c] = m_new == -CUDART_INF_F ? 0.f : -m_new;
                        sm.fac[g][c] = fac;
                    }
                    named_barrier_sync(kBarHalf0 + g, 128);
                    if (!first) {
                        // what was summed so far, here and in O, once the last block's P V is there
                        // (a weight that overflowed leaves a sum that is none, and a factor 0)
                        const float4 *fc = reinterpret_cast<const float4 *>(sm.fac[g]);
#pragma unroll
                        for (int x = 0; x < NH / 2; ++x) {
                            const float2 f = reinterpret_cast<const float2 *>(fc)[x];
                            scale_sums(sum[x], f.x, f.y);
                        }
                        wait(ok, &sm.pv_done[(j - kStep) & 1], (j - kStep) >> 1, a.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int c8 = 0; c8 < NH; c8 += 8) {
                            uint32_t o[8];
                            tmem_ld(o_at + (uint32_t)c8, o);
                            tmem_ld_wait();
                            const float4 f = fc[c8 / 4], f2 = fc[c8 / 4 + 1];
                            const float fs[8] = {f.x, f.y, f.z, f.w, f2.x, f2.y, f2.z, f2.w};
#pragma unroll
                            for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fs[x]);
                            tmem_st(o_at + (uint32_t)c8, o);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                }
                // the weights of block j, once the products that read their place are done
                const int before = j - 2;
                if (before >= 0) wait(ok, &sm.pv_done[before & 1], before >> 1, a.err);
                const uint64_t sign2 = pack2(sign, sign);
                float top = 0.f;
#pragma unroll
                for (int ch = 0; ch < NCH; ++ch) {
                    if (ch * CH >= live) break;  // (the same for the whole warp)
                    load(ch);
                    const float4 *nm = reinterpret_cast<const float4 *>(&sm.negm[g][ch * CH]);
#pragma unroll
                    for (int c = 0; c < CH; c += 8) {
                        if (ch * CH + c >= live) break;
                        uint32_t pk[4];
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            const float4 n = nm[c / 4 + k / 2];
                            const float2 x0 = unpack2(fma2(
                                pack2(__uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1])), mult2,
                                pack2(n.x, n.y)));
                            const float2 x1 = unpack2(fma2(
                                pack2(__uint_as_float(s[c + 2 * k + 2]), __uint_as_float(s[c + 2 * k + 3])), mult2,
                                pack2(n.z, n.w)));
                            const float u0 = ex2_approx(x0.x), v0 = ex2_approx(x0.y);
                            const float u1 = ex2_approx(x1.x), v1 = ex2_approx(x1.y);
                            const int at2 = (ch * CH + c) / 2 + k;
                            sum[at2] = fma2(pack2(u0, v0), sign2, sum[at2]);
                            sum[at2 + 1] = fma2(pack2(u1, v1), sign2, sum[at2 + 1]);
                            top = max3(max3(top, u0, v0), u1, v1);
                            pk[k] = pack_f16x2(u0, v0);  // a weight keeps 11 bits
                            pk[k + 1] = pack_f16x2(u1, v1);
                        }
                        *reinterpret_cast<uint4 *>(pt + p_at<NP>(t, (c0 + ch * CH + c) / 8)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                }
                if (raise) break;  // (no weight is above 2^5)
                if (sign < 0.f) {
                    sign = 1.f, raise = true;
                    continue;
                }
                if (!barrier_any(kBarHalf0 + g, 128, top > kMaxWeight)) break;
                sign = -1.f;
            }
            tc_fence_before();
            warp_arrive(&sm.s_empty[sb]);
            fence_proxy_async_smem();
            warp_arrive(&sm.p_full[j & 1]);
        }
        // ------------------------------------------------ the unit's epilogue
        const bool whole = p.n == p.nb;
        const int slot = 2 * (int)blockIdx.x + (p.x == w.x ? 0 : 1);
        const size_t row0 = (size_t)p.b * a.n_q * a.Hq + (size_t)p.h * a.G;
        // the groups with a block of this unit (their O hold something)
        const bool has0 = !kAlt || p.n > 1 || (j0 & 1) == 0, has1 = kAlt && (p.n > 1 || (j0 & 1) == 1);
        j0 += p.n;
#pragma unroll
        for (int c = 0; c < NH; c += 8) {  // (eight at a time: registers)
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float2 f = unpack2(sum[(c + k) / 2]);
                v[k] = f.x, v[k + 1] = f.y;
            }
            column_sums<8>(v, lane);
            if (lane < 8) sm.sums[unit & 1][g][quad][c + lane] = v[0];
        }
        if (kAlt) named_barrier_sync(kBarSoft, 256);
        else named_barrier_sync(kBarHalf0 + g, 128);
        // the columns g * kEC .. of both groups' results, a column a lane: their
        // common maximum and sum, and what each O is multiplied by
        constexpr int EC = C::kEC, CE = EC < 32 ? EC : 32, NE = EC / CE;
        const int e0 = g * EC;
        float w0[NE], w1[NE];
#pragma unroll
        for (int ch = 0; ch < NE; ++ch) {
            const int r = e0 + ch * CE + (lane & (CE - 1)), c = kAlt ? r : r - e0, ga = kAlt ? 0 : g;
            auto total = [&](int gg) {
                const float(*q)[64] = sm.sums[unit & 1][gg];
                return (q[0][c] + q[1][c]) + (q[2][c] + q[3][c]);
            };
            float m0 = has0 ? sm.m[unit & 1][ga][c] : -CUDART_INF_F, l0 = has0 ? total(ga) : 0.f;
            const float m1 = has1 ? sm.m[unit & 1][1][c] : -CUDART_INF_F, l1 = has1 ? total(1) : 0.f;
            const float m = fmaxf(m0, m1);
            w0[ch] = m0 == m ? 1.f : ex2_approx(m0 - m);
            w1[ch] = m1 == m ? 1.f : ex2_approx(m1 - m);
            const float l = l0 * w0[ch] + l1 * w1[ch];
            if (whole) {
                const float inv = l > 0.f ? fv / l : 0.f;
                w0[ch] *= inv, w1[ch] *= inv;
            }
            if (quad == 0 && lane < CE && r < a.M) {
                if (!whole) reinterpret_cast<float2 *>(a.part_ml)[(size_t)slot * a.M + r] = make_float2(m, l);
                else if (a.lse) a.lse[row0 + sm.row_off[r]] = (m + __log2f(l)) * kLn2;
            }
        }
        wait(ok, &sm.o_full, unit, a.err);
        tc_fence_after();
        // turned in this group's part of the weights' place, whose products are all
        // done (the next unit's first weights wait for a barrier of the group)
        float *turn = reinterpret_cast<float *>(kAlt ? sm.p[g] : sm.p[0] + g * kSlab);
#pragma unroll
        for (int ch = 0; ch < NE; ++ch) {
            if (e0 + ch * CE >= a.M) break;
            uint32_t o[CE];
            tmem_ld(lanes + kTmemO + (uint32_t)((has0 ? 0 : NP) + e0 + ch * CE), o);
            tmem_ld_wait();
            const float wa = has0 ? w0[ch] : w1[ch];
#pragma unroll
            for (int c = 0; c < CE; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, wa, c));
            if (has0 && has1) {
                uint32_t o1[CE];
                tmem_ld(lanes + kTmemO + (uint32_t)(NP + e0 + ch * CE), o1);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < CE; ++c)
                    o[c] = __float_as_uint(fmaf(__uint_as_float(o1[c]), __shfl_sync(0xffffffffu, w1[ch], c),
                                                __uint_as_float(o[c])));
            }
            if (NE == 1) {  // O is in registers
                tc_fence_before();
                warp_arrive(&sm.o_empty);
            }
            if (ch > 0) named_barrier_sync(kBarHalf0 + g, 128);
            if (t < D) {
#pragma unroll
                for (int c = 0; c < CE; ++c) turn[c * D + t] = __uint_as_float(o[c]);
            }
            named_barrier_sync(kBarHalf0 + g, 128);
            const int rows = min(CE, a.M - e0 - ch * CE);
#pragma unroll 1
            for (int c = quad; c < rows; c += 4) {
                if (lane >= D / 4) break;
                const int r = e0 + ch * CE + c;
                const float4 v = reinterpret_cast<const float4 *>(turn + c * D)[lane];
                if (whole)
                    reinterpret_cast<uint2 *>(a.out + (row0 + sm.row_off[r]) * D)[lane] =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                else
                    reinterpret_cast<float4 *>(a.part_acc + ((size_t)slot * a.M + r) * D)[lane] = v;
            }
        }
        if (NE > 1 || e0 >= a.M) {
            tc_fence_before();
            warp_arrive(&sm.o_empty);
        }
        last = p.f == 0 && !whole;
    }
    // A pair that begins in this CTA's share and goes on behind it: its parts are
    // joined by the next kernel.
    if (warp == 4 && lane == 0) {
        Fp4Join d = {0, 0, 0, 0};
        if (last > 0) {
            const long long W = sm.work, nsh = shares_of(W);
            const Piece &p = cur.unit();
            d.b = p.b, d.h = p.h, d.slot = 2 * (int)blockIdx.x + (p.x == w.x ? 0 : 1);
            d.parts = (int)(((p.x + p.nb) * nsh - 1) / W) - (int)blockIdx.x + 1;
        }
        a.joins[blockIdx.x] = d;
    }
}

template <int D, int NP>
__global__ void __launch_bounds__(Cfg<D, NP>::kThreads, 1)
    fp4_attn_kernel(const __grid_constant__ CUtensorMap mq0, const __grid_constant__ CUtensorMap mq1,
                    const __grid_constant__ Fp4AttnArgs a) {
    using C = Cfg<D, NP>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, NP> &sm =
        *reinterpret_cast<Smem<D, NP> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel waits for this one's end
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_ready[i], 2);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.p_full[i], C::kAlt ? 4 : 8);
            mbar_init(&sm.pv_done[i], 1);
        }
        for (int i = 0; i < C::kVBufs; ++i) {
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int i = 0; i < C::kSBufs; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], C::kAlt ? 4 : 8);
        }
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.o_empty, 8);
        fence_mbar_init();
    }
    if (warp == C::kQueryWarp && lane == 0) {
        prefetch_tensormap(&mq0);
        prefetch_tensormap(&mq1);
    }
    // query rows past M are never copied: zeros
    for (int i = tid; i < (int)sizeof(sm.q) / 16; i += C::kThreads)
        reinterpret_cast<uint4 *>(sm.q[0])[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < a.M) sm.row_off[tid] = tid / a.G * a.Hq + tid % a.G;
    fence_proxy_async_smem();
    if (warp == C::kPvWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // the number of blocks, and where this CTA's share of them begins
    const int per = (a.B + C::kThreads - 1) / C::kThreads;
    const int lo = min(tid * per, a.B), hi = min(lo + per, a.B);
    long long mine = 0;
    for (int b = lo; b < hi; ++b) {
        const int n = blocks_of(a, __ldg(a.context_lens + b));
        if (n == 0 && blockIdx.x == 0) raise_error(a.err, SVPA_DEVERR_BAD_VALUE);
        mine += (long long)n * a.Hkv;
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) sm.scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long W = 0, before = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
        if (i == warp) before = W;
        W += sm.scan[i];
    }
    const int nsh = shares_of(W);
    const long long xs = (int)blockIdx.x < nsh ? (long long)blockIdx.x * W / nsh : W;
    const long long xe = (int)blockIdx.x < nsh ? (long long)(blockIdx.x + 1) * W / nsh : W;
    before += incl - mine;
    if (xs < xe && xs >= before && xs < before + mine) {
        long long x = before;
        int b = lo;
        while (true) {
            const int nb = blocks_of(a, __ldg(a.context_lens + b));
            if (xs < x + (long long)nb * a.Hkv) {
                sm.b0 = b, sm.h0 = (int)((xs - x) / nb), sm.f0 = (int)((xs - x) % nb);
                break;
            }
            x += (long long)nb * a.Hkv;
            ++b;
        }
    }
    if (tid == 0) sm.work = W;
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    Walk w;
    w.b = w.h = w.f = w.nb = w.L = 0;
    w.x = xs, w.left = xe - xs;
    if (xs < xe) w.b = sm.b0, w.h = sm.h0, w.f = sm.f0;
    Piece p;
    bool ok = true;

    if (warp < 4) {
        regs_dec<C::kRegsDecode>();
        decode_role<D, NP>(sm, a, w, tmem, 0, C::kAlt ? 1 : 2);
    } else if (warp < 12) {
        regs_inc<C::kRegsSoftmax>();
        softmax_role<D, NP>(sm, a, w, tmem);
    } else if (C::kAlt && warp < 16) {
        regs_dec<C::kRegsDecode>();
        decode_role<D, NP>(sm, a, w, tmem, 1, 2);
    } else {
        regs_dec<C::kRegsIssue>();
        if (warp == C::kQueryWarp || warp == C::kQueryWarp + 3) {
            // ============================================ the queries: copied, and turned to f16
            const int tid = (warp == C::kQueryWarp ? 0 : 32) + lane;
            const uint64_t pol = policy_evict_first();
            int unit = 0;
    #pragma unroll 1
            for (; w.next(a, p); ++unit) {
                const float kf = fp4_factor(a.k_factor, p.h, a.err);
                if (warp == C::kQueryWarp) {
                    if (unit >= C::kQBufs) wait(ok, &sm.q_empty[unit % C::kQBufs], unit / C::kQBufs - 1, a.err);
                    if (ok && lane == 0) {
                        uint64_t *bar = &sm.q_full[unit % C::kQBufs];
                        mbar_arrive_expect_tx(bar, (uint32_t)(a.M * D * 2));
                        tma_load_4d(sm.q[unit % C::kQBufs], &mq0, 0, p.h * a.G, 0, p.b, bar, pol);
                        if (D == 128)
                            tma_load_4d(sm.q[unit % C::kQBufs] + NP * 128, &mq1, 0, p.h * a.G, 0, p.b, bar, pol);
                    }
                    __syncwarp();
                }
                // (also when an earlier wait ran out: what was copied has to land)
                bool landed = true;
                if (ok) wait(landed, &sm.q_full[unit % C::kQBufs], unit / C::kQBufs, a.err);
                ok = ok && landed;
                prepare_queries<D, NP>(sm, a, unit % C::kQBufs, unit, kf, tid);
                fence_proxy_async_smem();
                warp_arrive(&sm.q_ready[unit % C::kQBufs]);
            }
        } else if (warp == C::kScoreWarp) {
            // ============================================ S^T = K Q^T
            const uint32_t id = idesc(NP, 0, 0);
            int j = 0, unit = 0;
    #pragma unroll 1
            for (; ok && w.next(a, p); ++unit) {
    #pragma unroll 1
                for (int i = 0; i < p.n; ++i, ++j) {
                    const int sb = j % C::kSBufs;
                    if (i == 0) wait(ok, &sm.q_ready[unit % C::kQBufs], unit / C::kQBufs, a.err);
                    if (j >= C::kSBufs) wait(ok, &sm.s_empty[sb], j / C::kSBufs - 1, a.err);
                    wait(ok, &sm.k_full[j & 1], j >> 1, a.err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t qd = umma_desc_sw128(smem_u32(sm.q[unit % C::kQBufs]), 16, 1024);
                    if (elect_one()) {
    #pragma unroll 1
                        for (int k = 0; k < D / 16; ++k)
                            umma_bf16_tmem_a(tmem + kTmemS + (uint32_t)(sb * NP), tmem + kTmemK + 64 * (j & 1) + 8 * k,
                                             desc_at(qd, (k >> 2) * NP * 128 + (k & 3) * 32), id,
                                             k == 0 ? 0u : 1u);
                        umma_commit(&sm.k_empty[j & 1]);
                        umma_commit(&sm.s_full[sb]);
                        if (i == p.n - 1) umma_commit(&sm.q_empty[unit % C::kQBufs]);
                    }
                    __syncwarp();
                }
            }
            // the last arrivals land before the barriers are given up
            if (ok && j > 0) {
                wait(ok, &sm.k_empty[(j - 1) & 1], (j - 1) >> 1, a.err);
                wait(ok, &sm.q_empty[(unit - 1) % C::kQBufs], (unit - 1) / C::kQBufs, a.err);
            }
        } else if (warp == C::kPvWarp) {
            // ============================================ O^T += V^T P^T
            const uint32_t id = idesc(NP, 1, 1);
            constexpr uint32_t row = NP < 64 ? 2 * NP : 128;  // bytes of a token's weights
            int j = 0, unit = 0;
    #pragma unroll 1
            for (; ok && w.next(a, p); ++unit) {
    #pragma unroll 1
                for (int i = 0; i < p.n; ++i, ++j) {
                    const int vb = j % C::kVBufs;
                    if (i == 0 && unit > 0) wait(ok, &sm.o_empty, unit - 1, a.err);
                    wait(ok, &sm.v_full[vb], j / C::kVBufs, a.err);
                    wait(ok, &sm.p_full[j & 1], j >> 1, a.err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = umma_desc_sw128(smem_u32(sm.v[vb]), kSlab, 1024);
                    const uint64_t pd = p_desc<NP>(smem_u32(sm.p[j & 1]));
                    const uint32_t o = tmem + kTmemO + (C::kAlt ? (j & 1) * NP : 0);
                    const bool first = i < (C::kAlt ? 2 : 1);
                    if (elect_one()) {
    #pragma unroll 1
                        for (int k = 0; k < kNB / 16; ++k)
                            umma_bf16(o, desc_at(vd, k * 2048), desc_at(pd, k * 16 * row), id,
                                      first && k == 0 ? 0u : 1u);
                        umma_commit(&sm.pv_done[j & 1]);
                        umma_commit(&sm.v_empty[vb]);
                        if (i == p.n - 1) umma_commit(&sm.o_full);
                    }
                    __syncwarp();
                }
            }
            if (ok && j > 0) {
                wait(ok, &sm.pv_done[(j - 1) & 1], (j - 1) >> 1, a.err);
                wait(ok, &sm.v_empty[(j - 1) % C::kVBufs], (j - 1) / C::kVBufs, a.err);
                wait(ok, &sm.o_full, unit - 1, a.err);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::kPvWarp) tmem_dealloc(tmem, kTmemCols);
}

// The parts of the pairs that were cut between CTAs, a row a warp: the parts'
// sums and accumulators weighted by their reference maxima.  CTA x of the grid
// has the pair that begins in share x and goes on behind it, if there is one.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) fp4_join_kernel(const __grid_constant__ Fp4AttnArgs a) {
    const int r = (int)blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Fp4Join d = a.joins[blockIdx.x];
    if (d.parts == 0 || r >= a.M) return;
    const float fv = fp4_factor(a.v_factor, d.h, a.err);
    constexpr int kAtOnce = 4;
    float m = -CUDART_INF_F, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < d.parts; k0 += kAtOnce) {
        float2 ml[kAtOnce];
        float4 v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            ml[k] = make_float2(-CUDART_INF_F, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k >= d.parts) continue;
            // (the parts behind the first are the first pieces of their CTAs)
            const size_t row = (size_t)(k0 + k == 0 ? d.slot : 2 * ((int)blockIdx.x + k0 + k)) * a.M + r;
            ml[k] = reinterpret_cast<const float2 *>(a.part_ml)[row];
            if (lane < D / 4) v[k] = reinterpret_cast<const float4 *>(a.part_acc + row * D)[lane];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (ml[k].x == -CUDART_INF_F) continue;  // none, or one without a visible token
            const float mn = fmaxf(m, ml[k].x), fo = ex2_approx(m - mn), fn = ex2_approx(ml[k].x - mn);
            l = l * fo + ml[k].y * fn;
            o.x = o.x * fo + v[k].x * fn, o.y = o.y * fo + v[k].y * fn;
            o.z = o.z * fo + v[k].z * fn, o.w = o.w * fo + v[k].w * fn;
            m = mn;
        }
    }
    const float inv = l > 0.f ? fv / l : 0.f;
    const size_t row = (size_t)d.b * a.n_q * a.Hq + (size_t)d.h * a.G + (size_t)(r / a.G) * a.Hq + r % a.G;
    if (lane < D / 4)
        reinterpret_cast<uint2 *>(a.out + row * D)[lane] =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (lane == 0 && a.lse) a.lse[row] = (m + __log2f(l)) * kLn2;
}

template <int D, int NP>
cudaError_t launch(const CUtensorMap *mq, const Fp4AttnArgs &a, cudaStream_t st) {
    using C = Cfg<D, NP>;
    using S = Smem<D, NP>;
    static_assert(C::kStages >= 2 && sizeof(S) + 1024 <= 232448, "fp4_attn_kernel shared memory");
    static_assert(offsetof(S, negm) % 16 == 0 && offsetof(S, ks) % 128 == 0 && offsetof(S, kc) % 1024 == 0 &&
                      offsetof(S, v) % 1024 == 0 && offsetof(S, p) % 1024 == 0,
                  "tiles start on their swizzle's boundary");
    const size_t smem = sizeof(S) + 1024;
    static DeviceMemo<int> attr_set;  // the shared-memory opt-in, once per device
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(fp4_attn_kernel<D, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    fp4_attn_kernel<D, NP><<<fp4_attn_grid(), C::kThreads, smem, st>>>(mq[0], mq[1], a);
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess) return launched;
    // a programmatic dependent launch: its CTAs are there when the parts are
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)fp4_attn_grid(), (unsigned)((a.M + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_join_kernel<D>, a);
}

template <int D>
cudaError_t launch_d(const CUtensorMap *mq, const Fp4AttnArgs &a, cudaStream_t st) {
    if (a.M <= 16) return launch<D, 16>(mq, a, st);
    if (a.M <= 32) return launch<D, 32>(mq, a, st);
    if (a.M <= 64) return launch<D, 64>(mq, a, st);
    return launch<D, 128>(mq, a, st);
}

}  // namespace

int fp4_attn_grid() { return sm_count(); }

cudaError_t launch_paged_verify_attn_fp4(const CUtensorMap *mq, const Fp4AttnArgs &a, int D, cudaStream_t st) {
    return D == 64 ? launch_d<64>(mq, a, st) : launch_d<128>(mq, a, st);
}

}  // namespace svpa
