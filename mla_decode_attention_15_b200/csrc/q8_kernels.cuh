// Absorbed-MQA decode over a latent cache held in 8 bits (e4m3) with one fp32
// scale per page of 64 tokens (and per KV head; the latent cache has one):
//
//   row_t = scale[page(t)] * e4m3 row t            (576 values, 576 bytes)
//   z_t   = softmax_scale * <q, row_t>,  out = sum_t softmax(z)_t row_t[0:512]
//
// in the transposed order of decode_kernels.cuh: S^T = K Q^T, softmax along the
// KV axis, O^T = V^T P^T.  Both products run as tcgen05 kind::f8f6f4 straight
// on the cache's bytes; nothing is widened on the way.
//
// The other operands lose nothing to 8 bits either, because in the transposed
// order the query columns are the MMA's N, and an MMA of N <= 64 occupies the
// tensor pipe as long as one of N = 16.  So Q and P enter as sums of e4m3
// terms, the terms side by side as further columns:
//   - Q.  A bf16 value has 8 significant bits, an e4m3 value 4.  With x scaled by a
//     power of two per query row (its largest magnitude then lies in (224, 448]),
//     hi = e4m3(x) leaves a remainder of at most 4 significant bits, which
//     lo = e4m3(16 (x - hi)) holds exactly.  Only values below 2^-14 of the
//     row's largest are rounded, by at most 2^-21 of it.  S^T = S_hi + S_lo / 16.
//   - P.  x = 16 p s / (the largest p s of the query column so far; s the page's
//     scale) is rounded to fp16 (11 bits, half a step is 2^-12 of the weight: an
//     eighth of the rounding of a bf16 result) and cut into three e4m3 terms, each
//     16 times the remainder of the one before, which hold those 11 bits exactly;
//     values below 2^-6 lose at most 2^-18 absolutely, 2^-22 of the largest.
//     O^T = O_0 + O_1 / 16 + O_2 / 256.
// The page's scale s is a factor of the score of its tokens and of their value
// rows, so it enters the exponent of P and costs no pass over the data.  The running
// reference m of a column is that of the sum w = z log2 e + log2 s, which is what is stored: a page
// whose scale is large but whose tokens have no weight moves nothing.  The
// sum of the weights, of x / s, stands against the same reference, so
// out = O / l, and whatever w is rounded by, numerator and sum share it.
//
// Work split.  A step is 128 tokens (two pages; M = 128 in GEMM1), cut into four
// boxes of 128 latent columns (16 KB each, 128-byte swizzle) and the 64 RoPE
// columns (8 KB).  Box c is both K columns [128 c, 128 c + 128) of GEMM1 and the
// d_v chunk c of GEMM2 (read MN-major).  The ring holds them two boxes to a slot,
// and GEMM2 frees a slot as soon as both of its chunks are done.  The plan, the
// walk over work items, the partial slots and the combine are those of
// decode_kernels.cuh (64-token units, with an overhead per item of their own).
// Query groups are 16 or 32 columns; more query columns are several groups that
// walk each range of pages side by side, one CTA per group, so that all but the
// first read of a page hit L2.
//
// What bounds it, on B200 (event-timed, caches warm):
//   - 16 requests x 64K x 16 heads, 605 MB: 121 us, 5.0 TB/s of the 6.55 TB/s of a
//     plain copy.  A steady step keeps up with the loads; the rest is the first
//     items' Q split and last items' epilogue, the combine (7 us by itself), and the
//     clock, which the power limit lowers in a long run.
//   - 32 requests x 8-32K x 2 tokens x 128 heads, 365 GFLOP on 395 MB: 562 us, 0.65 PFLOP/s of
//     the sums as defined (0.40 of the measured bf16 rate).  A step's
//     tensor work (two Q terms, three P terms of 32 columns) is 1,760 cycles; its softmax,
//     a chain of TMEM read, exponentials, three conversions and the store of P^T,
//     about 2,950.
//   - 16 requests x 1-16K x 2 tokens x 16 heads, 81 MB: 39 us; 1 x 1K: 11.3 us.  An item's
//     fixed parts: plan, Q split, first step, epilogue, combine.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "cache_kernels.cuh"
#include "decode_kernels.cuh"

namespace mla {

constexpr int kQ8Row = kDqk;                    // bytes per token
constexpr int kQ8PageBytes = kPage * kQ8Row;    // 36,864
constexpr int kQ8Step = 2 * kPage;              // tokens per step
constexpr int kQ8BoxBytes = kQ8Step * 128;      // 128 tokens x 128 latent columns
constexpr int kQ8SlotBytes = 2 * kQ8BoxBytes;   // ring slot: two boxes, half of a step's latent columns
constexpr int kQ8RopeBytes = kQ8Step * 64;      // 128 tokens x 64 RoPE columns
constexpr int kQ8Boxes = 4;
constexpr int kQ8Halves = 2;                    // slots per step
constexpr int kQ8Terms = 3;                     // e4m3 terms of P
// x = 2^kQ8Bias p: the largest weight is 2^kQ8Bias, and a weight may grow
// 2^kQ8Grow above it before O^T is rescaled; 2^(bias + grow) <= 448.
constexpr float kQ8Bias = 4.0f;
constexpr float kQ8Grow = 4.8f;
// The Q warps wait for most of an item; they leave the issue slots alone meanwhile.
constexpr int kQ8Nap = 200, kQ8MaxNaps = 1 << 22;  // ns; about a second
// Where a page's scale is below this share of the largest so far, its tokens may carry all
// the weight and yet x may vanish: their part of the sum is then computed without x.
constexpr float kQ8FarScale = 0x1p-60f;
// A range's sum of weights is counted in 1 / scale, which fp32 holds (with 2^20 tokens) down
// to scales of 2^-100; with a page below that in the range, in units of 2^50.
constexpr float kQ8SmallScale = 0x1p-100f;
constexpr int kQ8SmallUnit = -50;
constexpr float kQ8Unset = -3.402823466e38f;    // running max before the first visible token: below every score

struct Q8Params : FwdParams {
    const __nv_bfloat16* q;   // [B * N][576]
    const float* kv_scales;   // [num_blocks]
};

template <int NG>
struct Q8Cfg {
    // Query columns of a softmax thread.  Eight warps serve either group: fewer
    // columns per thread shorten a step's serial part (16 columns, 8 instead of 16 per
    // thread: b1 x 1K 19.2 -> 15.8 us, b16 x 64K 131 -> 126 us), but a third and fourth
    // warp per scheduler only contend (32 columns, 8 per thread: 565 -> 825 us).
    static constexpr int kCols = NG / 2;
    static constexpr int kColGroups = 2;                    // softmax groups of 4 warps
    static constexpr int kFirstQ = 4;                       // warps 4..7 split Q
    static constexpr int kFirstSoftmax = 8;
    static constexpr int kThreads = 32 * (kFirstSoftmax + 4 * kColGroups);
    // 512 threads leave 128 registers each at launch.  With 16 columns the softmax
    // needs more: the issuing and the Q warps give some of theirs (warpgroups: issue, Q,
    // softmax twice).
    static constexpr bool kSplitRegs = kCols == 16;
    static constexpr int kRegsIssue = 64, kRegsQ = 96, kRegsSoftmax = 176;
    static_assert(kThreads == 512 && kRegsIssue + kRegsQ + 2 * kRegsSoftmax <= 4 * 128, "register split");
    static constexpr int kQN = 2 * NG;                      // S^T columns: hi, lo
    static constexpr int kNP = kQ8Terms * NG;               // O^T columns per d_v chunk
    // The ring holds two and a half steps.  A step's slots stay taken from its loads
    // through GEMM1, the softmax and GEMM2, so with two steps the loads of one
    // wait for the GEMM2 of the other; 32-column groups, whose Q takes 36 KB, make
    // room for the half by one buffer of P^T instead of two.
    static constexpr int kSlots = 5;                        // ring of 32 KB slots
    static constexpr int kRopeSlots = NG == 16 ? 3 : 2;     // RoPE columns of a step
    static constexpr int kPBufs = NG == 16 ? 2 : 1;
    // shared memory
    static constexpr int kBoxOff = 0;
    static constexpr int kRopeOff = kBoxOff + kSlots * kQ8SlotBytes;
    static constexpr int kQOff = kRopeOff + kRopeSlots * kQ8RopeBytes;
    static constexpr int kQBytes = kQN * kDqk;
    static constexpr int kPOff = kQOff + kQBytes;
    static constexpr int kPBytes = kQ8Step * kNP;
    static constexpr int kRedOff = kPOff + kPBufs * kPBytes;     // float [NG][4]
    static constexpr int kSumOff = kRedOff + NG * 16;       // float [NG][4]
    static constexpr int kQsOff = kSumOff + NG * 16;        // float [2][NG]: row scale x softmax scale x log2 e, by item
    static constexpr int kVoteOff = kQsOff + 2 * NG * 4;    // uint32 [2][8]
    static constexpr int kBarOff = kVoteOff + 64;
    static constexpr int kNumBars = 64;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kPlanMetaOff = kMiscOff + 16;
    static constexpr int kBytes = kPlanMetaOff + (kMetaWords + 8) * 4;
    // Plans of up to kSmallPlan work items keep their prefix where P^T goes, and one
    // idle warp publishes them while the others begin; the first P^T waits for it.
    static constexpr int kSmallPlan = kPBufs * kPBytes / 4 - 48;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
    static_assert(kQOff % 1024 == 0 && kPOff % 128 == 0 && kPBytes % 128 == 0, "operand alignment");
    // larger plans: the slots past the first step's
    static constexpr int kInlinePlanMaxBG = (kSlots - kQ8Halves) * kQ8SlotBytes / 4 - 48;
    // TMEM columns
    static constexpr int kSCol = 0;
    static constexpr int kOCol = 2 * kQN;
    static constexpr int kTmemUsed = kOCol + kQ8Boxes * kNP;
    static_assert(kTmemUsed <= 512, "TMEM budget");
    static constexpr int kTmemCols = 512;
};

constexpr int kQ8MaxSlots = 5;
enum Q8Bar {
    kQbQFull = 0, kQbQEmpty, kQbSFull0, kQbSFull1, kQbSEmpty0, kQbSEmpty1, kQbPFull0, kQbPFull1, kQbPEmpty0, kQbPEmpty1,
    kQbOEmpty, kQbDone1, kQbDone2, kQbQSeen, kQbPlan,
    kQbVote0,                            // [2 parities][2 column groups]
    kQbMax0 = kQbVote0 + 4,              // [2 column groups]
    kQbSum0 = kQbMax0 + 2,               // [2 column groups]
    kQbFull0 = kQbSum0 + 2,
    kQbEmpty0 = kQbFull0 + kQ8MaxSlots,
    kQbCount = kQbEmpty0 + kQ8MaxSlots
};
static_assert(kQbCount <= Q8Cfg<16>::kNumBars, "barrier slots");

// ------------------------------------------------------------------ PTX
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// D[tmem] (+)= A . B, kind::f8f6f4.  The descriptors come as their two words: only
// the low one (the address) changes from MMA to MMA.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of kind::f8f6f4 with e4m3 A/B and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t h2) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
    return r;
}

// W (8 or 16) values reduced over the 32 lanes of a warp; lane l returns value l W / 32.
template <bool kMax, int W>
__device__ __forceinline__ float reduce_cols(const float (&x)[W], int lane) {
    float v[W];
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = x[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const int h = W * off / 32;  // values left after this step; below one, a plain reduction
        const bool upper = (lane & off) != 0;
        if (h >= 1) {
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float send = upper ? v[i] : v[i + h];
                const float keep = upper ? v[i + h] : v[i];
                const float got = __shfl_xor_sync(kFullMask, send, off);
                v[i] = kMax ? fmaxf(keep, got) : keep + got;
            }
        } else {
            const float got = __shfl_xor_sync(kFullMask, v[0], off);
            v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return v[0];
}
template <int W>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[W]) {
    if constexpr (W == 8) tmem_ld_x8(taddr, v);
    else tmem_ld_x16(taddr, v);
}
template <int W>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[W]) {
    if constexpr (W == 8) tmem_st_x8(taddr, v);
    else tmem_st_x16(taddr, v);
}

// ------------------------------------------------------------------ producer
// Physical page of logical page j; a bad entry is reported and read as page 0.
__device__ __forceinline__ int q8_page(const Q8Params& p, const Item& item, int j) {
    int phys = __ldg(p.block_table + (size_t)item.b * p.max_blocks + j);
    if ((unsigned)phys >= (unsigned)p.num_blocks) {
        atomicOr(p.status, MLA_STATUS_BAD_BLOCK_TABLE);
        phys = 0;
    }
    return phys;
}

// Loads half hf of a step of one or two pages into a ring slot: boxes 2 hf and
// 2 hf + 1, and with the second half the RoPE columns.
template <int NG>
__device__ __forceinline__ void q8_load(const CUtensorMap* kv_map, const CUtensorMap* rope_map, uint8_t* smem, uint32_t slot,
                                        uint32_t rope_slot, int hf, int ph0, int ph1, uint64_t policy) {
    using C = Q8Cfg<NG>;
    const uint32_t bar = smem_addr(smem + C::kBarOff) + 8 * (kQbFull0 + slot);
    const uint32_t dst = smem_addr(smem + C::kBoxOff) + slot * kQ8SlotBytes;
    const uint32_t page = kQ8SlotBytes / 2 + (hf ? kQ8RopeBytes / 2 : 0);  // bytes of one page
    mbar_arrive_expect_tx(bar, ph1 >= 0 ? 2 * page : page);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        tma_load_3d_hint(dst + c * kQ8BoxBytes, kv_map, bar, 128 * (2 * hf + c), 0, ph0, policy);
        if (ph1 >= 0)
            tma_load_3d_hint(dst + c * kQ8BoxBytes + kQ8BoxBytes / 2, kv_map, bar, 128 * (2 * hf + c), 0, ph1, policy);
    }
    if (hf) {
        const uint32_t rd = smem_addr(smem + C::kRopeOff) + rope_slot * kQ8RopeBytes;
        tma_load_3d_hint(rd, rope_map, bar, kDv, 0, ph0, policy);
        if (ph1 >= 0) tma_load_3d_hint(rd + kQ8RopeBytes / 2, rope_map, bar, kDv, 0, ph1, policy);
    }
}

template <int NG>
__device__ void q8_producer(const CUtensorMap* kv_map, const CUtensorMap* rope_map, const Q8Params& p, const int32_t* meta,
                            uint8_t* smem, const Ctl& ctl, bool first_issued) {
    using C = Q8Cfg<NG>;
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    const uint64_t policy = p.share > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    WorkIter it;
    it.init(meta, p);
    Item item;
    uint32_t n = 0, rope = 0;              // halves issued (or left out by the test hook)
    const bool stall = p.test_stall != 0;
    bool ok = true;
    while (ok && it.next(p, item)) {
        for (int j = item.p0; ok && j < item.p1; j += 2) {
            if (n == 0 && (first_issued || stall)) {  // issued before the wait on the previous grid, or left out
                n = kQ8Halves;
                rope = 1;
                continue;
            }
            const int ph0 = q8_page(p, item, j);
            const int ph1 = j + 1 < item.p1 ? q8_page(p, item, j + 1) : -1;
#pragma unroll 1
            for (int hf = 0; hf < kQ8Halves; ++hf, ++n) {
                const uint32_t slot = n % C::kSlots;
                // (a step's RoPE slot is free when the slots of the step kRopeSlots before are)
                ok = wait_bounded(bar0 + 8 * (kQbEmpty0 + slot), ((n / C::kSlots) & 1) ^ 1, ctl);
                if (!ok) break;
                q8_load<NG>(kv_map, rope_map, smem, slot, rope, hf, ph0, ph1, policy);
            }
            if (++rope == C::kRopeSlots) rope = 0;
        }
    }
    if (!ok) {
        // Let the copies already issued land before the CTA exits.
        for (uint32_t k = 0; k < C::kSlots; ++k) {
            const uint32_t count = n > k ? (n - k + C::kSlots - 1) / C::kSlots : 0;
            if (count > (stall && k < kQ8Halves ? 1u : 0u)) wait_drain(bar0 + 8 * (kQbFull0 + k), (count - 1) & 1);
        }
    }
}

// ------------------------------------------------------------------ Q split
// Cuts a query row into hi and lo terms, 8 lanes per row.  The result is GEMM1's
// K-major B operand without swizzle: 16-byte pieces, piece (k, n) of K bytes
// [16 k, 16 k + 16) and column n at (k * kQN + n) * 16; `dst` is piece (0, n) of the
// row's hi term, `row` null for a column past the last.  Every CTA runs this once before
// anything else can start, with a cold instruction cache, so it is a loop of a few
// instructions: unrolled over the row it took 4,200
// cycles (32 columns: 7,900).
template <int NG>
__device__ __forceinline__ void q8_split_row(const __nv_bfloat16* row, uint8_t* dst, float* scale_out, float scale_log2) {
    using C = Q8Cfg<NG>;
    const int lane8 = threadIdx.x & 7;
    uint4 raw[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    if (row != nullptr) {
        // (plain loads: a read-only load may be scheduled above the wait on the grid that wrote q)
#pragma unroll
        for (int i = 0; i < 9; ++i) raw[i] = reinterpret_cast<const uint4*>(row)[i * 8 + lane8];
    }
    uint32_t top = 0;  // two bf16 magnitudes as bits: non-finite values are the largest
#pragma unroll
    for (int i = 0; i < 9; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                     __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)));
    uint32_t amax = max(top << 16, top & 0x7fff0000u);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFullMask, amax, o));
    const int ex = amax == 0 ? 0 : max(e4m3_scale_exp(amax), -100);
    // a row with an infinity or a NaN becomes NaN: so do its scores
    const float inv = amax >= kInfBits ? __int_as_float(0x7fffffff) : pow2f(-ex);
    if (lane8 == 0) *scale_out = (amax >= kInfBits ? 1.f : pow2f(ex)) * scale_log2;
    uint8_t* d = dst + (lane8 >> 1) * (C::kQN * 16) + (lane8 & 1) * 8;
#pragma unroll 1
    for (int i = 0; i < 9; ++i) {
        const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // scaled to at most 448, fp16 holds the 8 bits down to 2^-17, and its
            // last place (2^-24) is far below the last place of lo
            const __half2 x = __floats2half2_rn(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xffff0000u) * inv);
            const uint32_t h = e4m3x2_h2(as_u32(x));
            const uint32_t l = e4m3x2_h2(as_u32(__hmul2(__hsub2(x, as_h2(h2_of_e4m3x2(h))), __float2half2_rn(16.f))));
            if (e & 1) {
                hi[e >> 1] |= h << 16;
                lo[e >> 1] |= l << 16;
            } else {
                hi[e >> 1] = h;
                lo[e >> 1] = l;
            }
        }
        *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(d + NG * 16) = make_uint2(lo[0], lo[1]);
        d += 4 * C::kQN * 16;  // 64 columns on
#pragma unroll
        for (int k = 0; k < 8; ++k) raw[k] = raw[k + 1];
    }
    fence_proxy_async_smem();
    __syncwarp();
}
template <int NG>
__device__ __forceinline__ void q8_split(const Q8Params& p, const Item& item, uint8_t* smem, int col, uint32_t q_it) {
    using C = Q8Cfg<NG>;
    const int gc = item.g * NG + col;
    q8_split_row<NG>(gc < p.N ? p.q + ((size_t)item.b * p.N + gc) * kDqk : nullptr, smem + C::kQOff + col * 16,
                     reinterpret_cast<float*>(smem + C::kQsOff) + (q_it & 1) * NG + col, p.scale_log2);
}

// Four warps split each item's Q, 16 rows at a time, while the previous item's
// softmax and epilogue run.  Of the first item, which the whole CTA waits for, softmax
// warps take the rows past the first 16.
template <int NG>
__device__ void q8_split_q(const Q8Params& p, const int32_t* meta, uint8_t* smem, const Ctl& ctl) {
    using C = Q8Cfg<NG>;
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    const int tid = threadIdx.x - 32 * C::kFirstQ;
    WorkIter it;
    it.init(meta, p);
    Item item;
    uint32_t q_it = 0;
    while (it.next(p, item)) {
        if (q_it > 0) {
            // GEMM1 of the previous item has read its Q, and its softmax has begun
            // (so it is past its wait on kQbQFull, and done with the row scales of
            // the item before).
            for (int i = 0; i < kQ8MaxNaps && !mbar_try_wait(bar0 + 8 * kQbQEmpty, (q_it & 1) ^ 1) && !*ctl.abort_flag; ++i)
                __nanosleep(kQ8Nap);
            if (!wait_warp(bar0 + 8 * kQbQEmpty, (q_it & 1) ^ 1, ctl)) return;
            if (!wait_warp(bar0 + 8 * kQbQSeen, (q_it & 1) ^ 1, ctl)) return;
        }
        const int rows = q_it == 0 ? 16 : NG;
#pragma unroll 1
        for (int r = 0; r < rows; r += 16) {
            q8_split<NG>(p, item, smem, r + (tid >> 3), q_it);
            if ((tid & 31) == 0) mbar_arrive(bar0 + 8 * kQbQFull);
        }
        ++q_it;
    }
}

// ------------------------------------------------------------------ MMA issuers
// The issuing warps run converged and elect a lane for each MMA: the operands of
// tcgen05.mma are uniform registers, and in code that one thread runs alone the
// compiler has to move every operand there.  Measured on B200 (cycles from one MMA to
// the next): issued by a lone thread with computed descriptors 90, elected 40 (M = 128,
// N = 32), 44 (N = 48), 48 (N = 64) and 56 (N = 96); K-major and MN-major operands, swizzled or
// not, cost the same.

// S^T[128 x 2 NG] = K[128 x 576] . [Q_hi | Q_lo]^T.
template <int NG>
__device__ void q8_gemm1(const Q8Params& p, const int32_t* meta, uint8_t* smem, uint32_t tmem, const Ctl& ctl) {
    using C = Q8Cfg<NG>;
    constexpr uint32_t kIdesc = idesc_e4m3_f32(kQ8Step, C::kQN, 0, 0);
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    const uint64_t a0 = smem_desc(smem_addr(smem + C::kBoxOff), 16, 1024, kSwizzle128);
    const uint64_t r0 = smem_desc(smem_addr(smem + C::kRopeOff), 16, 512, kSwizzle64);
    const uint64_t b0 = smem_desc(smem_addr(smem + C::kQOff), C::kQN * 16, 128, kSwizzleNone);
    const uint32_t a_hi = (uint32_t)(a0 >> 32), r_hi = (uint32_t)(r0 >> 32), b_hi = (uint32_t)(b0 >> 32);
    const uint32_t b_lo = (uint32_t)b0;
    WorkIter it;
    it.init(meta, p);
    Item item;
    uint32_t s_it = 0, q_it = 0, slot = 0, phase = 0, rope = 0;
    bool ok = true;
    while (ok && it.next(p, item)) {
        ok = wait_warp(bar0 + 8 * kQbQFull, q_it & 1, ctl);
        if (!ok) break;
        for (int j = item.p0; j < item.p1; j += 2) {
            const int sb = s_it & 1;
            ok = wait_warp(bar0 + 8 * (kQbSEmpty0 + sb), ((s_it >> 1) & 1) ^ 1, ctl);
            if (!ok) break;
            const uint32_t d = tmem + C::kSCol + sb * C::kQN;
#pragma unroll
            for (int hf = 0; hf < kQ8Halves; ++hf) {
                ok = wait_warp(bar0 + 8 * (kQbFull0 + slot), phase, ctl);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a_lo = (uint32_t)a0 + slot * (kQ8SlotBytes >> 4);
                const uint32_t r_lo = (uint32_t)r0 + rope * (kQ8RopeBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        umma_f8(d, a_lo + (k >> 2) * (kQ8BoxBytes >> 4) + 2 * (k & 3), a_hi, b_lo + (16 * hf + 2 * k) * C::kQN,
                                b_hi, kIdesc, hf + k > 0);
                    if (hf == kQ8Halves - 1) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            umma_f8(d, r_lo + 2 * k, r_hi, b_lo + (8 * kQ8Boxes + 2 * k) * C::kQN, b_hi, kIdesc, 1);
                        umma_commit(bar0 + 8 * (kQbSFull0 + sb));
                        if (j + 2 >= item.p1) umma_commit(bar0 + 8 * kQbQEmpty);
                    }
                }
                __syncwarp();
                if (++slot == C::kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (++rope == C::kRopeSlots) rope = 0;
            ++s_it;
        }
        ++q_it;
    }
}

// O^T chunk c [128 x 3 NG] += V^T (box c, read MN-major) . P^T (MN-major without
// swizzle: 16-byte pieces of 16 columns, 128 tokens apart by 2 KB).
template <int NG>
__device__ void q8_gemm2(const Q8Params& p, const int32_t* meta, uint8_t* smem, uint32_t tmem, const Ctl& ctl) {
    using C = Q8Cfg<NG>;
    constexpr uint32_t kIdesc = idesc_e4m3_f32(128, C::kNP, 1, 1);
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    const uint64_t a0 = smem_desc(smem_addr(smem + C::kBoxOff), kQ8BoxBytes, 1024, kSwizzle128);
    const uint64_t b0 = smem_desc(smem_addr(smem + C::kPOff), 128, kQ8Step * 16, kSwizzleNone);
    const uint32_t a_hi = (uint32_t)(a0 >> 32), b_hi = (uint32_t)(b0 >> 32);
    WorkIter it;
    it.init(meta, p);
    Item item;
    uint32_t s_it = 0, item_it = 0, slot = 0;
    bool ok = true;
    while (ok && it.next(p, item)) {
        for (int j = item.p0; j < item.p1; j += 2) {
            const uint32_t pb = s_it % C::kPBufs;
            ok = wait_warp(bar0 + 8 * (kQbPFull0 + pb), (s_it / C::kPBufs) & 1, ctl);
            if (!ok) break;
            if (j == item.p0) {
                ok = wait_warp(bar0 + 8 * kQbOEmpty, (item_it & 1) ^ 1, ctl);
                if (!ok) break;
            }
            tc_fence_after();
            const uint32_t b_lo = (uint32_t)b0 + pb * (C::kPBytes >> 4);
            const uint32_t more = j == item.p0 ? 0u : 1u;
#pragma unroll
            for (int hf = 0; hf < kQ8Halves; ++hf) {
                const uint32_t a_lo = (uint32_t)a0 + slot * (kQ8SlotBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < kQ8Step / 32; ++k)
                            umma_f8(tmem + C::kOCol + (2 * hf + c) * C::kNP, a_lo + c * (kQ8BoxBytes >> 4) + k * (4096 >> 4), a_hi,
                                    b_lo + k * (512 >> 4), b_hi, kIdesc, k == 0 ? more : 1u);
                    umma_commit(bar0 + 8 * (kQbEmpty0 + slot));
                    if (hf + 1 == kQ8Halves) umma_commit(bar0 + 8 * (kQbPEmpty0 + pb));
                }
                __syncwarp();
                if (++slot == C::kSlots) slot = 0;
            }
            ++s_it;
        }
        if (!ok) break;
        ++item_it;
    }
}

// What an issuing warp's MMAs still write is done before TMEM is released, on the
// normal and the abort path alike (a commit with nothing outstanding arrives at once).
__device__ __forceinline__ void q8_drain(uint32_t bar) {
    if (elect_one()) umma_commit(bar);
    __syncwarp();
    wait_drain(bar, 0);
}

// ------------------------------------------------------------------ softmax
// W weights x (fp16 range) as three e4m3 terms, each term's W bytes term_stride apart.
template <int W>
__device__ __forceinline__ void q8_store_p(const float (&x)[W], uint8_t* dst, int term_stride) {
    uint32_t w[kQ8Terms][W / 4];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int t = 0; t < kQ8Terms; ++t) {
            const uint32_t v = e4m3x2_h2(as_u32(h));
            if (i & 1) w[t][i >> 1] |= v << 16;
            else w[t][i >> 1] = v;
            // the remainder is exact in fp16: at most 7 significant bits
            if (t + 1 < kQ8Terms) h = __hmul2(__hsub2(h, as_h2(h2_of_e4m3x2(v))), __float2half2_rn(16.f));
        }
    }
#pragma unroll
    for (int t = 0; t < kQ8Terms; ++t) {
        if constexpr (W == 8) *reinterpret_cast<uint2*>(dst + t * term_stride) = make_uint2(w[t][0], w[t][1]);
        else *reinterpret_cast<uint4*>(dst + t * term_stride) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
    }
}

template <int NG>
__device__ void q8_softmax(const Q8Params& p, const int32_t* meta, uint8_t* smem, uint32_t tmem, const Ctl& ctl,
                           bool plan_in_p) {
    using C = Q8Cfg<NG>;
    constexpr int W = C::kCols;
    const int lane = threadIdx.x & 31;
    const int wq = (threadIdx.x >> 5) & 3;                       // TMEM lane quadrant
    const int cg = ((threadIdx.x >> 5) - C::kFirstSoftmax) >> 2;  // columns [W cg, W cg + W)
    const int row = 32 * wq + lane;                              // token of the step
    const uint32_t tm = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    float* red = reinterpret_cast<float*>(smem + C::kRedOff) + cg * W * 4;   // [W][4]: a step's maxima
    float* sums = reinterpret_cast<float*>(smem + C::kSumOff) + cg * W * 4;  // [W][4]
    const float* qs_ring = reinterpret_cast<const float*>(smem + C::kQsOff) + cg * W;
    uint32_t* vote = reinterpret_cast<uint32_t*>(smem + C::kVoteOff) + cg * 4;
    constexpr int kTermStride = NG * kQ8Step;
    uint8_t* pbase = smem + C::kPOff + (cg * W / 16) * 16 * kQ8Step + row * 16 + cg * W % 16;
    const bool causal2 = p.causal && p.s_q > 1;
    auto arrive = [&](uint32_t bar) {  // once per warp, after all of its lanes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    WorkIter it;
    it.init(meta, p);
    Item item;
    uint32_t s_it = 0, item_it = 0, max_it = 0;
    bool ok = true;
    while (ok && it.next(p, item)) {
        if constexpr (NG > 16) {
            if (item_it == 0 && cg == 0) {
                q8_split<NG>(p, item, smem, 16 + (row >> 3), 0);
                arrive(bar0 + 8 * kQbQFull);
            }
        }
        ok = wait_warp(bar0 + 8 * kQbQFull, item_it & 1, ctl);
        if (!ok) break;
        arrive(bar0 + 8 * kQbQSeen);
        const float4* qs4 = reinterpret_cast<const float4*>(qs_ring + (item_it & 1) * NG);
        const int gc0 = item.g * NG + cg * W;  // first query column of the group
        // Table entries are fetched two steps ahead and page scales one, so
        // that no step waits for either.
        const int32_t* bt = p.block_table + (size_t)item.b * p.max_blocks;
        auto entry = [&](int j) { return __ldg(bt + (j < item.p1 ? j : item.p1 - 1)); };
        auto page_scale = [&](int phys) -> float {
            // (a scale of 0 goes with zeros: any other one keeps its tokens' weights finite)
            const float s = __ldg(p.kv_scales + ((unsigned)phys < (unsigned)p.num_blocks ? phys : 0));
            return s > 0.f ? s : kQ8SmallScale;
        };
        float sc0 = page_scale(entry(item.p0)), sc1 = page_scale(entry(item.p0 + 1));
        int ph0 = entry(item.p0 + 2), ph1 = entry(item.p0 + 3);
        float m[W], l[W];
#pragma unroll
        for (int c = 0; c < W; ++c) {
            m[c] = kQ8Unset;
            l[c] = 0.f;
        }
        float R = 0.f;  // the largest scale so far
        float lks = 0.f, back = 0.f, of_ks = -1.f;
        float small = kQ8SmallScale;  // 0 once l counts in units of 2^kQ8SmallUnit
        auto unit = [&]() { return small > 0.f ? 0 : kQ8SmallUnit; };
        for (int j = item.p0; j < item.p1; j += 2) {
            const float nx0 = page_scale(ph0), nx1 = page_scale(ph1);
            ph0 = entry(j + 4);
            ph1 = entry(j + 5);
            const float ks = wq < 2 ? sc0 : sc1;  // this token's page
            R = fmaxf(R, fmaxf(sc0, sc1));
            if (ks != of_ks) {  // (page scales seldom differ)
                of_ks = ks;
                lks = log2f(ks);
                back = (ks < small ? pow2f(kQ8SmallUnit) : pow2f(unit())) / ks;  // x -> its part of the sum
            }
            const int sb = s_it & 1;
            ok = wait_warp(bar0 + 8 * (kQbSFull0 + sb), (s_it >> 1) & 1, ctl);
            if (!ok) break;
            tc_fence_after();
            float z[W];
            {
                float lo[W];
                const uint32_t s = tm + C::kSCol + sb * C::kQN + cg * W;
                tmem_ld_cols(s, z);
                tmem_ld_cols(s + NG, lo);
                tmem_ld_wait();
                tc_fence_before();
                arrive(bar0 + 8 * (kQbSEmpty0 + sb));
#pragma unroll
                for (int c4 = 0; c4 < W / 4; ++c4) {
                    const float4 f = qs4[c4];
                    z[4 * c4 + 0] = fmaf(fmaf(lo[4 * c4 + 0], 0.0625f, z[4 * c4 + 0]), f.x * ks, lks);
                    z[4 * c4 + 1] = fmaf(fmaf(lo[4 * c4 + 1], 0.0625f, z[4 * c4 + 1]), f.y * ks, lks);
                    z[4 * c4 + 2] = fmaf(fmaf(lo[4 * c4 + 2], 0.0625f, z[4 * c4 + 2]), f.z * ks, lks);
                    z[4 * c4 + 3] = fmaf(fmaf(lo[4 * c4 + 3], 0.0625f, z[4 * c4 + 3]), f.w * ks, lks);
                }
            }
            const int t = j * kPage + row;
            const int end = (j + 2 < item.p1 ? j + 2 : item.p1) * kPage;  // tokens of the step
            const int lim0 = item.L - (causal2 ? 1 : 0);
            if (end > lim0 || j + 2 > item.p1) {
                // The step holds tokens that some column does not see (past the
                // length, the causal rule, or no second page).
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    const int lim = causal2 && gc0 + c < p.heads ? lim0 : item.L;
                    if (t >= lim || t >= end) z[c] = -INFINITY;
                }
            }
            // Does any x exceed the running reference by more than 2^kQ8Grow?
            // (The difference of two close numbers is exact; the sum of a large one and 4.8 is not.)
            // The first step, which sets the reference, exchanges its maxima at once.
            const bool first = j == item.p0;
            const uint32_t vbar = bar0 + 8 * (kQbVote0 + (s_it & 1) * 2 + cg);
            auto post_maxima = [&]() {
                const float wmax = reduce_cols<true>(z, lane);
                if (lane % (32 / W) == 0) red[lane / (32 / W) * 4 + wq] = wmax;
            };
            if (first) {
                post_maxima();
            } else {
                bool grow = ks < small;  // (the unit of the sum changes as the references do)
#pragma unroll
                for (int c = 0; c < W; ++c) grow |= z[c] - m[c] > kQ8Grow;
                const uint32_t gw = __any_sync(kFullMask, grow) ? 1u : 0u;
                if (lane == 0) vote[(s_it & 1) * 8 + wq] = gw;
            }
            arrive(vbar);
            ok = wait_warp(vbar, (s_it >> 1) & 1, ctl);
            if (!ok) break;
            bool grown = first;
            if (!first) {
                const uint4 v4 = *reinterpret_cast<const uint4*>(vote + (s_it & 1) * 8);
                grown = (v4.x | v4.y | v4.z | v4.w) != 0;  // the same for the group's four warps
            }
            if (grown) {
                // Move the references and rescale what is accumulated.
                if (!first) {
                    post_maxima();
                    arrive(bar0 + 8 * (kQbMax0 + cg));
                    ok = wait_warp(bar0 + 8 * (kQbMax0 + cg), max_it & 1, ctl);
                    ++max_it;
                    if (!ok) break;
                }
                float alpha[W];
                float to_unit = 1.f;
                if (fminf(sc0, sc1) < small) {
                    to_unit = pow2f(kQ8SmallUnit);
                    if (ks >= small) back *= to_unit;
                    small = 0.f;
                }
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    // (without branches: a column that stays has a = 2^0.  A reference may
                    // move further than fp32's exponents reach while the sum, whose
                    // unit is 1 / scale, still counts: its factor is applied in two halves)
                    const float4 r4 = *reinterpret_cast<const float4*>(red + c * 4);
                    const float mx = fmaxf(fmaxf(r4.x, r4.y), fmaxf(r4.z, r4.w));
                    const float to = mx - m[c] > kQ8Grow ? mx : m[c];
                    const float a = ex2_approx(0.5f * (m[c] - to));
                    m[c] = to;
                    l[c] = l[c] * a * a * to_unit;
                    alpha[c] = a * a;
                }
                if (j > item.p0) {
                    const uint32_t prev = s_it - 1;
                    ok = wait_warp(bar0 + 8 * (kQbPEmpty0 + prev % C::kPBufs), (prev / C::kPBufs) & 1, ctl);
                    if (!ok) break;
                    tc_fence_after();
                    constexpr int U = 48 / W;  // accumulators at a time
#pragma unroll 1
                    for (int i = 0; i < kQ8Boxes * kQ8Terms; i += U) {
                        float o[U][W];
                        const uint32_t ta = tm + C::kOCol + i * NG + cg * W;
#pragma unroll
                        for (int u = 0; u < U; ++u) tmem_ld_cols(ta + u * NG, o[u]);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < U; ++u) {
#pragma unroll
                            for (int c = 0; c < W; ++c) o[u][c] *= alpha[c];
                            tmem_st_cols(ta + u * NG, o[u]);
                        }
                    }
                    tmem_st_wait();
                }
            }
            if (ks >= R * kQ8FarScale) {
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    z[c] = ex2_approx(z[c] - m[c] + kQ8Bias);
                    l[c] = fmaf(z[c], back, l[c]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    const float w = z[c] - m[c] + kQ8Bias;
                    l[c] += ex2_approx(w - lks + (float)unit());
                    z[c] = ex2_approx(w);
                }
            }
            const uint32_t pb = s_it % C::kPBufs;
            ok = wait_warp(bar0 + 8 * (kQbPEmpty0 + pb), ((s_it / C::kPBufs) & 1) ^ 1, ctl);
            if (!ok) break;
            if (plan_in_p) {  // the plan's scratch lies there until it is published
                ok = wait_warp(bar0 + 8 * kQbPlan, 0, ctl);
                if (!ok) break;
                plan_in_p = false;
            }
            q8_store_p(z, pbase + pb * C::kPBytes, kTermStride);
            if (j + 2 >= item.p1 && t >= (end < item.L ? end : item.L)) {
                // Rows behind the sequence, or of an absent second page: their
                // weights are zero, but what lies there (stale rows, or no row
                // at all) may be NaN, so the row is cleared for GEMM2.
                if (cg == 0) {
#pragma unroll 1
                    for (int c = 0; c < kQ8Boxes; ++c) {
                        const uint32_t slot = (s_it * kQ8Halves + (c >> 1)) % C::kSlots;
                        uint4* d = reinterpret_cast<uint4*>(smem + C::kBoxOff + slot * kQ8SlotBytes +
                                                            (c & 1) * kQ8BoxBytes + row * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[i] = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(bar0 + 8 * (kQbPFull0 + pb));
            sc0 = nx0;
            sc1 = nx1;
            ++s_it;
        }
        if (!ok) break;

        // ---- epilogue ----
        {
            const float wsum = reduce_cols<false>(l, lane);
            if (lane % (32 / W) == 0) sums[lane / (32 / W) * 4 + wq] = wsum;
        }
        arrive(bar0 + 8 * (kQbSum0 + cg));
        ok = wait_warp(bar0 + 8 * (kQbSum0 + cg), item_it & 1, ctl);
        if (!ok) break;
        const uint32_t last = s_it - 1;
        float inv[W], m_own = 0.f, l_own = 0.f;
#pragma unroll
        for (int c = 0; c < W; ++c) {
            const float4 s4 = *reinterpret_cast<const float4*>(sums + c * 4);
            const float ls = (s4.x + s4.y) + (s4.z + s4.w);
            inv[c] = ls == 0.f ? 0.f : rcp_approx(ls);
            m_own = row == c ? m[c] : m_own;
            l_own = row == c ? ls : l_own;
        }
        if (row < W && gc0 + row < p.N) {
            const int gc = gc0 + row;
            // (the exponents are added first: the sum's unit is a scale's inverse, and what is
            // left of large ones is small)
            int e;
            const float part = log2f(frexpf(l_own, &e));
            const float lse = l_own == 0.f ? -INFINITY : ((m_own + ((float)(e - unit()) - kQ8Bias)) + part) * kLn2;
            if (item.unsplit) {
                const int sq = gc >= p.heads ? 1 : 0;  // (at most two query tokens)
                p.lse[((size_t)item.b * p.heads + (gc - sq * p.heads)) * p.s_q + sq] = lse;
            } else if (item.slot >= 0) {
                // (the combine's maximum passes over a NaN; an infinity makes its
                // weights NaN, and so the merged row)
                p.lpart[(size_t)item.slot * NG + cg * W + row] = isnan(lse) ? INFINITY : lse;
            }
        }
        ok = wait_warp(bar0 + 8 * (kQbPEmpty0 + last % C::kPBufs), (last / C::kPBufs) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        // Output column d of the chunk is this thread's lane: 32 lanes store 32
        // consecutive values of one query column.
        const bool f32 = !item.unsplit || p.out_f32;
        const int cols = item.unsplit ? p.N - gc0 : item.slot >= 0 ? W : 0;
        const size_t base = (item.unsplit ? (size_t)item.b * p.N + gc0 : (size_t)item.slot * NG + cg * W) * kDv + row;
        float* dst = (item.unsplit ? static_cast<float*>(p.out) : p.opart) + base;
        __nv_bfloat16* dst16 = static_cast<__nv_bfloat16*>(p.out) + base;
        const float scale = pow2f(unit());
#pragma unroll 1
        for (int ch = 0; ch < kQ8Boxes; ++ch) {
            float o[W], o1[W], o2[W];
            const uint32_t ta = tm + C::kOCol + ch * C::kNP + cg * W;
            tmem_ld_cols(ta, o);
            tmem_ld_cols(ta + NG, o1);
            tmem_ld_cols(ta + 2 * NG, o2);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < W; ++c) o[c] = fmaf(fmaf(o2[c], 0.0625f, o1[c]), 0.0625f, o[c]) * inv[c] * scale;
            if (f32) {
#pragma unroll
                for (int c = 0; c < W; ++c)
                    if (c < cols) dst[c * kDv] = o[c];
            } else {
#pragma unroll
                for (int c = 0; c < W; ++c)
                    if (c < cols) dst16[c * kDv] = __float2bfloat16_rn(o[c]);
            }
            dst += 128;
            dst16 += 128;
        }
        if (!item.unsplit && item.slot < 0 && row == 0) atomicOr(p.status, MLA_STATUS_BAD_SCHEDULE);
        tc_fence_before();
        arrive(bar0 + 8 * kQbOEmpty);
        ++item_it;
    }
}

// publish_plan_in_cta for one warp: this CTA's row of the plan, the rows of the work items
// whose first page it holds, and CTA 0's header and prefix.
__device__ void q8_publish(const FwdParams& p, int NG, const int32_t* prefix, const int32_t* plan_s) {
    const int lane = threadIdx.x & 31;
    const int k = blockIdx.x / p.share, G = gridDim.x / p.share, BG = p.BG;
    const bool writer = blockIdx.x % p.share == 0;  // group 0 of a shared range writes its rows
    const int64_t T = plan_s[kPlanT];
    if (lane < kMetaWords && writer) p.plan_out[kHdrWords + (size_t)k * kMetaWords + lane] = plan_s[lane];
    int32_t* bginfo = p.plan_out + bg_offset_words(G);
    int slots = 0;
    for (int bg = lane; bg < BG; bg += 32) {
        const int P = pages_in_prefix(prefix, bg, p.overhead);
        const int ns = num_splits_of(prefix, bg, P, T, p.overhead);
        if (ns > 1) slots += ns;
        int owner = P > 0 ? first_cta_of(prefix, bg, T, p.overhead) : 0;
        if (owner > G - 1) owner = G - 1;
        if (owner == k && writer) {
            bginfo[kBgWords * bg] = ns > 1 ? first_split_slot(prefix, bg, T, p.overhead) : 0;
            bginfo[kBgWords * bg + 1] = ns;
        }
    }
    if (blockIdx.x != 0) return;
    int32_t* pg = p.plan_out + prefix_offset_words(G, BG);
    for (int i = lane; i <= BG; i += 32) pg[i] = prefix[i];
    slots = __reduce_add_sync(kFullMask, slots);
    if (lane == 0) {
        int32_t* h = p.plan_out;
        h[kHdrMagic] = kSchedMagic;
        h[kHdrG] = G;
        h[kHdrBG] = BG;
        h[kHdrHg] = p.Hg;
        h[kHdrNG] = NG;
        h[kHdrSlots] = slots;
        h[kHdrT] = (int)T;
        h[kHdrW] = plan_s[kPlanW];
        h[kHdrBatch] = BG / p.Hg;
        h[kHdrMaxBlocks] = p.max_blocks;
        h[kHdrShift] = kPageShift;
        h[kHdrShareHg] = p.share;
        for (int i = kHdrShareHg + 1; i < kHdrWords; ++i) h[i] = 0;
        if (plan_s[kPlanBad]) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    }
}

// ------------------------------------------------------------------ kernel
template <int NG>
__global__ void __launch_bounds__(Q8Cfg<NG>::kThreads, 1)
    mla_decode_q8_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map,
                         const Q8Params p) {
    using C = Q8Cfg<NG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    const uint32_t bar0 = smem_addr(smem + C::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    int32_t* meta_s = reinterpret_cast<int32_t*>(smem + C::kPlanMetaOff);
    constexpr int kSm = 4 * C::kColGroups;  // softmax warps (a warp arrives once)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kQbCount; ++i) {
            uint32_t count = 1;
            if (i == kQbSEmpty0 || i == kQbSEmpty1 || i == kQbPFull0 || i == kQbPFull1 || i == kQbOEmpty || i == kQbQSeen)
                count = kSm;
            if (i >= kQbVote0 && i < kQbFull0) count = 4;
            if (i == kQbQFull) count = NG / 4;  // 4 rows per warp
            mbar_init(bar0 + 8 * i, count);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    if (p.plan_out != nullptr)
        for (int i = 32 * threadIdx.x; i < p.BG / p.Hg; i += 32 * blockDim.x) prefetch_l2_line(p.seqlens + i);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The plan from the lengths, and the first step's pages, before the wait on
    // the grid before this one (see mla_decode_fwd_kernel).
    const bool small_plan = p.BG <= C::kSmallPlan;
    int32_t* plan_scratch =
        reinterpret_cast<int32_t*>(smem + (small_plan ? C::kPOff : C::kBoxOff + kQ8Halves * kQ8SlotBytes));
    bool first_issued = false;
    if (p.plan_out != nullptr) {
        build_plan_in_cta(p, plan_scratch, meta_s);
        if (threadIdx.x == 0 && p.test_stall == 0) {
            WorkIter it;
            it.init(meta_s, p);
            Item item;
            if (it.next(p, item)) {
                const int32_t* bt = p.block_table + (size_t)item.b * p.max_blocks + item.p0;
                const int ph0 = __ldg(bt), ph1 = item.p0 + 1 < item.p1 ? __ldg(bt + 1) : -1;
                // (a bad entry is left to the producer, which reports it after the wait)
                if ((unsigned)ph0 < (unsigned)p.num_blocks &&
                    (item.p0 + 1 >= item.p1 || (unsigned)ph1 < (unsigned)p.num_blocks)) {
                    const uint64_t policy = p.share > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
                    for (int hf = 0; hf < kQ8Halves; ++hf) q8_load<NG>(&kv_map, &rope_map, smem, hf, 0, hf, ph0, ph1, policy);
                    first_issued = true;
                }
            }
        }
    }
    griddep_wait();
    const uint32_t tmem = *tmem_slot;
    const int32_t* meta;
    if (p.plan_out != nullptr) {
        if (!small_plan) {
            fence_proxy_async_smem();  // the scratch, before copies land there
            publish_plan_in_cta(p, NG, plan_scratch, meta_s);
        }
        meta = meta_s;
    } else {
        const int32_t* hdr = p.sched;
        if (hdr[kHdrMagic] != kSchedMagic || hdr[kHdrG] != p.G || hdr[kHdrBG] != p.BG || hdr[kHdrHg] != p.Hg ||
            hdr[kHdrNG] != NG || hdr[kHdrShift] != kPageShift || hdr[kHdrShareHg] != p.share) {
            if (threadIdx.x == 0) atomicOr(p.status, MLA_STATUS_BAD_SCHEDULE);
            if (warp == 1) {
                tc_fence_after();
                tmem_dealloc(tmem, C::kTmemCols);
            }
            return;
        }
        meta = hdr + kHdrWords + (size_t)(blockIdx.x / p.share) * kMetaWords;
    }
    const Ctl ctl{abort_flag, p.status};
    if (warp >= C::kFirstSoftmax) {
        if constexpr (C::kSplitRegs) setmaxnreg_inc<C::kRegsSoftmax>();
        q8_softmax<NG>(p, meta, smem, tmem, ctl, p.plan_out != nullptr && small_plan);
    } else if (warp >= C::kFirstQ) {
        if constexpr (C::kSplitRegs) setmaxnreg_dec<C::kRegsQ>();
        q8_split_q<NG>(p, meta, smem, ctl);
    } else {
        if constexpr (C::kSplitRegs) setmaxnreg_dec<C::kRegsIssue>();
        if (warp == 0) {
            if (lane == 0) q8_producer<NG>(&kv_map, &rope_map, p, meta, smem, ctl, first_issued);
        } else if (warp == 1) {
            q8_gemm1<NG>(p, meta, smem, tmem, ctl);
            q8_drain(bar0 + 8 * kQbDone1);
        } else if (warp == 2) {
            q8_gemm2<NG>(p, meta, smem, tmem, ctl);
            q8_drain(bar0 + 8 * kQbDone2);
        } else if (p.plan_out != nullptr && small_plan) {
            q8_publish(p, NG, plan_scratch, meta_s);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar0 + 8 * kQbPlan);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace mla
