// pda_quant.cuh -- the split kernel of decode over an 8-bit cache.
//
// The plan, the producer warp, the prefetch warp and the merge of split units
// are those of the bf16 split kernel (pda_kernels.cuh); the stage loader and
// the consumers are this file's.  With codes k, v and row scales ks, vs,
//   s_t = scale ks_t (q . k_t),   o = sum_t e^(s_t) vs_t v_t / sum_t e^(s_t),
// so nothing is dequantised: K scales multiply the scores, V scales the
// weights.  HBM sees D + 4 bytes per row and the tensor cores see codes:
//   * e4m3, S^T = K q^T: q, scaled by a power of two per row so that its largest
//     lies in [128, 256), splits into two e4m3 parts, hi + lo / 32, with sums of
//     their own.  A residual is 8 at most, so 32 of it still fit, and what e4m3
//     cannot hold lies below its smallest step of 2^-9: the parts hold all eight
//     significant bits of values from 2^-7 on, 2^-14 of the largest, and smaller
//     ones to 2^-15, 2^-22 of it.  Two m16n8k32 products take K's bytes as they
//     lie in shared memory.
//   * int8: codes become fp16 exactly (the byte placed under 0x64 reads as
//     1024 + u) for m16n8k16, q in fp16 with the same power-of-two scale.
//   * O^T += V^T P^T (m16n8k16): ldmatrix transposes pairs of bytes, so a lane
//     gets columns 2g, 2g + 1 of two tokens; they become rows g and g + 8 of
//     the product's A operand, which only permutes the rows of O.
// A weight that multiplies V is p' = 2^(s + log2 vs - m'), with the reference
// m' following the maximum of s + log2 vs, so that p' stays inside fp16
// whatever the V scales are; the sum of weights adds 2^(s - m'), which may be
// as small as 2^-116 or as large as 2^74 (see kSumBias).  (m', l, o) is an
// online-softmax state like any other: o / l and merges do not depend on the
// reference.  For bf16 outputs p' enters the product as fp16, off by 2^-11 of it
// at most: an eighth of the output's own half step.  For fp32 outputs (FINE) it
// enters as two fp16 parts, off by 2^-22, at twice the products with V (32
// sequences of 4096 tokens: 54.2 us for 53.1, 4 queries on 2456: 66.3 for 63.7).
// References sit kRefBias below the maximum they were taken at and move when a
// maximum passes them by more than kRefBias + kLazyLog2, so p' < 2^14 and what
// fp16 flushes is 2^-31 of the largest weight.
#pragma once

#include <cuda_fp16.h>

#include "pda_kernels.cuh"
#include "pda_quant.h"

namespace pda {

constexpr float kRefBias = 6.f;
constexpr float kLowPart = 32.f;  // times the residual of a q element in e4m3
// V scales below 2^-60 count as this (the codes of a scale of 0 are 0; others'
// elements are off by 448 * 2^-60 = 4e-16 at most), and scales of finite values
// are below 2^122 (2^128 / 127).  A row's p' is 2^(kRefBias + kLazyLog2) at
// most, so it adds 2^74 or less to the sum of weights, and 2^31 rows 2^105; the
// row of the largest score adds at least 2^(kRefBias - 122) = 2^-116, as its own
// p' or another's reaches the reference.  A warp's sum is kept times 2^kSumBias,
// so both ends, and rows 2^-30 of the largest, stay inside fp32.  References of
// states that merge lie up to 2^182 apart: their sums are scaled in two steps.
constexpr float kLeastScale = 8.6736174e-19f;
constexpr float kSumBias = 20.f;

template <int D, int NT>
struct QuantCfg {
    static constexpr int kWarps = quant_warps(D, NT);
    static constexpr int kRW = kWarps / NT;             // warps of a q tile
    static constexpr int kRT = quant_row_tiles(D, NT);
    static constexpr int kST = quant_stage_rows(D, NT);
    static constexpr int kMainThreads = (kWarps + 1) * 32;
    static constexpr int kThreads = kMainThreads + 32;  // + the prefetch warp
    static constexpr int kRB = D < 128 ? D : 128;       // bytes of a row in one swizzled slab
    static constexpr int kSlabs = D / kRB;
    static constexpr int kTileBytes = kST * D;
    static constexpr int kSOff = 2 * kTileBytes;        // the rows' scales: per block [K bs][V bs] floats
    static constexpr int kQOff = kSOff + kST * 8;       // the q rows
    static constexpr int kStageBytes = quant_stage_bytes(D, NT);
    static constexpr int kStages = quant_stages(D, NT);
    static constexpr int kK = D / 32;                   // 32-column steps of a row
    static_assert(kStageBytes % 1024 == 0, "stages start on swizzle spans");
    static_assert(kWarps * 8 * (D + 4) * 4 <= kStageBytes && kRW * 16 <= 4 * kMaxRowsPerWalk, "the staged states fit a stage");
};

// A stage holds blocks of 1 << lbs rows back to back (one of kST rows when the
// rows came one by one), each [K][V] (or V first) of [slabs][rows][kRB bytes].
// Row t's offset within the K or V parts, slab 0, and the XOR of the chunk
// index in a row at byte offset `off` of the stage: the TMA swizzle takes it
// from address bits 7.. (three of them for 128-byte rows, two for 64-byte
// rows); stages start on 1024-byte spans.
template <int D>
__device__ __forceinline__ uint32_t quant_row_off(int t, int lbs) {
    constexpr int RB = D < 128 ? D : 128;
    return ((uint32_t)(t >> lbs) << lbs) * (2u * D) + (uint32_t)(t & ((1 << lbs) - 1)) * RB;
}
template <int D>
__device__ __forceinline__ int quant_swz(uint32_t off) {
    return (int)(off >> 7) & (D == 64 ? 3 : 7);
}

template <int D, int NT>
struct QuantLoader {
    using C = QuantCfg<D, NT>;
    // at most 64 blocks (the producer's window of block ids), 32 where a lane takes one
    static __device__ __forceinline__ int blocks_per_stage(const SplitParams& p) {
        return min(C::kST / p.bs, p.row_gather ? 64 : 32);
    }
    static __device__ __forceinline__ uint32_t arrivals(const SplitParams& p) { return p.row_gather ? 33u : 1u; }
    // scales come four blocks to a copy where a stage has room for four
    static __device__ __forceinline__ bool four(const SplitParams& p) { return 4 * p.bs <= C::kST; }
    static __device__ __forceinline__ uint32_t tx_bytes(const SplitParams& p, int32_t n, int) {
        const uint32_t scaled = four(p) ? (uint32_t)(n + 3) & ~3u : (uint32_t)n;
        return p.row_gather == 0 ? ((uint32_t)n * (2u * D) + scaled * 8u) * p.bs : 0u;
    }
    static __device__ __forceinline__ uint32_t q_bytes(const SplitParams&, int nr) { return (uint32_t)(nr * D * 2); }
    static __device__ __forceinline__ void load_q(const SplitParams& p, uint32_t sK, int k, const uint16_t* q,
                                                  uint32_t full) {
        bulk_load(sK + C::kQOff + (uint32_t)(k * p.G * D * 2), q, (uint32_t)(p.G * D * 2), full);
    }
    template <typename WinId>
    static __device__ __forceinline__ void issue(const SplitParams& sp, uint32_t sK, int32_t n, int rows, int32_t rel,
                                                 int kvh, uint32_t full, uint64_t pol, int lane, const WinId& win_id) {
        const QuantParams& p = static_cast<const QuantParams&>(sp);
        const int bs = p.bs;
        const uint32_t sS = sK + C::kSOff;
        auto checked = [&](int32_t id) {
            if (id < 0 || (int64_t)id >= p.num_blocks) {
                atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
                id = 0;  // stays in bounds; the flag marks the result invalid
            }
            return id;
        };
        const int lbs = 31 - __clz(bs);
        if (p.row_gather == 0) {
            // lane i copies block i.  A warp's copies go out one lane after another, 80
            // to 100 cycles each, and with three a block (K, V, scales) that alone was
            // 2100 of a stage's 3000 cycles at block size 16: hence one joined box for
            // K and V, and the scales of four blocks to a copy.  (Scales by cp.async
            // took 900 cycles a stage; a uniform loop with one elected lane issuing
            // was slower than the lanes.)
            const int32_t id = checked(win_id(rel + min(lane, n - 1)));
            if (lane < n) {
                const uint32_t dst = sK + ((uint32_t)lane << lbs) * (2u * D);
                if (p.joined) {
                    tma_load_5d(dst, &p.tm_k, 0, 0, p.box_head * kvh, 0, id, full, pol);
                } else {
                    tma_load_5d(dst, &p.tm_k, 0, 0, 0, kvh, id, full, pol);
                    tma_load_5d(dst + (uint32_t)bs * D, &p.tm_v, 0, 0, 0, kvh, id, full, pol);
                }
            }
            if (four(p)) {
                const int32_t row = id * p.Hkv + kvh;  // lanes from n on repeat the last
                const int32_t r1 = __shfl_down_sync(0xffffffffu, row, 1), r2 = __shfl_down_sync(0xffffffffu, row, 2);
                const int32_t r3 = __shfl_down_sync(0xffffffffu, row, 3);
                if ((lane & 3) == 0 && lane < n)
                    tma_gather4(sS + ((uint32_t)lane << (lbs + 3)), &p.tm_k1, 0, row, r1, r2, r3, full, pol);
            } else if (lane < n) {
                bulk_load(sS + ((uint32_t)lane << (lbs + 3)), p.scales + (((int64_t)id * p.Hkv + kvh) << (lbs + 1)), 8u * bs,
                          full);
            }
        } else {
            const int lp = lbs > 0 ? lbs - 1 : 0;  // log2 of a block's 16-byte pieces (8 bytes for one token)
            for (int i0 = 0; i0 < n << lp; i0 += 32) {
                const int i = min(i0 + lane, (n << lp) - 1), blk = i >> lp;
                const int32_t id = checked(win_id(rel + blk));
                const float* s = p.scales + (((int64_t)id * p.Hkv + kvh) << (lbs + 1));
                if (i0 + lane < n << lp) {
                    if (lbs > 0) cp_async_16(sS + 16u * i, s + 4 * (i - (blk << lp)));
                    else cp_async_8(sS + 8u * i, s);
                }
            }
            // rows one by one in 16-byte chunks, written as one block of kST rows
            constexpr int CH = D / 16, RPI = 32 / CH;
            const int c = lane % CH, sub = lane / CH;
            const uint8_t* kb = reinterpret_cast<const uint8_t*>(p.k_base) + (int64_t)kvh * p.kvh_s + c * 16;
            const uint8_t* vb = reinterpret_cast<const uint8_t*>(p.v_base) + (int64_t)kvh * p.kvh_s + c * 16;
            constexpr int CPS = C::kRB / 16;
            for (int t0 = 0; t0 < rows; t0 += RPI) {
                const int t = t0 + sub;
                const int32_t wid = win_id(rel + (min(t, rows - 1) >> lbs));
                if (t < rows) {
                    const int64_t off = (int64_t)checked(wid) * p.blk_s + (int64_t)(t & (bs - 1)) * p.tok_s;
                    const uint32_t r = (uint32_t)(c / CPS) * (C::kST * C::kRB) + (uint32_t)t * C::kRB;
                    const uint32_t dst = sK + r + (uint32_t)(((c % CPS) ^ quant_swz<D>(r)) << 4);
                    cp_async_16(dst, kb + off);
                    cp_async_16(dst + C::kTileBytes, vb + off);
                }
            }
            cp_async_mbar_arrive_noinc(full);
        }
    }
};

template <int D, int NT>
struct TouchQuant {  // a block's rows of a kv head and their scales, towards L2
    static __device__ __forceinline__ int stage_rows(const SplitParams&) { return QuantCfg<D, NT>::kST; }
    static __device__ __forceinline__ void block(const SplitParams& sp, int32_t kvh, int32_t id) {
        const QuantParams& p = static_cast<const QuantParams&>(sp);
        if (p.joined) {
            tma_prefetch_5d(&p.tm_k, 0, 0, p.box_head * kvh, 0, id);
        } else {
            tma_prefetch_5d(&p.tm_k, 0, 0, 0, kvh, id);
            tma_prefetch_5d(&p.tm_v, 0, 0, 0, kvh, id);
        }
        bulk_prefetch(p.scales + ((int64_t)id * p.Hkv + kvh) * 2 * p.bs, 8u * p.bs);
    }
};

// The states that the W warps of a segment staged, st_m / st_l [warp][16 rows]
// and, of the tile's 8 rows, st_o [warp][8][D + 4]: the combined state of q row
// h, row hr of the tile.
template <int D, int W>
struct UnitSlices {
    const float *st_m, *st_l, *st_o;
    __device__ __forceinline__ void operator()(int h, int hr, int d4, float& M, float& Ls, float4& Os) const {
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, st_m[w * 16 + h]);
        if (M == kNegInf) return;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float d = st_m[w * 16 + h] - M, f = ex2(d);
            const float4 v = *reinterpret_cast<const float4*>(st_o + (size_t)(w * 8 + hr) * (D + 4) + d4);
            Ls += scale_sum(st_l[w * 16 + h], d);
            Os.x += v.x * f; Os.y += v.y * f; Os.z += v.z * f; Os.w += v.w * f;
        }
    }
};

// CTAs that a call's work is split over.  A unit of s stages in n pieces takes
// a s / n to stream and c n for the one CTA that merges them, four a round trip:
// n = sqrt(a s / c) is best, 2.4 sqrt(s) as measured, or 2.4 sqrt(units stages)
// CTAs over all units of a call; twice that for blocks below 8 tokens, whose
// stages take about four times as long; never less than a stage each.  One
// sequence of one kv head of 128 at 2, 2.4, 3, 4 sqrt: 2000 tokens 13.1, 13.5,
// 13.7, 15.1 us (79 over the whole grid), 32768 29.2, 29.4, 31.0, 35.7 (119), a
// million 134, 135, 150, 160; eight kv heads, 8192 tokens 17.2, 16.3, 16.2, 17.8.
// Two sequences of 2800 tokens, two kv heads of 256, blocks of one token: 35.4,
// 31.8, 30.2, 28.4, with a stage each 27.7.
// The prefetch warp cuts the work by the whole grid all the same: where fewer
// CTAs walk it, a CTA warms blocks that another one walks.  Cut by these CTAs
// instead, 8192 tokens of one kv head took 15.2 us for 15.1, 4 x 3000 of four
// 14.25 for 14.2, half a million of one 70.6 for 73.3; with no prefetch 15.0,
// 14.25 and 69.6 (replayed back to back, the first two from L2).
template <bool MQ, int ST>
__device__ __forceinline__ int64_t quant_plan_ctas(const SplitParams& p, const int32_t* pfx) {
    const int64_t stages = ((int64_t)pfx[p.B] * p.Hkv * p.bs + ST - 1) / ST, units = (int64_t)p.B * p.Hkv;
    const int64_t best = (int64_t)((p.bs < 8 ? 4.8f : 2.4f) * sqrtf((float)stages * (float)units));
    return min((int64_t)gridDim.x, max(min(stages, best), (int64_t)rows_per_seq<MQ>(p)));
}

// Two fp16 values from bytes lo, hi (0..3) of x.  int8: x holds code ^ 0x80;
// the byte under 0x64 reads as 1024 + code + 128.
template <int FMT, int lo, int hi>
__device__ __forceinline__ uint32_t half2_of(uint32_t x) {
    static_assert(FMT == kInt8, "int8");
    uint32_t h = __byte_perm(x, 0x64646464u, 0x4040 | lo | (hi << 8)), d;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x64806480u));  // 1152
    return d;
}

// The A fragment of 16 rows x 16 columns of K from the two registers of one
// 16-byte chunk (rows 0-7, rows 8-15): bytes 0, 1 are k slots 2t, 2t + 1 and
// bytes 2, 3 slots 2t + 8, 2t + 9, the order q's fragments follow.
__device__ __forceinline__ void k_fragment_int8(uint32_t r0, uint32_t r1, uint32_t (&a)[4]) {
    r0 ^= 0x80808080u;
    r1 ^= 0x80808080u;
    a[0] = half2_of<kInt8, 0, 1>(r0);
    a[1] = half2_of<kInt8, 0, 1>(r1);
    a[2] = half2_of<kInt8, 2, 3>(r0);
    a[3] = half2_of<kInt8, 2, 3>(r1);
}

// The A fragment of V^T, 16 columns x 16 tokens, from the transposed registers
// of one 16-byte chunk (tokens 0-7, tokens 8-15): bytes 0, 2 are column 2g of
// tokens 2t, 2t + 1 (row g), bytes 1, 3 column 2g + 1 (row g + 8).
template <int FMT>
__device__ __forceinline__ void v_fragment(uint32_t r0, uint32_t r1, uint32_t (&a)[4]) {
    if constexpr (FMT == kE4m3) {
        const uint32_t x = __byte_perm(r0, 0, 0x3120), y = __byte_perm(r1, 0, 0x3120);
        a[0] = e4m3x2_to_f16x2((uint16_t)x);
        a[1] = e4m3x2_to_f16x2((uint16_t)(x >> 16));
        a[2] = e4m3x2_to_f16x2((uint16_t)y);
        a[3] = e4m3x2_to_f16x2((uint16_t)(y >> 16));
    } else {
        r0 ^= 0x80808080u;
        r1 ^= 0x80808080u;
        a[0] = half2_of<kInt8, 0, 2>(r0);
        a[1] = half2_of<kInt8, 1, 3>(r0);
        a[2] = half2_of<kInt8, 0, 2>(r1);
        a[3] = half2_of<kInt8, 1, 3>(r1);
    }
}

// 0xff in the bytes of x that are NaN codes of e4m3.
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Where chunk c (16 bytes) of row r lies in a stage's V part at sV, before the
// swizzle of a row's chunks.
template <int D>
__device__ __forceinline__ uint32_t quant_chunk(uint32_t sV, int r, int c, int lbs) {
    constexpr int RB = D < 128 ? D : 128, CPS = RB / 16;
    return sV + quant_row_off<D>(r, lbs) + (((uint32_t)(c / CPS) * RB) << lbs) + (uint32_t)(c % CPS) * 16;
}
// Whether rows r .. r + n - 1 hold a NaN code (one warp's answer).
template <int D>
__device__ __forceinline__ bool any_nan_code(uint32_t sV, int r, int n, int lbs, int lane) {
    uint32_t any = 0;
#pragma unroll 1
    for (int u = lane; u < n * (D / 16); u += 32) {
        uint32_t x[4];
        lds_v4(quant_chunk<D>(sV, r + u / (D / 16), u % (D / 16), lbs), x);
        any |= nan_codes(x[0]) | nan_codes(x[1]) | nan_codes(x[2]) | nan_codes(x[3]);
    }
    return __any_sync(0xffffffffu, any != 0);
}
// NaN codes in values that only some of the queries of a walk see would give the
// others NaN, as 0 * NaN.  In rows r .. r + n - 1 (one warp's) of a stage's V part
// at sV they become 0, and the columns of O that they make NaN for this lane's
// queries, which see the first from0 + 1 and from1 + 1 of these rows, are noted
// until the segment ends: bits 4 i + 2 c, + 1 are columns 16 i + 2 g and the next
// of its c-th query.  Walks whose last rows hold no such codes only look for
// them: 4 queries on 2456 tokens 62.0 us for 61.8 without, 2 queries at head size
// 256 42.4 for 41.3.
template <int W, int RW>
struct NanNotes {
    uint64_t cols[W * 32];  // [thread]
    uint64_t bars[RW];      // of the warps that share KV rows
    uint32_t phase[W];
};
template <int D, int NT, class Notes>
__device__ __forceinline__ void hide_nan_codes(Notes* notes, uint32_t sV, int r, int n, int lbs, int from0, int from1,
                                            bool paired, int thread, uint32_t* err, volatile int* abort_flag) {
    constexpr int CH = D / 16, CPS = D < 128 ? CH : 8;
    const int lane = thread & 31, warp = thread >> 5;
    const auto chunk = [&](int i, int c) { return quant_chunk<D>(sV, r + i, c, lbs); };
    uint64_t cols = notes->cols[thread];
    for (int i = 0; i < n; ++i)
        for (int c = 0; c < CH; ++c) {
            const int at = c / CPS * CPS + (c % CPS ^ quant_swz<D>(chunk(i, c / CPS * CPS)));
            uint32_t x[4];
            lds_v4(chunk(i, at), x);
            const int g = lane >> 2;
            const uint32_t bad = nan_codes(g < 2 ? x[0] : g < 4 ? x[1] : g < 6 ? x[2] : x[3]) >> (16 * (g & 1));
            const uint32_t two = (bad & 1u) | (bad >> 7 & 2u);
            cols |= (uint64_t)((i <= from0 ? two : 0u) | (i <= from1 ? two << 2 : 0u)) << (4 * c);
        }
    notes->cols[thread] = cols;
    __syncwarp();
    if (NT > 1 && paired) {  // the warp of the other q rows looks at these codes too
        uint32_t phase = notes->phase[warp];
        consumer_sync(smem_u32(&notes->bars[warp % (sizeof(notes->bars) / 8)]), phase, err, abort_flag);
        __syncwarp();
        if (lane == 0) notes->phase[warp] = phase;
    }
    for (int u = lane; u < n * CH; u += 32) {
        const uint32_t at = chunk(u / CH, u % CH);
        uint32_t x[4];
        lds_v4(at, x);
        sts_v4(at, x[0] & ~nan_codes(x[0]), x[1] & ~nan_codes(x[1]), x[2] & ~nan_codes(x[2]), x[3] & ~nan_codes(x[3]));
    }
    fence_proxy_async_smem();  // generic writes before the next TMA
    __syncwarp();
}

// Out of line: head size 256 has no registers left for it (2 queries 42.6 us,
// 44.0 inlined; at head size 128 43.2 and 41.4).
template <int D, int NT, class Notes>
__device__ __noinline__ void hide_nan_codes_apart(Notes* notes, uint32_t sV, int r, int n, int lbs, int from0, int from1,
                                                  bool paired, int thread, uint32_t* err, volatile int* abort_flag) {
    hide_nan_codes<D, NT>(notes, sV, r, n, lbs, from0, from1, paired, thread, err, abort_flag);
}

// A unit's q rows in the stage (bf16, 8 NT of them, those from nr on zero),
// scaled by a power of two each and turned in place into the lanes' B
// fragments [tile of 8 rows][32-column step][lane] of 16 bytes: e4m3, four high
// parts of columns 4t .. and 16 + 4t .., then their low parts; int8, the same
// columns in fp16.  `back` takes the factor that undoes each row's power of
// two, times the score scale.  A warp takes a row, an eighth of the work of
// every warp preparing all of its own fragments, whose reads at a row's stride
// also met on the same banks; both run once a unit and are fetched cold (16 q
// rows, 2456 tokens: 67.5 -> 66.7 us).
template <int D, int FMT, int NT, int W>
__device__ __forceinline__ bool quant_q_fragments(uint8_t* at, float* back, int nr, float scale, int warp, int lane,
                                                  uint32_t cbar, uint32_t& cphase, uint32_t* err,
                                                  volatile int* abort_flag) {
    constexpr int R = 8 * NT / W, N4 = D / 4, J = (N4 + 31) / 32;  // rows a warp, runs of four columns a row, and a lane
    static_assert(R * W == 8 * NT, "the rows divide over the warps");
    uint2 raw[R][J];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int row = r * W + warp, c4 = lane + 32 * j;
            raw[r][j] = row < nr && c4 < N4 ? *reinterpret_cast<const uint2*>(at + (row * D + 4 * c4) * 2) : make_uint2(0u, 0u);
        }
    if (!consumer_sync(cbar, cphase, err, abort_flag)) return false;  // every row is read
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = r * W + warp;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t x = raw[r][j].x, y = raw[r][j].y;
            top = max(top, max(max(x & 0x7fffu, (x >> 16) & 0x7fffu), max(y & 0x7fffu, (y >> 16) & 0x7fffu)));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // the row's largest magnitude lies in [2^e, 2^(e+1)): multiply by 2^(7-e)
        const int e = max((int)(top >> 7) - 127, -119);
        const float mult = __int_as_float((127 + 7 - e) << 23);
        if (lane == 0)  // infinities and NaN: NaN
            back[row] = top < 0x7f80u ? scale * __int_as_float((127 - 7 + e) << 23) : __int_as_float(0x7fffffff);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c4 = lane + 32 * j;
            const float x0 = bf16_lo(raw[r][j].x) * mult, x1 = bf16_hi(raw[r][j].x) * mult;
            const float x2 = bf16_lo(raw[r][j].y) * mult, x3 = bf16_hi(raw[r][j].y) * mult;
            uint32_t u, v;
            if constexpr (FMT == kE4m3) {
                const uint32_t h01 = pack_e4m3x2(x0, x1), h23 = pack_e4m3x2(x2, x3);
                const uint32_t b01 = e4m3x2_to_f16x2((uint16_t)h01), b23 = e4m3x2_to_f16x2((uint16_t)h23);
                const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&b01));
                const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&b23));
                u = h01 | (h23 << 16);
                v = pack_e4m3x2(kLowPart * (x0 - s.x), kLowPart * (x1 - s.y)) |
                    (pack_e4m3x2(kLowPart * (x2 - w.x), kLowPart * (x3 - w.y)) << 16);
            } else {
                u = pack_f16x2(x0, x1);
                v = pack_f16x2(x2, x3);
            }
            if (c4 < N4) {
                const int i = (c4 >> 2) & 1;
                uint32_t* d = reinterpret_cast<uint32_t*>(at) +
                              (((row >> 3) * (D / 32) + (c4 >> 3)) * 32 + (row & 7) * 4 + (c4 & 3)) * 4;
                d[FMT == kE4m3 ? i : 2 * i] = u;
                d[FMT == kE4m3 ? 2 + i : 2 * i + 1] = v;
            }
        }
    }
    fence_proxy_async_smem();  // generic writes before the next TMA into this stage
    return consumer_sync(cbar, cphase, err, abort_flag);
}

template <int D, int FMT, int NT, int MODE, bool FINE, class Notes>
__device__ __forceinline__ void run_quant_consumer(const QuantParams& p, uint32_t base_s, uint8_t* base,
                                                   const SmemLayout& L, const StageMeta* meta, const int32_t* pfx,
                                                   volatile int* abort_flag, const GroupRange* group,
                                                   Notes* notes, int warp, int lane) {
    using C = QuantCfg<D, NT>;
    constexpr int S = C::kStages, RT = C::kRT, K = C::kK;
    constexpr int kThreadsC = C::kWarps * 32, kOStride = D + 4;
    constexpr bool MQ = is_multi(MODE), kHide = MQ && FMT == kE4m3;
    const uint32_t full0 = base_s + L.bars, empty0 = full0 + 8 * S;
    const int g = lane >> 2, t = lane & 3;
    // warps 0 .. kRW - 1 take the first eight q rows, the next kRW the others, all of a stage's KV rows
    const int tile = NT > 1 ? warp / C::kRW : 0, rw = NT > 1 ? warp % C::kRW : warp;
    const int r0 = rw * 16 * RT;
    const int G = p.G;
    const int lbr = 31 - __clz(p.bs);                       // the cache's blocks
    const int lbs = p.row_gather ? 31 - __clz(C::kST) : lbr;  // the tile's blocks
    const uint32_t hs = (uint32_t)C::kRB << lbs;            // bytes between slabs of a block
    // ldmatrix lane addresses, alike for K and (transposed) V: matrices are rows
    // 0-7, rows 8-15 of chunk c, then of chunk c + 1
    const int row = r0 + (lane & 15), cpar = lane >> 4;
    const uint32_t part = (uint32_t)D << lbs;               // bytes between a block's K and V
    const uint32_t k_at = p.v_first ? part : 0u, v_at = p.v_first ? 0u : part;
    constexpr int CPS = C::kRB / 16;  // 16-byte chunks per slab row
    // Byte offsets in a stage of this lane's chunk `cpar` of its row, slab h, in K
    // and V; chunk 2 kk + cpar of a 32-column step lies at the offset XOR 32 kk
    // (rows start on multiples of their slab's bytes).  Row tiles are `tile_at`
    // apart and share the swizzle.
    uint32_t k_off[C::kSlabs], v_off[C::kSlabs];
#pragma unroll
    for (int h = 0; h < C::kSlabs; ++h) {
        const uint32_t ro = quant_row_off<D>(row, lbs) + h * hs;
        k_off[h] = ro + k_at + (uint32_t)((cpar ^ quant_swz<D>(ro + k_at)) << 4);
        v_off[h] = ro + v_at + (uint32_t)((cpar ^ quant_swz<D>(ro + v_at)) << 4);
    }
    const uint32_t tile_at = quant_row_off<D>(row + 16, lbs) - quant_row_off<D>(row, lbs);
    auto step = [](const uint32_t (&at)[C::kSlabs], int kk) { return at[(2 * kk) / CPS] ^ (uint32_t)((2 * kk) % CPS << 4); };
    // this lane's rows g, g + 8 of each tile: where their K scale is, in floats
    uint32_t s_off[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tr = r0 + 16 * r + 8 * i + g;
            s_off[r][i] = (uint32_t)(((tr >> lbr) << (lbr + 1)) + (tr & (p.bs - 1)));
        }

    float o[2 * K][4];
    uint32_t qf[K][4];
    float f[2] = {0.f, 0.f}, m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * K; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) qf[i][0] = qf[i][1] = qf[i][2] = qf[i][3] = 0u;
    // causal queries of this lane's score columns
    const int qc[2] = {MQ ? (8 * tile + 2 * t) / G : 0, MQ ? (8 * tile + 2 * t + 1) / G : 0};
    const uint32_t cbar = base_s + L.cbar;
    float* q_back = reinterpret_cast<float*>(base + L.st_x);  // [16 rows]
    uint32_t cphase = 0;
    int stage = 0;
    uint32_t phase = 0;
    int32_t ticket = 0;
    const int ct = warp * 32 + lane;
    zero_empty_rows<D, kThreadsC>(p, pfx, ct);

    while (true) {
        if (*abort_flag) break;
        if (!mbar_wait_bounded(full0 + 8 * stage, phase, kWaitLimitNs)) {
            atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
            *abort_flag = 1;
            break;
        }
        const StageMeta md = meta[stage];
        if (md.flags & kDone) break;
        // the last stage of a piece of a split unit draws the piece's ticket (see run_consumer)
        if (warp == 0 && lane == 0 && (md.flags & kSegEnd) && !(md.flags & kWholeUnit))
            ticket = atomicAdd(p.unit_sync + 2 * (md.b * p.Hkv + md.kvh), 1);
        const uint32_t s0 = base_s + (uint32_t)stage * C::kStageBytes;
        const uint32_t sV = s0 + v_at;
        const uint8_t* bytes = base + (s0 - base_s);

        if (md.flags & kSegBegin) {
            if (!quant_q_fragments<D, FMT, NT, C::kWarps>(base + (s0 - base_s) + C::kQOff, q_back, MQ ? md.nr : G,
                                                          p.scale_log2, warp, lane, cbar, cphase, p.err, abort_flag))
                break;
            const uint4* frags = reinterpret_cast<const uint4*>(bytes + C::kQOff) + tile * K * 32 + lane;
#pragma unroll
            for (int kk = 0; kk < K; ++kk) {
                const uint4 w = frags[kk * 32];
                qf[kk][0] = w.x; qf[kk][1] = w.y; qf[kk][2] = w.z; qf[kk][3] = w.w;
            }
            f[0] = q_back[8 * tile + 2 * t];
            f[1] = q_back[8 * tile + 2 * t + 1];
            m[0] = m[1] = kNegInf;
            l[0] = l[1] = 0.f;
            if constexpr (kHide) notes->cols[ct] = 0;
#pragma unroll
            for (int i = 0; i < 2 * K; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        if (r0 < md.n_valid && (NT == 1 || 8 * tile < md.nr)) {
            const bool partial = r0 + 16 * RT > md.n_valid;
            const int pos0 = MQ ? md.j0 * p.bs + r0 : 0;
            const bool diagonal = MQ && pos0 + 16 * RT - 1 > md.lim;  // some queries do not see some of these rows
            if (FMT == kE4m3 && (MQ ? partial || diagonal : partial)) {
                // rows behind the end may hold NaN codes, and 0 * NaN would poison P V
                for (int u = lane; u < (r0 + 16 * RT - md.n_valid) * (D / 16); u += 32) {
                    const int r = md.n_valid + u / (D / 16), c = u % (D / 16);
                    const uint32_t a = sV + quant_row_off<D>(r, lbs) + (uint32_t)(c / CPS) * hs + (uint32_t)((c % CPS) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                }
                if constexpr (kHide) {
                    const int later = max(0, md.lim + 1 - pos0);  // the first row that some query does not see
                    const int n = min(16 * RT, md.n_valid - r0) - later;
                    if (any_nan_code<D>(sV, r0 + later, n, lbs, lane)) {
                        constexpr auto hide = D == 256 ? hide_nan_codes_apart<D, NT, Notes> : hide_nan_codes<D, NT, Notes>;
                        hide(notes, sV, r0 + later, n, lbs, md.lim - pos0 - later + qc[0], md.lim - pos0 - later + qc[1],
                             md.nr > 8, ct, p.err, abort_flag);
                    }
                }
                __syncwarp();
            }
            float ks[RT][2], lv[RT][2], lw[RT][2];
            const float* sp = reinterpret_cast<const float*>(bytes + C::kSOff);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ks[r][i] = sp[s_off[r][i]];
                    float vs = sp[s_off[r][i] + p.bs];
                    if (partial && r0 + 16 * r + 8 * i + g >= md.n_valid) vs = 1.f;
                    lv[r][i] = lg2(max_nan(vs, kLeastScale));
                    // log2 of what takes p' to the sum of weights.  fminf drops a NaN, which
                    // stays in lv: the scores of a row of scale NaN are NaN, but a causal
                    // query that does not see it adds 0.
                    lw[r][i] = fminf(kSumBias - lv[r][i], kSumBias + 60.f);
                }
            float x[RT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float acc[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][i] = acc[1][i] = 0.f;
#pragma unroll
                for (int kk = 0; kk < K; ++kk) {
                    uint32_t w[4];
                    ldsm_x4(s0 + r * tile_at + step(k_off, kk), w);
                    if constexpr (FMT == kE4m3) {
                        mma_e4m3_16832(acc[0], w, qf[kk][0], qf[kk][1]);
                        mma_e4m3_16832(acc[1], w, qf[kk][2], qf[kk][3]);
                    } else {
                        uint32_t a[4], b[4];
                        k_fragment_int8(w[0], w[1], a);
                        k_fragment_int8(w[2], w[3], b);
                        mma_f16_16816(acc[0], a, qf[kk][0], qf[kk][1]);
                        mma_f16_16816(acc[1], b, qf[kk][2], qf[kk][3]);
                    }
                }
                // x: the score in base-2 units plus log2 of the row's V scale
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[r][i] = fmaf(FMT == kE4m3 ? fmaf(acc[1][i], 1.f / kLowPart, acc[0][i]) : acc[0][i] + acc[1][i],
                                   ks[r][i >> 1] * f[i & 1], lv[r][i >> 1]);
            }
            if (partial) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (r0 + 16 * r + 8 * (i >> 1) + g >= md.n_valid) x[r][i] = kNegInf;
            }
            if (MQ && diagonal) {  // column c is query c / G of the row: no later tokens
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pos0 + 16 * r + 8 * (i >> 1) + g > md.lim + qc[i & 1]) x[r][i] = kNegInf;
            }
            // the references move only when a weight would pass 2^(kRefBias + kLazyLog2);
            // the columns' maxima are taken only then
            float top[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                top[c] = fmaxf(x[0][c], x[0][c + 2]);
#pragma unroll
                for (int r = 1; r < RT; ++r) top[c] = fmaxf(top[c], fmaxf(x[r][c], x[r][c + 2]));
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] + (kLazyLog2 + kRefBias) || top[1] > m[1] + (kLazyLog2 + kRefBias))) {
                float a[2];  // an empty column (m = -inf): 0
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], s));
                    const bool up = top[c] > m[c] + (kLazyLog2 + kRefBias);
                    const float to = up ? top[c] - kRefBias : m[c];
                    a[c] = up ? ex2(m[c] - to) : 1.f;
                    if (up) l[c] = scale_sum(l[c], m[c] - to);
                    m[c] = to;
                }
#pragma unroll
                for (int i = 0; i < 2 * K; ++i) {
                    o[i][0] *= a[0]; o[i][1] *= a[1]; o[i][2] *= a[0]; o[i][3] *= a[1];
                }
            }
            const float u0 = m[0] == kNegInf ? 0.f : m[0];
            const float u1 = m[1] == kNegInf ? 0.f : m[1];
            uint32_t pb[RT][2], pl[RT][2];  // weights, and (FINE) what fp16 leaves of them
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float d0 = x[r][0] - u0, d1 = x[r][1] - u1, d2 = x[r][2] - u0, d3 = x[r][3] - u1;
                const float p0 = ex2(d0), p1 = ex2(d1), p2 = ex2(d2), p3 = ex2(d3);
                l[0] += ex2(d0 + lw[r][0]) + ex2(d2 + lw[r][1]);
                l[1] += ex2(d1 + lw[r][0]) + ex2(d3 + lw[r][1]);
                const uint32_t h01 = pack_f16x2(p0, p1), h23 = pack_f16x2(p2, p3);
                pb[r][0] = movmatrix_trans(h01);
                pb[r][1] = movmatrix_trans(h23);
                if constexpr (FINE) {
                    const float2 b01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
                    const float2 b23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
                    pl[r][0] = movmatrix_trans(pack_f16x2(p0 - b01.x, p1 - b01.y));
                    pl[r][1] = movmatrix_trans(pack_f16x2(p2 - b23.x, p3 - b23.y));
                }
            }
#pragma unroll
            for (int kk = 0; kk < K; ++kk)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint32_t w[4], a[4], b[4];
                    ldsm_x4_trans(s0 + r * tile_at + step(v_off, kk), w);
                    v_fragment<FMT>(w[0], w[1], a);
                    v_fragment<FMT>(w[2], w[3], b);
                    mma_f16_16816(o[2 * kk], a, pb[r][0], pb[r][1]);
                    mma_f16_16816(o[2 * kk + 1], b, pb[r][0], pb[r][1]);
                    if constexpr (FINE) {
                        mma_f16_16816(o[2 * kk], a, pl[r][0], pl[r][1]);
                        mma_f16_16816(o[2 * kk + 1], b, pl[r][0], pl[r][1]);
                    }
                }
            if (FMT == kE4m3 && partial) fence_proxy_async_smem();  // generic writes before the next TMA
        }
        if (md.flags & kSegEnd) {
            // the warps' states merge through this stage's memory; roles as in run_consumer
            float* st_m = reinterpret_cast<float*>(base + L.st_m);  // [warp][16 rows]
            float* st_l = reinterpret_cast<float*>(base + L.st_l);
            int32_t* st_role = reinterpret_cast<int32_t*>(base + L.st_x) + 2 * kMaxGroup;
            float* st_o = reinterpret_cast<float*>(base + (s0 - base_s));  // [warp][8][kOStride]
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], s);
            if (!consumer_sync(cbar, cphase, p.err, abort_flag)) break;  // all reads of the stage done
            const RowInfo ri = row_info<MQ>(p, md.b);
            StageMeta me = md;
            me.nr = ri.cnt * G;
            UnitPieces pc;
            pc.cf = 0; pc.su = 0; pc.n = 1; pc.every = true;
            const GroupRange grs = *group;  // of units in pieces
            if (!(md.flags & kWholeUnit)) pc = unit_pieces(pfx, md.b, md.kvh, p.Hkv, p.unit_cost, grs);
            int role = kRoleAbort;
            bool stop = false;
            const uint64_t nan_cols = kHide ? notes->cols[ct] : 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // a warp's states of its eight rows
                const int hr = 2 * t + c, h = 8 * tile + hr;
                if (h >= me.nr) continue;
                if (g == 0) {
                    // a NaN sum must not hide behind an empty reference
                    st_m[rw * 16 + h] = l[c] == l[c] ? m[c] : 0.f;
                    st_l[rw * 16 + h] = l[c] * (1.f / (1 << (int)kSumBias));
                }
                float* r = st_o + (size_t)(warp * 8 + hr) * kOStride + 2 * g;
#pragma unroll
                for (int i = 0; i < 2 * K; ++i) {
                    float2 v = make_float2(o[i][c], o[i][2 + c]);
                    if constexpr (kHide) {
                        const uint32_t bad = (uint32_t)(nan_cols >> (4 * i + 2 * c));
                        if (bad & 1u) v.x = __int_as_float(0x7fffffff);
                        if (bad & 2u) v.y = __int_as_float(0x7fffffff);
                    }
                    *reinterpret_cast<float2*>(r + 16 * i) = v;
                }
            }
            // one copy of the merge's code for both tiles: code that runs once a unit is fetched cold
#pragma unroll 1
            for (int n = 0; n < NT && 8 * n < me.nr; ++n) {
                if (!rows_tile_merge<D, kThreadsC, 8, true>(
                        p, me, n, ct, ticket, pc, grs, ri,
                        UnitSlices<D, C::kRW>{st_m, st_l, st_o + (size_t)n * C::kRW * 8 * kOStride}, st_role, cbar, cphase,
                        abort_flag, role)) {
                    stop = true;
                    break;
                }
            }
            if (stop) break;
            if (!consumer_sync(cbar, cphase, p.err, abort_flag)) break;
            if (role == kRoleStore && ct == 0) red_release_gpu_add(p.unit_sync + 2 * (md.b * p.Hkv + md.kvh) + 1, 1);
            fence_proxy_async_smem();  // staging writes before the next TMA into this stage
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * stage);
        if (++stage == S) { stage = 0; phase ^= 1u; }
    }
}

template <int D, int FMT, int NT, int MODE, bool FINE>
__global__ void __maxnreg__(168) quant_split_kernel(const __grid_constant__ QuantParams p) {
    using C = QuantCfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ GroupRange group;  // of this CTA
    constexpr bool kHide = is_multi(MODE) && FMT == kE4m3;
    __shared__ NanNotes<kHide ? C::kWarps : 1, kHide ? C::kRW : 1> notes;
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_s - raw_s);
    const SmemLayout L = smem_layout_of(C::kStageBytes, kOneShot, C::kStages, p.B);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* pfx = reinterpret_cast<int32_t*>(base + L.pfx);
    int32_t* scan = reinterpret_cast<int32_t*>(base + L.scan);
    StageMeta* meta = reinterpret_cast<StageMeta*>(base + L.meta);
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(base_s + L.bars + 8 * s, QuantLoader<D, NT>::arrivals(p));
            mbar_init(base_s + L.bars + 8 * (C::kStages + s), C::kWarps);
        }
        mbar_init(base_s + L.cbar, C::kWarps * 32);
        if (kHide)
            for (int i = 0; i < C::kRW; ++i) mbar_init(smem_u32(notes.bars + i), NT * 32);
        fence_mbar_init();
        abort_flag = 0;
    }
    if (kHide && tid < C::kWarps) notes.phase[tid] = 0;
    if (tid == C::kWarps * 32 && p.row_gather == 0) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_k1);
        if (!p.joined) prefetch_tensormap(&p.tm_v);
    }
    if (warp == C::kMainThreads / 32) {  // the prefetch warp: joins nothing below
        if (p.prefetch) prefetch_first_stages<MODE, TouchQuant<D, NT>>(p, lane);
        return;
    }
    pdl_wait_primary();
    pdl_launch_dependents();
    const int32_t nv_max = build_prefix<is_multi(MODE), C::kMainThreads>(p, pfx, scan);
    int64_t begin, end;
    int64_t ctas = gridDim.x;
    const bool by_unit = unit_mode((int64_t)p.B * p.Hkv, ctas, real_blocks(nv_max, p.unit_cost), C::kST, p.bs);
    if (!by_unit) ctas = quant_plan_ctas<is_multi(MODE), C::kST>(p, pfx);
    const GroupRange gr = cta_range<MODE>(p, pfx, nv_max, C::kST, ctas, &begin, &end);
    if (tid == 0 && !by_unit) group = gr;  // out of registers; the syncs of the first unit's q rows order it
    if (warp == C::kWarps) {
        run_producer<C, QuantLoader<D, NT>, D, MODE>(p, base_s, L, pfx, meta, &abort_flag, begin, end, lane);
        return;
    }
    run_quant_consumer<D, FMT, NT, MODE, FINE>(p, base_s, base, L, meta, pfx, &abort_flag, &group, &notes, warp, lane);
}

template <int D, int FMT, int NT, int MODE, bool FINE>
cudaError_t launch_quant_as(const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    using C = QuantCfg<D, NT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(p.prefetch ? C::kThreads : C::kMainThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quant_split_kernel<D, FMT, NT, MODE, FINE>, p);
}

// visit(instance) of the form, or `none` where it does not exist: one tile of
// q rows has a form for single queries, head size 256 no second tile.
template <int FMT, int NT, int MODE, bool FINE>
struct QuantInstance {
    static constexpr int fmt = FMT, nt = NT, mode = MODE;
    static constexpr bool fine = FINE;
};
template <int D, int FMT, bool FINE, class R, class Visit>
R visit_quant_tiles(const QuantForm& form, R none, const Visit& visit) {
    if (form.n_tiles == 1)
        return form.multi ? visit(QuantInstance<FMT, 1, kMulti, FINE>()) : visit(QuantInstance<FMT, 1, kOneShot, FINE>());
    if constexpr (D <= 128)
        if (form.n_tiles == 2) return visit(QuantInstance<FMT, 2, kMulti, FINE>());
    return none;
}
template <int D, class R, class Visit>
R visit_quant(const QuantForm& form, R none, const Visit& visit) {
    if (form.format == kE4m3)
        return form.fine ? visit_quant_tiles<D, kE4m3, true>(form, none, visit)
                         : visit_quant_tiles<D, kE4m3, false>(form, none, visit);
    return form.fine ? visit_quant_tiles<D, kInt8, true>(form, none, visit)
                     : visit_quant_tiles<D, kInt8, false>(form, none, visit);
}

template <int D>
const void* quant_fn(const QuantForm& form) {
    return visit_quant<D>(form, (const void*)nullptr, [](auto i) {
        using I = decltype(i);
        return reinterpret_cast<const void*>(&quant_split_kernel<D, I::fmt, I::nt, I::mode, I::fine>);
    });
}

template <int D>
cudaError_t launch_quant_of(const QuantForm& form, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return visit_quant<D>(form, cudaErrorInvalidValue, [&](auto i) {
        using I = decltype(i);
        return launch_quant_as<D, I::fmt, I::nt, I::mode, I::fine>(p, grid, smem, stream);
    });
}

}  // namespace pda
