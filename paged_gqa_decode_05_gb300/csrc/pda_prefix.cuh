// pda_prefix.cuh -- attention of a group of sequences over the prefix they
// share, on the tcgen05 tensor cores.
//
// The q rows of a group and kv head (its sequences x queries x G heads) meet
// every token of the prefix, so they are tiles of 128 rows of a matrix product:
//   S = Q K^T   (M = 128 q rows, N = a tile of kT tokens; Q and K in shared
//                memory, S in tensor memory)
//   softmax     (a thread per q row, 128 lanes of tensor memory: no shuffles;
//                it reads its row of S and writes P over it, as bf16 high and
//                low parts, p = hi + lo to 2^-17)
//   O += P V    (P as the A operand in tensor memory, V as an MN-major B)
// and the result is an online-softmax state (m, l, o) per row, which join_kernel
// (pda_weights.cu) joins with those of the sequences' own tokens.
//
// Work: units (pair of q tiles, kv head) of one position per token tile, cut
// evenly over one CTA per SM.  Each CTA runs two streams of four softmax warps
// with two S and an O each.  A unit of two q tiles gives each stream one, so
// that a tile of K and V serves 256 q rows; a unit of one q tile gives the
// streams alternate token tiles, and their states join at the segment's end.
// A stream's next S is there when it has written a P.  Head size 256, whose O
// takes half the tensor memory, runs one stream.
//
// K and V go through rings of slots (PrefixRing), in the order in which the
// products use them (K runs two tiles before V), so that every slot but those in
// use is one on its way.  Four loader warps, two for K and two for V, fill 32 rows of a
// slot each, with TMA boxes of up to 32 rows and one 64-column slab, or, for
// block sizes below 8, row by row with 16-byte cp.async in the same swizzle.
// (Row by row for all, a call over 32768 tokens of 8 kv heads of 128 took 101 us
// for 79: a slot's copies kept a warp 1900 cycles.)  Rows behind the prefix's end
// and of bad block ids are zero-filled, by coordinates outside the pool where
// boxes load.  The codes of 8-bit caches land in the warp's own part of their
// slot, which spreads them to bf16 there; bf16 holds them exactly (4 and 8
// significant bits).  K scales multiply the scores, V scales the weights; weights
// are taken 2^-40 times, as they reach 2^8 (the reference lags), scales 2^122 and
// codes 448, and the sum over any number of tokens stays inside fp32.
//
// Bounds.  One q tile in bf16: memory; 32768 tokens of 8 kv heads of 128 (134 MB,
// 19.8 us at the measured copy rate) take 20 us of token tiles, with 3 before the
// first and 2 behind the last.  Two q tiles in 8 bits: the softmax; 16384 tokens of
// 8 kv heads and 512 rows take 74 us (26 at the products' rate), 28 tiles of 64 tokens
// a stream, each of 2300 cycles to the maximum (capped), 1450 for the weights and 500 of
// waits.  No pipe is full (fp32 35 %, exponentials 26 %, tensor 33 %, issue slots 53 %): a
// scheduler's two softmax warps have 0.9 ready between them.  Sixteen softmax warps
// instead of eight: 155 us a call for 124; P's parts 16 tokens wide instead of 32: no
// faster; all of a row unrolled: slower, its code no longer stays in the instruction
// caches.
#pragma once

#include <cuda_fp16.h>

#include "pda_kernels.cuh"
#include "pda_prefix.h"
#include "pda_ring.h"

namespace pda {

constexpr int kPlanHere = 16;  // groups whose plan is kept in shared memory
constexpr uint64_t kDrainLimitNs = 10000000ull;  // a copy lands in microseconds; a phase since reused does not show

template <int D, int FMT>
struct PrefixCfg {
    static constexpr int kT = kPrefixTile;               // tokens of a tile
    static constexpr int kStreams = prefix_streams(D);
    static constexpr int kSoftWarps = 4 * kStreams, kLoadWarps = 4;
    static constexpr int kThreads = (kSoftWarps + kLoadWarps + kStreams) * 32;  // + a warp a stream that issues products
    static constexpr int kSlotBytes = kT * D * 2;        // K or V of a tile
    static constexpr int kQTileBytes = 128 * D * 2;
    static constexpr int kSlots = D == 64 ? 20 : D == 256 ? (FMT == kBf16 ? 5 : 4) : FMT == kBf16 ? 10 : 9;
    // ring of scales, [K | V][kT] a tile: from when K's slot is filled until the
    // softmax, 4 + kSlots / 2 tiles at most
    static constexpr int kRing = 16, kScaleTiles = FMT == kBf16 ? 0 : kRing;
    static constexpr int kRW = kT / 2;                   // rows of a loader warp
    // tensor memory: two S of a stream, then its O
    static constexpr uint32_t kTmO = 256;
    static_assert(kStreams * 2 * kT <= 256 && kStreams * D <= 256, "tensor memory columns");
    static_assert(kScaleTiles == 0 || kScaleTiles > 4 + kSlots / 2, "scales of the tiles under way");
    // shared memory after the 1024-byte aligned base
    static constexpr uint32_t kSlot0 = kStreams * kQTileBytes;
    static constexpr uint32_t kScale0 = kSlot0 + kSlots * kSlotBytes;
    static constexpr uint32_t kBars = kScale0 + kScaleTiles * kT * 8;
    // full, empty [kSlots], landed [kSlots][half of the rows] (8-bit), S and P
    // [stream][2], P V [stream], then the rest
    static constexpr uint32_t kFull = kBars, kEmpty = kFull + 8 * kSlots, kLanded = kEmpty + 8 * kSlots;
    static constexpr uint32_t kS = kLanded + 8 * kSlots * (FMT == kBf16 ? 0 : 2), kP = kS + 32, kPV = kP + 32,
                              kO = kPV + 16, kQ = kO + 8, kSync = kQ + 8, kFin = kSync + 8, kTm = kFin + 8, kEnd = kTm + 16;
    static constexpr uint32_t kSmem = kEnd + (1024 - 16);  // (dynamic shared memory starts on 16 bytes)
    static_assert(kSmem + (kPlanHere + 1) * sizeof(PrefixGroup) + 16 <= 232448, "shared memory of an SM");
};

// One run of a CTA over token tiles of a unit.
struct PrefixSegment {
    int start, end;   // the group's first sequence, the one behind its last
    int rows;         // its q rows of a kv head
    int tokens;       // of the prefix
    int kvh, pair;
    int j0, n;        // token tiles j0 .. j0 + n - 1
    int64_t slot;     // of its state
    bool dual;        // two q tiles
};

template <int D, int FMT>
struct PrefixWalk {
    using C = PrefixCfg<D, FMT>;
    int64_t pos, end;
    __device__ __forceinline__ PrefixWalk(const PrefixParams& p, const PrefixGroup* groups) {
        const int64_t W = groups[p.n_groups].work, P = prefix_ctas(W, groups[p.n_groups].unit, gridDim.x), c = blockIdx.x;
        pos = c < P ? cta_begin(c, W, P) : 0;
        end = c < P ? cta_begin(c + 1, W, P) : 0;
    }
    __device__ __forceinline__ bool next(const PrefixParams& p, const PrefixGroup* groups, PrefixSegment& s) {
        if (pos >= end) return false;
        int lo = 0, hi = p.n_groups - 1;  // the last group that starts at or before pos (groups without work precede)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (groups[mid].work <= pos) lo = mid; else hi = mid - 1;
        }
        const PrefixGroup g = groups[lo];
        const int rem = (int)pos - g.work, unit = rem / g.tiles;
        s.start = g.start;
        s.end = groups[lo + 1].start;
        s.rows = (s.end - g.start) * p.q_len * p.G;
        s.tokens = g.blocks << p.lbs;
        s.pair = unit / p.Hkv;
        s.kvh = unit - s.pair * p.Hkv;
        s.j0 = rem - unit * g.tiles;
        s.n = min(g.tiles - s.j0, (int)(end - pos));
        s.slot = (int64_t)g.unit + unit + blockIdx.x;
        s.dual = C::kStreams == 2 && s.rows > (2 * s.pair + 1) * 128;
        pos += s.n;
        return true;
    }
};

// The plan of the groups.  Every CTA makes all of it, in shared memory or, where
// there are more than kPlanHere groups, in the call's scratch: the same values,
// so that each reads its own stores.  Run by one warp.
template <int D, int FMT>
__device__ __forceinline__ void prefix_plan(const PrefixParams& p, PrefixGroup* groups, int lane) {
    using C = PrefixCfg<D, FMT>;
    // a group's entries, loaded together; the first 32 groups' once
    struct Entry { int32_t start, end, blocks; };
    auto entry = [&](int g) {
        Entry e = {};
        if (g <= p.n_groups) e.start = e.end = group_start(p.starts, g, p.n_groups, p.B);
        if (g < p.n_groups) {
            e.end = group_start(p.starts, g + 1, p.n_groups, p.B);
            e.blocks = p.shared[g];
        }
        return e;
    };
    auto wrong = [&](const Entry& e) {  // (bad_group)
        return e.start < 0 || e.start > p.B || e.end < e.start || e.blocks < 0 || e.blocks > p.table_stride;
    };
    const Entry mine = entry(lane);
    bool bad = wrong(mine);
    for (int g = lane + 32; g <= p.n_groups; g += 32) bad |= wrong(entry(g));
    const bool none = __any_sync(0xffffffffu, bad);  // (the decode of the own tokens has raised the flag)
    int32_t units = 0, work = 0;  // of the groups before
    for (int g0 = 0; g0 <= p.n_groups; g0 += 32) {
        const int g = g0 + lane;
        PrefixGroup out = {};
        if (!none) {
            const Entry e = g0 == 0 ? mine : entry(g);
            out.start = e.start;
            out.blocks = e.blocks;
            out.pairs = ((e.end - e.start) * p.q_len * p.G + 128 * C::kStreams - 1) / (128 * C::kStreams);
            // (a prefix of 2^31 tokens and more is longer than any sequence: nobody shares it)
            const int64_t tokens = (int64_t)out.blocks << p.lbs;
            out.tiles = out.pairs > 0 && tokens <= INT32_MAX ? (int32_t)((tokens + C::kT - 1) / C::kT) : 0;
        }
        const int32_t u = out.tiles > 0 ? out.pairs * p.Hkv : 0, w = u * out.tiles;
        int32_t us = u, wsum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t a = __shfl_up_sync(0xffffffffu, us, o), b = __shfl_up_sync(0xffffffffu, wsum, o);
            if (lane >= o) { us += a; wsum += b; }
        }
        out.unit = units + us - u;
        out.work = work + wsum - w;
        if (g <= p.n_groups) groups[g] = out;
        units += __shfl_sync(0xffffffffu, us, 31);
        work += __shfl_sync(0xffffffffu, wsum, 31);
    }
}

// 16 bytes, or 16 zero bytes where !use.
__device__ __forceinline__ void cp_async_16_or_0(uint32_t dst, const void* src, bool use) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(use ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_4_or_0(uint32_t dst, const void* src, bool use) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(use ? 4 : 0) : "memory");
}

// Four codes as bf16, which holds them exactly.
template <int FMT>
__device__ __forceinline__ void codes_to_bf16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    uint32_t a, b;
    if constexpr (FMT == kE4m3) {
        a = e4m3x2_to_f16x2((uint16_t)x);
        b = e4m3x2_to_f16x2((uint16_t)(x >> 16));
    } else {
        // the byte under 0x64 reads as 1024 + code + 128
        const uint32_t u = x ^ 0x80808080u, c = 0x64806480u;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(c));
        asm("sub.f16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(c));
    }
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    lo = pack_bf16x2(fa.x, fa.y);
    hi = pack_bf16x2(fb.x, fb.y);
}

// A bounded wait whose outcome the warp shares.
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity) ? 1 : 0)) return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimitNs) ? 1 : 0) != 0;
}

// ------------------------------------------------------------------ loaders

// The first of the sequences start + 1 .. end - 1 that shares a prefix of `tokens`, or
// -1, by one warp, 32 at a time.  (A call, as few segments need it.)
static __device__ __noinline__ int32_t later_lead(const int32_t* lens, int32_t start, int32_t end, int32_t q_len, int64_t tokens) {
    const int lane = threadIdx.x & 31;
    for (int32_t b0 = start + 1; b0 < end; b0 += 32) {
        const uint32_t found = __ballot_sync(0xffffffffu, b0 + lane < end && sees_prefix(lens[min(b0 + lane, end - 1)], q_len, tokens));
        if (found) return b0 + __ffs((int)found) - 1;
    }
    return -1;
}

// Loader warp w fills 32 rows (half w & 1) of the slots of K (w < 2) or of V.
template <int D, int FMT>
__device__ __forceinline__ void prefix_load(const PrefixParams& p, const PrefixGroup* groups, uint32_t base, uint8_t* smem,
                                            volatile int* abort_flag, int w, int lane, uint32_t& filled, uint32_t& parities) {
    using C = PrefixCfg<D, FMT>;
    constexpr int RW = C::kRW, ES = FMT == kBf16 ? 2 : 1;  // rows of this warp; bytes of an element
    constexpr int CH = D * ES / 16, RPI = 32 / CH;         // 16-byte chunks of a row; rows of an instruction
    constexpr int RC = D < 128 ? D : 128;                  // codes of a row in one piece (8-bit)
    static_assert(RW == 32 && RPI >= 1, "a lane a row");
    const bool k = w < 2;
    const int half = w & 1, row0 = half * RW;
    const uint8_t* pool = k ? p.k_base : p.v_base;
    const CUtensorMap* map = k ? &p.tm_k : &p.tm_v;
    const uint64_t once = policy_evict_first(), keep = policy_evict_normal();  // rows that one unit reads, or several
    const int chunk = lane % CH, sub = lane / CH;
    const int bs = 1 << p.lbs, rb = min(bs, RW);  // rows of a block, of a box
    // The tile to fill and, looked up a tile ahead, the block id of this lane's
    // row of it as read (checked when it is used, so that nothing waits for it).
    constexpr int32_t kNoRow = INT32_MIN;
    PrefixWalk<D, FMT> walk(p, groups);
    PrefixSegment s = {}, s2 = {};
    bool more = walk.next(p, groups, s), more2 = more && walk.next(p, groups, s2);
    int32_t id_next = kNoRow;
    // The row of the table that holds a segment's blocks: the first one of its group
    // whose sequence shares the prefix (the others' rows are their own, and what lies
    // behind their lengths is not read); -1: none, nobody looks at the tiles.
    int32_t lead = -1;
    auto look_up = [&](const PrefixSegment& at, int tile) {
        const int64_t t = (int64_t)tile * C::kT + row0 + lane;
        id_next = t < at.tokens && lead >= 0 ? p.table[(int64_t)lead * p.table_stride + (t >> p.lbs)] : kNoRow;
    };
    // (nearly always the group's first: its ids are on their way beside its length.
    // In the plan instead, which every warp waits for, two groups of eight sequences
    // behind 1000 tokens take 16.0 us for 15.6.)
    auto first_look = [&](const PrefixSegment& at) {
        lead = at.start;
        look_up(at, at.j0);
        if (!sees_prefix(p.lens[at.start], p.q_len, at.tokens)) {
            lead = later_lead(p.lens, at.start, at.end, p.q_len, at.tokens);
            look_up(at, at.j0);
        }
    };
    if (more) first_look(s);
    // (8-bit) codes in their slot: up to 128 of a row at a time over the warp's part of a slab each
    auto code_at = [&](uint32_t slot, int r, int c) {
        return slot + (uint32_t)(c / RC) * (C::kT * 128) + (uint32_t)(row0 * 128 + r * RC + c % RC);
    };
    auto convert = [&](uint32_t slot) {
        if constexpr (FMT != kBf16) {
            constexpr int N = RW * D / 16 / 32;  // 16-code chunks of a lane
            uint32_t x[N][4];
#pragma unroll
            for (int i = 0; i < N; ++i) lds_v4(code_at(slot, (lane + 32 * i) / CH, (lane + 32 * i) % CH * 16), x[i]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = lane + 32 * i, t = row0 + at / CH, c = 2 * (at % CH);  // row, first 8-column chunk
                const uint32_t row = slot + (uint32_t)(c >> 3) * (C::kT * 128) + (uint32_t)t * 128;
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) codes_to_bf16<FMT>(x[i][e], y[2 * e], y[2 * e + 1]);
                sts_v4(row + (uint32_t)(((c & 7) ^ (t & 7)) << 4), y[0], y[1], y[2], y[3]);
                sts_v4(row + (uint32_t)((((c & 7) + 1) ^ (t & 7)) << 4), y[4], y[5], y[6], y[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (lane_wait(bar, parity)) return true;
        atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
        *abort_flag = 1;
        return false;
    };
    PrefixRing<C::kSlots, C::kStreams == 2> ring;
    uint32_t tiles = 0, segs = 0;   // tiles that are filled; segments before
    uint32_t issued = 0, spread = 0, queue = 0;  // (8-bit) slots filled, converted; lane l & 31: the l-th one's 2 slot + phase
    int i = 0;                      // tile of the segment
    bool ok = true;
    while (ok && (more || spread != issued)) {
        const bool shared = s.dual || C::kStreams == 1;  // by both streams
        const int st = shared ? 0 : i & 1, own = shared ? i : i >> 1, items = shared ? s.n : (s.n - st + 1) / 2;
        uint32_t phase;
        const uint32_t at = ring.slot(shared, st, k ? ring.k_use(own) : ring.v_use(own, items), phase);
        const uint32_t slot = base + C::kSlot0 + at * C::kSlotBytes, empty = base + C::kEmpty + 8 * at, parity = phase ^ 1u;
        bool can = more;
        if (can && i == 0 && segs > 0) {  // a segment's first, once every product of the one before is done
            if (FMT != kBf16 && spread != issued) can = __all_sync(0xffffffffu, mbar_test_wait(base + C::kO, (segs - 1) & 1u));
            else if (!(ok = wait(base + C::kO, (segs - 1) & 1u))) break;
        }
        if (FMT != kBf16 && can && spread != issued) can = __all_sync(0xffffffffu, mbar_test_wait(empty, parity));
        if (can) {
            if (!(ok = wait(empty, parity))) break;
            const int tile = s.j0 + i;
            int32_t id = id_next;
            if (i + 1 < s.n) look_up(s, tile + 1);
            else if (more2) first_look(s2);
            if (id < 0 || (int64_t)id >= p.num_blocks) {
                if (id != kNoRow) atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
                id = -1;  // zeros
            }
            const uint32_t bar = FMT == kBf16 ? base + C::kFull + 8 * at : base + C::kLanded + 8 * (2 * at + half);
            const uint32_t to = base + C::kScale0 + (FMT == kBf16 ? 0 : tiles % C::kRing) * (C::kT * 8) + (uint32_t)row0 * 4;
            if (p.boxes) {
                // lane b * pieces + h: box b, piece h of its columns
                constexpr int kPieces = FMT == kBf16 ? D / 64 : D / RC;
                const int b = lane / kPieces, h = lane % kPieces, r = min(b * rb, RW - 1);
                const bool box = b * rb < RW;
                const int32_t bid = __shfl_sync(0xffffffffu, id, r);
                const bool scaled = FMT != kBf16 && k && box && h == 0;
                uint32_t bytes = RW * D * ES;
                if constexpr (FMT != kBf16) bytes += __popc(__ballot_sync(0xffffffffu, scaled && bid >= 0)) * 2u * rb * 4u;
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (box) {
                    const int in = (row0 + r) & (bs - 1);  // the box's first row in its block (tiles hold whole blocks)
                    if (scaled) {
                        const float* sc = p.scales + (((((int64_t)bid * p.Hkv + s.kvh) * 2) << p.lbs) + in);
                        if (bid >= 0) {
                            bulk_load(to + 4 * r, sc, 4 * rb, bar);
                            bulk_load(to + C::kT * 4 + 4 * r, sc + bs, 4 * rb, bar);
                        } else {
                            for (int e = 0; e < rb; e += 4) {
                                sts_v4(to + 4 * (r + e), 0u, 0u, 0u, 0u);
                                sts_v4(to + C::kT * 4 + 4 * (r + e), 0u, 0u, 0u, 0u);
                            }
                        }
                    }
                    const uint32_t dst = FMT == kBf16 ? slot + (uint32_t)h * (C::kT * 128) + (uint32_t)(row0 + r) * 128
                                                      : code_at(slot, r, h * RC);
                    // (the id past the last one is outside the view: zeros)
                    tma_load_5d(dst, map, 0, in, h, s.kvh, bid < 0 ? (int32_t)p.num_blocks : bid, bar,
                                s.dual || s.pair > 0 ? keep : once);
                }
            } else {
                const int in = (row0 + lane) & (bs - 1);
                const int64_t off = id < 0 ? -1 : (int64_t)id * p.blk_s + (int64_t)in * p.tok_s + (int64_t)s.kvh * p.kvh_s;
                if (FMT != kBf16 && k) {
                    const float* sc = p.scales + (id < 0 ? 0 : ((((int64_t)id * p.Hkv + s.kvh) * 2) << p.lbs) + in);
                    cp_async_4_or_0(to + 4 * lane, sc, id >= 0);
                    cp_async_4_or_0(to + C::kT * 4 + 4 * lane, sc + (id < 0 ? 0 : bs), id >= 0);
                }
#pragma unroll 2
                for (int r0 = 0; r0 < RW; r0 += RPI) {
                    const int r = r0 + sub, t = row0 + r;
                    const int64_t o = __shfl_sync(0xffffffffu, off, r);
                    const uint32_t dst = FMT == kBf16 ? slot + (uint32_t)(chunk >> 3) * (C::kT * 128) + (uint32_t)t * 128 +
                                                            (uint32_t)(((chunk & 7) ^ (t & 7)) << 4)
                                                      : code_at(slot, r, chunk * 16);
                    cp_async_16_or_0(dst, pool + (o < 0 ? 0 : o * ES) + chunk * 16, o >= 0);
                }
                cp_async_mbar_arrive_noinc(bar);
            }
            ++tiles;
            filled |= 1u << at;
            parities = (parities & ~(1u << at)) | phase << at;
            if constexpr (FMT != kBf16) {
                if (lane == (int)(issued & 31u)) queue = 2 * at + phase;
                ++issued;
            }
            if (++i == s.n) {
                if (more2) ring.next(shared, s.n);
                ++segs;
                i = 0;
                s = s2;
                more = more2;
                more2 = more && walk.next(p, groups, s2);
            }
        } else if constexpr (FMT != kBf16) {
            const uint32_t m = __shfl_sync(0xffffffffu, queue, spread & 31u), c = m >> 1;
            if (!(ok = wait(base + C::kLanded + 8 * (2 * c + half), m & 1u))) break;
            if (k) {  // K's scales times what every score is multiplied by
                __syncwarp();  // (another lane's zeros, of a bad block id, among them)
                float* ks = reinterpret_cast<float*>(smem + C::kScale0) + spread % C::kRing * (2 * C::kT) + row0 + lane;
                *ks *= p.score_mult;
            }
            convert(base + C::kSlot0 + c * C::kSlotBytes);
            if (lane == 0) mbar_arrive(base + C::kFull + 8 * c);
            ++spread;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ products

// The products of stream st.  A warp each, so that one's waits pass under the
// other's products (one warp for both streams: a call over 32768 tokens of 8 kv
// heads of 128 and 128 q rows 70 us for 63).
template <int D, int FMT>
__device__ __forceinline__ void prefix_mma(const PrefixParams& p, const PrefixGroup* groups, uint32_t base,
                                           volatile int* abort_flag, uint32_t tmem, int st) {
    using C = PrefixCfg<D, FMT>;
    constexpr uint32_t idS = umma_idesc_bf16(128, C::kT, false), idO = umma_idesc_bf16(128, D, true);
    PrefixWalk<D, FMT> walk(p, groups);
    PrefixSegment s;
    PrefixRing<C::kSlots, C::kStreams == 2> ring;
    uint32_t segs = 0;
    bool every_before = false;
    int n_before = 0;
    uint32_t sn = 0, pn = 0;        // S and P V issued
    const bool one = elect_one();
    const uint32_t tS0 = tmem + st * 2 * C::kT, tO = tmem + C::kTmO + st * D;
    const uint32_t kS = base + C::kS + 16 * st, kP = base + C::kP + 16 * st;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (lane_wait(bar, parity)) return true;
        if (one) atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
        *abort_flag = 1;
        return ok = false;
    };
    while (ok && walk.next(p, groups, s)) {
        // item k of this stream: tile k (two q tiles, or one stream) or every other one
        const bool every = s.dual || C::kStreams == 1;
        const int items = every ? s.n : (s.n - st + 1) / 2;
        if (segs > 0) ring.next(every_before, n_before);
        const uint64_t q = umma_sdesc(base + (s.dual ? st : 0) * C::kQTileBytes, 16, 1024);
        if (!wait(base + C::kQ, segs & 1u)) break;
        ++segs;
        // S of item k comes before P V of item k - 1: two S ahead of their P V
#pragma unroll 1
        for (int k = -2; ok && k < items; ++k) {
            if (k >= 0) {
                uint32_t phase;
                const uint32_t slot = ring.slot(every, st, ring.v_use(k, items), phase), buf = pn & 1u;
                if (!wait(base + C::kFull + 8 * slot, phase)) break;
                if (!wait(kP + 8 * buf, (pn >> 1) & 1u)) break;
                fence_proxy_async_smem();  // cp.async writes of the loaders, and of the q rows
                tc_fence_after();
                const uint32_t tP = tS0 + buf * C::kT;
                const uint64_t v = umma_sdesc(base + C::kSlot0 + slot * C::kSlotBytes, C::kT * 128, 1024);
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < C::kT / 16; ++ks) {
                        const uint32_t part = tP + ks / 2 * 32 + ks % 2 * 8;
                        umma_bf16_ts(tO, part, v + 128 * ks, idO, ks > 0 || k > 0);  // 16 rows of 128 bytes
                        umma_bf16_ts(tO, part + 16, v + 128 * ks, idO, true);
                    }
                    umma_commit(base + C::kEmpty + 8 * slot);
                    if (C::kStreams == 2 && !s.dual) mbar_arrive(base + C::kEmpty + 8 * slot);  // for the other stream
                    umma_commit(base + C::kPV + 8 * st);
                    if (k == items - 1) umma_commit(base + C::kO);
                }
                __syncwarp();
                ++pn;
            }
            const int i = k + 2;
            if (i < items) {
                uint32_t phase;
                const uint32_t slot = ring.slot(every, st, ring.k_use(i), phase), buf = sn & 1u;
                if (!wait(base + C::kFull + 8 * slot, phase)) break;
                fence_proxy_async_smem();
                tc_fence_after();
                const uint32_t tS = tS0 + buf * C::kT;
                const uint64_t kk = umma_sdesc(base + C::kSlot0 + slot * C::kSlotBytes, 16, 1024);
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)  // 32 bytes a step, slabs of 128 and of kT rows
                        umma_bf16_ss(tS, q + (ks >> 2) * (128 * 8) + (ks & 3) * 2, kk + (ks >> 2) * (C::kT * 8) + (ks & 3) * 2,
                                     idS, ks > 0);
                    umma_commit(kS + 8 * buf);
                    umma_commit(base + C::kEmpty + 8 * slot);
                    if (C::kStreams == 2 && !s.dual) mbar_arrive(base + C::kEmpty + 8 * slot);
                }
                __syncwarp();
                ++sn;
            }
        }
        if (one && ok && items == 0) mbar_arrive(base + C::kO);
        every_before = every;
        n_before = s.n;
    }
    // every product has completed before the tensor memory is freed
    if (one) umma_commit(base + C::kFin);
    __syncwarp();
    if (!lane_wait(base + C::kFin, 0) && one) atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
}

// ------------------------------------------------------------------ softmax

// 2 N columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_row(uint32_t taddr, float2 (&v)[N]) {
#pragma unroll
    for (int c = 0; c < 2 * N; c += 16) {
        uint32_t* r = reinterpret_cast<uint32_t*>(v) + c;
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + c)
            : "memory");
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // (no use of the loaded registers moves ahead of the wait)
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i].x), "+f"(v[i].y));
}

// A tile under a wide cap, in place: this thread's row at `t` becomes what times its
// multiplier (the score scale, 8-bit: with the K scale) is the capped score, so that
// the passes below know nothing of it (two roundings more).  A call where no part of
// the row is in registers, four columns at a time, so that its code is small: with the
// series beside the other cap's code 64 sequences behind 16384 tokens in e4m3, at a cap
// of 50, took 126.8 us for 117.8 without it; so 119.8.
template <int FMT>
__device__ __noinline__ void prefix_wide_cap(uint32_t t, const float* kscale, float mult, float cap) {
    const float unit = cap * 0.34657359f;  // ln 2 / 2: z back to the score
#pragma unroll 1
    for (int c = 0; c < kPrefixTile; c += 4) {
        float x[4];
        uint32_t* r = reinterpret_cast<uint32_t*>(x);
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(t + c) : "memory");
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm volatile("" : "+f"(x[i]));  // (not used ahead of the wait)
            const float f = FMT == kBf16 ? mult : kscale[c + i], z = x[i] * f;
            x[i] = f == 0.f ? z : capped_wide(cap, z * unit, z) / f;
        }
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                     ::"r"(t + c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    }
    tmem_wait_st();
}

template <int D, int FMT>
__device__ __forceinline__ void prefix_softmax(const PrefixParams& p, const PrefixGroup* groups, uint32_t base, uint8_t* smem, volatile int* abort_flag,
                                               uint32_t tmem, int warp, int lane) {
    using C = PrefixCfg<D, FMT>;
    constexpr int kT = C::kT, kPart = 32;
    constexpr float kDown = FMT == kBf16 ? 0.f : 40.f, kBack = FMT == kBf16 ? 1.f : 1.0995116e12f;  // 2^40
    const int st = warp >> 2, w = warp & 3, row = 32 * w + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * w) << 16);
    float* ml = reinterpret_cast<float*>(smem);  // [stream][2][128], over the q rows once they are used
    PrefixWalk<D, FMT> walk(p, groups);
    PrefixSegment s;
    const bool plain = p.cap == 0.f && p.slopes == nullptr;
    uint32_t tile0 = 0, segs = 0, done = 0, cphase = 0;  // done: items of this stream
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (lane_wait(bar, parity)) return true;
        atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
        *abort_flag = 1;
        return false;
    };
    auto sync_all = [&]() {
        const bool ok = consumer_sync(base + C::kSync, cphase, p.err, abort_flag);
        return __all_sync(0xffffffffu, ok ? 1 : 0) != 0;
    };
    while (walk.next(p, groups, s)) {
        const int tile = s.pair * C::kStreams + (s.dual ? st : 0);
        // the segment's q rows, in the swizzle of the products' operand: a
        // stream its own tile, or both streams one
        {
            const int threads = s.dual ? 128 : 128 * C::kStreams, t0 = s.dual ? row : warp * 32 + lane;
            const uint32_t sQ = base + (s.dual ? st : 0) * C::kQTileBytes;
            const int g0 = tile * 128, bq0 = g0 / p.G, h0 = g0 - bq0 * p.G;
            const uint32_t over = 65536u / p.G + 1;  // x / G = x * over >> 16 for x < 136
            const uint16_t* q0 = p.q + (((int64_t)s.start * p.q_len + bq0) * p.Hq + s.kvh * p.G) * D;
#pragma unroll 1
            for (int i = t0; i < 128 * (D / 8); i += threads) {
                const int r = i / (D / 8), c = i % (D / 8);
                const int x = h0 + r, bq = (int)((uint32_t)x * over >> 16), h = x - bq * p.G;
                const bool use = g0 + r < s.rows;
                cp_async_16_or_0(sQ + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                                 use ? q0 + (int64_t)bq * p.Hq * D + h * D + c * 8 : p.q, use);
            }
            cp_async_mbar_arrive_noinc(base + C::kQ);
        }
        // this thread's q row: whether its sequence shares the prefix (else the decode of the
        // own tokens takes it), and its bias
        const int g = tile * 128 + row;
        int vis = 0, own = 0;
        float slope = 0.f;
        if (g < s.rows) {
            const int bq = g / p.G, h = g - bq * p.G, b = bq / p.q_len, qi = bq - b * p.q_len;
            const int32_t len = p.lens[s.start + b];
            own = max(len, 0) - p.q_len + qi;
            vis = sees_prefix(len, p.q_len, s.tokens) ? s.tokens : 0;
            if (p.slopes) slope = p.slopes[s.kvh * p.G + h] * 1.4426950408889634f;
        }
        const bool idle = tile * 128 + 32 * w >= s.rows;  // a warp without rows
        const int items = s.dual ? 2 * s.n : s.n;
        float m = kNegInf, l = 0.f;
        for (int k = st; k < items; k += C::kStreams) {
            const int jj = s.dual ? k >> 1 : k;
            const uint32_t buf = done & 1u, tS = tl + st * 2 * kT + buf * kT;
            if (!wait(base + C::kS + 16 * st + 8 * buf, (done >> 1) & 1u)) return;
            tc_fence_after();
            if (!idle) {
                const int t0 = (s.j0 + jj) * kT, seen = vis - t0;  // the tile's first token; tokens of it in sight
                // scores in base-2 units, a part of the row at a time (unrolled, the loop
                // would not stay in the instruction caches beside the other warps'); what
                // is more than a product goes back to tensor memory for the second pass
                const bool cut = __any_sync(0xffffffffu, seen < kT), bare = FMT == kBf16 && plain && !cut;
                const float* kscale = reinterpret_cast<const float*>(smem + C::kScale0) +
                                      (FMT == kBf16 ? 0 : (tile0 + jj) % C::kRing * (2 * kT));
                const float f = bare ? p.score_mult : 1.f;
                if (p.wide_cap != 0.f) prefix_wide_cap<FMT>(tS, kscale, p.score_mult, p.wide_cap);
                float top = kNegInf;
#pragma unroll 1
                for (int c = 0; c < kT; c += kPart) {
                    float2 v[kPart / 2];
                    tmem_ld_row(tS + c, v);
                    float two[2] = {kNegInf, kNegInf};
                    if (!bare) {
                        // times the score scale (8-bit: and the K scale), under a cap over half of it
#pragma unroll
                        for (int i = 0; i < kPart / 2; i += 2) {
                            float4 x = make_float4(p.score_mult, p.score_mult, p.score_mult, p.score_mult);
                            if constexpr (FMT != kBf16) x = *reinterpret_cast<const float4*>(kscale + c + 2 * i);
                            v[i] = __fmul2_rn(v[i], make_float2(x.x, x.y));
                            v[i + 1] = __fmul2_rn(v[i + 1], make_float2(x.z, x.w));
                        }
                        if (p.cap != 0.f) {
                            // (see capped; four scores share a reciprocal, which takes twice an
                            // exponential's time: at 2^30 and above tanh is 1, and four fit fp32)
                            float high = kNegInf;
#pragma unroll
                            for (int i = 0; i < kPart / 2; ++i) high = fmaxf(high, fmaxf(v[i].x, v[i].y));
                            if (__any_sync(0xffffffffu, high > 30.f)) {
#pragma unroll
                                for (int i = 0; i < kPart / 2; ++i) v[i] = make_float2(min_nan(v[i].x, 30.f), min_nan(v[i].y, 30.f));
                            }
                            const float2 one = make_float2(1.f, 1.f), c0 = make_float2(p.cap, p.cap),
                                         c2 = make_float2(-2.f * p.cap, -2.f * p.cap);
#pragma unroll
                            for (int i = 0; i < kPart / 2; i += 2) {
                                const float2 a = __fadd2_rn(make_float2(ex2(v[i].x), ex2(v[i].y)), one);
                                const float2 b = __fadd2_rn(make_float2(ex2(v[i + 1].x), ex2(v[i + 1].y)), one);
                                const float2 ab = __fmul2_rn(a, b);
                                const float x = rcp_approx(ab.x * ab.y);
                                const float2 q = __fmul2_rn(make_float2(ab.y, ab.x), make_float2(x, x));  // 1 / ab
                                v[i] = __ffma2_rn(__fmul2_rn(q, b), c2, c0);
                                v[i + 1] = __ffma2_rn(__fmul2_rn(q, a), c2, c0);
                            }
                            if (!p.slopes && !cut)  // (the cap does not decrease)
                                two[0] = fmaf(-2.f * p.cap, rcp_approx(1.f + ex2(fminf(high, 30.f))), p.cap);
                        }
                        if (p.slopes) {
                            const float far = (float)(t0 + c - own);
#pragma unroll
                            for (int i = 0; i < kPart / 2; ++i)
                                v[i] = __ffma2_rn(make_float2(slope, slope), make_float2(far + (float)(2 * i), far + (float)(2 * i + 1)), v[i]);
                        }
                        if (cut) {
#pragma unroll
                            for (int i = 0; i < kPart / 2; ++i) {
                                if (2 * i >= seen - c) v[i].x = kNegInf;
                                if (2 * i + 1 >= seen - c) v[i].y = kNegInf;
                            }
                        }
                        const float* x = reinterpret_cast<const float*>(v);
#pragma unroll
                        for (int i = 0; i < kPart; i += 16) tmem_st16(tS + c + i, *reinterpret_cast<const float(*)[16]>(x + i));
                    } else {
#pragma unroll
                        for (int i = 0; i < kPart / 2; ++i) v[i] = __fmul2_rn(v[i], make_float2(f, f));
                    }
                    if (p.cap == 0.f || p.slopes || cut) {  // (else the cap's largest is known)
#pragma unroll
                        for (int i = 0; i < kPart / 2; ++i) {
                            two[0] = fmaxf(two[0], v[i].x);
                            two[1] = fmaxf(two[1], v[i].y);
                        }
                    }
                    top = fmaxf(top, fmaxf(two[0], two[1]));
                }
                if (!bare) tmem_wait_st();
                // lazy reference (kLazyLog2); O is scaled once this stream's last product with V is done
                const bool up = top > m + kLazyLog2, scale_o = up && m != kNegInf;
                // (waited for every time, long over as a rule: a parity tells a phase from the one
                // before only to who has seen that)
                if (done > 0 && !wait(base + C::kPV + 8 * st, (done - 1u) & 1u)) return;
                if (__any_sync(0xffffffffu, scale_o)) {
                    tc_fence_after();
                    const float a = scale_o ? ex2(m - top) : 1.f;
                    l *= a;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(tl + C::kTmO + st * D + c, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= a;
                        tmem_st16(tl + C::kTmO + st * D + c, o);
                    }
                }
                if (up) m = top;
                const float u = (m == kNegInf ? 0.f : m) + kDown;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int c = 0; c < kT; c += kPart) {  // P over its part of S: high parts, then low parts
                    float2 v[kPart / 2];
                    uint32_t hi[kPart / 2], lo[kPart / 2];
                    tmem_ld_row(tS + c, v);
#pragma unroll
                    for (int i = 0; i < kPart / 2; ++i) {
                        const float2 x = __ffma2_rn(v[i], make_float2(f, f), make_float2(-u, -u));
                        float2 e = make_float2(ex2(x.x), ex2(x.y));
                        sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                        if constexpr (FMT != kBf16) e = __fmul2_rn(e, *reinterpret_cast<const float2*>(kscale + kT + c + 2 * i));
                        hi[i] = pack_bf16x2(e.x, e.y);
                        const float2 r = __ffma2_rn(make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])), make_float2(-1.f, -1.f), e);
                        lo[i] = pack_bf16x2(r.x, r.y);
                    }
                    tmem_st16u(tS + c, hi);
                    tmem_st16u(tS + c + kPart / 2, lo);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
            }
            ++done;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + C::kP + 16 * st + 8 * buf);
        }
        // ---- the segment's end: every product of it is done
        if (!wait(base + C::kO, segs & 1u)) return;
        ++segs;
        tile0 += s.n;
        tc_fence_after();
        m = seen_reference(m, l);
        const bool joined = C::kStreams == 2 && !s.dual;
        float f0 = 1.f, f1 = 0.f;
        bool two = false;
        if (joined) {  // the streams' states of the same rows
            ml[st * 256 + row] = m;
            ml[st * 256 + 128 + row] = l;
            if (!sync_all()) return;
            two = items > 1;
            const float m0 = ml[row], m1 = two ? ml[256 + row] : kNegInf;
            m = fmaxf(m0, m1);
            f0 = m0 == kNegInf ? 0.f : ex2(m0 - m);
            f1 = m1 == kNegInf ? 0.f : ex2(m1 - m);
            l = ml[128 + row] * f0 + (two ? ml[256 + 128 + row] * f1 : 0.f);
        }
        // Slabs of 64 columns (32 at head size 64) go out through the q rows' memory,
        // a stream's own tile of it, as bulk copies: [slab][row][columns], the 16-byte
        // pieces of a row XORed with its index (8 rows in a column would meet on
        // four banks; written from registers a lane its row, a store's 32 rows are 32
        // sectors).
        constexpr int kCols = prefix_slab(D), kRowBytes = kCols * 4;
        static_assert(128 * kRowBytes <= C::kQTileBytes, "a slab fits a q tile");
        const int64_t at = s.slot * C::kStreams + (s.dual ? st : 0);
        const uint32_t stage = base + st * C::kQTileBytes;
        if (joined && !sync_all()) return;  // (the states just read lie there)
#pragma unroll 1
        for (int slab = idle ? D / kCols : joined ? st : 0; slab < D / kCols; slab += joined ? 2 : 1) {
            if (!joined && slab > 0) {  // the warp's copy before has read its rows' memory
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            }
#pragma unroll 1
            for (int c = 0; c < kCols; c += 16) {
                float o[16], x[16];
                tmem_ld16(tl + C::kTmO + (joined ? 0 : st * D) + slab * kCols + c, o);
                if (two) tmem_ld16(tl + C::kTmO + D + slab * kCols + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i] = (o[i] * f0 + (two ? x[i] * f1 : 0.f)) * kBack;
                    if (m == kNegInf) o[i] = 0.f;  // a row that sees none of these tokens
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    sts_v4(stage + row * kRowBytes + ((((c + i) >> 2) ^ (row & 7)) << 4), __float_as_uint(o[i]), __float_as_uint(o[i + 1]),
                           __float_as_uint(o[i + 2]), __float_as_uint(o[i + 3]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)  // this warp's 32 rows
                bulk_store(p.part_o + ((at * (D / kCols) + slab) * 128 + 32 * w) * kCols, stage + w * 32 * kRowBytes, 32 * kRowBytes);
        }
        if (g < s.rows && (!joined || st == 0))
            reinterpret_cast<float2*>(p.part_ml)[at * 128 + row] = make_float2(m, l * kBack);
        if (lane == 0) bulk_wait_read();  // before the next segment's q rows
        __syncwarp();
        tc_fence_before();
        if (!sync_all()) return;  // both streams have read both states
    }
}

__device__ __forceinline__ PrefixSeq prefix_seq(const PrefixParams& p, const PrefixGroup* groups, int b) {
    int lo = 0, hi = p.n_groups;  // the first entry that starts past b
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (groups[mid].start <= b) lo = mid + 1; else hi = mid;
    }
    PrefixSeq s = {};
    if (lo > 0 && b < groups[p.n_groups].start) {
        const PrefixGroup g = groups[lo - 1];
        const PrefixGroup all = groups[p.n_groups];
        s = {g.start, g.blocks, g.tiles, g.unit, g.work, all.work, (int32_t)prefix_ctas(all.work, all.unit, gridDim.x), 0};
    }
    return s;
}

template <int D, int FMT>
__global__ void __launch_bounds__(PrefixCfg<D, FMT>::kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
    using C = PrefixCfg<D, FMT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ PrefixGroup plan[kPlanHere + 1];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(base + C::kFull + 8 * i, FMT == kBf16 && !p.boxes ? 64 : 2);
            mbar_init(base + C::kEmpty + 8 * i, C::kStreams);
        }
        if (FMT != kBf16)
            for (int i = 0; i < C::kSlots * 2; ++i) mbar_init(base + C::kLanded + 8 * i, p.boxes ? 1 : 32);
        for (int i = 0; i < 4; ++i) {
            mbar_init(base + C::kS + 8 * i, 1);
            mbar_init(base + C::kP + 8 * i, 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(base + C::kPV + 8 * i, 1);
        mbar_init(base + C::kO, C::kStreams);
        mbar_init(base + C::kQ, C::kSoftWarps * 32);
        mbar_init(base + C::kSync, C::kSoftWarps * 32);
        mbar_init(base + C::kFin, C::kStreams);
        fence_mbar_init();
        abort_flag = 0;
    }
    constexpr int kMmaWarp = C::kSoftWarps + C::kLoadWarps;
    if (p.boxes && threadIdx.x == C::kSoftWarps * 32) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(base + C::kTm, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    // Launched behind the decode of the sequences' own tokens, which waited for all
    // before it and hands this kernel nothing: it starts as SMs come free.  It
    // waits for that decode before it ends, so that the join, which waits for this
    // kernel, finds both done.
    pdl_launch_dependents();
    PrefixGroup* groups = p.n_groups <= kPlanHere ? plan : p.groups;
    if (warp == 0) prefix_plan<D, FMT>(p, groups, lane);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::kTm);
    uint32_t filled = 0, parities = 0;  // of a loader: the slots it filled, the phase of each
    if (warp < C::kSoftWarps) {
        prefix_softmax<D, FMT>(p, groups, base, smem, &abort_flag, tmem, warp, lane);
        if (lane == 0) bulk_wait();  // the states are written before the kernel ends
        tc_fence_before();
    } else if (warp < kMmaWarp) {
        prefix_load<D, FMT>(p, groups, base, smem, &abort_flag, warp - C::kSoftWarps, lane, filled, parities);
    } else {
        // what the sequences' own decode needs of the plan, while the first rows are on their way
        if (warp == kMmaWarp)
            for (int b = blockIdx.x * 32 + lane; b < p.B; b += gridDim.x * 32) p.seqs[b] = prefix_seq(p, groups, b);
        __syncwarp();
        prefix_mma<D, FMT>(p, groups, base, &abort_flag, tmem, warp - kMmaWarp);
    }
    __syncthreads();
    if (abort_flag) {  // a wait gave up: copies may be on their way to slots that nobody waits for any more
        const int half = (warp - C::kSoftWarps) & 1;
        for (int i = 0; i < C::kSlots; ++i)
            if (filled & (1u << i))
                mbar_wait_bounded(base + (FMT == kBf16 ? C::kFull + 8 * i : C::kLanded + 8 * (2 * i + half)), (parities >> i) & 1u,
                                  kDrainLimitNs);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    pdl_wait_primary();
}

template <int D, int FMT>
PrefixShape prefix_shape_as() {
    using C = PrefixCfg<D, FMT>;
    return {reinterpret_cast<const void*>(&prefix_kernel<D, FMT>), C::kThreads, (int)C::kSmem};
}
template <int D>
PrefixShape prefix_shape_of(int format) {
    return format == kBf16 ? prefix_shape_as<D, kBf16>() : format == kE4m3 ? prefix_shape_as<D, kE4m3>() : prefix_shape_as<D, kInt8>();
}

template <int D, int FMT>
cudaError_t launch_prefix_as(const PrefixParams& p, int ctas, cudaStream_t stream) {
    using C = PrefixCfg<D, FMT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_kernel<D, FMT>, p);
}
template <int D>
cudaError_t launch_prefix_of(int format, const PrefixParams& p, int ctas, cudaStream_t stream) {
    return format == kBf16   ? launch_prefix_as<D, kBf16>(p, ctas, stream)
           : format == kE4m3 ? launch_prefix_as<D, kE4m3>(p, ctas, stream)
                             : launch_prefix_as<D, kInt8>(p, ctas, stream);
}

}  // namespace pda
