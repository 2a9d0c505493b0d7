// pda_cache.cu -- the kernels around the decode: norm and rotation of q / k
// heads, the cache write and the cache read-back.
//
// All three move rows of D elements (one head of one token) and do a few
// operations per element, so HBM bounds them once there are enough rows, and
// the chain of dependent loads (starts -> lengths -> block id / rotation row
// -> store) bounds small calls.
#include <cuda_fp16.h>

#include "pda_cache.h"
#include "pda_kernels.cuh"

namespace pda {

#define PDA_DEVERR_BAD_POSITION_ 0x8u
// 64, 128, 256: 450k tokens of 8 heads of 128 read back in 452, 410, 414 us, 64
// tokens appended and 2900 read in 10.4, 9.3, 9.9.
constexpr int kHeadsThreads = 128;

// Where row t of a packed batch belongs: its sequence b, the end of the
// sequence's rows and its length.  Warp-wide.  Up to 32 sequences the lanes
// fetch every start and length at once (one round trip) and search the starts
// with shuffles; a longer list leaves a span of B / 32 entries to a serial
// search.
struct Place {
    int32_t b, begin, end, len;
};
__device__ __forceinline__ Place find_seq(const CacheRef& c, int64_t t, int lane) {
    const int32_t step = (c.B + 31) / 32, at = lane * step;
    const int32_t v = at < c.B ? c.starts[at] : 0x7fffffff;
    const int32_t len = at < c.B ? c.lens[at] : 0;
    const int32_t last = c.starts[c.B];
    int32_t i = 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const int32_t x = __shfl_sync(0xffffffffu, v, i + w);
        if (x <= t && (i + w) * step < c.B) i += w;
    }
    Place p;
    p.b = i;
    p.begin = __shfl_sync(0xffffffffu, v, i);
    p.end = __shfl_sync(0xffffffffu, v, (i + 1) & 31);
    p.len = __shfl_sync(0xffffffffu, len, i);
    if (step == 1) {
        if (i + 1 >= c.B) p.end = last;
        return p;
    }
    int32_t lo = i * step, hi = min(lo + step, c.B) - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (c.starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    p.b = lo;
    p.begin = c.starts[lo];
    p.end = c.starts[lo + 1];
    p.len = c.lens[lo];
    return p;
}
// The same for equal shares.
__device__ __forceinline__ Place share_of(const CacheRef& c, int64_t t, bool in) {
    Place p;
    p.b = (int32_t)(in ? div_floor(t, c.rows_each) : 0);
    p.begin = (int32_t)(p.b * c.rows_each);
    p.end = (int32_t)(p.begin + c.rows_each);
    p.len = c.lens[p.b];
    return p;
}

// Pairs of fp32 values in one register pair: two operations an instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 unpack2(uint32_t x) { return f2(bf16_lo(x), bf16_hi(x)); }
__device__ __forceinline__ uint32_t pack2(F2 a) {
    float x, y;
    split(a, x, y);
    return pack_bf16x2(x, y);
}

// E elements (4 or 8) of bf16 as they lie in memory.
template <int E>
struct Run {
    uint32_t w[E / 2];
};
template <int E>
__device__ __forceinline__ Run<E> load_run(const uint16_t* s) {
    Run<E> r;
    if constexpr (E == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(s);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(s);
        r.w[0] = x.x; r.w[1] = x.y;
    }
    return r;
}
template <int E>
__device__ __forceinline__ void store_run(void* d, const uint32_t* w) {
    if constexpr (E == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
}

template <int E>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int at, F2 (&out)[E / 2]) {
    if (f32) {
        const float2* s = reinterpret_cast<const float2*>(static_cast<const float*>(w) + at);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) out[e] = f2(s[e].x, s[e].y);
    } else {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(w) + at);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) out[e] = unpack2(s[e]);
    }
}

// A row's scale and the factor that takes its values to codes.  Infinities
// and NaN sort above every finite magnitude as bit patterns.
template <int FMT>
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float* inv, bool* keep) {
    constexpr float kMax = FMT == kE4m3 ? 448.f : 127.f;
    constexpr uint32_t kTiny = 27u << 23;  // 2^-100
    const float amax = __uint_as_float(amax_bits);
    *keep = amax_bits >= kTiny && amax_bits < 0x7f800000u;
    *inv = *keep ? __fdiv_rn(kMax, amax) : 0.f;
    return *keep ? __fdiv_rn(amax, kMax) : amax_bits < kTiny ? 0.f : __uint_as_float(0x7fffffffu);
}

// Four codes from two pairs.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(F2 p, F2 q, F2 inv) {
    float x[4];
    split(mul2(p, inv), x[0], x[1]);
    split(mul2(q, inv), x[2], x[3]);
    if constexpr (FMT == kE4m3) {
        return pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16);
    } else {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = max(-127, min(127, __float2int_rn(x[i])));
            r |= (uint32_t)(c & 0xff) << (8 * i);
        }
        return r;
    }
}

// ---- norm, rotation and cache write
//
// D / (2 E) lanes share a row; a lane holds two runs of E columns, chosen so
// that it owns both halves of its E rotation pairs (columns E l.. and
// rotary/2 + E l.. when the pairs are half a rotation apart), so the rotation
// moves nothing between lanes and a lane reads E cosines and E sines.
// Arithmetic is on pairs of fp32 values, two to an instruction.

// Where a token's keys and values go.
struct Spot {
    int64_t off;   // elements into the pools, of kv head 0
    int32_t blk, slot;
    bool write;    // false: no such place (flagged)
};

template <int D, int FMT, int E>
struct RowWork {
    static constexpr int TPR = D / (2 * E), H = E / 2;
    const HeadsParams& p;
    int l;               // lane of the row
    uint32_t gmask;      // the row's lanes
    bool turn;           // this lane's columns rotate
    int a_at, b_at;      // first columns of the two runs
    F2 cs[H], sn[H];
    const void* weight = nullptr;
    F2 wa[H], wb[H];     // the norm weights in use
    F2 a[H], b[H];       // this lane's part of a row

    __device__ __forceinline__ RowWork(const HeadsParams& p_, int thread) : p(p_) {
        const int lane = thread & 31;
        l = thread % TPR;
        gmask = TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1u) << (lane & ~(TPR - 1));
        const int rl = p.rotary / (2 * E);  // lanes that rotate
        turn = l < rl;
        const bool halves = turn && !p.interleaved;
        a_at = E * (halves ? l : 2 * l);
        b_at = E * (halves ? l + rl : 2 * l + 1);
    }
    // cosines and sines from a row of the table (global or shared memory)
    __device__ __forceinline__ void load_turn(const float* row) {
        if (!turn) return;
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
            const float4 c = reinterpret_cast<const float4*>(row + E * l)[e];
            const float4 s = reinterpret_cast<const float4*>(row + E * l + p.rotary / 2)[e];
            cs[2 * e] = f2(c.x, c.y);
            cs[2 * e + 1] = f2(c.z, c.w);
            sn[2 * e] = f2(s.x, s.y);
            sn[2 * e + 1] = f2(s.z, s.w);
        }
    }
    __device__ __forceinline__ void set(const Run<E>& x, const Run<E>& y) {
#pragma unroll
        for (int e = 0; e < H; ++e) {
            a[e] = unpack2(x.w[e]);
            b[e] = unpack2(y.w[e]);
        }
    }
    __device__ __forceinline__ void prepare(const void* w) {
        if (w) {
            if (weight != w) {
                load_weight<E>(w, p.weights_f32 != 0, a_at, wa);
                load_weight<E>(w, p.weights_f32 != 0, b_at, wb);
                weight = w;
            }
            F2 sq = f2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < H; ++e) sq = fma2(b[e], b[e], fma2(a[e], a[e], sq));
            float s0, s1;
            split(sq, s0, s1);
            float ss = s0 + s1;
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(gmask, ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
            const F2 i2 = f2(inv, inv);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                a[e] = mul2(mul2(a[e], i2), wa[e]);
                b[e] = mul2(mul2(b[e], i2), wb[e]);
            }
        }
        if (!turn) return;
        const F2 minus = f2(-1.f, -1.f);
        if (p.interleaved) {
            // pairs lie side by side: gather two of them into (evens, odds)
#pragma unroll
            for (int e = 0; e < H; ++e) {
                F2& u = 2 * e < H ? a[2 * e] : b[2 * e - H];
                F2& v = 2 * e + 1 < H ? a[2 * e + 1] : b[2 * e + 1 - H];
                float u0, u1, v0, v1;
                split(u, u0, u1);
                split(v, v0, v1);
                const F2 x = f2(u0, v0), y = f2(u1, v1);
                const F2 nx = fma2(mul2(y, sn[e]), minus, mul2(x, cs[e])), ny = fma2(x, sn[e], mul2(y, cs[e]));
                float x0, x1, y0, y1;
                split(nx, x0, x1);
                split(ny, y0, y1);
                u = f2(x0, y0);
                v = f2(x1, y1);
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const F2 x = a[e];
                a[e] = fma2(mul2(b[e], sn[e]), minus, mul2(x, cs[e]));
                b[e] = fma2(x, sn[e], mul2(b[e], cs[e]));
            }
        }
    }
    __device__ __forceinline__ void put16(uint16_t* d) const {
        uint32_t w[H];
#pragma unroll
        for (int e = 0; e < H; ++e) w[e] = pack2(a[e]);
        store_run<E>(d + a_at, w);
#pragma unroll
        for (int e = 0; e < H; ++e) w[e] = pack2(b[e]);
        store_run<E>(d + b_at, w);
    }
    // a K (which 0) or V (which 1) row of kv head h into its slot
    __device__ __forceinline__ void put_cache(int which, int h, const Spot& at) const {
        if constexpr (FMT == kBf16) {
            put16(reinterpret_cast<uint16_t*>(which ? p.c.v : p.c.k) + at.off + (int64_t)h * p.c.kvh);
        } else if constexpr (FMT != kNoCache) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < H; ++e) {
                float x, y;
                split(a[e], x, y);
                top = max(top, max(__float_as_uint(x) & 0x7fffffffu, __float_as_uint(y) & 0x7fffffffu));
                split(b[e], x, y);
                top = max(top, max(__float_as_uint(x) & 0x7fffffffu, __float_as_uint(y) & 0x7fffffffu));
            }
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(gmask, top, o));
            float inv;
            bool keep;
            const float scale = row_scale<FMT>(top, &inv, &keep);
            const F2 i2 = f2(inv, inv);
            uint8_t* d = (which ? p.c.v : p.c.k) + at.off + (int64_t)h * p.c.kvh;
            uint32_t ca[E / 4], cb[E / 4];
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                ca[e] = keep ? codes4<FMT>(a[2 * e], a[2 * e + 1], i2) : 0u;
                cb[e] = keep ? codes4<FMT>(b[2 * e], b[2 * e + 1], i2) : 0u;
            }
            if constexpr (E == 8) {
                *reinterpret_cast<uint2*>(d + a_at) = make_uint2(ca[0], ca[1]);
                *reinterpret_cast<uint2*>(d + b_at) = make_uint2(cb[0], cb[1]);
            } else {
                *reinterpret_cast<uint32_t*>(d + a_at) = ca[0];
                *reinterpret_cast<uint32_t*>(d + b_at) = cb[0];
            }
            if (l == 0) p.c.scales[((((int64_t)at.blk * p.Hkv + h) * 2 + which) << p.c.lbs) + at.slot] = scale;
        }
    }
    // row r of token t (its elements set) to where it goes
    __device__ __forceinline__ void finish(int64_t t, int r, int nq, int nk, const Spot& at) {
        if (r < nq) {
            prepare(p.q_weight);
            put16(p.q_out.p + t * p.q_out.tok + r * p.q_out.head);
        } else if (r < nq + nk) {
            prepare(p.k_weight);
            if constexpr (FMT == kNoCache) put16(p.k_out.p + t * p.k_out.tok + (r - nq) * p.k_out.head);
            else if (at.write) put_cache(0, r - nq, at);
        } else {
            if (at.write) put_cache(1, r - nq - nk, at);
        }
    }
};

// A new token's index in its sequence (negative: padding) and its spot, given
// its place in the batch.  `flag`: this thread reports what is wrong.
__device__ __forceinline__ Spot spot_of(const HeadsParams& p, const Place& at, int64_t idx, bool flag) {
    Spot s = {0, 0, (int32_t)idx & ((1 << p.c.lbs) - 1), false};
    const int64_t j = idx >> p.c.lbs;
    if (j >= p.c.table_stride) {
        if (flag) atomicOr(p.err, PDA_DEVERR_BAD_POSITION_);
        return s;
    }
    s.blk = p.c.table[(int64_t)at.b * p.c.table_stride + j];
    s.write = s.blk >= 0 && s.blk < p.c.num_blocks;
    if (!s.write && flag) atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
    s.off = (int64_t)s.blk * p.c.blk + (int64_t)s.slot * p.c.tok;
    return s;
}
// The rotation row of token t at index idx of its sequence.
__device__ __forceinline__ int32_t turn_row(const HeadsParams& p, int64_t t, int64_t idx, bool flag) {
    int64_t pos = p.positions ? p.positions[t] : idx;
    if (pos < 0 || pos >= p.max_pos) {
        if (flag) atomicOr(p.err, PDA_DEVERR_BAD_POSITION_);
        pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    return (int32_t)pos;
}

// Little work, or any alignment: a group of lanes takes kRows rows of one token
// straight from memory.  Latency counts (loads of the rows go out before the
// token's place is looked up), and many small groups hide it better than few
// with more rows each: a 32-token step of 48 rows takes 3.7 us with two rows a
// group, 4.8 with four.  What is left of such a step is one chain of dependent
// loads and the launch itself.
constexpr int kRows = 2;
template <int D, int FMT>
__global__ void __launch_bounds__(kHeadsThreads, 8) heads_kernel(const __grid_constant__ HeadsParams p) {
    constexpr int E = 4;
    using Work = RowWork<D, FMT, E>;
    const int nq = p.q.p ? p.Hq : 0, nk = p.k.p ? p.Hkv : 0, nv = FMT != kNoCache ? p.Hkv : 0;
    const int rows = nq + nk + nv, spans = (rows + kRows - 1) / kRows;
    const int64_t item = (int64_t)blockIdx.x * (kHeadsThreads / Work::TPR) + threadIdx.x / Work::TPR;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t t = div_floor(item, spans);
    const bool in = t < p.T;
    const int first = (int)(item - t * spans) * kRows, last = min(first + kRows, rows);
    Work work(p, threadIdx.x);
    Run<E> xa[kRows], xb[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = first + i;
        if (in && r < last) {
            const uint16_t* s = r < nq ? p.q.p + t * p.q.tok + r * p.q.head
                              : r < nq + nk ? p.k.p + t * p.k.tok + (r - nq) * p.k.head
                                            : p.v.p + t * p.v.tok + (r - nq - nk) * p.v.head;
            xa[i] = load_run<E>(s + work.a_at);
            xb[i] = load_run<E>(s + work.b_at);
        }
    }
    bool live = in;
    int64_t idx = 0;
    Spot at = {0, 0, 0, false};
    if constexpr (FMT != kNoCache) {
        const Place place = p.c.starts ? find_seq(p.c, t, threadIdx.x & 31) : share_of(p.c, t, in);
        idx = (int64_t)place.len - place.end + t;
        live = live && t < place.end && t >= place.begin && idx >= 0;
        if (live && last > nq) at = spot_of(p, place, idx, work.l == 0);
    }
    if (!live) return;
    if (p.cos_sin) work.load_turn(p.cos_sin + (int64_t)turn_row(p, t, idx, work.l == 0) * p.rotary);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (first + i >= last) break;
        work.set(xa[i], xb[i]);
        work.finish(t, first + i, nq, nk, at);
    }
}

// Many tokens: one persistent CTA per SM streams them through a ring of
// shared-memory slots, a token's rows (and its row of cosines and sines) to a
// slot.  A producer warp looks 32 tokens up at a time and issues their bulk
// copies, teams of warps take the slots in turn and write straight to memory.
// The copies in flight do not depend on occupancy; loading rows to registers
// instead, with 32 warps an SM, came to 3.9 TB/s on 8191 tokens of 72 heads of
// 128 and no arrangement of rows per thread passed it.  HBM bounds it: those
// tokens take 51 us (5.9 TB/s read and written), ragged prompts of 24
// sequences (20k tokens of 32 + 2 * 8 heads, e4m3 cache) 79 us (5.8 TB/s).
//
// Slots of kSmallSlot bytes and more: teams of three warps (teams of 2 and 4
// took 53.5 and 52 us on the first), copies issued by one lane after another.
// The first fill is paced: kFillPace bytes a cycle and SM are about the share
// of HBM that reads get once stores run too.  Issued all at once, the copies
// delay each other, the first slot lands late and the stores start late (4096
// tokens of 40 heads of 128: 19.4 us at once, 18.1 paced; 12 bytes 18.0, 9
// bytes 18.6).
// Smaller slots: each warp a team of its own and kIssue lanes issuing at once,
// since one lane's issue (0.3 us a token) and a team's turn are longer than
// their traffic takes (8000 tokens of 16 + 2 * 2 heads of 128 appended: 20.1
// us, as large slots 25.5; of 20 + 2 * 4 heads, past the border, 27.2 and 24.6).
//
// A slot belongs to one team (slots are a multiple of the teams at work): the
// team that waits for a slot's next token has itself seen the previous one
// land.  Copies land in any order, so another team could be a whole turn of
// the slot ahead and take the barrier's older phase for the one it waits for.
constexpr int kRingWarps = 15, kMaxSlots = 30, kIssue = 4;
constexpr uint32_t kFillPace = 16;
constexpr int kRingThreads = (kRingWarps + 1) * 32;
static_assert(kMaxSlots <= 32, "the first fill is the producer's first 32 tokens");
static_assert(32 % kIssue == 0, "lanes that issue together belong to one look-up");
struct SlotMeta {
    Spot at;
    int32_t t;  // -1: padding
};

template <int D, int FMT>
__global__ void __launch_bounds__(kRingThreads) heads_ring_kernel(const __grid_constant__ HeadsParams p) {
    constexpr int E = 8;
    using Work = RowWork<D, FMT, E>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * kMaxSlots];
    __shared__ SlotMeta meta[kMaxSlots];
    __shared__ int abort_flag;
    const uint32_t ring = (smem_u32(smem_raw) + 127u) & ~127u;
    const uint8_t* ring_p = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t bars0 = smem_u32(bars);
    const int nq = p.q.p ? p.Hq : 0, nk = p.k.p ? p.Hkv : 0, nv = FMT != kNoCache ? p.Hkv : 0;
    const int rows = nq + nk + nv, S = p.slots;
    const uint32_t turn_bytes = (uint32_t)p.rotary * 4u, slot_bytes = (uint32_t)rows * (2u * D) + turn_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(bars0 + 8 * s, 1);
            mbar_init(bars0 + 8 * (S + s), p.team_warps);
        }
        fence_mbar_init();
        abort_flag = 0;
    }
    __syncthreads();
    pdl_wait_primary();
    pdl_launch_dependents();
    const int32_t n = (int32_t)((p.T - blockIdx.x + gridDim.x - 1) / gridDim.x);  // tokens blockIdx.x, + gridDim.x, ..
    if (warp == kRingWarps) {
        // side by side (one fused projection's output): one copy brings all of a token
        const bool joined = nq && nk && p.k.p == p.q.p + nq * D && p.k.tok == p.q.tok &&
                            (!nv || (p.v.p == p.k.p + nk * D && p.v.tok == p.q.tok));
        for (int32_t i0 = 0; i0 < n; i0 += 32) {
            // lane i: token i0 + i
            const int32_t mine = i0 + lane;
            const int64_t t = (int64_t)blockIdx.x + (int64_t)mine * gridDim.x;
            bool live = mine < n;
            int64_t idx = 0;
            Spot at = {0, 0, 0, false};
            if constexpr (FMT != kNoCache) {
                const Place place = p.c.starts ? find_seq(p.c, t, lane) : share_of(p.c, t, live);
                idx = (int64_t)place.len - place.end + t;
                live = live && t < place.end && t >= place.begin && idx >= 0;
                if (live) at = spot_of(p, place, idx, true);
            }
            const int32_t turn = live && p.rotary ? turn_row(p, t, idx, true) : 0;
            const int s = mine % S;
            const uint32_t phase = (uint32_t)(mine / S) & 1u, full = bars0 + 8 * s, dst = ring + (uint32_t)s * slot_bytes;
            // lanes i .. i + w - 1 issue their tokens; false: a wait ran out
            const auto issue = [&](int i, int w) -> bool {
                int issued = 0, stop = 0;
                if (lane >= i && lane < i + w && mine < n) {
                    if (*(volatile int*)&abort_flag || !mbar_wait_bounded(bars0 + 8 * (S + s), phase ^ 1u, kWaitLimitNs)) {
                        stop = 1;
                    } else {
                        meta[s].at = at;
                        meta[s].t = live ? (int32_t)t : -1;
                        issued = 1;
                        mbar_arrive_expect_tx(full, live ? slot_bytes : 0u);
                        if (live) {
                            uint32_t to = dst;
                            if (joined) {
                                bulk_load(to, p.q.p + t * p.q.tok, (uint32_t)(rows * 2 * D), full);
                            } else {
                                if (nq) bulk_load(to, p.q.p + t * p.q.tok, (uint32_t)(nq * 2 * D), full);
                                to += (uint32_t)(nq * 2 * D);
                                if (nk) bulk_load(to, p.k.p + t * p.k.tok, (uint32_t)(nk * 2 * D), full);
                                to += (uint32_t)(nk * 2 * D);
                                if (nv) bulk_load(to, p.v.p + t * p.v.tok, (uint32_t)(nv * 2 * D), full);
                            }
                            if (turn_bytes)
                                bulk_load(dst + (uint32_t)(rows * 2 * D), p.cos_sin + (int64_t)turn * p.rotary, turn_bytes,
                                          full);
                        }
                    }
                }
                if (!__any_sync(0xffffffffu, stop)) return true;
                // report it, and leave once the copies issued have landed
                const uint32_t out = __ballot_sync(0xffffffffu, issued);
                if (lane == 0) {
                    atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
                    abort_flag = 1;
                    for (int32_t k = max(0, i0 + i - S); k < i0 + i + w; ++k)
                        if (k < i0 + i || (out >> (k - i0)) & 1u)
                            mbar_wait_bounded(bars0 + 8 * (k % S), (k / S) & 1, kWaitLimitNs);
                }
                return false;
            };
            int i = 0;
            const int w = p.team_warps == 1 ? kIssue : 1;
            if (i0 == 0) {
                const int64_t t0 = clock64();
                for (; i + w <= S && i < n; i += w) {
                    while (clock64() - t0 < (int64_t)(i * slot_bytes / kFillPace)) {
                    }
                    if (!issue(i, w)) return;
                }
            }
            for (; i < 32 && i0 + i < n; i += w)
                if (!issue(i, w)) return;
        }
        return;
    }
    const int TW = p.team_warps, team = warp / TW, member = warp % TW;
    constexpr int G = 32 / Work::TPR;  // rows a warp takes at once
    Work work(p, threadIdx.x);
    const int teams = min(kRingWarps / TW, S);
    if (team >= teams) return;
    for (int32_t i = team; i < n; i += teams) {
        const int s = i % S;
        if (!mbar_wait_bounded(bars0 + 8 * s, (i / S) & 1, kWaitLimitNs)) {
            if (lane == 0) {
                atomicOr(p.err, PDA_DEVERR_TIMEOUT_);
                *(volatile int*)&abort_flag = 1;
            }
            return;
        }
        const SlotMeta m = meta[s];
        if (m.t >= 0) {
            const uint8_t* slot = ring_p + (size_t)s * slot_bytes;
            if (p.rotary) work.load_turn(reinterpret_cast<const float*>(slot + (size_t)rows * 2 * D));
            for (int r = member * G + lane / Work::TPR; r < rows; r += TW * G) {
                const uint16_t* x = reinterpret_cast<const uint16_t*>(slot) + r * D;
                work.set(load_run<E>(x + work.a_at), load_run<E>(x + work.b_at));
                work.finish(m.t, r, nq, nk, m.at);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars0 + 8 * (S + s));
    }
}

// Read-back: D / 16 lanes share a row of 16 elements each; a group takes HC
// of a token's 2 Hkv rows, whose loads go out together.  Two bytes are written
// for each byte read, and HBM bounds it: 450k tokens of 8 heads of 128 (int8,
// blocks of 32; 0.9 GB read, 1.9 written) take 410 us, 6.8 TB/s, the rate
// of a plain copy.  A small call is bound by its chain of loads: lengths, block
// id, codes.
template <int D, int FMT, bool F32, int HC>
__global__ void __launch_bounds__(kHeadsThreads) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int TPR = D / 16;
    const int lane = threadIdx.x & 31, l = threadIdx.x % TPR;
    const int nk = p.k_out ? p.Hkv : 0, nv = p.v_out ? p.Hkv : 0;
    const int rows = nk + nv, chunks = (rows + HC - 1) / HC;
    const int64_t item = (int64_t)blockIdx.x * (kHeadsThreads / TPR) + threadIdx.x / TPR;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t t = div_floor(item, chunks);
    const int r0 = (int)(item - t * chunks) * HC;
    bool live = t < p.rows;
    const Place place = p.c.starts ? find_seq(p.c, t, lane) : share_of(p.c, t, live);
    const int32_t b = place.b;
    const int64_t at = t - place.begin;
    live = live && at >= 0 && t < place.end;
    if (live && at == 0 && r0 == 0 && l == 0 && (place.len < 0 || place.len > (int64_t)p.c.table_stride << p.c.lbs))
        atomicOr(p.err, PDA_DEVERR_BAD_LENGTH_);  // whichever of its rows are asked for
    if (!live || at >= place.len) return;
    const int64_t j = at >> p.c.lbs;
    const int slot = (int)at & ((1 << p.c.lbs) - 1);
    if (j >= p.c.table_stride) {
        if (l == 0) atomicOr(p.err, PDA_DEVERR_BAD_LENGTH_);
        return;
    }
    const int32_t blk = p.c.table[(int64_t)b * p.c.table_stride + j];
    const bool bad = blk < 0 || blk >= p.c.num_blocks;
    if (bad && l == 0) atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
    const int64_t off = (int64_t)blk * p.c.blk + (int64_t)slot * p.c.tok + 16 * l;

    constexpr int W = FMT == kBf16 ? 2 : 1;  // 16-byte words of 16 elements
    uint4 raw[HC][W];
    float scale[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const int r = r0 + i, which = r >= nk, h = which ? r - nk : r;
        scale[i] = 1.f;
#pragma unroll
        for (int w = 0; w < W; ++w) raw[i][w] = make_uint4(0, 0, 0, 0);
        if (r >= rows || bad) continue;
        const int64_t o = off + (int64_t)h * p.c.kvh;
        const uint8_t* s = (which ? p.c.v : p.c.k) + (FMT == kBf16 ? 2 * o : o);
#pragma unroll
        for (int w = 0; w < W; ++w) raw[i][w] = __ldcg(reinterpret_cast<const uint4*>(s) + w);
        if constexpr (FMT != kBf16)
            scale[i] = p.c.scales[((((int64_t)blk * p.Hkv + h) * 2 + which) << p.c.lbs) + slot];
    }
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const int r = r0 + i, which = r >= nk, h = which ? r - nk : r;
        if (r >= rows) break;
        float x[16];
        if constexpr (FMT == kBf16) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t v[4] = {raw[i][w].x, raw[i][w].y, raw[i][w].z, raw[i][w].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[8 * w + 2 * e] = bf16_lo(v[e]);
                    x[8 * w + 2 * e + 1] = bf16_hi(v[e]);
                }
            }
        } else {
            const uint32_t v[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (FMT == kE4m3) {
                    const uint32_t lo = e4m3x2_to_f16x2((uint16_t)v[e]), hi = e4m3x2_to_f16x2((uint16_t)(v[e] >> 16));
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    x[4 * e] = a.x; x[4 * e + 1] = a.y; x[4 * e + 2] = c.x; x[4 * e + 3] = c.y;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[4 * e + k] = (float)(int8_t)(v[e] >> (8 * k));
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= scale[i];
        }
        const int64_t o = (t * p.Hkv + h) * D + 16 * l;
        void* out = which ? p.v_out : p.k_out;
        if constexpr (F32) {
            float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + o);
#pragma unroll
            for (int w = 0; w < 4; ++w) d[w] = make_float4(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
        } else {
            uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + o);
#pragma unroll
            for (int w = 0; w < 2; ++w)
                d[w] = make_uint4(pack_bf16x2(x[8 * w], x[8 * w + 1]), pack_bf16x2(x[8 * w + 2], x[8 * w + 3]),
                                  pack_bf16x2(x[8 * w + 4], x[8 * w + 5]), pack_bf16x2(x[8 * w + 6], x[8 * w + 7]));
        }
    }
}

namespace {

template <typename P>
cudaError_t launch_grid(void (*kernel)(const P), const P& p, int64_t grid, int threads, size_t smem,
                        cudaStream_t stream) {
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// `items` groups of `lanes` lanes.
template <typename P>
cudaError_t launch_rows(void (*kernel)(const P), const P& p, int64_t items, int lanes, cudaStream_t stream) {
    return launch_grid(kernel, p, (items * lanes + kHeadsThreads - 1) / kHeadsThreads, kHeadsThreads, 0, stream);
}

// A token's heads as one bulk copy: side by side, on 16-byte boundaries.
bool one_copy(const Heads& h, int D) {
    return !h.p || (h.head == D && h.tok % 8 == 0 && reinterpret_cast<uintptr_t>(h.p) % 16 == 0);
}
bool runs_of_8(const Heads& h) {
    return !h.p || (h.tok % 8 == 0 && h.head % 8 == 0 && reinterpret_cast<uintptr_t>(h.p) % 16 == 0);
}

constexpr int kRingBytes = 200 * 1024;  // of an SM's 227 KB
// Bytes of heads from which the ring pays.  Short of it a launch is over before
// the ring is under way: 512 tokens of 40 heads of 128 (5.2 MB) take 4.6 us
// straight, 4.9 through the ring; 1024 (10.5 MB) 8.9 and 7.9; 4096 26.0 and
// 18.1.  And bytes of a slot: 8000 tokens of 10 heads of 64 (1.5 KB) take 9.6
// straight, 11.4 through the ring, of 12 such heads (1.8 KB) 16.4 and 13.8.
constexpr int64_t kRingWork = 8 << 20;
constexpr int kSmallSlot = 6144, kLeastSlot = 1792;

template <int D, int FMT>
cudaError_t launch_heads_of(HeadsParams p, cudaStream_t stream) {
    const int rows = (p.q.p ? p.Hq : 0) + (p.k.p ? p.Hkv : 0) + (FMT != kNoCache ? p.Hkv : 0);
    const int slot = rows * 2 * D + p.rotary * 4;
    p.team_warps = slot < kSmallSlot ? 1 : 3;
    const int teams = kRingWarps / p.team_warps, most = p.team_warps == 1 ? kMaxSlots : 20;
    p.slots = kRingBytes / slot < most ? kRingBytes / slot : most;
    if (p.slots > teams) p.slots -= p.slots % teams;
    if (p.T * rows * 2 * D >= kRingWork && slot >= kLeastSlot && p.slots >= 4 && p.rotary % 16 == 0 && one_copy(p.q, D) && one_copy(p.k, D) &&
        one_copy(p.v, D) && runs_of_8(p.q_out) && runs_of_8(p.k_out)) {
        return launch_grid(heads_ring_kernel<D, FMT>, p, p.sms, kRingThreads, (size_t)p.slots * slot + 128, stream);
    }
    return launch_rows(heads_kernel<D, FMT>, p, p.T * ((rows + kRows - 1) / kRows), D / 8, stream);
}

template <int D, int FMT>
cudaError_t ring_attributes() {
    return cudaFuncSetAttribute(heads_ring_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 128);
}
template <int D>
cudaError_t heads_setup_of() {
    cudaError_t e = ring_attributes<D, kNoCache>();
    if (e == cudaSuccess) e = ring_attributes<D, kBf16>();
    if (e == cudaSuccess) e = ring_attributes<D, kE4m3>();
    if (e == cudaSuccess) e = ring_attributes<D, kInt8>();
    return e;
}

template <int D>
cudaError_t launch_heads_fmt(int format, const HeadsParams& p, cudaStream_t stream) {
    switch (format) {
        case kNoCache: return launch_heads_of<D, kNoCache>(p, stream);
        case kBf16: return launch_heads_of<D, kBf16>(p, stream);
        case kE4m3: return launch_heads_of<D, kE4m3>(p, stream);
        case kInt8: return launch_heads_of<D, kInt8>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int D, int FMT>
cudaError_t launch_read_of(bool f32, const ReadParams& p, cudaStream_t stream) {
    // two rows a group: 410 us for 450k tokens of 8 heads of 128, four 437, one 548
    constexpr int HC = 2;
    const int rows = (p.k_out ? p.Hkv : 0) + (p.v_out ? p.Hkv : 0);
    const int64_t items = p.rows * ((rows + HC - 1) / HC);
    return f32 ? launch_rows(read_kernel<D, FMT, true, HC>, p, items, D / 16, stream)
               : launch_rows(read_kernel<D, FMT, false, HC>, p, items, D / 16, stream);
}

template <int D>
cudaError_t launch_read_fmt(int format, bool f32, const ReadParams& p, cudaStream_t stream) {
    switch (format) {
        case kBf16: return launch_read_of<D, kBf16>(f32, p, stream);
        case kE4m3: return launch_read_of<D, kE4m3>(f32, p, stream);
        case kInt8: return launch_read_of<D, kInt8>(f32, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t heads_setup(int D) {
    return D == 64 ? heads_setup_of<64>() : D == 128 ? heads_setup_of<128>() : heads_setup_of<256>();
}

cudaError_t launch_heads(int D, int format, const HeadsParams& p, cudaStream_t stream) {
    switch (D) {
        case 64: return launch_heads_fmt<64>(format, p, stream);
        case 128: return launch_heads_fmt<128>(format, p, stream);
        case 256: return launch_heads_fmt<256>(format, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_read(int D, int format, bool out_f32, const ReadParams& p, cudaStream_t stream) {
    switch (D) {
        case 64: return launch_read_fmt<64>(format, out_f32, p, stream);
        case 128: return launch_read_fmt<128>(format, out_f32, p, stream);
        case 256: return launch_read_fmt<256>(format, out_f32, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pda
