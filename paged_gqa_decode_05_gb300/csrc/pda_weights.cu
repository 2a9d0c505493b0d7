// pda_weights.cu -- the sums of attention weights beside a cache, and the
// head-size dispatch of the scored and shared-prefix kernels.
//
//   out[t, g] = (t is one of the queries' own tokens ? 0 : in[t, g])
//             + sum over the queries i that see t and the G q heads h of kv
//               head g of 2^(s_iht - m_ih) / l_ih
// with the scores s that the decode wrote (base-2 units; -inf where a query
// does not see the token) and the (m, l) of its output rows.  The decode holds
// a score in registers once, long before its row's l is known, so it writes
// 4 bytes a score (G of them beside a token's 2 D of K and V, and soon enough
// read back to come from L2) where a second pass over K would read 2 D again.
// Bound by those reads and by the sums' own 8 bytes a token.
#include "pda_prefix.h"
#include "pda_ptx.cuh"
#include "pda_scored.h"

namespace pda {

#define PDA_DECLARE_SCORED(FORMAT, D)                                                                       \
    ScoredShape scored_shape_##FORMAT##_d##D(const ScoredForm& f);                                          \
    cudaError_t launch_scored_##FORMAT##_d##D(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, \
                                              cudaStream_t stream);
#define PDA_FOR_SCORED(F) F(bf16, 64) F(bf16, 128) F(bf16, 256) F(e4m3, 64) F(e4m3, 128) F(e4m3, 256) F(int8, 64) F(int8, 128) F(int8, 256)
PDA_FOR_SCORED(PDA_DECLARE_SCORED)

namespace {
constexpr int bf16 = kBf16, e4m3 = kE4m3, int8 = kInt8;
}

ScoredShape scored_shape(int D, const ScoredForm& f) {
#define PDA_SCORED_SHAPE(FORMAT, DIM) if (f.format == FORMAT && D == DIM) return scored_shape_##FORMAT##_d##DIM(f);
    PDA_FOR_SCORED(PDA_SCORED_SHAPE)
    return {};
}

cudaError_t launch_scored(int D, const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
#define PDA_SCORED_LAUNCH(FORMAT, DIM) \
    if (f.format == FORMAT && D == DIM) return launch_scored_##FORMAT##_d##DIM(f, p, grid, smem, stream);
    PDA_FOR_SCORED(PDA_SCORED_LAUNCH)
    return cudaErrorInvalidValue;
}

#define PDA_DECLARE_PREFIX(D)              \
    PrefixShape prefix_shape_d##D(int format); \
    cudaError_t launch_prefix_d##D(int format, const PrefixParams& p, int ctas, cudaStream_t stream);
PDA_DECLARE_PREFIX(64)
PDA_DECLARE_PREFIX(128)
PDA_DECLARE_PREFIX(256)

PrefixShape prefix_shape(int D, int format) {
    switch (D) {
        case 64: return prefix_shape_d64(format);
        case 128: return prefix_shape_d128(format);
        case 256: return prefix_shape_d256(format);
        default: return {};
    }
}

cudaError_t launch_prefix(int D, int format, const PrefixParams& p, int ctas, cudaStream_t stream) {
    switch (D) {
        case 64: return launch_prefix_d64(format, p, ctas, stream);
        case 128: return launch_prefix_d128(format, p, ctas, stream);
        case 256: return launch_prefix_d256(format, p, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

namespace {

cudaLaunchConfig_t pdl_config(int grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// A CTA takes chunks of kThreads * kTok tokens of a (sequence, kv head), kTok a
// thread with their loads together, kCtas a SM.  Whole decodes of 32 sequences of
// 4096 tokens, and of 64 of 128 to 32768 with 8 q rows: 128 threads 97.7 and 176.4
// us, 256 101.1 and 180.8; (another board) 5, 8 and 16 CTAs a SM 97.0, 99.4, 101.5 and
// 192, 184, 187; 3 tokens a thread 99.5 and 187, 6 101.1 and 185.5.
constexpr int kCtas = 8, kThreads = 128, kTok = 4, kChunk = kThreads * kTok;

__host__ __device__ __forceinline__ int32_t chunks_of(int32_t n) { return (int32_t)(((uint32_t)n + kChunk - 1) / kChunk); }

// A score's weight, z the (-m, -log2 l) of its row: 0 where the query does not see the
// token, whatever that row's sum is.
__device__ __forceinline__ float weight(float s, const float2& z) {
    return s == __int_as_float(0xff800000) ? 0.f : ex2((s + z.x) + z.y);
}

// A launch row's q rows are taken kSub at a time.  kSR: kSub where rows_per_slot is
// a multiple of 8 or of 4 (a token's scores in one or two loads), 0: any.  kOne:
// a launch row is one step (with the steps' arithmetic for all, 2.8 M tokens of 8
// q rows took 190.8 us for 183.6).
template <int kSR, bool kOne>
__global__ void __launch_bounds__(kThreads) weights_kernel(const WeightsParams p) {
    __shared__ int32_t pfx[kMaxLaunchBatch + 1];  // chunks before each sequence, one kv head
    __shared__ int32_t sums[kThreads / 32];
    constexpr int kSub = kSR > 0 ? kSR : kMaxGroup;
    __shared__ alignas(16) float2 ml[2][kSub];  // (-m, -log2 l) of the q rows
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Launched behind the decode, which waited for all before it: lengths, tables and
    // the sums so far are there, so the plan and the first chunk's sums are read
    // under its end; only its scores and row sums are waited for.
    const int32_t most = (int32_t)min((int64_t)p.table_stride << p.lbs, (int64_t)0x7fffffff);
    auto tokens = [&](int b) { return min(max(p.lens[b], 0), most); };
    constexpr int kPer = kMaxLaunchBatch / kThreads;
    const int per = (p.B + kThreads - 1) / kThreads;  // <= kPer
    int32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (k < per && tid * per + k < p.B) mine += chunks_of(tokens(tid * per + k));
    int32_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int32_t run = x - mine;
    for (int w = 0; w < warp; ++w) run += sums[w];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int b = tid * per + k;
        if (k < per && b < p.B) {
            pfx[b] = run;
            run += chunks_of(tokens(b));
            if (b == p.B - 1) pfx[p.B] = run;
        }
    }
    __syncthreads();
    const int64_t chunks = (int64_t)pfx[p.B] * p.Hkv;
    const int64_t T = (int64_t)p.table_stride << p.lbs;
    const int SR = kOne && kSR > 0 ? kSR : p.rows_per_slot, subs = kOne ? 1 : (SR + kSub - 1) / kSub, mask = (1 << p.lbs) - 1;
    const int steps = (p.q_len + p.qp - 1) / p.qp * subs;  // a step: kSub rows, from sub_of on, of launch row step / subs
    bool waited = false;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        int lo = 0, hi = p.B - 1;  // the largest b with pfx[b] * Hkv <= c
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)pfx[mid] * p.Hkv <= c) lo = mid; else hi = mid - 1;
        }
        const int b = lo, n = pfx[b + 1] - pfx[b];
        const int rem = (int)(c - (int64_t)pfx[b] * p.Hkv);
        const int kvh = rem / n, t0 = (rem - kvh * n) * kChunk + tid;  // this thread's tokens: t0 + k kThreads
        const int32_t raw = p.lens[b], len = tokens(b);
        const int32_t* ids = p.table + (int64_t)b * p.table_stride;
        int32_t id[kTok];
        float4 v[kTok][kSR > 0 ? kSR / 4 : 1];
        float w[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int t = t0 + k * kThreads;
            id[k] = t < len ? ids[t >> p.lbs] : -1;
            w[k] = 0.f;
        }
        auto sub_of = [&](int e) { return kOne ? 0 : e % subs * kSub; };
        auto row_of = [&](int e) { return kOne ? e : e / subs; };
        auto scores_of = [&](int e) {
            return p.scores + ((((int64_t)row_of(e) * p.B + b) * p.Hkv + kvh) * T + t0) * SR + sub_of(e);
        };
        auto queries_of = [&](int r) { return min(p.qp, p.q_len - r * p.qp); };
        auto rows_of = [&](int e) { return min(kSub, queries_of(row_of(e)) * p.G - sub_of(e)); };  // (may be none)
        auto seen_of = [&](int e) { return min(len, raw - p.q_len + row_of(e) * p.qp + queries_of(row_of(e))); };  // by the launch row
        auto fetch = [&](int r) {
            if (tid < rows_of(r)) {
                const float2 z = __ldcg(reinterpret_cast<const float2*>(p.row_ml) +
                                        ((int64_t)b * p.q_len + row_of(r) * p.qp + (sub_of(r) + tid) / p.G) * p.Hq +
                                        kvh * p.G + (sub_of(r) + tid) % p.G);
                // (a query that sees nothing has scores of -inf only: weights of 0)
                ml[r & 1][tid] = z.y == 0.f ? make_float2(0.f, 0.f) : make_float2(-z.x, -lg2(z.y));
            }
            if constexpr (kSR > 0) {
                const float* s = scores_of(r);
                const int seen = seen_of(r);
#pragma unroll
                for (int k = 0; k < kTok; ++k)
                    if (t0 + k * kThreads < seen) {
#pragma unroll
                        for (int i = 0; i < kSR / 4; ++i) v[k][i] = __ldcs(reinterpret_cast<const float4*>(s + (int64_t)k * kThreads * SR) + i);
                    }
            }
        };
        // (loads in the order of what hangs on them: scores, of no id, before what lies at the ids)
        const bool first = !waited;
        if (!first) fetch(0);
        int64_t at[kTok];  // -1: no token, or a bad block id (the decode raised the flag)
        float old[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            at[k] = id[k] >= 0 && id[k] < p.num_blocks ? (((int64_t)id[k] * p.Hkv + kvh) << p.lbs) + ((t0 + k * kThreads) & mask) : -1;
            old[k] = at[k] >= 0 && p.in && t0 + k * kThreads < raw - p.q_len ? __ldcg(p.in + at[k]) : 0.f;
        }
        if (first) {
            pdl_wait_primary();
            pdl_launch_dependents();
            waited = true;
            fetch(0);
        }
        for (int r = 0; r < steps; ++r) {
            if (r > 0) fetch(r);
            const int rows = rows_of(r), seen = seen_of(r);
            __syncthreads();  // (the other half of ml is read until the next row's barrier)
            if constexpr (kSR > 0) {
                float2 sum[kTok];
#pragma unroll
                for (int k = 0; k < kTok; ++k) sum[k] = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kSR; i += 2) {
                    const float4 z = *reinterpret_cast<const float4*>(&ml[r & 1][i]);
                    const bool both = i + 1 < rows;
                    if (i < rows) {
#pragma unroll
                        for (int k = 0; k < kTok; ++k) {
                            const float4 f = v[k][i / 4];
                            float2 y = i % 4 == 0 ? make_float2(f.x, f.y) : make_float2(f.z, f.w);
                            y = __fadd2_rn(__fadd2_rn(y, make_float2(z.x, z.z)), make_float2(z.y, z.w));
                            sum[k] = __fadd2_rn(sum[k], make_float2(ex2(y.x), both ? ex2(y.y) : 0.f));
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kTok; ++k)
                    if (t0 + k * kThreads < seen) {
                        float x = sum[k].x + sum[k].y;
                        if (x != x) {  // rare: -inf plus a NaN sum's logarithm is NaN (again in the same order)
                            float even = 0.f, odd = 0.f;
                            const float* s = scores_of(r) + (int64_t)k * kThreads * SR;
#pragma unroll 1
                            for (int i = 0; i < rows; i += 2) {
                                even += weight(__ldcs(s + i), ml[r & 1][i]);
                                if (i + 1 < rows) odd += weight(__ldcs(s + i + 1), ml[r & 1][i + 1]);
                            }
                            x = even + odd;
                        }
                        w[k] += x;
                    }
            } else {
                const float* s = scores_of(r);
                float sum[kTok];
#pragma unroll
                for (int k = 0; k < kTok; ++k) sum[k] = 0.f;
                for (int i = 0; i < rows; ++i) {
                    const float2 z = ml[r & 1][i];
#pragma unroll
                    for (int k = 0; k < kTok; ++k)
                        if (t0 + k * kThreads < seen) sum[k] += weight(s[(int64_t)k * kThreads * SR + i], z);
                }
#pragma unroll
                for (int k = 0; k < kTok; ++k) w[k] += sum[k];
            }
        }
        // summed apart from the old sum, whose last place may be above a weight's first
#pragma unroll
        for (int k = 0; k < kTok; ++k)
            if (at[k] >= 0) p.out[at[k]] = old[k] + w[k];
        if (steps & 1) __syncthreads();  // the next chunk's first row takes the half that the last one reads
    }
    if (!waited) {
        pdl_wait_primary();
        pdl_launch_dependents();
    }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const int64_t most = (int64_t)p.B * p.Hkv * chunks_of((int32_t)((int64_t)p.table_stride << p.lbs));
    const cudaLaunchConfig_t cfg = pdl_config((int)(most < sms * kCtas ? most : sms * kCtas), kThreads, stream, &attr);
    const int SR = p.rows_per_slot;
    const auto kernel = SR == 8       ? weights_kernel<8, true>
                        : SR == 4     ? weights_kernel<4, true>
                        : SR < 8      ? weights_kernel<0, true>
                        : SR % 8 == 0 ? weights_kernel<8, false>
                        : SR % 4 == 0 ? weights_kernel<4, false> : weights_kernel<0, false>;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---- joining a shared prefix
//
// out = o / l of the prefix's pieces and the state of the sequence's own tokens.
// A thread takes four columns of an output row and, where rows are few, every
// kJ-th piece, eight of them a round trip; a prefix that fills the GPU leaves about
// 152 / units pieces.  Whole calls behind 8192 tokens, 8 kv heads of 128, with a CTA a
// row and a row a thread's columns: 1024 rows 34.1 and 36.6 us, 1536 46.1 and 46.7, 2048
// 52.4 and 51.8, 4096 74.5 and 69.5; 4 kv heads of 64 in e4m3 34.1 and 37.7, 42.1 and
// 42.8, 45.1 and 44.5, 69.9 and 61.7.
// (In the split kernel's segment ends instead, it cost that kernel its registers:
// 32 sequences of 4096 tokens without any prefix 89 us for 81.)

namespace {

__device__ __forceinline__ void join(float& M, float& L, float4& O, float m, float l, const float4& o) {
    const float t = fmaxf(M, m);
    if (t == __int_as_float(0xff800000)) return;  // both empty
    // references may lie further apart than fp32's exponents reach, and the sums still matter
    const float fa = ex2(M - t), fb = ex2(m - t), ha = ex2(0.5f * (M - t)), hb = ex2(0.5f * (m - t));
    L = L * ha * ha + l * hb * hb;
    O.x = O.x * fa + o.x * fb;
    O.y = O.y * fa + o.y * fb;
    O.z = O.z * fa + o.z * fb;
    O.w = O.w * fa + o.w * fb;
    M = t;
}

template <int D, int THREADS, int kJ>
__global__ void __launch_bounds__(THREADS) join_kernel(const JoinParams p) {
    constexpr int kC = D / 4, kIn = kJ > 1 ? 8 : 16;  // threads of a row's columns; pieces in flight
    __shared__ float4 others[kJ][kC];
    __shared__ float2 other_ml[kJ][kC];
    pdl_wait_primary();
    pdl_launch_dependents();
    static_assert(kJ == 1 || THREADS == kC * kJ, "a row a CTA, or a row a thread's columns");
    const int64_t row = kJ > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (THREADS / kC) + threadIdx.x / kC;
    const int c = threadIdx.x % kC, part = kJ > 1 ? threadIdx.x / kC : 0;
    if (kJ == 1 && row >= p.rows) return;
    const int per = p.q_len * p.Hq, b = (int)(row / per), in = (int)(row - (int64_t)b * per), qi = in / p.Hq, head = in - qi * p.Hq;
    // (from L2 all: the CTA may have come to its SM before they were written)
    const int4 lo = __ldcg(reinterpret_cast<const int4*>(p.seqs + b)), hi = __ldcg(reinterpret_cast<const int4*>(p.seqs + b) + 1);
    const PrefixSeq s = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float M = __int_as_float(0xff800000), L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part == 0) {
        const float2 own = __ldcg(reinterpret_cast<const float2*>(p.row_ml) + row);
        O = __ldcg(reinterpret_cast<const float4*>(p.row_o) + row * kC + c);
        M = own.x;
        L = own.y;
    }
    if (s.tiles > 0) {
        constexpr int kSub = prefix_streams(D);  // q tiles of a slot
        const int kvh = head / p.G, r = ((b - s.start) * p.q_len + qi) * p.G + head - kvh * p.G, tile = r >> 7;
        const int unit = tile / kSub * p.Hkv + kvh;
        const int64_t first = s.work + (int64_t)unit * s.tiles;
        const int c0 = (int)cta_of_block(first, s.total, s.ctas), n = (int)cta_of_block(first + s.tiles - 1, s.total, s.ctas) - c0 + 1;
        const int64_t at = (((int64_t)s.unit + unit + c0) * kSub + tile % kSub) * 128 + (r & 127);
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at;
        constexpr int kPieces = prefix_slab(D) / 4;  // 16-byte pieces of a row in a slab, XORed with the row
        const float4* po = reinterpret_cast<const float4*>(p.part_o) + (at - (r & 127)) * kC +
                           (c / kPieces * 128 + (r & 127)) * kPieces + (c % kPieces ^ (r & 7));
        for (int k0 = part; k0 < n; k0 += kIn * kJ) {
            float2 si[kIn];
            float4 oi[kIn];
#pragma unroll
            for (int k = 0; k < kIn; ++k) {
                si[k] = make_float2(__int_as_float(0xff800000), 0.f);
                oi[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k * kJ < n) {
                    si[k] = __ldcg(ml + (int64_t)(k0 + k * kJ) * kSub * 128);
                    oi[k] = __ldcg(po + (int64_t)(k0 + k * kJ) * kSub * 128 * kC);
                }
            }
#pragma unroll
            for (int k = 0; k < kIn; ++k) join(M, L, O, si[k].x, si[k].y, oi[k]);
        }
        if (kJ > 1 && part > 0) {
            others[part][c] = O;
            other_ml[part][c] = make_float2(M, L);
        }
        if (kJ > 1) __syncthreads();
        if (part == 0)
            for (int k = 1; k < kJ; ++k) join(M, L, O, other_ml[k][c].x, other_ml[k][c].y, others[k][c]);
    }
    if (part > 0) return;
    // (a NaN sum gives NaN, no sum 0)
    const float4 v = L != 0.f ? make_float4(O.x / L, O.y / L, O.z / L, O.w / L) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.out_f32) reinterpret_cast<float4*>(p.out_f32)[row * kC + c] = v;
    else reinterpret_cast<uint2*>(p.out)[row * kC + c] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

}  // namespace

template <int D>
cudaError_t launch_join_as(const JoinParams& p, cudaStream_t stream) {
    constexpr int kC = D / 4, kT = 128;
    const bool few = p.rows < 2048;
    const int64_t grid = few ? p.rows : (p.rows * kC + 127) / 128;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config((int)grid, few ? kT : 128, stream, &attr);
    return cudaLaunchKernelEx(&cfg, few ? join_kernel<D, kT, kT / kC> : join_kernel<D, 128, 1>, p);
}

cudaError_t launch_join(int D, const JoinParams& p, cudaStream_t stream) {
    return D == 64 ? launch_join_as<64>(p, stream) : D == 128 ? launch_join_as<128>(p, stream) : launch_join_as<256>(p, stream);
}

}  // namespace pda
