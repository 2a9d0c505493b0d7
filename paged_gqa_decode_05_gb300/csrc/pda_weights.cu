// pda_weights.cu -- the sums of attention weights beside a cache, and the
// head-size dispatch of the kScored and shared-prefix kernels.
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

#define PDA_DECLARE_SCORED(D)                                                   \
    ScoredShape scored_shape_d##D(int st, int format, bool fine);               \
    cudaError_t launch_scored_d##D(int st, int format, bool fine, const QuantParams& p, int grid, size_t smem, \
                                   cudaStream_t stream);
PDA_DECLARE_SCORED(64)
PDA_DECLARE_SCORED(128)
PDA_DECLARE_SCORED(256)

ScoredShape scored_shape(int D, int st, int format, bool fine) {
    switch (D) {
        case 64: return scored_shape_d64(st, format, fine);
        case 128: return scored_shape_d128(st, format, fine);
        case 256: return scored_shape_d256(st, format, fine);
        default: return {};
    }
}

cudaError_t launch_scored(int D, int st, int format, bool fine, const QuantParams& p, int grid, size_t smem,
                          cudaStream_t stream) {
    switch (D) {
        case 64: return launch_scored_d64(st, format, fine, p, grid, smem, stream);
        case 128: return launch_scored_d128(st, format, fine, p, grid, smem, stream);
        case 256: return launch_scored_d256(st, format, fine, p, grid, smem, stream);
        default: return cudaErrorInvalidValue;
    }
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

constexpr int kThreads = 256;  // tokens of a chunk: one (sequence, kv head)'s

__global__ void __launch_bounds__(kThreads) weights_kernel(const WeightsParams p) {
    __shared__ int32_t pfx[kMaxLaunchBatch + 1];  // chunks before each sequence, one kv head
    __shared__ int32_t sums[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int32_t most = (int32_t)min((int64_t)p.table_stride << p.lbs, (int64_t)0x7fffffff);
    auto tokens = [&](int b) { return min(max(p.lens[b], 0), most); };
    constexpr int kPer = kMaxLaunchBatch / kThreads;
    const int per = (p.B + kThreads - 1) / kThreads;  // <= kPer
    int32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (k < per && tid * per + k < p.B) mine += (int32_t)(((int64_t)tokens(tid * per + k) + kThreads - 1) / kThreads);
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
            run += (int32_t)(((int64_t)tokens(b) + kThreads - 1) / kThreads);
            if (b == p.B - 1) pfx[p.B] = run;
        }
    }
    __syncthreads();
    const int64_t chunks = (int64_t)pfx[p.B] * p.Hkv;
    const int64_t T = (int64_t)p.table_stride << p.lbs;
    const int Qr = (p.q_len + p.qp - 1) / p.qp;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        int lo = 0, hi = p.B - 1;  // the largest b with pfx[b] * Hkv <= c
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)pfx[mid] * p.Hkv <= c) lo = mid; else hi = mid - 1;
        }
        const int b = lo, n = pfx[b + 1] - pfx[b];
        const int64_t rem = c - (int64_t)pfx[b] * p.Hkv;
        const int kvh = (int)(rem / n);
        const int64_t t = (rem - (int64_t)kvh * n) * kThreads + tid;
        const int32_t raw = p.lens[b], len = tokens(b);
        if (t >= len) continue;
        const int32_t id = p.table[(int64_t)b * p.table_stride + (t >> p.lbs)];
        const bool good = id >= 0 && id < p.num_blocks;  // the decode raised the flag
        const int64_t at = (((int64_t)id * p.Hkv + kvh) << p.lbs) + (t & ((1 << p.lbs) - 1));
        const float old = good && p.in && t < (int64_t)raw - p.q_len ? p.in[at] : 0.f;
        float w = 0.f;  // summed apart from the old sum, whose last place may be above a weight's first
        for (int r = 0; r < Qr; ++r) {
            const int first = r * p.qp, cnt = min(p.qp, p.q_len - first);
            if (t >= (int64_t)raw - p.q_len + first + cnt) continue;  // past what the launch row's queries see
            const float* s = p.scores + ((((int64_t)r * p.B + b) * p.Hkv + kvh) * T + t) * p.rows_per_slot;
            const float2* ml = reinterpret_cast<const float2*>(p.row_ml) + ((int64_t)b * p.q_len + first) * p.Hq + kvh * p.G;
            auto add = [&](int col, float score) {
                const float2 z = __ldg(ml + (int64_t)(col / p.G) * p.Hq + col % p.G);
                if (score != __int_as_float(0xff800000)) w += ex2((score - z.x) - lg2(z.y));
            };
            if ((p.rows_per_slot & 3) == 0) {
                for (int i = 0; i < cnt * p.G; i += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(s + i);
                    add(i, v.x);
                    if (i + 1 < cnt * p.G) add(i + 1, v.y);
                    if (i + 2 < cnt * p.G) add(i + 2, v.z);
                    if (i + 3 < cnt * p.G) add(i + 3, v.w);
                }
            } else {
                for (int i = 0; i < cnt * p.G; ++i) add(i, s[i]);
            }
        }
        if (good) p.out[at] = old + w;
    }
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms * 8), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_kernel, p);
}

}  // namespace pda
