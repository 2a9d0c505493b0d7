// pda_quant.cu -- decode over an 8-bit cache: one CTA per (query row, q head),
// its warps striding over the tokens with an online softmax each, merged in
// shared memory.
#include <cuda_fp16.h>

#include "pda_kernels.cuh"
#include "pda_quant.h"

namespace pda {

constexpr int kQuantWarps = 8;

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
    if constexpr (FMT == kE4m3) {
        const uint32_t h = e4m3x2_to_f16x2((uint16_t)(c & 0xff));
        return __half2float(__low2half(*reinterpret_cast<const __half2*>(&h)));
    } else {
        return (float)(int8_t)c;
    }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kQuantWarps * 32) quant_kernel(const __grid_constant__ QuantParams p) {
    constexpr int E = D / 32;  // elements per lane
    __shared__ float sm[kQuantWarps], sl[kQuantWarps], so[kQuantWarps][D];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, row = blockIdx.y, b = row / p.q_len, i = row - b * p.q_len, kvh = h / p.G;
    int32_t len = p.c.lens[b];
    const int64_t cap = (int64_t)p.c.table_stride << p.c.lbs;
    if (len < 0 || len > cap) {
        if (threadIdx.x == 0) atomicOr(p.err, PDA_DEVERR_BAD_LENGTH_);
        len = len < 0 ? 0 : (int32_t)cap;
    }
    const int32_t n = len - p.q_len + 1 + i;  // tokens seen
    float q[E], o[E], m = kNegInf, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_lo(p.q[((int64_t)row * p.Hq + h) * D + lane * E + e]);
        o[e] = 0.f;
    }
    for (int t = warp; t < n; t += kQuantWarps) {
        int32_t blk = p.c.table[(int64_t)b * p.c.table_stride + (t >> p.c.lbs)];
        const int slot = t & ((1 << p.c.lbs) - 1);
        float ks = 0.f, vs = 0.f;
        if (blk < 0 || blk >= p.c.num_blocks) {
            if (lane == 0) atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
            blk = 0;
        } else {
            const float* s = p.c.scales + (((int64_t)blk * p.Hkv + kvh) * 2 << p.c.lbs) + slot;
            ks = s[0];
            vs = s[1 << p.c.lbs];
        }
        const int64_t off = (int64_t)blk * p.c.blk + (int64_t)slot * p.c.tok + (int64_t)kvh * p.c.kvh + lane * E;
        float s = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s += q[e] * code_value<FMT>(p.c.k[off + e]);
            v[e] = code_value<FMT>(p.c.v[off + e]) * vs;
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= ks * p.scale_log2;
        const float mn = fmaxf(m, s), f = m == kNegInf ? 0.f : ex2(m - mn), w = ex2(s - mn);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * v[e];
        m = mn;
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    float M = kNegInf;
    for (int w = 0; w < kQuantWarps; ++w) M = fmaxf(M, sm[w]);
    for (int d = threadIdx.x; d < D; d += kQuantWarps * 32) {
        float L = 0.f, O = 0.f;
        for (int w = 0; w < kQuantWarps; ++w) {
            const float f = sm[w] == kNegInf ? 0.f : ex2(sm[w] - M);
            L += sl[w] * f;
            O += so[w][d] * f;
        }
        const float r = L != 0.f ? O / L : 0.f;
        const int64_t at = ((int64_t)row * p.Hq + h) * D + d;
        if (p.out_f32) static_cast<float*>(p.out)[at] = r;
        else static_cast<uint16_t*>(p.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
    }
}

cudaError_t launch_quant(int D, int format, const QuantParams& p, cudaStream_t stream) {
    const dim3 grid(p.Hq, p.c.B * p.q_len);
    const int threads = kQuantWarps * 32;
#define PDA_QUANT_CASE(DD)                                                                   \
    if (D == DD) {                                                                           \
        if (format == kE4m3) quant_kernel<DD, kE4m3><<<grid, threads, 0, stream>>>(p);       \
        else quant_kernel<DD, kInt8><<<grid, threads, 0, stream>>>(p);                       \
        return cudaGetLastError();                                                           \
    }
    PDA_QUANT_CASE(64)
    PDA_QUANT_CASE(128)
    PDA_QUANT_CASE(256)
#undef PDA_QUANT_CASE
    return cudaErrorInvalidValue;
}

}  // namespace pda
