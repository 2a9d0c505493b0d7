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
constexpr int kHeadsThreads = 256;

// The sequence that owns row t: the largest b in [0, B) with starts[b] <= t.
// Warp-wide: the lanes fetch 32 evenly spaced entries at once and search them
// with shuffles, so up to 32 sequences cost one round trip; a longer list
// leaves a span of B / 32 entries for a serial search.
__device__ __forceinline__ int32_t find_seq(const int32_t* starts, int32_t B, int64_t t, int lane) {
    const int32_t step = (B + 31) / 32;
    const int32_t at = lane * step;
    const int32_t v = at < B ? starts[at] : 0x7fffffff;
    int32_t i = 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const int32_t x = __shfl_sync(0xffffffffu, v, i + w);
        if (x <= t && (i + w) * step < B) i += w;
    }
    int32_t lo = i * step, hi = min(lo + step, B) - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A row's 8 elements of this lane, as two runs a, b of four.
struct Eight {
    float a[4], b[4];
};

__device__ __forceinline__ Eight unpack(uint2 a, uint2 b) {
    Eight x;
    x.a[0] = bf16_lo(a.x); x.a[1] = bf16_hi(a.x); x.a[2] = bf16_lo(a.y); x.a[3] = bf16_hi(a.y);
    x.b[0] = bf16_lo(b.x); x.b[1] = bf16_hi(b.x); x.b[2] = bf16_lo(b.y); x.b[3] = bf16_hi(b.y);
    return x;
}

__device__ __forceinline__ uint2 pack4(const float (&x)[4]) {
    return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, float (&out)[4]) {
    if (f32) {
        const float2 x = reinterpret_cast<const float2*>(w)[2 * c], y = reinterpret_cast<const float2*>(w)[2 * c + 1];
        out[0] = x.x; out[1] = x.y; out[2] = y.x; out[3] = y.y;
    } else {
        const uint2 x = reinterpret_cast<const uint2*>(w)[c];
        out[0] = bf16_lo(x.x); out[1] = bf16_hi(x.x); out[2] = bf16_lo(x.y); out[3] = bf16_hi(x.y);
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

template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float inv) {
    if constexpr (FMT == kE4m3) {
        return pack_e4m3x2(x[0] * inv, x[1] * inv) | (pack_e4m3x2(x[2] * inv, x[3] * inv) << 16);
    } else {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = max(-127, min(127, __float2int_rn(x[i] * inv)));
            r |= (uint32_t)(c & 0xff) << (8 * i);
        }
        return r;
    }
}

// Norm, rotation and cache write.  D / 8 lanes share a row; a lane holds two
// runs of four columns, chosen so that it owns both halves of its four
// rotation pairs (columns 4l.. and rotary/2 + 4l.. when the pairs are half a
// rotation apart), so the rotation moves nothing between lanes and a lane
// reads four cosines and four sines.  A group of lanes takes HC rows of one
// token: their loads are in flight together, and the token's sequence, block
// and rotation are looked up once for them.
template <int D, int FMT, int HC>
__global__ void __launch_bounds__(kHeadsThreads) heads_kernel(const __grid_constant__ HeadsParams p) {
    constexpr int TPR = D / 8;
    const int lane = threadIdx.x & 31, l = threadIdx.x % TPR;
    const uint32_t gmask = TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1u) << (lane & ~(TPR - 1));
    const int nq = p.q.p ? p.Hq : 0, nk = p.k.p ? p.Hkv : 0, nv = FMT != kNoCache ? p.Hkv : 0;
    const int rows = nq + nk + nv;
    const int chunks = (rows + HC - 1) / HC;
    const int64_t item = (int64_t)blockIdx.x * (kHeadsThreads / TPR) + threadIdx.x / TPR;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t t = div_floor(item, chunks);
    const bool in = t < p.T;
    const int r0 = (int)(item - t * chunks) * HC;

    // columns of the two runs
    const int rl = p.rotary >> 3;  // lanes that rotate
    const bool turn = p.cos_sin != nullptr && l < rl;
    const int c0 = p.interleaved || l >= rl || !p.cos_sin ? 2 * l : l;  // past the rotation: 2 rl + 2 (l - rl)
    const int c1 = p.interleaved || l >= rl || !p.cos_sin ? c0 + 1 : l + rl;

    uint2 xa[HC], xb[HC];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const int r = r0 + i;
        if (in && r < rows) {
            const uint16_t* s = r < nq ? p.q.p + t * p.q.tok + r * p.q.head
                              : r < nq + nk ? p.k.p + t * p.k.tok + (r - nq) * p.k.head
                                            : p.v.p + t * p.v.tok + (r - nq - nk) * p.v.head;
            xa[i] = *reinterpret_cast<const uint2*>(s + 4 * c0);
            xb[i] = *reinterpret_cast<const uint2*>(s + 4 * c1);
        }
    }

    // the token's place
    int32_t pos = 0;
    bool live = in;
    int64_t slot_off = 0;
    int32_t blk = 0, slot = 0;
    bool write = false;
    if constexpr (FMT != kNoCache) {
        int32_t b;
        int64_t end;
        if (p.c.starts) {
            b = find_seq(p.c.starts, p.c.B, t, lane);
            end = p.c.starts[b + 1];
            live = live && t < end && t >= p.c.starts[0];
        } else {
            b = (int32_t)(in ? div_floor(t, p.c.rows_each) : 0);
            end = (b + 1) * p.c.rows_each;
        }
        const int64_t at = (int64_t)p.c.lens[b] - end + t;
        live = live && at >= 0;
        pos = (int32_t)at;
        const int64_t j = at >> p.c.lbs;
        slot = pos & ((1 << p.c.lbs) - 1);
        if (live && r0 + HC > nq) {
            bool bad = j >= p.c.table_stride;
            if (bad) {
                if (l == 0) atomicOr(p.err, PDA_DEVERR_BAD_POSITION_);
            } else {
                blk = p.c.table[(int64_t)b * p.c.table_stride + j];
                bad = blk < 0 || blk >= p.c.num_blocks;
                if (bad && l == 0) atomicOr(p.err, PDA_DEVERR_BAD_BLOCK_ID_);
            }
            write = !bad;
            slot_off = (int64_t)blk * p.c.blk + (int64_t)slot * p.c.tok;
        }
    }
    if (!live) return;
    float cs[4], sn[4];
    if (p.cos_sin) {
        if (p.positions) pos = p.positions[t];
        if (pos < 0 || pos >= p.max_pos) {
            if (l == 0) atomicOr(p.err, PDA_DEVERR_BAD_POSITION_);
            pos = pos < 0 ? 0 : p.max_pos - 1;
        }
        if (turn) {
            const float* row = p.cos_sin + (int64_t)pos * p.rotary + 4 * l;
            const float4 c = *reinterpret_cast<const float4*>(row);
            const float4 s = *reinterpret_cast<const float4*>(row + p.rotary / 2);
            cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
            sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        }
    }
    // `x`: this lane's part of a q or k head
    auto prepare = [&](Eight& x, const void* weight) {
        if (weight) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) ss += x.a[e] * x.a[e] + x.b[e] * x.b[e];
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(gmask, ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
            float wa[4], wb[4];
            load_weight(weight, p.weights_f32 != 0, c0, wa);
            load_weight(weight, p.weights_f32 != 0, c1, wb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x.a[e] = x.a[e] * inv * wa[e];
                x.b[e] = x.b[e] * inv * wb[e];
            }
        }
        if (!turn) return;
        if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float& u = e < 2 ? x.a[2 * e] : x.b[2 * e - 4];
                float& w = e < 2 ? x.a[2 * e + 1] : x.b[2 * e - 3];
                const float y = u * cs[e] - w * sn[e];
                w = w * cs[e] + u * sn[e];
                u = y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = x.a[e] * cs[e] - x.b[e] * sn[e];
                x.b[e] = x.b[e] * cs[e] + x.a[e] * sn[e];
                x.a[e] = y;
            }
        }
    };
    auto put_heads = [&](const Heads& h, int64_t head, const Eight& x) {
        uint16_t* d = h.p + t * h.tok + head * h.head;
        *reinterpret_cast<uint2*>(d + 4 * c0) = pack4(x.a);
        *reinterpret_cast<uint2*>(d + 4 * c1) = pack4(x.b);
    };
    // a K (which 0) or V (which 1) row of kv head `h` into its slot
    auto put_cache = [&](int which, int h, const Eight& x) {
        if constexpr (FMT == kBf16) {
            uint16_t* d = reinterpret_cast<uint16_t*>(which ? p.c.v : p.c.k) + slot_off + (int64_t)h * p.c.kvh;
            *reinterpret_cast<uint2*>(d + 4 * c0) = pack4(x.a);
            *reinterpret_cast<uint2*>(d + 4 * c1) = pack4(x.b);
        } else if constexpr (FMT != kNoCache) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = max(top, max(__float_as_uint(x.a[e]) & 0x7fffffffu, __float_as_uint(x.b[e]) & 0x7fffffffu));
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(gmask, top, o));
            float inv;
            bool keep;
            const float scale = row_scale<FMT>(top, &inv, &keep);
            uint8_t* d = (which ? p.c.v : p.c.k) + slot_off + (int64_t)h * p.c.kvh;
            *reinterpret_cast<uint32_t*>(d + 4 * c0) = keep ? codes4<FMT>(x.a, inv) : 0u;
            *reinterpret_cast<uint32_t*>(d + 4 * c1) = keep ? codes4<FMT>(x.b, inv) : 0u;
            if (l == 0) p.c.scales[((((int64_t)blk * p.Hkv + h) * 2 + which) << p.c.lbs) + slot] = scale;
        }
    };
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const int r = r0 + i;
        if (r >= rows) break;
        Eight x = unpack(xa[i], xb[i]);
        if (r < nq) {
            prepare(x, p.q_weight);
            put_heads(p.q_out, r, x);
        } else if (r < nq + nk) {
            prepare(x, p.k_weight);
            if constexpr (FMT == kNoCache) put_heads(p.k_out, r - nq, x);
            else if (write) put_cache(0, r - nq, x);
        } else {
            if (write) put_cache(1, r - nq - nk, x);
        }
    }
}

// Read-back: D / 16 lanes share a row of 16 elements each; a group takes HC
// of a token's 2 Hkv rows.
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
    int32_t b;
    int64_t begin, end;
    if (p.c.starts) {
        b = find_seq(p.c.starts, p.c.B, t, lane);
        begin = p.c.starts[b];
        end = p.c.starts[b + 1];
    } else {
        b = (int32_t)(live ? div_floor(t, p.c.rows_each) : 0);
        begin = b * p.c.rows_each;
        end = begin + p.c.rows_each;
    }
    const int64_t at = t - begin;
    live = live && at >= 0 && t < end && at < p.c.lens[b];
    if (!live) return;
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

// `items` groups of D / per_lane lanes.
template <typename P>
cudaError_t launch_rows(void (*kernel)(const P), const P& p, int64_t items, int lanes, cudaStream_t stream) {
    const int64_t grid = (items * lanes + kHeadsThreads - 1) / kHeadsThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kHeadsThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int FMT>
cudaError_t launch_heads_of(const HeadsParams& p, cudaStream_t stream) {
    const int rows = (p.q.p ? p.Hq : 0) + (p.k.p ? p.Hkv : 0) + (FMT != kNoCache ? p.Hkv : 0);
    constexpr int HC = 4;
    return launch_rows(heads_kernel<D, FMT, HC>, p, p.T * ((rows + HC - 1) / HC), D / 8, stream);
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
    constexpr int HC = 4;
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
