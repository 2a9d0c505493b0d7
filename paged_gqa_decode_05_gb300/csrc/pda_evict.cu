// pda_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// choose_kernel: a CTA per (sequence, kv head).  The tokens between the first
// and the last ones that stay anyway are ranked by their sums as 32-bit keys of
// the same order; the key of the last one to stay is found digit by digit, 11
// bits each from the highest in which the keys differ, from histograms in shared
// memory, until the keys that are left are few enough to compare each with all.
// Sums of one size differ late, so that one digit leaves a few where the exponent
// alone would leave hundreds.  Ties go to the lowest index: warps own consecutive runs of tokens
// and count theirs before they write.
//
// move_kernel: rows to other blocks, in any order.  pack_kernel: rows to the
// front of their own blocks.  There token kept[i] moves to i <= kept[i], so a
// source is never behind its destination: a CTA that takes a unit's rows in
// order may read as far ahead as it likes and overwrites only what it, or an
// earlier step of its own, has read.  K and V, and parts of their rows, are
// independent of each other, which is where its CTAs come from.
#include "pda_evict.h"
#include "pda_params.h"
#include "pda_ptx.cuh"

namespace pda {

namespace {

constexpr uint32_t kBadBlock = 0x1u, kBadLength = 0x2u;
constexpr int kDigit = 11, kBins = 1 << kDigit, kFew = 128;
constexpr uint32_t kForced = 0xffffffffu;

struct Unit {
    int b, kvh;
    int32_t n, m;  // tokens, tokens that stay
    bool bad;
};
__device__ __forceinline__ Unit unit_of(const EvictParams& p, int64_t u) {
    Unit r;
    r.b = (int)(u / p.Hkv);
    r.kvh = (int)(u - (int64_t)r.b * p.Hkv);
    const int32_t len = p.lens[r.b];
    const int64_t most = (int64_t)p.table_stride << p.lbs;
    r.bad = len < 0 || len > most;
    r.n = (int32_t)min((int64_t)max(len, 0), most);
    r.m = min(r.n, p.keep);
    return r;
}

// A sum as a key of the same order: NaN the largest but for tokens that stay anyway, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xfffffffeu;
    const uint32_t x = __float_as_uint(w + 0.f);
    return (x & 0x80000000u) ? ~x : x | 0x80000000u;
}

// The slot of token t, in block `id`: block * bs + place in the block, or -1 (a bad block id).
__device__ __forceinline__ int64_t slot_of(const EvictParams& p, int32_t id, int32_t t) {
    if (id < 0 || (int64_t)id >= p.num_blocks) {
        atomicOr(p.err, kBadBlock);
        return -1;
    }
    return ((int64_t)id << p.lbs) + (t & ((1 << p.lbs) - 1));
}
__device__ __forceinline__ int64_t weight_at(const EvictParams& p, int64_t slot, int kvh) {
    return ((((slot >> p.lbs) * p.Hkv) + kvh) << p.lbs) + (slot & ((1 << p.lbs) - 1));
}
__device__ __forceinline__ int64_t scale_at(const EvictParams& p, int64_t slot, int kvh, int which) {
    return (((((slot >> p.lbs) * p.Hkv) + kvh) * 2 + which) << p.lbs) + (slot & ((1 << p.lbs) - 1));
}
__device__ __forceinline__ int64_t row_at(const EvictParams& p, int64_t slot, int kvh) {
    return (slot >> p.lbs) * p.blk + (slot & ((1 << p.lbs) - 1)) * p.tok + kvh * p.kvh;
}

__device__ __forceinline__ int warp_sums(int x) {  // of the lanes up to this one
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The sum over the block's threads before this one.  `sums` holds a word per warp.
template <int THREADS>
__device__ __forceinline__ int block_before(int x, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, y = warp_sums(x);
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    const int z = warp_sums(lane < THREADS / 32 ? sums[lane] : 0);
    const int before = __shfl_sync(0xffffffffu, z, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + y - x;
}

// The key of token t of a unit, from memory.  (A call where it is rare: beside the
// keys in shared memory its code would be most of what the search fetches.)
__device__ __noinline__ uint32_t far_key(const float* weights, const int32_t* row, int64_t num_blocks, int32_t lbs, int32_t Hkv,
                                         int32_t kvh, int32_t t, bool forced) {
    if (forced) return kForced;
    const int32_t id = row[t >> lbs];
    const bool bad = id < 0 || (int64_t)id >= num_blocks;  // (flagged when the keys were first read)
    return key_of(bad ? 0.f : weights[(((int64_t)id * Hkv + kvh) << lbs) + (t & ((1 << lbs) - 1))]);
}

// cached: how many keys fit behind the histogram.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) choose_kernel(const EvictParams p, int32_t cached) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kBins];
    __shared__ int sums[THREADS / 32], eqs[THREADS / 32];
    __shared__ uint32_t least[THREADS / 32], most[THREADS / 32];
    __shared__ int digit, above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int32_t* row = p.table + (int64_t)(blockIdx.x / p.Hkv) * p.table_stride;
    int32_t ids[4];  // of the first tokens, looked up beside the length
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t e = (tid + i * THREADS) >> p.lbs;
        ids[i] = e < p.table_stride ? row[e] : -1;
    }
    const Unit u = unit_of(p, blockIdx.x);
    if (tid == 0 && u.kvh == 0) {
        p.new_lens[u.b] = u.m;
        if (u.bad) atomicOr(p.err, kBadLength);
    }
    int32_t* kept = p.kept + (int64_t)blockIdx.x * p.keep;
    if (u.n <= p.keep) {
        for (int64_t i = tid; i < p.keep; i += THREADS) kept[i] = i < u.n ? (int32_t)i : -1;  // (keep may be near 2^31)
        return;
    }
    auto load_key = [&](int32_t t, int32_t id) {
        const int64_t s = slot_of(p, id, t);
        if (t < p.first || t >= u.n - p.recent) return kForced;
        return key_of(s < 0 ? 0.f : p.weights[weight_at(p, s, u.kvh)]);
    };
    for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
    uint32_t low = kForced, high = 0;  // of the keys between
    auto seen = [&](uint32_t k) {
        if (k == kForced) return;
        low = min(low, k);
        high = max(high, k);
    };
    const int32_t here = min(u.n, cached);
    for (int32_t t = tid; t < here; t += 4 * THREADS) {  // four loads in flight
        uint32_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t >= 4 * THREADS && t + i * THREADS < here) ids[i] = row[(t + i * THREADS) >> p.lbs];
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = t + i * THREADS < here ? load_key(t + i * THREADS, ids[i]) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i * THREADS < here) {
                keys[t + i * THREADS] = k[i];
                seen(k[i]);
            }
    }
    for (int32_t t = here + tid; t < u.n; t += THREADS) seen(load_key(t, row[t >> p.lbs]));
    auto key = [&](int32_t t) {
        return t < cached ? keys[t]
                          : far_key(p.weights, row, p.num_blocks, p.lbs, p.Hkv, u.kvh, t, t < p.first || t >= u.n - p.recent);
    };
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
        least[warp] = low;
        most[warp] = high;
    }
    __syncthreads();
    low = __reduce_min_sync(0xffffffffu, least[lane % (THREADS / 32)]);
    high = __reduce_max_sync(0xffffffffu, most[lane % (THREADS / 32)]);
    // The key of the last one to stay: `prefix` but for its lowest `bits`, and
    // `left` of the keys that begin so still to take.  (None to take: the largest
    // key, of which none stays.)
    int left = p.keep - p.first - p.recent, bits = left > 0 ? 32 - __clz(low ^ high) : 0;
    uint32_t prefix = bits == 32 ? 0u : high >> bits << bits;
#pragma unroll 1
    while (bits > 0) {
        const int take = min(bits, kDigit), shift = bits - take, bins = 1 << take;
        const uint32_t mask = bits == 32 ? 0u : ~0u << bits;
        for (int32_t t0 = 0; t0 < u.n; t0 += THREADS) {
            const int32_t t = t0 + tid;
            const uint32_t k = t < u.n ? key(t) : kForced;
            const bool mine = k != kForced && (k & mask) == prefix;
            const uint32_t bin = (k >> shift) & (uint32_t)(bins - 1);
            // one addition for a warp of equal digits, which would meet on one bin otherwise
            const uint32_t bin0 = __shfl_sync(0xffffffffu, bin, 0);
            if (__all_sync(0xffffffffu, mine && bin == bin0)) {
                if (lane == 0) atomicAdd(&hist[bin], 32);
            } else if (mine) {
                atomicAdd(&hist[bin], 1);
            }
        }
        __syncthreads();
        // bins in descending order: thread i takes a run of them
        constexpr int kPer = kBins / THREADS;
        int count[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int d = bins - 1 - (tid * kPer + i);
            count[i] = d >= 0 ? hist[d] : 0;
            sum += count[i];
        }
        int before = block_before<THREADS>(sum, sums);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (before < left && left <= before + count[i]) {
                digit = bins - 1 - (tid * kPer + i);
                above = before;
            }
            before += count[i];
        }
        __syncthreads();
        prefix |= (uint32_t)digit << shift;
        left -= above;
        bits = shift;
        const int same = hist[digit];
        __syncthreads();
        if (same == left || bits == 0) break;  // all of them stay
        if (same > kFew) {
            for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
            __syncthreads();
            continue;
        }
        // Few keys: each is compared with all, by kEach threads; the one with fewer than
        // `left` above it, and as many with its equals, is the last.
        uint32_t* few = reinterpret_cast<uint32_t*>(hist);
        if (tid == 0) above = 0;
        __syncthreads();
        for (int32_t t = tid; t < u.n; t += THREADS) {
            const uint32_t k = key(t);
            if (k != kForced && k >> bits == prefix >> bits) few[atomicAdd(&above, 1)] = k;
        }
        __syncthreads();
        constexpr int kEach = THREADS / kFew;
        const int mine = tid / kEach;
        const uint32_t k = mine < same ? few[mine] : 0u;
        int more = 0, equal = 0;
        if (warp * 32 / kEach < same)  // (whole warps)
            for (int i = tid % kEach; i < same; i += kEach) {
                const uint32_t x = few[i];
                more += x > k;
                equal += x == k;
            }
#pragma unroll
        for (int o = 1; o < kEach; o <<= 1) {
            more += __shfl_xor_sync(0xffffffffu, more, o);
            equal += __shfl_xor_sync(0xffffffffu, equal, o);
        }
        if (mine < same && tid % kEach == 0 && more < left && left <= more + equal) {
            digit = (int)k;
            above = more;
        }
        __syncthreads();
        prefix = (uint32_t)digit;
        left -= above;
        break;
    }
    // Every key above `prefix` stays, and the first `left` of its own.
    const int32_t run = ((u.n + THREADS - 1) / THREADS) * 32;  // tokens of a warp
    const int32_t lo = min(u.n, warp * run), hi = min(u.n, lo + run);
    int more = 0, equal = 0;
    for (int32_t t = lo + lane; t < hi; t += 32) {
        const uint32_t k = key(t);
        more += k > prefix;
        equal += k == prefix;
    }
    more = __reduce_add_sync(0xffffffffu, more);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sums[warp] = more;
        eqs[warp] = equal;
    }
    __syncthreads();
    int at = warp_sums(lane < warp ? sums[lane] : 0), taken = warp_sums(lane < warp ? eqs[lane] : 0);
    at = __shfl_sync(0xffffffffu, at, 31);
    taken = __shfl_sync(0xffffffffu, taken, 31);
    at += min(taken, left);
    for (int32_t t0 = lo; t0 < hi; t0 += 32) {
        const int32_t t = t0 + lane;
        const uint32_t k = t < hi ? key(t) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, t < hi && k == prefix), below = (1u << lane) - 1u;
        const bool stays = t < hi && (k > prefix || (k == prefix && taken + __popc(eq & below) < left));
        const uint32_t ones = __ballot_sync(0xffffffffu, stays);
        if (stays) kept[at + __popc(ones & below)] = t;
        at += __popc(ones);
        taken += __popc(eq);
    }
}

__device__ __forceinline__ uint4 ld16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// 64 destination rows of a unit to other blocks.
constexpr int kMoveThreads = 256, kMoveRows = 64;
template <int RB>  // bytes of a row
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p, int32_t chunks) {
    constexpr int CH = 2 * RB / 16;                                // 16-byte pieces of a token: K, then V
    constexpr int N = kMoveRows * CH / kMoveThreads;               // pieces of a thread
    constexpr int U = N < 8 ? N : 8;                               // in flight
    __shared__ int64_t src[kMoveRows], dst[kMoveRows];
    // (launched behind choose_kernel, which waited for all before it: lengths and
    // tables are there, and only `kept` is waited for)
    const int64_t unit = blockIdx.x / chunks;
    const int32_t i0 = (int32_t)(blockIdx.x % chunks) * kMoveRows;
    const Unit u = unit_of(p, unit);
    const int tid = threadIdx.x;
    const int32_t i = i0 + tid;
    int64_t b = -1;
    if (tid < kMoveRows && i < u.m) b = slot_of(p, p.out_table[(int64_t)u.b * p.out_stride + (i >> p.lbs)], i);
    pdl_wait_primary();
    pdl_launch_dependents();
    if (i0 >= u.m) return;
    if (tid < kMoveRows) {
        int64_t a = -1;
        if (i < u.m) {
            const int32_t t = __ldcg(p.kept + unit * p.keep + i);
            a = slot_of(p, p.table[(int64_t)u.b * p.table_stride + (t >> p.lbs)], t);
            if (b >= 0) {
                p.weights[weight_at(p, b, u.kvh)] = a < 0 ? 0.f : p.weights[weight_at(p, a, u.kvh)];
                if (p.scales)
                    for (int w = 0; w < 2; ++w)
                        p.scales[scale_at(p, b, u.kvh, w)] = a < 0 ? 0.f : p.scales[scale_at(p, a, u.kvh, w)];
            }
        }
        src[tid] = a < 0 ? -1 : row_at(p, a, u.kvh);
        dst[tid] = b < 0 ? -1 : row_at(p, b, u.kvh);
    }
    __syncthreads();
#pragma unroll 1
    for (int k0 = 0; k0 < N; k0 += U) {
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = (k0 + k) * kMoveThreads + tid, r = e / CH, c = e % CH;
            const int64_t s = src[r];
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (s >= 0) x[k] = ld16((c < CH / 2 ? p.k : p.v) + s + (c % (CH / 2)) * 16);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = (k0 + k) * kMoveThreads + tid, r = e / CH, c = e % CH;
            const int64_t d = dst[r];
            if (d >= 0) *reinterpret_cast<uint4*>((c < CH / 2 ? p.k : p.v) + d + (c % (CH / 2)) * 16) = x[k];
        }
    }
}

// A unit's K or V rows, SB bytes of each, to the front of its blocks: steps of
// R rows in order, the next step's loads ahead of this one's stores.
constexpr int kPackThreads = 256;
template <int SB>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const EvictParams p, int32_t parts) {
    constexpr int CH = SB / 16, U = 8, R = U * kPackThreads / CH;  // pieces of a row, of a thread; rows of a step
    __shared__ int64_t src[2][R], dst[2][R];
    const int64_t unit = blockIdx.x / (2 * parts);
    const int which = (int)(blockIdx.x / parts) & 1, part = (int)(blockIdx.x % parts);
    const Unit u = unit_of(p, unit);  // (as in move_kernel)
    pdl_wait_primary();
    pdl_launch_dependents();
    if (u.n <= p.keep) return;  // nothing moves
    const int tid = threadIdx.x;
    uint8_t* pool = (which ? p.v : p.k) + part * SB;
    const int32_t* row = p.table + (int64_t)u.b * p.table_stride;
    const int32_t* kept = p.kept + unit * p.keep;
    uint4 x[2][U];
    constexpr int kF = R / kPackThreads > 0 ? R / kPackThreads : 1;  // rows whose place a thread looks up
    float w[2][kF], sc[2][kF];
    int64_t wd[2][kF], sd[2][kF];
    auto load = [&](int s, int32_t i0) {  // step s & 1
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            const int r = f * kPackThreads + tid;
            wd[s][f] = sd[s][f] = -1;
            if (r < R) {
                int64_t a = -1, b = -1;
                const int32_t i = i0 + r;
                bool moves = false;
                if (i < u.m) {
                    const int32_t t = __ldcg(kept + i);
                    moves = t != i;
                    if (moves) {
                        a = slot_of(p, row[t >> p.lbs], t);
                        b = slot_of(p, row[i >> p.lbs], i);
                    }
                }
                if (part == 0 && b >= 0) {
                    if (which == 0) {
                        wd[s][f] = weight_at(p, b, u.kvh);
                        w[s][f] = a < 0 ? 0.f : p.weights[weight_at(p, a, u.kvh)];
                    }
                    if (p.scales) {
                        sd[s][f] = scale_at(p, b, u.kvh, which);
                        sc[s][f] = a < 0 ? 0.f : p.scales[scale_at(p, a, u.kvh, which)];
                    }
                }
                src[s][r] = a < 0 ? -1 : row_at(p, a, u.kvh);
                dst[s][r] = b < 0 ? -1 : row_at(p, b, u.kvh);
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = k * kPackThreads + tid, r = e / CH, c = e % CH;
            x[s][k] = make_uint4(0u, 0u, 0u, 0u);
            if (src[s][r] >= 0) x[s][k] = ld16(pool + src[s][r] + c * 16);
        }
    };
    auto store = [&](int s) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = k * kPackThreads + tid, r = e / CH, c = e % CH;
            if (dst[s][r] >= 0) *reinterpret_cast<uint4*>(pool + dst[s][r] + c * 16) = x[s][k];
        }
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            if (wd[s][f] >= 0) p.weights[wd[s][f]] = w[s][f];
            if (sd[s][f] >= 0) p.scales[sd[s][f]] = sc[s][f];
        }
    };
    load(0, 0);
#pragma unroll 1
    for (int32_t i0 = 0; i0 < u.m; i0 += 2 * R) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t i = i0 + s * R;
            if (i >= u.m) break;
            if (i + R < u.m) load(s ^ 1, i + R);  // (its barrier, or the one below, orders every load of this step before its stores)
            else __syncthreads();
            store(s);
            __syncthreads();
        }
    }
}

template <class K, class... Args>
cudaError_t launch(K kernel, int64_t grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
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
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMostKeys = 49152;  // 192 KB of keys beside the histogram

}  // namespace

cudaError_t evict_setup() {
    return cudaFuncSetAttribute(choose_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    const int64_t units = (int64_t)p.B * p.Hkv, tokens = (int64_t)p.table_stride << p.lbs;
    cudaError_t e;
    // threads for 4 tokens each, up to 1024.  Whole calls with 256 and with 1024 threads:
    // 256 units of 4096 tokens 114.6 and 98.5 us, 512 of 1000 55.4 and 58.3, 32 of 500
    // 7.65 and 7.95
    if (tokens <= 1024) e = launch(choose_kernel<256>, units, 256, (size_t)tokens * 4, stream, p, (int32_t)tokens);
    else {
        const int32_t cached = (int32_t)(tokens < kMostKeys ? tokens : kMostKeys);
        e = launch(choose_kernel<1024>, units, 1024, (size_t)cached * 4, stream, p, cached);
    }
    if (e != cudaSuccess) return e;
    if (!p.in_place) {
        const int32_t most = (int32_t)(tokens < p.keep ? tokens : p.keep), chunks = (most + kMoveRows - 1) / kMoveRows;
        switch (p.row_bytes) {
            case 64: return launch(move_kernel<64>, units * chunks, kMoveThreads, 0, stream, p, chunks);
            case 128: return launch(move_kernel<128>, units * chunks, kMoveThreads, 0, stream, p, chunks);
            case 256: return launch(move_kernel<256>, units * chunks, kMoveThreads, 0, stream, p, chunks);
            case 512: return launch(move_kernel<512>, units * chunks, kMoveThreads, 0, stream, p, chunks);
            default: return cudaErrorInvalidValue;
        }
    }
    // 128-byte parts of rows (a step then takes 128 rows), or of 64 bytes where CTAs are few
    const int32_t row = p.row_bytes < 128 ? p.row_bytes : 128;
    const int32_t part = units * 2 * (p.row_bytes / row) >= 2 * p.sms ? row : 64, parts = p.row_bytes / part;
    switch (part) {
        case 64: return launch(pack_kernel<64>, units * 2 * parts, kPackThreads, 0, stream, p, parts);
        case 128: return launch(pack_kernel<128>, units * 2 * parts, kPackThreads, 0, stream, p, parts);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pda
