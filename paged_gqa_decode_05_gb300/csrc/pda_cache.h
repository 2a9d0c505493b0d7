// pda_cache.h -- parameter blocks and launch entry points of the kernels
// around the decode (pda_cache.cu): norm and rotation of q / k heads, the
// cache write, the cache read-back.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pda {

// One byte of cache format in the kernels: none (no cache behind the call) or
// PDA_CACHE_*.
enum CacheFormat : int { kNoCache = -1, kBf16 = 0, kE4m3 = 1, kInt8 = 2 };

// The cache and the sequences that index it.
struct CacheRef {
    uint8_t* k;
    uint8_t* v;
    float* scales;            // [num_blocks, Hkv, 2, bs]; null for bf16
    int64_t num_blocks;
    int64_t blk, tok, kvh;    // strides in elements
    const int32_t* table;     // [B, table_stride]
    int32_t table_stride;
    int32_t lbs;              // log2(block size)
    const int32_t* lens;      // [B]
    const int32_t* starts;    // [B + 1] or null: rows_each rows per sequence
    int64_t rows_each;
    int32_t B;
};

struct Heads {
    uint16_t* p;              // bf16 [tokens, heads, D]; null: none
    int64_t tok, head;        // strides in elements
};

struct HeadsParams {
    Heads q, k, v, q_out, k_out;
    const void* q_weight;     // [D] bf16, or fp32 when weights_f32; null: no norm
    const void* k_weight;
    const float* cos_sin;     // [max_pos, rotary] fp32; null: no rotation
    const int32_t* positions; // [T] or null: the token's index in its sequence
    CacheRef c;
    int64_t T;                // tokens
    int32_t Hq, Hkv;
    int32_t weights_f32;
    float eps;
    int32_t max_pos, rotary, interleaved;
    int32_t sms;
    int32_t slots;            // of the ring (set at launch)
    int32_t team_warps;  // warps that share a slot
    uint32_t* err;
};

struct ReadParams {
    CacheRef c;
    void* k_out;              // [rows, Hkv, D] bf16 or fp32; null: none
    void* v_out;
    int64_t rows;
    int32_t Hkv;
    uint32_t* err;
};

// Launch attributes for a head size on the current device.
cudaError_t heads_setup(int D);
// format kNoCache: norm_rope (outputs q_out, k_out); otherwise append.
cudaError_t launch_heads(int D, int format, const HeadsParams& p, cudaStream_t stream);
cudaError_t launch_read(int D, int format, bool out_f32, const ReadParams& p, cudaStream_t stream);

}  // namespace pda
