// pda_evict.h -- eviction: the kernels that choose the tokens a sequence keeps
// and that move their rows (pda_evict.cu).
#pragma once

#include "pda_cache.h"

namespace pda {

struct EvictParams {
    uint8_t* k;
    uint8_t* v;
    float* scales;            // [num_blocks, Hkv, 2, bs]; null for bf16
    float* weights;           // [num_blocks, Hkv, bs]
    int64_t num_blocks;
    int64_t blk, tok, kvh;    // strides in bytes
    const int32_t* table;     // [B, table_stride]
    const int32_t* out_table; // [B, out_stride]; the table itself: in place
    const int32_t* lens;      // [B]
    int32_t* kept;            // [B, Hkv, keep]
    int32_t* new_lens;        // [B]
    uint32_t* err;
    int32_t table_stride, out_stride, lbs;
    int32_t B, Hkv, keep, first, recent;
    int32_t row_bytes;        // of a token's key or value, one kv head
    bool in_place;
    int32_t sms;
};

cudaError_t evict_setup();
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace pda
