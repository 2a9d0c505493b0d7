// pda_prefix.h -- the kernel that walks the prefix a group of sequences
// shares, once for all their queries (pda_prefix.cuh): parameters, plan
// limits and launch entry points.
#pragma once

#include "pda_cache.h"
#include "pda_params.h"

namespace pda {

struct PrefixParams {
    CUtensorMap tm_k, tm_v;     // boxes of min(block size, 32) rows (encode_box in pda_scored_api.cu); with `boxes`
    const uint16_t* q;          // [B, q_len, Hq, D] bf16
    const uint8_t* k_base;      // pools, elements of the cache's format
    const uint8_t* v_base;
    const float* scales;        // [num_blocks, Hkv, 2, bs]; 8-bit formats
    int64_t blk_s, tok_s, kvh_s, num_blocks;
    const int32_t* table;       // [B, table_stride]
    const int32_t* lens;        // [B]
    const int32_t* shared;      // [n_groups] blocks
    const int32_t* starts;      // [n_groups + 1] or null: B / n_groups sequences each
    PrefixGroup* groups;        // [n_groups + 1] out
    PrefixSeq* seqs;            // [B] out
    float* part_o;              // [slots][streams][D / slab][128][slab], pieces of 4 XORed with the row
    float* part_ml;             // [slots][streams][128][2]
    uint32_t* err;
    int32_t table_stride, lbs;
    int32_t boxes;              // rows come as TMA boxes (block sizes from 8), else one by one
    int32_t B, q_len, Hq, Hkv, G, n_groups;
    float score_mult;           // score scale in base-2 units; under a cap, what capped() takes the exponential of
    float cap, wide_cap;        // in base-2 units (Scoring)
    const float* slopes;
};

struct PrefixShape {
    const void* fn;
    int threads, smem;
};
PrefixShape prefix_shape(int D, int format);
cudaError_t launch_prefix(int D, int format, const PrefixParams& p, int ctas, cudaStream_t stream);

// Joins the pieces of the prefixes with the states of the sequences' own tokens.
struct JoinParams {
    const PrefixSeq* seqs;      // [B]
    const float* row_ml;        // [rows][2], [rows][D]: states of the own tokens
    const float* row_o;
    const float* part_ml;       // as in PrefixParams
    const float* part_o;
    uint16_t* out;              // [rows][D] bf16, or
    float* out_f32;             // fp32 when not null
    int64_t rows;               // B * q_len * Hq
    int32_t q_len, Hq, Hkv, G;
};
cudaError_t launch_join(int D, const JoinParams& p, cudaStream_t stream);

// Units of a call at most: pairs of q tiles (single ones at head size 256) per
// kv head, one more for every group whose rows do not fill their last.
PDA_HD int64_t prefix_units(int D, int64_t rows, int64_t groups, int64_t Hkv) {
    return Hkv * (rows / (128 * prefix_streams(D)) + groups);
}

}  // namespace pda
