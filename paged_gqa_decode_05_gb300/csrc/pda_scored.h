// pda_scored.h -- decode with scored attention (capped, distance-biased),
// with the attention weight of every cached token, and over a shared prefix:
// the kernels' shapes and launch entry points (kernels in pda_scored.cuh and
// pda_weights.cu, one translation unit per head size for the former).
#pragma once

#include "pda_quant.h"

namespace pda {

struct ScoredShape {
    const void* fn;  // null: no such instance
    int threads;     // with the prefetch warp
    int stage_rows, stages;
    uint32_t stage_bytes;
    int max_rows;    // launch rows of a launch
    uint32_t smem(int B) const { return smem_layout_of(stage_bytes, kScored, stages, B).total; }
};

// An instance: stages of st rows (bf16 caches), a cache format, the q rows of a
// launch row (1: one query; 8: several causal ones; bf16 at head sizes up to 128
// 16 and 32), and (8-bit caches) weights in two fp16 parts, for calls whose output is
// in fp32 (the states that a shared prefix's bf16 outputs come from take one, too).
struct ScoredForm {
    int st, format, rows;
    bool fine;
};
ScoredShape scored_shape(int D, const ScoredForm& form);
// p is a QuantParams; bf16 kernels take its SplitParams.
cudaError_t launch_scored(int D, const ScoredForm& form, const QuantParams& p, int grid, size_t smem, cudaStream_t stream);

// The sums of attention weights of a decode's cached tokens.
struct WeightsParams {
    const float* scores;      // [Qr launch rows of each sequence, row-major][Hkv][table_stride * bs][rows_per_slot]
    const float* row_ml;      // [B * q_len * Hq][2]
    const float* in;          // [num_blocks, Hkv, bs] or null (zeros)
    float* out;               // [num_blocks, Hkv, bs]
    const int32_t* table;
    const int32_t* lens;
    uint32_t* err;
    int64_t num_blocks;
    int32_t table_stride, lbs;
    int32_t B, q_len, qp, rows_per_slot, Hq, Hkv, G;
};
cudaError_t launch_weights(const WeightsParams& p, int sms, cudaStream_t stream);

}  // namespace pda
