// pda_quant.h -- parameter block and launch entry point of decode over an
// 8-bit cache.
#pragma once

#include "pda_cache.h"

namespace pda {

struct QuantParams {
    const uint16_t* q;  // [B, q_len, Hq, D] bf16
    CacheRef c;
    void* out;          // [B, q_len, Hq, D] bf16, or fp32
    int32_t out_f32;
    int32_t q_len;
    int32_t Hq, Hkv, G;
    float scale_log2;
    uint32_t* err;
};

cudaError_t launch_quant(int D, int format, const QuantParams& p, cudaStream_t stream);

}  // namespace pda
