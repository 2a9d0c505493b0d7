// pda_ctx.h -- the context behind the C ABI and the helpers that every
// translation unit of the API shares.
#pragma once

#include <cudaTypedefs.h>

#include "pda.h"
#include "pda_launch.h"

#define PDA_EXPORT extern "C" __attribute__((visibility("default")))

namespace pda {

// Sets the calling thread's pda_last_error() and returns st.
pda_status fail(pda_status st, const char* fmt, ...);
pda_status cuda_fail(cudaError_t e, const char* what);
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
// scale * log2(e), with NaN standing for 1/sqrt(D).
pda_status check_scale(float scale, int D, float* scale_log2);
pda_status check_plan_size(int64_t rows, int32_t table_width, int32_t unit_cost);

}  // namespace pda

struct pda_pool_key {  // what a pool's tensor maps are encoded from
    const void* k = nullptr;
    const void* v = nullptr;
    int64_t num_blocks = 0, blk = 0, tok = 0, kvh = 0;
};

struct pda_ctx {
    pda_dims dims;
    int32_t G = 0;
    int device = 0;
    int num_sms = 0;
    int stages = 0;
    int stage_rows = 64;  // split-kernel shape: KV rows per stage
    int ctas_per_sm = 0;
    int split_ctas = 0;
    int smem_max = 0;
    int64_t slots = 0;
    int64_t part_rows = 0;  // q rows the partial-state buffers hold (all slots)
    // Row form of multi-query (one / two 16-row q tiles): grid and pipeline
    // depth; a grid of 0 when the shape does not exist (head size 256).
    int rows_ctas[2] = {0, 0};
    int rows_stages[2] = {0, 0};
    // The tcgen05 row form (launch rows of 17 to 32 q rows): grid and depth
    // (0: not on this shape), and whether calls take it (pda_set_multi_tc; off
    // by default: measured slower than the mma.sync row form).
    int tc_ctas = 0;
    int tc_stages = 0;
    bool multi_tc = false;
    float* part_o = nullptr;
    float* part_ml = nullptr;
    int32_t* unit_sync = nullptr;  // [chunk_b*Hkv][2] split-unit tickets and stored counts
    int64_t unit_sync_bytes = 0;
    uint32_t* err = nullptr;
    float* m_state = nullptr;
    float* l_state = nullptr;
    float* o_state = nullptr;
    cudaEvent_t ev_begin = nullptr, ev_split = nullptr, ev_end = nullptr;
    // Tiled lifecycle: tile steps since the last begin_step and the stream of
    // the last one; a tile step right behind another on the same stream reads
    // its inputs early (pda_set_tile_overlap turns that off).
    int64_t tile_steps = 0;
    cudaStream_t tile_stream = nullptr;
    bool tile_overlap = true;
    // The last pool's tensor maps: a decode loop over one cache encodes them
    // once (encoding costs host time on every call otherwise).
    bool maps_valid = false;
    pda_pool_key maps_key;
    int32_t maps_row_mode = 0;
    CUtensorMap map_k, map_v;
    CUtensorMap map_k1, map_v1;  // one-slab boxes (head size 128, block boxes): the tcgen05 form
    // Decode over 8-bit caches: grids with up to 8 and 16 packed q rows per
    // walk (0: not on this shape).
    int quant_ctas[2] = {0, 0};
};

namespace pda {
// Launch attributes and grids of the 8-bit kernels of a context's shape.
pda_status quant_setup(pda_ctx* ctx, int smem_optin);
// Causal multi-query decode over a bf16 cache of any stride triple.
pda_status decode_bf16_multi(pda_ctx* ctx, const pda_bf16* q, const pda_cache* cache, const int32_t* block_table,
                             int32_t max_blocks, const int32_t* seq_lens, int32_t batch, int32_t q_len, float scale,
                             pda_bf16* out, pda_stream stream);
}  // namespace pda
