// pda_quant.h -- decode over an 8-bit cache: the split kernel's shapes,
// parameters and launch entry points (kernels in pda_quant.cuh, one
// translation unit per head size).
#pragma once

#include "pda_cache.h"
#include "pda_params.h"

namespace pda {

// Shapes.  A consumer warp takes 16 KV rows of a stage per row tile, against
// eight packed q rows.  Head sizes up to 128 run two CTAs of 4 such warps per
// SM, two row tiles each; with 16 packed q rows (n_tiles 2) one CTA of 8, four
// to each tile of q rows, over stages that both tiles share; head size 256 one
// CTA of 8.  Measured against it, 32 sequences of 4096 tokens, 32 q and 8 kv
// heads of 128, e4m3 (52.6 us): one CTA of 8 warps 53.8, 8 warps of one row
// tile twice a SM (96 registers) 63.9, three CTAs at 128 registers 57.0, warps
// with a ring each 51 to 57 (and 107 to 120 where the lengths are ragged: 107
// here), two producer warps 53.9.  16 q rows, 4 queries on 2456 tokens: both
// tiles in one warp's registers, which shares the conversions of V, 67.6 us;
// two walks over the cache 65.4; this form 61.7 (int8 64.0, 72.4 and 66.5); it
// takes 62.0 (64.3) since its sums hold for every V scale.
PDA_HD constexpr int quant_warps(int D, int n_tiles) { return D == 256 || n_tiles == 2 ? 8 : 4; }
PDA_HD constexpr int quant_row_tiles(int D, int n_tiles) { return D == 256 ? 1 : 2; }
PDA_HD constexpr int quant_stage_rows(int D, int n_tiles) {
    return 16 * quant_warps(D, n_tiles) / n_tiles * quant_row_tiles(D, n_tiles);
}
PDA_HD constexpr int quant_stage_bytes(int D, int n_tiles) {  // whole swizzle spans
    return (quant_stage_rows(D, n_tiles) * (2 * D + 8) + 8 * n_tiles * D * 2 + 1023) / 1024 * 1024;
}
PDA_HD constexpr int quant_stages(int D, int n_tiles) { return n_tiles == 2 ? (D == 64 ? 8 : 5) : D == 64 ? 5 : 3; }
// Whether blocks load as boxes: a block's K and V rows of one kv head must
// fill whole 1024-byte spans (one box brings both where the pools' layout
// allows it, with `joined`; else a box each).
PDA_HD constexpr bool quant_boxes(int D, int bs, bool joined) { return (bs * D * (joined ? 2 : 1)) % 1024 == 0; }
// Plan blocks added to every unit (see pda_plan.h), in quarter stages: what the
// preparation of its q rows and its merge cost a CTA (6000 and 7000 of the
// 90000 cycles of a CTA with one unit of 30 stages).  64 sequences of 128 to
// 32768 tokens take 106.3, 106.1, 107.7, 110.5 us at 6, 9 to 12, 16, 28; 4
// queries on 2456 tokens each 61.1, 60.7, 61.3, 63.2 at 8, 12, 16, 24.  Blocks
// below 8 tokens come in so many copies that a stage takes as long as a unit's
// ends.
PDA_HD int32_t quant_unit_cost(int D, int n_tiles, int bs) {
    const int nb = quant_stage_rows(D, n_tiles) / bs, x4 = nb * (bs < 8 ? 2 : 12);
    return x4 < 4 ? 1 : x4 / 4;
}

struct QuantParams : SplitParams {
    const float* scales;  // [num_blocks, Hkv, 2, bs]
    // Box loads: tm_k brings a block's K and V rows of a kv head (V first when
    // v_first), head h at coordinate 2 of box_head * h; or, when !joined, tm_k
    // and tm_v bring them apart, h at coordinate 3.  tm_k1 views the scales as
    // [num_blocks * Hkv][2 bs] for row gathers.
    int32_t joined, v_first, box_head;
};

// An instance of the kernel.
struct QuantForm {
    int format;   // kE4m3 / kInt8
    int n_tiles;  // 1: up to 8 q rows per walk, 2: 16 (head sizes up to 128)
    bool multi;   // several causal queries per sequence
    bool fine;    // weights in two fp16 parts: fp32 outputs
};

struct QuantShape {
    const void* fn;   // null: no such instance
    int threads;      // with the prefetch warp
    int stage_rows, stages, stage_bytes;
    uint32_t smem(int B) const { return smem_layout_of((uint32_t)stage_bytes, kOneShot, stages, B).total; }
};

QuantShape quant_shape(int D, const QuantForm& form);
cudaError_t launch_quant(int D, const QuantForm& form, const QuantParams& p, int grid, size_t smem, cudaStream_t stream);

}  // namespace pda
