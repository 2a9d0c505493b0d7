// pda_scored_api.cu -- the C ABI of scored decode, of the sums of attention
// weights, of eviction by them and of decode over a shared prefix: argument
// checks, scratch layout and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pda_cache.h"
#include "pda_ctx.h"
#include "pda_evict.h"
#include "pda_prefix.h"
#include "pda_scored.h"

using pda::DeviceGuard;
using pda::aligned;
using pda::cuda_fail;
using pda::fail;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

bool overlap(const void* a, const void* b, int64_t bytes) {
    const int64_t d = (int64_t)((uintptr_t)a - (uintptr_t)b);
    return d < bytes && d > -bytes;
}

// Launch rows of scored decode: up to 8 q rows of a sequence each, or, over bf16
// caches of head sizes up to 128 where a sequence has more, up to 32 (one walk
// over K and V for four).  3 sequences of 8000 tokens with 40 q and 8 kv heads of
// 128 and 4 queries: 39.7 us, 62.8 in rows of 8; blocks of 4 tokens 52.6 and 88.8.
// Over 8-bit caches rows of 8 stay: their wider forms are bound by the consumer
// warps, not by the walks (12 rows, 5000 tokens of 256 in int8: 43.0 us for the
// wide form's 41.6 without scores).
struct Rows {
    int32_t qp, Qr, SR;  // queries per launch row, launch rows per sequence, q rows per launch row
    int32_t form;        // ScoredForm::rows
    int grid;
};
constexpr int kQuantGrid = 3;  // (scored_ctas)
Rows rows_of(const pda_ctx* ctx, bool bf16, int32_t q_len) {
    const int32_t G = ctx->dims.num_q_heads / ctx->dims.num_kv_heads;
    Rows r;
    int k = bf16 ? 0 : kQuantGrid;
    if (bf16 && q_len * G > pda::kMaxGroup && ctx->scored_ctas[2] > 0) {
        r.qp = std::min(q_len, pda::kMaxRowsPerWalk / G);
        k = r.qp * G <= 16 && ctx->scored_ctas[1] > 0 ? 1 : 2;
        r.form = 16 * k;
    } else {
        r.qp = std::max(1, std::min(q_len, pda::kMaxGroup / G));
        r.form = q_len > 1 ? pda::kMaxGroup : 1;
    }
    r.Qr = (q_len + r.qp - 1) / r.qp;
    r.SR = r.qp * G;
    r.grid = ctx->scored_ctas[k];
    return r;
}

// Sequences per launch: whole ones, as many as the kernel's launch rows and the
// partial states allow.
int32_t chunk_of(const pda_ctx* ctx, const Rows& r) {
    const int64_t fit = (ctx->part_rows / r.SR - r.grid) / ctx->dims.num_kv_heads;
    const int64_t most = r.form == 16 ? pda::max_launch_rows(pda::kScoredRows16) : pda::kMaxLaunchBatch;
    return (int32_t)(std::min(most, fit) / r.Qr);
}

struct Call {
    const pda_bf16* q;
    const pda_cache* cache;
    const int32_t* table;
    int32_t max_blocks;
    const int32_t* lens;
    int32_t batch, q_len;
    float scale;
    const pda_scoring* scoring;
    void* out;
    bool f32;
    cudaStream_t stream;
};

pda_status check_call(const pda_ctx* ctx, const Call& c) {
    pda_status st = pda::check_cache(c.cache);
    if (st != PDA_OK) return st;
    if (c.q_len < 1 || c.q_len > pda::kMaxLaunchBatch) return fail(PDA_ERR_INVALID_ARG, "q_len %d outside [1, %d]", c.q_len, pda::kMaxLaunchBatch);
    if (c.batch < 0 || (int64_t)c.batch * c.q_len > ctx->dims.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d x q_len %d outside [0, max_seqs=%d]", c.batch, c.q_len,
                    ctx->dims.max_seqs);
    if (c.scoring) {
        if (!(c.scoring->softcap >= 0.f) || std::isinf(c.scoring->softcap))
            return fail(PDA_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: none)");
        if (c.scoring->softcap > 0.f && (c.scoring->softcap < 1e-3f || c.scoring->softcap > 1e6f))
            return fail(PDA_ERR_INVALID_ARG, "softcap %g outside [1e-3, 1e6]", (double)c.scoring->softcap);
        if (!aligned(c.scoring->slopes, 4)) return fail(PDA_ERR_INVALID_ARG, "slopes must be 4-byte aligned");
    }
    if (c.batch == 0) return PDA_OK;
    if (!c.q || !aligned(c.q, 16) || !c.out || !aligned(c.out, 16))
        return fail(PDA_ERR_INVALID_ARG, "q and out must be non-NULL and 16-byte aligned");
    if (!c.table || !c.lens || !aligned(c.table, 4) || !aligned(c.lens, 4))
        return fail(PDA_ERR_INVALID_ARG, "block_table / seq_lens must be non-NULL and 4-byte aligned");
    if (c.max_blocks < 1) return fail(PDA_ERR_INVALID_ARG, "block table width must be >= 1 (got %d)", c.max_blocks);
    float scale_log2;
    return pda::check_scale(c.scale, ctx->dims.head_dim, &scale_log2);
}

pda_status record(const pda_ctx* ctx, cudaEvent_t ev, cudaStream_t stream) {
    if (!(ctx->ev_begin && ctx->ev_split && ctx->ev_end)) return PDA_OK;
    const cudaError_t e = cudaEventRecord(ev, stream);
    return e == cudaSuccess ? PDA_OK : cuda_fail(e, "cudaEventRecord");
}

// The split launches of a call.  sc: its Scoring, with buffers of the whole
// call; after(p, s0, n) follows each launch of sequences s0 .. s0 + n - 1.
template <class After>
pda_status run_scored(pda_ctx* ctx, const Call& c, const pda::Scoring& sc, const After& after) {
    const pda_dims& d = ctx->dims;
    const int D = d.head_dim, Hq = d.num_q_heads, bs = d.block_size;
    const bool bf16 = c.cache->format == PDA_CACHE_BF16;
    const Rows rows = rows_of(ctx, bf16, c.q_len);
    const pda::ScoredForm form = {ctx->stage_rows, c.cache->format, rows.form, !bf16 && c.f32};
    pda::QuantParams p = {};
    p.sc = sc;
    pda_status st = pda::check_scale(c.scale, D, &p.scale_log2);
    if (st != PDA_OK) return st;
    const pda::ScoredShape shape = pda::scored_shape(D, form);
    const int grid = rows.grid;
    if (rows.Qr > grid)
        return fail(PDA_ERR_INVALID_ARG, "q_len %d: more launch rows per sequence than CTAs (%d)", c.q_len, grid);
    const int32_t cost = rows.form == 1   ? pda::kCostDecode
                         : rows.form == 8 ? pda::kCostMultiN8
                         : rows.form == 16 ? pda::kCostRows16 : pda::kCostRows32;
    p.unit_cost = bf16 ? pda::unit_cost_blocks(ctx->stage_rows, D, bs, cost)
                       : pda::quant_unit_cost(D, 1, bs);
    if ((st = pda::check_plan_size((int64_t)c.batch * rows.Qr, c.max_blocks, p.unit_cost)) != PDA_OK) return st;
    const int32_t chunk = chunk_of(ctx, rows);
    if (chunk < 1)
        return fail(PDA_ERR_UNSUPPORTED, "q_len %d: a sequence's %d launch rows exceed the partial-state buffers", c.q_len,
                    rows.Qr);
    if (!bf16) pda::set_quant_pools(ctx, c.cache, &p);
    else if ((st = pda::set_bf16_pools(ctx, c.cache, &p)) != PDA_OK) return st;
    p.part_o = ctx->part_o;
    p.part_ml = ctx->part_ml;
    p.unit_sync = ctx->unit_sync;
    p.err = ctx->err;
    p.table_stride = c.max_blocks;
    p.q_len = c.q_len;
    p.qp = rows.qp;
    p.rows_per_slot = rows.SR;
    p.Hq = Hq;
    p.Hkv = d.num_kv_heads;
    p.G = ctx->G;
    p.bs = bs;
    // (the prefetch warp knows no blocks that a walk leaves out)
    p.prefetch = p.row_gather == 0 && bs >= 8 && rows.Qr == 1 && rows.form != 32 && !sc.shared;
    for (int32_t s0 = 0; s0 < c.batch; s0 += chunk) {
        const int32_t n = std::min(chunk, c.batch - s0);
        const int64_t rows0 = (int64_t)s0 * c.q_len * Hq;
        p.B = n * rows.Qr;
        p.q = c.q + rows0 * D;
        p.table = c.table + (int64_t)s0 * c.max_blocks;
        p.lens = c.lens + s0;
        p.out = c.f32 ? nullptr : static_cast<uint16_t*>(c.out) + rows0 * D;
        p.out_f32 = c.f32 ? static_cast<float*>(c.out) + rows0 * D : nullptr;
        p.sc.seq0 = s0;
        if (sc.row_o) {  // (the scores' own (m, l) are a launch's)
            p.sc.row_o = sc.row_o + rows0 * D;
            p.sc.row_ml = sc.row_ml + rows0 * 2;
        }
        const cudaError_t e = pda::launch_scored(D, form, p, grid, shape.smem(p.B), c.stream);
        if (e != cudaSuccess) return cuda_fail(e, "scored decode launch");
        if ((st = after(p, s0, n)) != PDA_OK) return st;
    }
    return PDA_OK;
}

pda::Scoring scoring_of(const pda_scoring* s) {
    pda::Scoring sc = {};
    if (!s) return sc;
    const float cap = s->softcap * kLog2e;
    (s->softcap > pda::kPlainCap ? sc.wide_cap : sc.cap) = cap;
    sc.inv_cap = s->softcap > 0.f ? 2.f * kLog2e / cap : 0.f;
    sc.slopes = s->slopes;
    return sc;
}

// Scratch of a decode that sums weights: the scores of one launch, and (m, l)
// of its output rows.
struct WeightsScratch {
    int64_t scores, row_ml, total;  // bytes; row_ml lies after the scores
};
WeightsScratch weights_scratch(const pda_ctx* ctx, bool bf16, int32_t batch, int32_t q_len, int32_t max_blocks) {
    const Rows r = rows_of(ctx, bf16, q_len);
    const int64_t n = std::min(batch, std::max(1, chunk_of(ctx, r)));
    WeightsScratch s;
    s.scores = round256(n * r.Qr * ctx->dims.num_kv_heads * (int64_t)max_blocks * ctx->dims.block_size * r.SR * 4);
    s.row_ml = round256(n * q_len * ctx->dims.num_q_heads * 8);
    s.total = s.scores + s.row_ml;
    return s;
}

pda_status check_weights_width(const pda_ctx* ctx, int32_t max_blocks) {
    if ((int64_t)max_blocks * ctx->dims.block_size <= (int64_t(1) << 30)) return PDA_OK;
    return fail(PDA_ERR_INVALID_ARG, "block table width %d is too large for sums of weights", max_blocks);
}

// Scratch of a shared prefix: the plan, the states of its pieces and those of
// the sequences' own tokens.
struct SharedScratch {
    int64_t groups, seqs, ml, o, row_ml, row_o, total;
};
SharedScratch shared_scratch(const pda_ctx* ctx, int32_t batch, int32_t q_len, int32_t n_groups) {
    const int D = ctx->dims.head_dim;
    const int64_t G = ctx->dims.num_q_heads / ctx->dims.num_kv_heads;
    const int64_t units = pda::prefix_units(D, batch * q_len * G, n_groups, ctx->dims.num_kv_heads);
    const int64_t rows = (units + ctx->num_sms) * pda::prefix_streams(D) * 128;
    SharedScratch s;
    s.groups = round256(((int64_t)n_groups + 1) * (int64_t)sizeof(pda::PrefixGroup));
    s.seqs = round256((int64_t)batch * (int64_t)sizeof(pda::PrefixSeq));
    s.ml = round256(rows * 8);
    s.o = round256(rows * D * 4);
    const int64_t out = (int64_t)batch * q_len * ctx->dims.num_q_heads;
    s.row_ml = round256(out * 8);
    s.row_o = round256(out * D * 4);
    s.total = s.groups + s.seqs + s.ml + s.o + s.row_ml + s.row_o;
    return s;
}

// A pool as boxes of the shared-prefix kernel: up to 32 rows of a block and kv
// head, one 64-column slab in the swizzle of the products' operands (bf16), or
// up to 128 codes a row as they are.
bool encode_box(const pda_dims& d, const void* base, const pda_cache* c, CUtensorMap* tm) {
    const bool bf16 = c->format == PDA_CACHE_BF16;
    const cuuint64_t es = bf16 ? 2 : 1, cols = bf16 ? 64 : std::min(d.head_dim, 128);
    const cuuint64_t dims[5] = {cols, (cuuint64_t)d.block_size, d.head_dim / cols, (cuuint64_t)d.num_kv_heads,
                                (cuuint64_t)c->num_blocks};
    const cuuint64_t strides[4] = {(cuuint64_t)c->tok_stride * es, cols * es, (cuuint64_t)c->kvh_stride * es,
                                   (cuuint64_t)c->blk_stride * es};
    const cuuint32_t box[5] = {(cuuint32_t)cols, (cuuint32_t)std::min(d.block_size, 32), 1, 1, 1}, one[5] = {1, 1, 1, 1, 1};
    return pda::tensor_map_encoder()(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 5,
                                     const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                     bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a cache for the shared-prefix kernel, encoded when it is another
// than the last call's.  (Blocks below 8 rows do not fill a swizzle span, and an
// id outside the pool, which reads as zeros, has to be an int32.)
void prefix_maps(pda_ctx* ctx, const pda_cache* c, pda::PrefixParams* p) {
    const pda_pool_key& k = ctx->prefix_key;
    if (!(ctx->prefix_valid && ctx->prefix_format == c->format && k.k == c->k_pool && k.v == c->v_pool &&
          k.num_blocks == c->num_blocks && k.blk == c->blk_stride && k.tok == c->tok_stride && k.kvh == c->kvh_stride)) {
        ctx->prefix_boxes = ctx->dims.block_size >= 8 && c->num_blocks < INT32_MAX && pda::tensor_map_encoder() &&
                            encode_box(ctx->dims, c->k_pool, c, &ctx->prefix_k) &&
                            encode_box(ctx->dims, c->v_pool, c, &ctx->prefix_v);
        ctx->prefix_key = {c->k_pool, c->v_pool, c->num_blocks, c->blk_stride, c->tok_stride, c->kvh_stride};
        ctx->prefix_format = c->format;
        ctx->prefix_valid = true;
    }
    p->boxes = ctx->prefix_boxes;
    if (p->boxes) {
        p->tm_k = ctx->prefix_k;
        p->tm_v = ctx->prefix_v;
    }
}

}  // namespace

pda_status pda::scored_setup(pda_ctx* ctx, int optin) {
    const int D = ctx->dims.head_dim;
    const auto setup = [&](const ScoredForm& form, int* per_sm) -> pda_status {
        const ScoredShape s = scored_shape(D, form);
        if (!s.fn) return fail(PDA_ERR_UNSUPPORTED, "no scored decode kernel");
        const int limit = (int)s.smem(s.max_rows);
        if (limit > optin)
            return fail(PDA_ERR_UNSUPPORTED, "needs %d bytes of shared memory per CTA (device allows %d)", limit, optin);
        int n = 0;
        cudaError_t e = cudaFuncSetAttribute(s.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(s.fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, s.fn, s.threads, limit);
        if (e != cudaSuccess) return cuda_fail(e, "scored decode attributes");
        if (n < 1) return fail(PDA_ERR_UNSUPPORTED, "scored decode kernel does not fit on an SM");
        *per_sm = std::min(*per_sm, n);
        return PDA_OK;
    };
    // the partial states of a context are sized for its other kernels' grids
    const int most[4] = {ctx->split_ctas, ctx->rows_ctas[0], ctx->rows_ctas[1], ctx->quant_ctas[0]};
    for (int k = 0; k < 4; ++k) {
        if (most[k] == 0) continue;
        int per_sm = 1 << 30;
        for (int f = 0; f < (k == 0 ? 2 : k == kQuantGrid ? 8 : 1); ++f) {
            const ScoredForm form = {ctx->stage_rows, k < kQuantGrid ? PDA_CACHE_BF16 : f & 1 ? PDA_CACHE_INT8 : PDA_CACHE_E4M3,
                                     k == 0             ? (f ? kMaxGroup : 1)
                                     : k == kQuantGrid ? (f & 2 ? kMaxGroup : 1) : 16 * k,
                                     (f & 4) != 0};
            if (const pda_status st = setup(form, &per_sm); st != PDA_OK) return st;
        }
        ctx->scored_ctas[k] = std::min(per_sm * ctx->num_sms, most[k]);
    }
    if (const cudaError_t e = evict_setup(); e != cudaSuccess) return cuda_fail(e, "eviction kernel attributes");
    for (int format : {PDA_CACHE_BF16, PDA_CACHE_E4M3, PDA_CACHE_INT8}) {
        const PrefixShape s = prefix_shape(D, format);
        if (s.smem > optin)
            return fail(PDA_ERR_UNSUPPORTED, "needs %d bytes of shared memory per CTA (device allows %d)", s.smem, optin);
        const cudaError_t e = cudaFuncSetAttribute(s.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem);
        if (e != cudaSuccess) return cuda_fail(e, "shared prefix kernel attributes");
    }
    return PDA_OK;
}

PDA_EXPORT pda_status pda_decode_scored_scratch(const pda_ctx* ctx, int32_t batch, int32_t q_len, int32_t max_blocks,
                                                int64_t* bytes) {
    if (!ctx || !bytes) return fail(PDA_ERR_INVALID_ARG, "NULL argument");
    if (batch < 0 || q_len < 1 || q_len > pda::kMaxLaunchBatch || max_blocks < 1 ||
        (int64_t)batch * q_len > ctx->dims.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d x q_len %d outside [0, max_seqs=%d] or table width %d < 1", batch, q_len,
                    ctx->dims.max_seqs, max_blocks);
    const pda_status st = check_weights_width(ctx, max_blocks);
    if (st == PDA_OK)  // over caches of any format
        *bytes = std::max(weights_scratch(ctx, true, batch, q_len, max_blocks).total,
                          weights_scratch(ctx, false, batch, q_len, max_blocks).total);
    return st;
}

PDA_EXPORT pda_status pda_decode_scored(pda_ctx* ctx, const pda_bf16* q, const pda_cache* cache,
                                        const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                        int32_t batch, int32_t q_len, float scale, const pda_scoring* scoring,
                                        const float* weights_in, float* weights_out, void* scratch, int64_t scratch_bytes,
                                        void* out, int32_t out_f32, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    const Call c = {q, cache, block_table, max_blocks, seq_lens, batch, q_len, scale, scoring, out, out_f32 != 0,
                    (cudaStream_t)stream};
    pda_status st = check_call(ctx, c);
    if (st != PDA_OK) return st;
    if (weights_in && !weights_out) return fail(PDA_ERR_INVALID_ARG, "weights_in without weights_out");
    if (!aligned(weights_in, 4) || !aligned(weights_out, 4))
        return fail(PDA_ERR_INVALID_ARG, "weights must be 4-byte aligned");
    if (weights_in && weights_in != weights_out &&
        overlap(weights_in, weights_out, cache->num_blocks * ctx->dims.num_kv_heads * ctx->dims.block_size * 4))
        return fail(PDA_ERR_INVALID_ARG, "weights_in must be weights_out, or apart from it");
    if (batch == 0) return PDA_OK;
    if (weights_out && (st = check_weights_width(ctx, max_blocks)) != PDA_OK) return st;
    const WeightsScratch ws = weights_scratch(ctx, cache->format == PDA_CACHE_BF16, batch, q_len, max_blocks);
    if (weights_out && (!scratch || !aligned(scratch, 16) || scratch_bytes < ws.total))
        return fail(PDA_ERR_INVALID_ARG, "weights need %lld bytes of 16-byte aligned scratch (got %lld)", (long long)ws.total,
                    (long long)scratch_bytes);
    DeviceGuard on(ctx->device);
    pda::Scoring sc = scoring_of(scoring);
    if (weights_out) {
        sc.scores = static_cast<float*>(scratch);
        sc.row_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + ws.scores);
    }
    ctx->tile_steps = 0;
    if ((st = record(ctx, ctx->ev_begin, c.stream)) != PDA_OK) return st;
    st = run_scored(ctx, c, sc, [&](const pda::SplitParams& p, int32_t, int32_t n) -> pda_status {
        if (!weights_out) return PDA_OK;
        pda::WeightsParams w = {};
        w.scores = sc.scores;
        w.row_ml = sc.row_ml;
        w.in = weights_in;
        w.out = weights_out;
        w.table = p.table;
        w.lens = p.lens;
        w.err = ctx->err;
        w.num_blocks = cache->num_blocks;
        w.table_stride = max_blocks;
        while ((1 << w.lbs) < p.bs) ++w.lbs;
        w.B = n;
        w.q_len = q_len;
        w.qp = p.qp;
        w.rows_per_slot = p.rows_per_slot;
        w.Hq = p.Hq;
        w.Hkv = p.Hkv;
        w.G = p.G;
        const cudaError_t e = pda::launch_weights(w, ctx->num_sms, c.stream);
        return e == cudaSuccess ? PDA_OK : cuda_fail(e, "attention weights launch");
    });
    if (st == PDA_OK) st = record(ctx, ctx->ev_split, c.stream);
    return st == PDA_OK ? record(ctx, ctx->ev_end, c.stream) : st;
}

PDA_EXPORT pda_status pda_decode_shared_scratch(const pda_ctx* ctx, int32_t batch, int32_t q_len, int32_t groups,
                                                int64_t* bytes) {
    if (!ctx || !bytes) return fail(PDA_ERR_INVALID_ARG, "NULL argument");
    if (batch < 0 || q_len < 1 || q_len > pda::kMaxLaunchBatch || (int64_t)batch * q_len > ctx->dims.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d x q_len %d outside [0, max_seqs=%d]", batch, q_len, ctx->dims.max_seqs);
    if (groups < 1 || groups > pda::kMaxLaunchBatch)
        return fail(PDA_ERR_INVALID_ARG, "groups %d outside [1, %d]", groups, pda::kMaxLaunchBatch);
    *bytes = shared_scratch(ctx, batch, q_len, groups).total;
    return PDA_OK;
}

PDA_EXPORT pda_status pda_decode_shared(pda_ctx* ctx, const pda_bf16* q, const pda_cache* cache,
                                        const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                        int32_t batch, int32_t q_len, const int32_t* shared_blocks, const int32_t* starts,
                                        int32_t groups, float scale, const pda_scoring* scoring, void* scratch,
                                        int64_t scratch_bytes, void* out, int32_t out_f32, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    const Call c = {q, cache, block_table, max_blocks, seq_lens, batch, q_len, scale, scoring, out, out_f32 != 0,
                    (cudaStream_t)stream};
    pda_status st = check_call(ctx, c);
    if (st != PDA_OK) return st;
    if (groups < 1 || groups > pda::kMaxLaunchBatch)
        return fail(PDA_ERR_INVALID_ARG, "groups %d outside [1, %d]", groups, pda::kMaxLaunchBatch);
    if (batch == 0) return PDA_OK;
    if (!shared_blocks || !aligned(shared_blocks, 4) || !aligned(starts, 4))
        return fail(PDA_ERR_INVALID_ARG, "shared_blocks must be non-NULL, it and starts 4-byte aligned");
    if (!starts && batch % groups != 0)
        return fail(PDA_ERR_INVALID_ARG, "without starts batch (%d) must be a multiple of groups (%d)", batch, groups);
    const pda_dims& d = ctx->dims;
    const int D = d.head_dim;
    const int64_t tiles = ((int64_t)max_blocks * d.block_size + pda::kPrefixTile - 1) / pda::kPrefixTile;
    const int64_t most = pda::prefix_units(D, (int64_t)batch * q_len * (d.num_q_heads / d.num_kv_heads), groups, d.num_kv_heads) * tiles;
    if (most > INT32_MAX)
        return fail(PDA_ERR_INVALID_ARG, "block table width %d is too large for a shared prefix", max_blocks);
    const SharedScratch ss = shared_scratch(ctx, batch, q_len, groups);
    if (!scratch || !aligned(scratch, 16) || scratch_bytes < ss.total)
        return fail(PDA_ERR_INVALID_ARG, "a shared prefix needs %lld bytes of 16-byte aligned scratch (got %lld)",
                    (long long)ss.total, (long long)scratch_bytes);
    DeviceGuard on(ctx->device);
    pda::PrefixParams pp = {};
    if ((st = pda::check_scale(scale, D, &pp.score_mult)) != PDA_OK) return st;
    uint8_t* base = static_cast<uint8_t*>(scratch);
    pda::Scoring sc = scoring_of(scoring);
    pp.q = q;
    pp.k_base = static_cast<const uint8_t*>(cache->k_pool);
    pp.v_base = static_cast<const uint8_t*>(cache->v_pool);
    pp.scales = cache->scales;
    pp.blk_s = cache->blk_stride;
    pp.tok_s = cache->tok_stride;
    pp.kvh_s = cache->kvh_stride;
    pp.num_blocks = cache->num_blocks;
    pp.table = block_table;
    pp.lens = seq_lens;
    pp.shared = shared_blocks;
    pp.starts = starts;
    pp.groups = reinterpret_cast<pda::PrefixGroup*>(base);
    pp.seqs = reinterpret_cast<pda::PrefixSeq*>(base + ss.groups);
    pp.part_ml = reinterpret_cast<float*>(base + ss.groups + ss.seqs);
    pp.part_o = reinterpret_cast<float*>(base + ss.groups + ss.seqs + ss.ml);
    pp.err = ctx->err;
    pp.table_stride = max_blocks;
    while ((1 << pp.lbs) < d.block_size) ++pp.lbs;
    pp.B = batch;
    pp.q_len = q_len;
    pp.Hq = d.num_q_heads;
    pp.Hkv = d.num_kv_heads;
    pp.G = ctx->G;
    pp.n_groups = groups;
    pp.cap = sc.cap;
    pp.wide_cap = sc.wide_cap;
    if (sc.inv_cap != 0.f) pp.score_mult *= sc.inv_cap;
    pp.slopes = sc.slopes;
    sc.shared = shared_blocks;
    sc.starts = starts;
    sc.n_groups = groups;
    sc.all_seqs = batch;
    sc.row_ml = reinterpret_cast<float*>(base + ss.groups + ss.seqs + ss.ml + ss.o);
    sc.row_o = reinterpret_cast<float*>(base + ss.groups + ss.seqs + ss.ml + ss.o + ss.row_ml);
    prefix_maps(ctx, cache, &pp);
    ctx->tile_steps = 0;
    if ((st = record(ctx, ctx->ev_begin, c.stream)) != PDA_OK) return st;
    // own tokens first: the prefix kernel's start, which needs nothing of them, passes under their end
    st = run_scored(ctx, c, sc, [](const pda::SplitParams&, int32_t, int32_t) -> pda_status { return PDA_OK; });
    if (st != PDA_OK) return st;
    if ((st = record(ctx, ctx->ev_split, c.stream)) != PDA_OK) return st;
    const int ctas = (int)std::min<int64_t>(most, ctx->num_sms);  // none that no plan gives work
    cudaError_t e = pda::launch_prefix(D, cache->format, pp, ctas, c.stream);
    if (e != cudaSuccess) return cuda_fail(e, "shared prefix launch");
    pda::JoinParams j = {};
    j.seqs = pp.seqs;
    j.row_ml = sc.row_ml;
    j.row_o = sc.row_o;
    j.part_ml = pp.part_ml;
    j.part_o = pp.part_o;
    j.out = out_f32 ? nullptr : static_cast<uint16_t*>(out);
    j.out_f32 = out_f32 ? static_cast<float*>(out) : nullptr;
    j.rows = (int64_t)batch * q_len * d.num_q_heads;
    j.q_len = q_len;
    j.Hq = d.num_q_heads;
    j.Hkv = d.num_kv_heads;
    j.G = ctx->G;
    e = pda::launch_join(D, j, c.stream);
    if (e != cudaSuccess) return cuda_fail(e, "shared prefix join launch");
    return st == PDA_OK ? record(ctx, ctx->ev_end, c.stream) : st;
}

PDA_EXPORT pda_status pda_evict(pda_ctx* ctx, const pda_cache* cache, float* weights, const int32_t* block_table,
                                int32_t max_blocks, const int32_t* seq_lens, int32_t batch, int32_t keep, int32_t first,
                                int32_t recent, const int32_t* out_table, int32_t out_blocks, int32_t* kept,
                                int32_t* new_lens, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    pda_status st = pda::check_cache(cache);
    if (st != PDA_OK) return st;
    const pda_dims& d = ctx->dims;
    if (batch < 0 || batch > d.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d outside [0, max_seqs=%d]", batch, d.max_seqs);
    if (keep < 1 || first < 0 || recent < 0 || (int64_t)first + recent > keep)
        return fail(PDA_ERR_INVALID_ARG, "keep %d must be >= 1 and hold first %d + recent %d tokens", keep, first, recent);
    if (batch == 0) return PDA_OK;
    if (!block_table || !seq_lens || !kept || !new_lens || !weights)
        return fail(PDA_ERR_INVALID_ARG, "weights, block_table, seq_lens, kept and new_lens must be non-NULL");
    for (const void* a : {(const void*)weights, (const void*)block_table, (const void*)seq_lens, (const void*)out_table,
                          (const void*)kept, (const void*)new_lens})
        if (!aligned(a, 4)) return fail(PDA_ERR_INVALID_ARG, "eviction arrays must be 4-byte aligned");
    if (overlap(new_lens, seq_lens, (int64_t)batch * 4)) return fail(PDA_ERR_INVALID_ARG, "new_lens must not overlap seq_lens");
    if (max_blocks < 1 || (out_table && out_blocks < 1))
        return fail(PDA_ERR_INVALID_ARG, "block table width must be >= 1 (got %d, %d)", max_blocks, out_blocks);
    const int64_t tokens = (int64_t)max_blocks * d.block_size;
    if (tokens > (int64_t(1) << 30)) return fail(PDA_ERR_INVALID_ARG, "block table width %d is too large", max_blocks);
    const bool in_place = !out_table || out_table == block_table;
    if (in_place && out_table && out_blocks != max_blocks)
        return fail(PDA_ERR_INVALID_ARG, "out_table is block_table but for its width");
    if (!in_place && (int64_t)out_blocks * d.block_size < std::min<int64_t>(keep, tokens))
        return fail(PDA_ERR_INVALID_ARG, "out_table's %d blocks do not hold %d tokens", out_blocks, keep);
    const int64_t chunks = (std::min<int64_t>(keep, tokens) + 63) / 64, units = (int64_t)batch * d.num_kv_heads;
    if (units * std::max<int64_t>(chunks, 16) > INT32_MAX) return fail(PDA_ERR_INVALID_ARG, "too many tokens to keep");
    const int es = cache->format == PDA_CACHE_BF16 ? 2 : 1;
    pda::EvictParams p = {};
    p.k = static_cast<uint8_t*>(cache->k_pool);
    p.v = static_cast<uint8_t*>(cache->v_pool);
    p.scales = cache->format == PDA_CACHE_BF16 ? nullptr : cache->scales;
    p.weights = weights;
    p.num_blocks = cache->num_blocks;
    p.blk = cache->blk_stride * es;
    p.tok = cache->tok_stride * es;
    p.kvh = cache->kvh_stride * es;
    p.table = block_table;
    p.out_table = in_place ? block_table : out_table;
    p.lens = seq_lens;
    p.kept = kept;
    p.new_lens = new_lens;
    p.err = ctx->err;
    p.table_stride = max_blocks;
    p.out_stride = in_place ? max_blocks : out_blocks;
    while ((1 << p.lbs) < d.block_size) ++p.lbs;
    p.B = batch;
    p.Hkv = d.num_kv_heads;
    p.keep = keep;
    p.first = first;
    p.recent = recent;
    p.row_bytes = d.head_dim * es;
    p.in_place = in_place;
    p.sms = ctx->num_sms;
    DeviceGuard on(ctx->device);
    ctx->tile_steps = 0;
    const cudaError_t e = pda::launch_evict(p, (cudaStream_t)stream);
    return e == cudaSuccess ? PDA_OK : cuda_fail(e, "eviction launch");
}
