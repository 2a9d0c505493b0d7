// pda_cache_api.cu -- the C ABI around the decode: q / k preparation, cache
// writes and read-backs, and decode over a cache of any format: argument
// checks and launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "pda_cache.h"
#include "pda_ctx.h"
#include "pda_quant.h"

using pda::DeviceGuard;
using pda::aligned;
using pda::check_cache;
using pda::cuda_fail;
using pda::fail;

namespace {

pda_status check_heads(const pda_heads* h, const char* name) {
    if (!h->data || !aligned(h->data, 8))
        return fail(PDA_ERR_INVALID_ARG, "%s must be non-NULL and 8-byte aligned", name);
    const int64_t s[2] = {h->tok_stride, h->head_stride};
    for (int64_t x : s)
        if (x <= 0 || x % 4 != 0 || x >= (int64_t(1) << 38))
            return fail(PDA_ERR_INVALID_ARG, "%s strides must be positive multiples of 4 elements (got %lld)", name,
                        (long long)x);
    return PDA_OK;
}

pda_status check_prep(const pda_prep* p, int D) {
    if (!p) return PDA_OK;
    if ((p->q_weight || p->k_weight) && !(p->eps >= 0.f && std::isfinite(p->eps)))
        return fail(PDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(p->q_weight, 8) || !aligned(p->k_weight, 8))
        return fail(PDA_ERR_INVALID_ARG, "norm weights must be 8-byte aligned");
    if (p->cos_sin) {
        if (!aligned(p->cos_sin, 16)) return fail(PDA_ERR_INVALID_ARG, "cos_sin must be 16-byte aligned");
        if (p->rotary_dim < 8 || p->rotary_dim > D || p->rotary_dim % 8 != 0)
            return fail(PDA_ERR_INVALID_ARG, "rotary_dim %d must be a multiple of 8 in [8, %d]", p->rotary_dim, D);
        if (p->max_positions < 1) return fail(PDA_ERR_INVALID_ARG, "max_positions must be >= 1");
    }
    return PDA_OK;
}

}  // namespace

pda_status pda::check_cache(const pda_cache* c) {
    if (!c) return fail(PDA_ERR_INVALID_ARG, "cache is NULL");
    if (c->format != PDA_CACHE_BF16 && c->format != PDA_CACHE_E4M3 && c->format != PDA_CACHE_INT8)
        return fail(PDA_ERR_INVALID_ARG, "unknown cache format %d", c->format);
    if (!c->k_pool || !c->v_pool || !aligned(c->k_pool, 16) || !aligned(c->v_pool, 16))
        return fail(PDA_ERR_INVALID_ARG, "k_pool / v_pool must be non-NULL and 16-byte aligned");
    if (c->num_blocks < 1 || c->num_blocks > INT32_MAX)
        return fail(PDA_ERR_INVALID_ARG, "num_blocks %lld outside [1, 2^31)", (long long)c->num_blocks);
    const int64_t unit = c->format == PDA_CACHE_BF16 ? 8 : 16;  // elements in 16 bytes
    const int64_t s[3] = {c->blk_stride, c->tok_stride, c->kvh_stride};
    for (int64_t x : s)
        if (x <= 0 || x % unit != 0 || x >= (int64_t(1) << 38))
            return fail(PDA_ERR_INVALID_ARG, "pool strides must be positive multiples of 16 bytes (got %lld elements)",
                        (long long)x);
    if (c->format != PDA_CACHE_BF16 && (!c->scales || !aligned(c->scales, 16)))
        return fail(PDA_ERR_INVALID_ARG, "scales must be non-NULL and 16-byte aligned for an 8-bit cache");
    return PDA_OK;
}

namespace {

pda_status check_sequences(const pda_ctx* ctx, const int32_t* table, int32_t max_blocks, const int32_t* lens,
                           int32_t batch, const int32_t* starts, int64_t rows) {
    if (batch < 0 || batch > ctx->dims.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d outside [0, max_seqs=%d]", batch, ctx->dims.max_seqs);
    if (rows < 0 || rows > INT32_MAX) return fail(PDA_ERR_INVALID_ARG, "token count outside [0, 2^31)");
    if (batch == 0 || rows == 0) return PDA_OK;
    if (!table || !lens || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4))
        return fail(PDA_ERR_INVALID_ARG, "block_table / seq_lens / starts must be 4-byte aligned, the first two non-NULL");
    if (max_blocks < 1) return fail(PDA_ERR_INVALID_ARG, "block table width must be >= 1 (got %d)", max_blocks);
    if (!starts && rows % batch != 0)
        return fail(PDA_ERR_INVALID_ARG, "without starts the token count (%lld) must be a multiple of batch (%d)",
                    (long long)rows, batch);
    return PDA_OK;
}

pda::CacheRef cache_ref(const pda_ctx* ctx, const pda_cache* c, const int32_t* table, int32_t max_blocks,
                        const int32_t* lens, int32_t batch, const int32_t* starts, int64_t rows) {
    pda::CacheRef r = {};
    r.k = static_cast<uint8_t*>(c->k_pool);
    r.v = static_cast<uint8_t*>(c->v_pool);
    r.scales = c->scales;
    r.num_blocks = c->num_blocks;
    r.blk = c->blk_stride;
    r.tok = c->tok_stride;
    r.kvh = c->kvh_stride;
    r.table = table;
    r.table_stride = max_blocks;
    while ((1 << r.lbs) < ctx->dims.block_size) ++r.lbs;
    r.lens = lens;
    r.starts = starts;
    r.rows_each = batch > 0 ? rows / batch : 0;
    r.B = batch;
    return r;
}

pda::Heads heads(const pda_heads* h) {
    if (!h) return {nullptr, 0, 0};
    return {h->data, h->tok_stride, h->head_stride};
}

void set_prep(pda::HeadsParams& p, const pda_prep* prep) {
    if (!prep) return;
    p.q_weight = prep->q_weight;
    p.k_weight = prep->k_weight;
    p.weights_f32 = prep->weights_f32;
    p.eps = prep->eps;
    p.cos_sin = prep->cos_sin;
    p.max_pos = prep->max_positions;
    p.rotary = prep->cos_sin ? prep->rotary_dim : 0;
    p.interleaved = prep->interleaved;
}

// 5-D views of 8-bit pools for TMA boxes that land as [head][slab][slot][128
// bytes] (64 at head size 64) with the swizzle of that width.
bool encode_view(const void* base, const cuuint64_t (&dims)[5], const cuuint64_t (&strides)[4],
                 const cuuint32_t (&box)[5], CUtensorMap* tm) {
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return pda::tensor_map_encoder()(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box,
                                     one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                     box[0] == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Joined: the distance between the pools is one more axis, {bytes of a row,
// bs slots, heads, K|V, num_blocks}, so that one copy brings a block's K and V
// rows; head size 256 has two slabs a row and puts slabs and heads on one
// axis, where heads lie side by side.  Returns false where the layout does
// not fit (or the driver refuses it).
bool encode_joined(const pda_dims& d, const pda_cache* c, CUtensorMap* tm) {
    const uintptr_t k = reinterpret_cast<uintptr_t>(c->k_pool), v = reinterpret_cast<uintptr_t>(c->v_pool);
    const uintptr_t first = std::min(k, v), apart = std::max(k, v) - first;
    if (apart == 0 || apart >= (uintptr_t(1) << 40)) return false;
    const cuuint64_t bs = (cuuint64_t)d.block_size, nb = (cuuint64_t)c->num_blocks, slabs = d.head_dim == 256 ? 2 : 1;
    const cuuint64_t tok = (cuuint64_t)c->tok_stride, kvh = (cuuint64_t)c->kvh_stride, blk = (cuuint64_t)c->blk_stride;
    const cuuint32_t row = d.head_dim < 128 ? (cuuint32_t)d.head_dim : 128u;
    if (slabs == 2 && kvh != 256) return false;
    return encode_view(reinterpret_cast<void*>(first), {row, bs, slabs * (cuuint64_t)d.num_kv_heads, 2, nb},
                       {tok, slabs == 2 ? 128 : kvh, apart, blk},
                       {row, (cuuint32_t)bs, (cuuint32_t)slabs, 2, 1}, tm);
}

// A view of one pool, {bytes of a slab, bs slots, slabs, heads, num_blocks}.
bool encode_apart(const pda_dims& d, const void* base, const pda_cache* c, CUtensorMap* tm) {
    const cuuint32_t row = d.head_dim < 128 ? (cuuint32_t)d.head_dim : 128u, slabs = (cuuint32_t)d.head_dim / row;
    return encode_view(base,
                       {row, (cuuint64_t)d.block_size, slabs, (cuuint64_t)d.num_kv_heads, (cuuint64_t)c->num_blocks},
                       {(cuuint64_t)c->tok_stride, row, (cuuint64_t)c->kvh_stride, (cuuint64_t)c->blk_stride},
                       {row, (cuuint32_t)d.block_size, slabs, 1, 1}, tm);
}

// The scales as rows of 2 bs floats, one per (block, kv head), for gathers.
bool encode_scales(const pda_dims& d, const pda_cache* c, CUtensorMap* tm) {
    const int64_t rows = c->num_blocks * d.num_kv_heads;
    if (rows > INT32_MAX) return false;
    const cuuint64_t floats = 2 * (cuuint64_t)d.block_size;
    const cuuint64_t dims[2] = {floats, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {4 * floats};
    const cuuint32_t box[2] = {(cuuint32_t)floats, 1}, one[2] = {1, 1};
    return pda::tensor_map_encoder()(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, c->scales, dims, strides, box, one,
                                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call's pools load: encodes the launch's maps, or returns false where
// boxes do not fit (then rows are copied one by one).
bool encode_boxes(const pda_dims& d, const pda_cache* c, pda::QuantParams* p) {
    if (!pda::tensor_map_encoder()) return false;
    if (d.block_size < 4) return false;  // four blocks' scales must fill the 128 bytes a copy starts on
    if (!encode_scales(d, c, &p->tm_k1)) return false;
    p->joined = pda::quant_boxes(d.head_dim, d.block_size, true) && encode_joined(d, c, &p->tm_k);
    return p->joined || (pda::quant_boxes(d.head_dim, d.block_size, false) && encode_apart(d, c->k_pool, c, &p->tm_k) &&
                         encode_apart(d, c->v_pool, c, &p->tm_v));
}

pda_status run_quant(pda_ctx* ctx, const pda_bf16* q, const pda_cache* c, const int32_t* table, int32_t max_blocks,
                     const int32_t* lens, int32_t batch, int32_t q_len, float scale, void* out, bool f32,
                     cudaStream_t stream) {
    pda::QuantParams p = {};
    pda_status st = pda::check_scale(scale, ctx->dims.head_dim, &p.scale_log2);
    if (st != PDA_OK) return st;
    const pda_dims& d = ctx->dims;
    const int D = d.head_dim, G = ctx->G, Hq = d.num_q_heads, Hkv = d.num_kv_heads, bs = d.block_size;
    // Queries of a sequence share one walk over its KV, 8 q rows of it or, where
    // there are more and the shape has it, 16.
    const int tiles = q_len * G > 8 && ctx->quant_ctas[1] > 0 ? 2 : 1;
    const int qp = std::max(1, std::min(q_len, 8 * tiles / G));
    const int Qr = (q_len + qp - 1) / qp;
    const pda::QuantForm form = {c->format, tiles, q_len > 1, f32};
    const pda::QuantShape shape = pda::quant_shape(D, form);
    const int grid = ctx->quant_ctas[tiles - 1];
    if (Qr > grid) return fail(PDA_ERR_INVALID_ARG, "q_len %d: more launch rows per sequence than CTAs (%d)", q_len, grid);
    p.unit_cost = pda::quant_unit_cost(D, tiles, bs);
    if ((st = pda::check_plan_size((int64_t)batch * q_len, max_blocks, p.unit_cost)) != PDA_OK) return st;
    pda::set_quant_pools(ctx, c, &p);
    p.part_o = ctx->part_o;
    p.part_ml = ctx->part_ml;
    p.unit_sync = ctx->unit_sync;
    p.err = ctx->err;
    p.table_stride = max_blocks;
    p.q_len = q_len;
    p.qp = qp;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = G;
    p.rows_per_slot = qp * G;
    p.bs = bs;
    p.prefetch = p.row_gather == 0 && bs >= 8 && Qr == 1;

    // launch rows per chunk (whole sequences), as many as the partial states allow
    const int64_t fit = (ctx->part_rows / p.rows_per_slot - grid) / p.Hkv;
    const int32_t rows_total = batch * Qr;
    const int32_t chunk = (int32_t)(std::min<int64_t>(pda::kMaxLaunchBatch, fit) / Qr) * Qr;
    if (chunk < 1)
        return fail(PDA_ERR_UNSUPPORTED, "q_len %d: a sequence's %d launch rows exceed the partial-state buffers", q_len,
                    Qr);
    const bool timing = ctx->ev_begin && ctx->ev_split && ctx->ev_end;
    if (timing)
        if (const cudaError_t e = cudaEventRecord(ctx->ev_begin, stream); e != cudaSuccess)
            return cuda_fail(e, "cudaEventRecord");
    for (int32_t c0 = 0; c0 < rows_total; c0 += chunk) {
        const int64_t s0 = c0 / Qr;  // first sequence of the chunk
        p.B = std::min(chunk, rows_total - c0);
        p.q = q + s0 * q_len * Hq * D;
        p.table = table + s0 * max_blocks;
        p.lens = lens + s0;
        p.out = f32 ? nullptr : static_cast<uint16_t*>(out) + s0 * q_len * Hq * D;
        p.out_f32 = f32 ? static_cast<float*>(out) + s0 * q_len * Hq * D : nullptr;
        const cudaError_t e = pda::launch_quant(D, form, p, grid, shape.smem(p.B), stream);
        if (e != cudaSuccess) return cuda_fail(e, "decode_cache launch");
    }
    if (timing)
        for (const cudaEvent_t ev : {ctx->ev_split, ctx->ev_end})
            if (const cudaError_t e = cudaEventRecord(ev, stream); e != cudaSuccess)
                return cuda_fail(e, "cudaEventRecord");
    ctx->tile_steps = 0;
    return PDA_OK;
}

}  // namespace

void pda::set_quant_pools(const pda_ctx* ctx, const pda_cache* c, QuantParams* p) {
    p->row_gather = encode_boxes(ctx->dims, c, p) ? 0 : 2;
    p->v_first = p->joined && c->v_pool < c->k_pool;
    p->box_head = ctx->dims.head_dim == 256 ? 2 : 1;
    p->num_blocks = c->num_blocks;
    p->k_base = static_cast<const uint16_t*>(c->k_pool);
    p->v_base = static_cast<const uint16_t*>(c->v_pool);
    p->blk_s = c->blk_stride;
    p->tok_s = c->tok_stride;
    p->kvh_s = c->kvh_stride;
    p->scales = c->scales;
}

pda_status pda::quant_setup(pda_ctx* ctx, int optin) {
    const int D = ctx->dims.head_dim;
    if (const cudaError_t e = heads_setup(D); e != cudaSuccess) return cuda_fail(e, "norm_rope / append attributes");
    for (int tiles = 1; tiles <= 2; ++tiles) {
        int per_sm = 1 << 30;
        for (int format : {PDA_CACHE_E4M3, PDA_CACHE_INT8})
            for (int k = 0; k < 4; ++k) {
                const QuantShape s = quant_shape(D, {format, tiles, (k & 1) != 0, (k & 2) != 0});
                if (!s.fn) { per_sm = 0; continue; }
                const int limit = (int)s.smem(kMaxLaunchBatch);
                if (limit > optin)
                    return fail(PDA_ERR_UNSUPPORTED, "needs %d bytes of shared memory per CTA (device allows %d)", limit,
                                optin);
                int n = 0;
                cudaError_t e = cudaFuncSetAttribute(s.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(s.fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
                if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, s.fn, s.threads, limit);
                if (e != cudaSuccess) return cuda_fail(e, "8-bit kernel attributes");
                per_sm = std::min(per_sm, n);
            }
        ctx->quant_ctas[tiles - 1] = per_sm * ctx->num_sms;
    }
    return ctx->quant_ctas[0] > 0 ? PDA_OK : fail(PDA_ERR_UNSUPPORTED, "8-bit kernel does not fit on an SM");
}

PDA_EXPORT pda_status pda_norm_rope(pda_ctx* ctx, const pda_heads* q, const pda_heads* k, const int32_t* positions,
                                    int64_t num_tokens, const pda_prep* prep, const pda_heads* q_out,
                                    const pda_heads* k_out, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    if (!prep) return fail(PDA_ERR_INVALID_ARG, "prep is NULL");
    if (num_tokens < 0 || num_tokens > INT32_MAX) return fail(PDA_ERR_INVALID_ARG, "token count outside [0, 2^31)");
    if (!q != !q_out || !k != !k_out) return fail(PDA_ERR_INVALID_ARG, "q and k each need an output, and it an input");
    if (!q && !k) return fail(PDA_ERR_INVALID_ARG, "neither q nor k given");
    pda_status st = check_prep(prep, ctx->dims.head_dim);
    if (st != PDA_OK) return st;
    if (num_tokens == 0) return PDA_OK;
    if ((q && ((st = check_heads(q, "q")) != PDA_OK || (st = check_heads(q_out, "q_out")) != PDA_OK)) ||
        (k && ((st = check_heads(k, "k")) != PDA_OK || (st = check_heads(k_out, "k_out")) != PDA_OK)))
        return st;
    if (prep->cos_sin && (!positions || !aligned(positions, 4)))
        return fail(PDA_ERR_INVALID_ARG, "the rotation needs positions (4-byte aligned)");
    pda::HeadsParams p = {};
    p.q = heads(q);
    p.k = heads(k);
    p.q_out = heads(q_out);
    p.k_out = heads(k_out);
    set_prep(p, prep);
    p.positions = positions;
    p.T = num_tokens;
    p.Hq = ctx->dims.num_q_heads;
    p.Hkv = ctx->dims.num_kv_heads;
    p.err = ctx->err;
    p.sms = ctx->num_sms;
    DeviceGuard on(ctx->device);
    ctx->tile_steps = 0;
    const cudaError_t e = pda::launch_heads(ctx->dims.head_dim, pda::kNoCache, p, (cudaStream_t)stream);
    return e == cudaSuccess ? PDA_OK : cuda_fail(e, "norm_rope launch");
}

PDA_EXPORT pda_status pda_append(pda_ctx* ctx, const pda_heads* k, const pda_heads* v, const pda_cache* cache,
                                 const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                 int32_t batch, const int32_t* starts, const int32_t* positions, int64_t num_tokens,
                                 const pda_prep* prep, const pda_heads* q, const pda_heads* q_out, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    pda_status st = check_cache(cache);
    if (st == PDA_OK) st = check_sequences(ctx, block_table, max_blocks, seq_lens, batch, starts, num_tokens);
    if (st == PDA_OK) st = check_prep(prep, ctx->dims.head_dim);
    if (st != PDA_OK) return st;
    if (!q != !q_out) return fail(PDA_ERR_INVALID_ARG, "q and q_out go together");
    if (batch == 0 || num_tokens == 0) return PDA_OK;
    if (!k || !v) return fail(PDA_ERR_INVALID_ARG, "k / v are NULL");
    if ((st = check_heads(k, "k")) != PDA_OK || (st = check_heads(v, "v")) != PDA_OK ||
        (q && ((st = check_heads(q, "q")) != PDA_OK || (st = check_heads(q_out, "q_out")) != PDA_OK)))
        return st;
    if (!aligned(positions, 4)) return fail(PDA_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    pda::HeadsParams p = {};
    p.q = heads(q);
    p.k = heads(k);
    p.v = heads(v);
    p.q_out = heads(q_out);
    set_prep(p, prep);
    p.positions = positions;
    p.c = cache_ref(ctx, cache, block_table, max_blocks, seq_lens, batch, starts, num_tokens);
    p.T = num_tokens;
    p.Hq = ctx->dims.num_q_heads;
    p.Hkv = ctx->dims.num_kv_heads;
    p.err = ctx->err;
    p.sms = ctx->num_sms;
    DeviceGuard on(ctx->device);
    ctx->tile_steps = 0;  // a following tile step reads what this writes: it must wait
    const cudaError_t e = pda::launch_heads(ctx->dims.head_dim, cache->format, p, (cudaStream_t)stream);
    return e == cudaSuccess ? PDA_OK : cuda_fail(e, "append launch");
}

PDA_EXPORT pda_status pda_read_cache(pda_ctx* ctx, const pda_cache* cache, const int32_t* block_table,
                                     int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                     const int32_t* starts, int64_t num_rows, void* k_out, void* v_out,
                                     int32_t out_f32, pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    pda_status st = check_cache(cache);
    if (st == PDA_OK) st = check_sequences(ctx, block_table, max_blocks, seq_lens, batch, starts, num_rows);
    if (st != PDA_OK) return st;
    if (batch == 0 || num_rows == 0) return PDA_OK;
    if ((!k_out && !v_out) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(PDA_ERR_INVALID_ARG, "k_out / v_out must be 16-byte aligned, one of them non-NULL");
    pda::ReadParams p = {};
    p.c = cache_ref(ctx, cache, block_table, max_blocks, seq_lens, batch, starts, num_rows);
    p.k_out = k_out;
    p.v_out = v_out;
    p.rows = num_rows;
    p.Hkv = ctx->dims.num_kv_heads;
    p.err = ctx->err;
    DeviceGuard on(ctx->device);
    ctx->tile_steps = 0;
    const cudaError_t e = pda::launch_read(ctx->dims.head_dim, cache->format, out_f32 != 0, p, (cudaStream_t)stream);
    return e == cudaSuccess ? PDA_OK : cuda_fail(e, "read_cache launch");
}

PDA_EXPORT pda_status pda_decode_cache(pda_ctx* ctx, const pda_bf16* q, const pda_cache* cache,
                                       const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                       int32_t batch, int32_t q_len, float scale, void* out, int32_t out_f32,
                                       pda_stream stream) {
    if (!ctx) return fail(PDA_ERR_INVALID_ARG, "ctx is NULL");
    pda_status st = check_cache(cache);
    if (st != PDA_OK) return st;
    const pda_dims& d = ctx->dims;
    if (q_len < 1) return fail(PDA_ERR_INVALID_ARG, "q_len %d must be >= 1", q_len);
    if (batch < 0 || (int64_t)batch * q_len > d.max_seqs)
        return fail(PDA_ERR_INVALID_ARG, "batch %d x q_len %d outside [0, max_seqs=%d]", batch, q_len, d.max_seqs);
    if (batch == 0) return PDA_OK;
    DeviceGuard on(ctx->device);
    if (cache->format == PDA_CACHE_BF16) {
        if (q_len > 1 && out_f32) return fail(PDA_ERR_UNSUPPORTED, "fp32 output of a bf16 cache needs q_len 1");
        if (q_len > 1)
            return pda::decode_bf16_multi(ctx, q, cache, block_table, max_blocks, seq_lens, batch, q_len, scale,
                                          static_cast<pda_bf16*>(out), stream);
        if (out_f32)
            return pda_decode_f32(ctx, q, static_cast<const pda_bf16*>(cache->k_pool),
                                  static_cast<const pda_bf16*>(cache->v_pool), cache->num_blocks, cache->blk_stride,
                                  cache->tok_stride, cache->kvh_stride, block_table, max_blocks, seq_lens, batch, scale,
                                  static_cast<float*>(out), stream);
        return pda_decode_strided(ctx, q, static_cast<const pda_bf16*>(cache->k_pool),
                                  static_cast<const pda_bf16*>(cache->v_pool), cache->num_blocks, cache->blk_stride,
                                  cache->tok_stride, cache->kvh_stride, block_table, max_blocks, seq_lens, batch, scale,
                                  static_cast<pda_bf16*>(out), stream);
    }
    if (!q || !aligned(q, 16) || !out || !aligned(out, 16))
        return fail(PDA_ERR_INVALID_ARG, "q and out must be non-NULL and 16-byte aligned");
    if (!block_table || !seq_lens || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return fail(PDA_ERR_INVALID_ARG, "block_table / seq_lens must be non-NULL and 4-byte aligned");
    if (max_blocks < 1) return fail(PDA_ERR_INVALID_ARG, "block table width must be >= 1 (got %d)", max_blocks);
    return run_quant(ctx, q, cache, block_table, max_blocks, seq_lens, batch, q_len, scale, out, out_f32 != 0,
                     (cudaStream_t)stream);
}
