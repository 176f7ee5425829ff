// Host side of the attention block's operators: argument checks, the handle's
// workspace, and the choice of kernels.
#include <math.h>
#include <stdio.h>

#include <new>

#include "paged.h"

namespace dfl {
dflash_status host_fail(dflash_status st, const char *msg);
dflash_status host_make_tmap_pages(CUtensorMap *tm, const void *ptr, int bytes, int head_dim, int slots, int heads,
                                   int64_t pages, int64_t slot_stride, int64_t head_stride, int64_t page_stride,
                                   int box_rows);
}

struct dflash_paged_ctx {
    dflash_paged_config cfg;
    int dev = 0, num_sms = 0;
    float *part_o = nullptr;
    float2 *part_ml = nullptr;
    int4 *merge = nullptr;
    unsigned *ticket = nullptr;
    int *err = nullptr;
    void *block = nullptr;  // the one allocation
};

namespace {

dflash_status paged_fail(dflash_status st, const char *fmt, long long a = 0, long long b = 0)
{
    char buf[256];
    snprintf(buf, sizeof buf, fmt, a, b);
    return dfl::host_fail(st, buf);
}

bool misaligned(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

// Rows [tokens, heads, head_dim] of 16-bit values: aligned, strides in whole 16 bytes.
bool bad_rows(const void *p, int64_t ts, int64_t hs)
{
    return !p || misaligned(p) || ts < 0 || hs < 0 || ts % 8 != 0 || hs % 8 != 0;
}

dflash_status check_transform(const dflash_qk_transform *t, int head_dim)
{
    if (t->rotary_dim < 0 || t->rotary_dim > head_dim || t->rotary_dim % 16 != 0)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim = %lld] (got %lld)",
                          head_dim, t->rotary_dim);
    if (t->rotary_dim > 0 && (!t->table || misaligned(t->table) || t->positions < 1 || t->positions >= (int64_t(1) << 31)))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "a rotation needs a 16-byte aligned table of 1 to 2^31 - 1 positions");
    if (t->interleaved != 0 && t->interleaved != 1)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %lld)", t->interleaved);
    if (misaligned(t->q_weight) || misaligned(t->k_weight))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "norm weights must be 16-byte aligned");
    if (!(t->eps >= 0.f) || isinf(t->eps)) return paged_fail(DFLASH_ERR_INVALID_ARG, "eps must be finite and >= 0");
    return DFLASH_OK;
}

void set_transform(dfl::PrepParams &p, const dflash_qk_transform *t)
{
    p.table = t->table;
    p.positions_n = static_cast<int>(t->positions);
    p.rotary = t->rotary_dim;
    p.interleaved = t->interleaved;
    p.eps = t->eps;
    p.q.weight = t->q_weight;
    p.k.weight = t->k_weight;
}

dflash_status check_call(dflash_paged_handle h, const dflash_paged_cache *c, const dflash_paged_batch *b)
{
    if (!h) return paged_fail(DFLASH_ERR_INVALID_ARG, "handle is NULL");
    if (!c || !b) return paged_fail(DFLASH_ERR_INVALID_ARG, "cache and batch must not be NULL");
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return paged_fail(DFLASH_ERR_CUDA, "querying the current device failed");
    if (dev != h->dev)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "the handle belongs to device %lld, the current device is %lld", h->dev, dev);
    if (b->batch < 0 || b->batch > h->cfg.max_batch)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "batch must be in [0, max_batch = %lld] (got %lld)", h->cfg.max_batch, b->batch);
    if (b->tokens < 0 || b->max_tokens < 0)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "tokens and max_tokens must be >= 0 (got %lld, %lld)", b->tokens, b->max_tokens);
    if (b->tokens > 1 << 30)  // (places less a window of up to 2^30 stay in 32 bits)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "tokens must be at most 2^30 (got %lld)", b->tokens);
    if (static_cast<int64_t>(b->tokens) * h->cfg.heads >= (int64_t(1) << 31))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "tokens * heads must be below 2^31 (got %lld * %lld)", b->tokens, h->cfg.heads);
    if (b->batch > 0 && (!b->cu_tokens || !b->lens || !b->page_table || b->table_cols < 1 || b->table_stride < 0))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "cu_tokens, lens and page_table must be given, table_cols >= 1, table_stride >= 0");
    if (!c->k || !c->v || misaligned(c->k) || misaligned(c->v))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "the cache's k and v must be given and 16-byte aligned");
    if (c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "num_pages must be in [1, 2^31) (got %lld)", c->num_pages);
    const int64_t unit = h->cfg.cache_dtype == DFLASH_E4M3 ? 16 : 8;
    for (int64_t s : {c->page_stride, c->slot_stride, c->head_stride})
        if (s < 0 || s % unit != 0)
            return paged_fail(DFLASH_ERR_INVALID_ARG, "cache strides must be multiples of %lld elements (got %lld)", unit, s);
    // (ordinary numbers: the reciprocal of a smaller one may be infinite)
    if (h->cfg.cache_dtype == DFLASH_E4M3 && !(c->k_scale > 0.f && c->v_scale > 0.f && isnormal(c->k_scale) && isnormal(c->v_scale)))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "an 8-bit cache needs ordinary fp32 numbers > 0 as k_scale and v_scale");
    return DFLASH_OK;
}

}  // namespace

// The current device (-1: none), for the binding, which compares it with the tensors' device.
extern "C" int dflash_paged_current_device(void)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

extern "C" dflash_status dflash_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride, void *q_out,
                                             int64_t qo_token_stride, int64_t qo_head_stride, const void *k,
                                             int64_t k_token_stride, int64_t k_head_stride, void *k_out,
                                             int64_t ko_token_stride, int64_t ko_head_stride, int32_t tokens,
                                             int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                             const dflash_qk_transform *transform, const int32_t *positions, void *stream)
{
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %lld)", head_dim);
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP16)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "dtype must be BF16 or FP16 (got %lld)", dtype);
    if (tokens < 0 || heads < 0 || kv_heads < 0)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "tokens and heads must be >= 0");
    if (static_cast<int64_t>(tokens) * (heads > kv_heads ? heads : kv_heads) >= (int64_t(1) << 31))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "tokens * heads must be below 2^31 (tokens = %lld)", tokens);
    if (!transform) return paged_fail(DFLASH_ERR_INVALID_ARG, "transform must not be NULL");
    dflash_status st = check_transform(transform, head_dim);
    if (st != DFLASH_OK) return st;
    if (transform->rotary_dim > 0 && !positions && tokens > 0)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "a rotation needs positions");
    const bool has_q = q && heads > 0, has_k = k && kv_heads > 0;
    if (tokens == 0 || (!has_q && !has_k)) return DFLASH_OK;
    if ((has_q && (bad_rows(q, q_token_stride, q_head_stride) || bad_rows(q_out, qo_token_stride, qo_head_stride))) ||
        (has_k && (bad_rows(k, k_token_stride, k_head_stride) || bad_rows(k_out, ko_token_stride, ko_head_stride))))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "q, k and their outputs must be 16-byte aligned, with strides of whole 16 bytes");
    dfl::PrepParams p;
    if (has_q) p.q = {q, q_out, q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, nullptr, heads};
    if (has_k) p.k = {k, k_out, k_token_stride, k_head_stride, ko_token_stride, ko_head_stride, nullptr, kv_heads};
    set_transform(p, transform);
    p.tokens = tokens;
    p.positions = positions;
    const cudaError_t e = dfl::launch_prep(p, head_dim, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return paged_fail(DFLASH_ERR_CUDA, "norm and rotation: the launch failed (error %lld)", e);
    return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_init(const dflash_paged_config *cfg, void *stream, dflash_paged_handle *out)
{
    if (!out) return paged_fail(DFLASH_ERR_INVALID_ARG, "out must not be NULL");
    *out = nullptr;
    if (!cfg) return paged_fail(DFLASH_ERR_INVALID_ARG, "cfg must not be NULL");
    if (cfg->kv_heads < 1 || cfg->heads < cfg->kv_heads || cfg->heads > 1024 || cfg->heads % cfg->kv_heads != 0)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "heads must be a multiple of kv_heads, at most 1024 (got %lld, %lld)",
                          cfg->heads, cfg->kv_heads);
    if (cfg->head_dim != 64 && cfg->head_dim != 128)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %lld)", cfg->head_dim);
    if (cfg->page_size < 16 || cfg->page_size > 1024 || cfg->page_size % 16 != 0)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "page_size must be a multiple of 16 in [16, 1024] (got %lld)", cfg->page_size);
    if (cfg->dtype != DFLASH_BF16 && cfg->dtype != DFLASH_FP16)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "dtype must be BF16 or FP16 (got %lld)", cfg->dtype);
    if (cfg->cache_dtype != cfg->dtype && cfg->cache_dtype != DFLASH_E4M3)
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "cache_dtype must be dtype or E4M3 (got %lld)", cfg->cache_dtype);
    if (cfg->max_batch < 1 || cfg->max_batch > 65536)
        return paged_fail(DFLASH_ERR_INVALID_ARG, "max_batch must be in [1, 65536] (got %lld)", cfg->max_batch);
    dflash_paged_ctx *c = new (std::nothrow) dflash_paged_ctx;
    if (!c) return paged_fail(DFLASH_ERR_CUDA, "out of host memory");
    c->cfg = *cfg;
    int major = 0, minor = 0, smem_optin = 0;
    if (cudaGetDevice(&c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, c->dev) != cudaSuccess) {
        delete c;
        return paged_fail(DFLASH_ERR_CUDA, "querying the current device failed");
    }
    if (major != 10 || minor != 3) {
        delete c;
        return paged_fail(DFLASH_ERR_UNSUPPORTED, "built for sm_103 (GB300); device is sm_%lld%lld", major, minor);
    }
    // Partial results: two slots per CTA of the larger of the two kernels' grids.
    const size_t rows = 2 * static_cast<size_t>(c->num_sms) * dfl::kTileRows;
    static_assert(dfl::kTileRows >= 2 * 32, "two CTAs of up to 32 rows per SM, or one of kTileRows");
    const size_t o_bytes = rows * cfg->head_dim * sizeof(float), ml_bytes = rows * sizeof(float2);
    const size_t merge_bytes = 2 * static_cast<size_t>(c->num_sms) * 3 * sizeof(int4);
    const size_t ticket_bytes = 3 * static_cast<size_t>(c->num_sms) * dfl::kTicketWarps * sizeof(unsigned);
    const size_t total = o_bytes + ml_bytes + merge_bytes + ticket_bytes + 256;
    if (dfl::prepare_attend_rows(smem_optin) != cudaSuccess || dfl::prepare_attend_tile(smem_optin) != cudaSuccess ||
        cudaMalloc(&c->block, total) != cudaSuccess) {
        delete c;
        cudaGetLastError();
        return paged_fail(DFLASH_ERR_CUDA, "setting up paged attention failed (workspace of %lld bytes)", total);
    }
    char *at = static_cast<char *>(c->block);
    c->part_o = reinterpret_cast<float *>(at);
    c->part_ml = reinterpret_cast<float2 *>(at + o_bytes);
    c->merge = reinterpret_cast<int4 *>(at + o_bytes + ml_bytes);
    c->ticket = reinterpret_cast<unsigned *>(at + o_bytes + ml_bytes + merge_bytes);
    c->err = reinterpret_cast<int *>(at + o_bytes + ml_bytes + merge_bytes + ticket_bytes);
    // (waited for: the first call may be on another stream)
    if (cudaMemsetAsync(c->ticket, 0, ticket_bytes + 256, static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaFree(c->block);
        delete c;
        return paged_fail(DFLASH_ERR_CUDA, "clearing the workspace failed");
    }
    *out = c;
    return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_append(dflash_paged_handle h, const dflash_paged_cache *cache,
                                             const dflash_paged_batch *batch, const void *k, int64_t k_token_stride,
                                             int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                             int64_t v_head_stride, const dflash_qk_transform *transform,
                                             const int32_t *positions, const void *q, int64_t q_token_stride,
                                             int64_t q_head_stride, void *q_out, int64_t qo_token_stride,
                                             int64_t qo_head_stride, void *stream)
{
    dflash_status st = check_call(h, cache, batch);
    if (st != DFLASH_OK) return st;
    if (transform && (st = check_transform(transform, h->cfg.head_dim)) != DFLASH_OK) return st;
    if (batch->batch == 0 || batch->tokens == 0) return DFLASH_OK;
    if (bad_rows(k, k_token_stride, k_head_stride) || bad_rows(v, v_token_stride, v_head_stride) ||
        (q && (bad_rows(q, q_token_stride, q_head_stride) || bad_rows(q_out, qo_token_stride, qo_head_stride))))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "k, v, q and q_out must be 16-byte aligned, with strides of whole 16 bytes");
    dfl::PrepParams p;
    if (q) p.q = {q, q_out, q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, nullptr, h->cfg.heads};
    p.k = {k, nullptr, k_token_stride, k_head_stride, 0, 0, nullptr, h->cfg.kv_heads};
    p.v = {v, nullptr, v_token_stride, v_head_stride, 0, 0, nullptr, h->cfg.kv_heads};
    if (transform) set_transform(p, transform);
    p.tokens = batch->tokens;
    p.positions = positions;
    p.append = 1;
    p.fp8 = h->cfg.cache_dtype == DFLASH_E4M3;
    p.cache = *cache;
    p.batch = *batch;
    p.page = h->cfg.page_size;
    p.err = h->err;
    const cudaError_t e = dfl::launch_prep(p, h->cfg.head_dim, h->cfg.dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return paged_fail(DFLASH_ERR_CUDA, "append: the launch failed (error %lld)", e);
    return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_attend(dflash_paged_handle h, const dflash_paged_cache *cache,
                                             const dflash_paged_batch *batch, const void *q, int64_t q_token_stride,
                                             int64_t q_head_stride, void *out, int64_t out_token_stride,
                                             int64_t out_head_stride, float *lse, int32_t causal, int32_t window,
                                             float scale, void *stream)
{
    const dflash_status st = check_call(h, cache, batch);
    if (st != DFLASH_OK) return st;
    if (causal != 0 && causal != 1) return paged_fail(DFLASH_ERR_INVALID_ARG, "causal must be 0 or 1 (got %lld)", causal);
    if (window < 0) return paged_fail(DFLASH_ERR_INVALID_ARG, "window must be >= 0 (got %lld)", window);
    if (!(scale > 0.f) || isinf(scale)) return paged_fail(DFLASH_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (batch->batch == 0 || batch->tokens == 0) return DFLASH_OK;
    if (bad_rows(q, q_token_stride, q_head_stride) || bad_rows(out, out_token_stride, out_head_stride))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "q and out must be 16-byte aligned, with strides of whole 16 bytes");
    if (q == out) return paged_fail(DFLASH_ERR_INVALID_ARG, "out must not overlap q");
    const bool fp8 = h->cfg.cache_dtype == DFLASH_E4M3;
    dfl::AttendParams p;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.o_ts = out_token_stride;
    p.o_hs = out_head_stride;
    p.k = cache->k;
    p.v = cache->v;
    p.page_stride = cache->page_stride;
    p.slot_stride = cache->slot_stride;
    p.head_stride = cache->head_stride;
    p.cu = batch->cu_tokens;
    p.lens = batch->lens;
    p.table = batch->page_table;
    p.table_stride = batch->table_stride;
    p.table_cols = batch->table_cols;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.B = batch->batch;
    p.tokens = batch->tokens;
    p.kv_heads = h->cfg.kv_heads;
    p.group = h->cfg.heads / h->cfg.kv_heads;
    p.page = h->cfg.page_size;
    p.by_group = dfl::FastDiv(p.group);
    p.by_page = dfl::FastDiv(p.page);
    p.causal = causal;
    p.window = window < (1 << 30) ? window : 1 << 30;  // (places are sums with it)
    p.scale_log2 = scale * 1.44269504088896341f * (fp8 ? cache->k_scale : 1.f);
    p.v_scale = fp8 ? cache->v_scale : 1.f;
    p.part_o = h->part_o;
    p.part_ml = h->part_ml;
    p.merge = h->merge;
    p.ticket = h->ticket;
    p.err = h->err;
    if (!isnormal(p.scale_log2))
        return paged_fail(DFLASH_ERR_INVALID_ARG, "scale (times k_scale) must be an ordinary fp32 number");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t most_rows = static_cast<int64_t>(batch->max_tokens) * p.group;
    cudaError_t e;
    int rows, grid;
    auto most_units = [&](int unit) { return (static_cast<int64_t>(p.table_cols) * p.page + unit - 1) / unit; };
    // In a call of no more than a unit a CTA the next launch's start-up may hide behind the merge; in a longer one its
    // CTAs would take the places of those that are still to come (a block of 8 after 2041 keys: 13.5 us a call, 14.3
    // without; 128 single tokens of 64-value heads: 110 us, 86 without).
    auto short_call = [&](int unit, int item_rows, int ctas) {
        return static_cast<double>(most_units(unit)) * ((most_rows + item_rows - 1) / item_rows) * p.B * p.kv_heads <= ctas;
    };
    // The few-row kernel keeps up to 32 rows of accumulators in registers and streams the keys near the memory's rate
    // (32 ragged sequences of 32 rows: 98 us, 84 with an 8-bit cache; by the other 107 and 115; of 4 rows: 86 and
    // 105). Beyond 32 it would read them once per 32 rows, where the tensor-memory kernel takes 256 (64 rows: 106 us,
    // by this one 158).
    if (most_rows > 32) {
        CUtensorMap tm_k, tm_v;
        const int box = dfl::tile_box_rows(p.page), bytes = fp8 ? 1 : 2;
        dflash_status st2 = dfl::host_make_tmap_pages(&tm_k, p.k, bytes, h->cfg.head_dim, p.page, p.kv_heads, p.num_pages,
                                                      p.slot_stride, p.head_stride, p.page_stride, box);
        if (st2 == DFLASH_OK)
            st2 = dfl::host_make_tmap_pages(&tm_v, p.v, bytes, h->cfg.head_dim, p.page, p.kv_heads, p.num_pages,
                                            p.slot_stride, p.head_stride, p.page_stride, box);
        if (st2 != DFLASH_OK) return st2;
        rows = dfl::kTileRows;
        grid = h->num_sms;
        dfl::set_lanes(p, grid, 1);
        p.merge_early = short_call(dfl::kTileUnit, rows, grid);
        e = dfl::launch_attend_tile(p, tm_k, tm_v, h->cfg.head_dim, h->cfg.dtype, fp8, grid, s);
    } else {
        // (With up to 8 rows by the variant for 16: 128 single tokens of an 8-bit cache 95 us, not 88; up to 16 by the
        // one for 32: 80 us, not 60.)
        rows = most_rows <= 8 ? 8 : (most_rows <= 16 ? 16 : 32);
        grid = (rows <= 16 ? 3 : 2) * h->num_sms;
        dfl::set_lanes(p, grid, p.kv_heads);
        p.merge_early = short_call(dfl::kRowsUnit, rows, grid);
        e = dfl::launch_attend_rows(p, h->cfg.head_dim, h->cfg.dtype, fp8, rows, grid, s);
    }
    // An item of few units is joined by the CTAs that share it.
    if (e == cudaSuccess && most_units(rows == dfl::kTileRows ? dfl::kTileUnit : dfl::kRowsUnit) > dfl::kTicketParts)
        e = dfl::launch_attend_merge(p, h->cfg.head_dim, h->cfg.dtype, rows, grid, rows == dfl::kTileRows, 3 * h->num_sms, s);
    if (e != cudaSuccess) return paged_fail(DFLASH_ERR_CUDA, "attention: a launch failed (error %lld)", e);
    return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_sync_status(dflash_paged_handle h, void *stream)
{
    if (!h) return paged_fail(DFLASH_ERR_INVALID_ARG, "handle is NULL");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int e = 0;
    if (cudaMemcpyAsync(&e, h->err, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return paged_fail(DFLASH_ERR_CUDA, "reading the device error word failed");
    if (e == 0) return DFLASH_OK;
    // (with the counters of split items, which a pipeline that gave up may have left behind)
    const size_t bytes = reinterpret_cast<char *>(h->err + 1) - reinterpret_cast<char *>(h->ticket);
    if (cudaMemsetAsync(h->ticket, 0, bytes, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return paged_fail(DFLASH_ERR_CUDA, "clearing the device error word failed");
    if (e & dfl::DEV_ERR_TIMEOUT)
        return paged_fail(DFLASH_ERR_TIMEOUT, "an attention pipeline wait exceeded its time bound (error word %lld)", e);
    return paged_fail(DFLASH_ERR_DEVICE_CHECK, "a page id, place or position was outside its table (error word %lld)", e);
}

extern "C" dflash_status dflash_paged_destroy(dflash_paged_handle h)
{
    if (!h) return DFLASH_OK;
    cudaDeviceSynchronize();
    cudaFree(h->block);
    delete h;
    return DFLASH_OK;
}
