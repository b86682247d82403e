// C ABI of trees of drafts and of the paged cache (declared in
// include/topk_cols.h): argument checks and dispatch to the kernels.  Nothing
// here allocates, synchronizes or aborts.
#include "topk_cols.h"

#include "topk_cache.hpp"

namespace {

constexpr int64_t kMax32 = 0x7FFFFFFF;
constexpr int64_t kMaxRows = (int64_t)1 << 26;   // columns times heads: a launch has at most 2^32 - 1 threads
constexpr int64_t kMaxPlanes = (int64_t)1 << 20; // layers times heads

bool misaligned(const void* p, uintptr_t bytes) { return (uintptr_t)p % bytes != 0; }
bool known_dtype(int32_t dtype) { return dtype == TOPK_BF16 || dtype == TOPK_F32; }
bool bad_stride(int64_t stride, int64_t unit) { return stride < 0 || stride % unit != 0; }
int answer(hipError_t e) { return e == hipSuccess ? TOPK_OK : TOPK_ERR_HIP; }

int make_parts(topk::Parts* parts, const int32_t* start, int64_t total, int64_t lanes) {
    if (misaligned(start, 4) || (!start && total % lanes != 0)) return TOPK_ERR_INVALID_ARG;
    parts->start = start;
    parts->total = (uint32_t)total;
    parts->each = start ? 1u : (uint32_t)(total / lanes);
    return TOPK_OK;
}

// Offset of the last slot of a layer.
unsigned __int128 last_slot(const topk_cache& c, int64_t block_stride, int64_t slot_stride) {
    return (unsigned __int128)(c.blocks - 1) * (uint64_t)block_stride + (unsigned __int128)(c.block_size - 1) * (uint64_t)slot_stride;
}

int check_cache(const topk_cache* c) {
    if (!c || c->layers < 1 || c->blocks < 1 || c->block_size < 1 || c->heads < 1 || c->dim < 16 || c->dim % 16 != 0)
        return TOPK_ERR_INVALID_ARG;
    if (c->format != TOPK_CACHE_BF16 && c->format != TOPK_CACHE_FP8) return TOPK_ERR_INVALID_ARG;
    if (!c->keys || !c->values || misaligned(c->keys, 16) || misaligned(c->values, 16)) return TOPK_ERR_INVALID_ARG;
    const int64_t unit = c->format == TOPK_CACHE_BF16 ? 8 : 16;
    if (bad_stride(c->layer_stride, unit) || bad_stride(c->block_stride, unit) || bad_stride(c->slot_stride, unit) ||
        bad_stride(c->head_stride, unit))
        return TOPK_ERR_INVALID_ARG;
    if (c->format == TOPK_CACHE_FP8 &&
        (!c->key_scales || !c->value_scales || c->scale_layer_stride < 0 || c->scale_block_stride < 0 ||
         c->scale_slot_stride < 0 || c->scale_head_stride < 0))
        return TOPK_ERR_INVALID_ARG;
    if (c->dim > TOPK_MAX_DIM || c->blocks > kMax32 / c->block_size || c->layers > kMaxPlanes / c->heads)
        return TOPK_ERR_UNSUPPORTED;
    // offsets within a layer are computed in 32 bits, of rows' 16-byte parts in units of those: the last one has to fit
    if ((last_slot(*c, c->block_stride / unit, c->slot_stride / unit) + (uint64_t)(c->dim / unit - 1)) >> 32 ||
        (c->format == TOPK_CACHE_FP8 && last_slot(*c, c->scale_block_stride, c->scale_slot_stride) >> 32))
        return TOPK_ERR_UNSUPPORTED;
    return TOPK_OK;
}

// The cache from `layer` on.
topk::Cache cache_at(const topk_cache& c, int64_t layer) {
    const int64_t size = c.format == TOPK_CACHE_BF16 ? 2 : 1;
    topk::Cache a = {c, topk::Divisor::of((uint32_t)c.block_size), (uint32_t)(c.block_stride * size / 16), (uint32_t)(c.slot_stride * size / 16),
                     (uint32_t)c.scale_block_stride, (uint32_t)c.scale_slot_stride};
    a.c.keys = static_cast<uint8_t*>(c.keys) + layer * c.layer_stride * size;
    a.c.values = static_cast<uint8_t*>(c.values) + layer * c.layer_stride * size;
    if (c.format == TOPK_CACHE_FP8) {
        a.c.key_scales = c.key_scales + layer * c.scale_layer_stride;
        a.c.value_scales = c.value_scales + layer * c.scale_layer_stride;
    }
    return a;
}

// What topk_cols_attend and topk_cols_attend_workspace check; `sizes`: no pointers.
int make_attend(topk::AttendArgs* to, const topk_cache* c, const topk_attend_args* a, bool sizes) {
    if (!a || a->lanes < 1 || a->C < 1 || a->table_ld < 1 || a->window < 0) return TOPK_ERR_INVALID_ARG;
    if (const int bad = check_cache(c)) return bad;
    if (a->layer < 0 || a->layer >= c->layers || a->heads < 1 || a->heads % c->heads != 0) return TOPK_ERR_INVALID_ARG;
    if (!(a->scale >= -0x1p127f && a->scale <= 0x1p127f)) return TOPK_ERR_INVALID_ARG;  // (its product with log2(e) is finite)
    if (bad_stride(a->q_stride, 8) || bad_stride(a->q_head_stride, 8) || bad_stride(a->out_stride, 8) ||
        bad_stride(a->out_head_stride, 8))
        return TOPK_ERR_INVALID_ARG;
    if (!sizes) {
        if (!a->q || !a->lens || !a->table || !a->out || misaligned(a->q, 16) || misaligned(a->lens, 4) ||
            misaligned(a->table, 4) || misaligned(a->out, 16) || misaligned(a->mask, 4) || misaligned(a->positions, 4) ||
            misaligned(a->workspace, 256))
            return TOPK_ERR_INVALID_ARG;
        if (a->mask && a->mask_ld < 1) return TOPK_ERR_INVALID_ARG;
    }
    if (a->lanes > TOPK_MAX_LANES || a->table_ld > kMax32 || (a->mask && a->mask_ld > kMax32) || a->C > kMaxRows / a->heads)
        return TOPK_ERR_UNSUPPORTED;
    to->cache = cache_at(*c, a->layer);
    to->a = *a;
    to->places = a->table_ld <= kMax32 / c->block_size ? (uint32_t)(a->table_ld * c->block_size) : (uint32_t)kMax32;
    return make_parts(&to->cols, a->col_start, a->C, a->lanes);
}

}  // namespace

extern "C" {

int topk_cols_tree(int64_t lanes, int64_t C, const int32_t* col_start, const int32_t* parents, const int32_t* lens,
                   uint32_t* mask, int64_t mask_ld, int32_t* positions, hipStream_t stream) {
    if (lanes < 1 || C < 1 || mask_ld < 1 || !parents || !mask || !positions) return TOPK_ERR_INVALID_ARG;
    if (misaligned(parents, 4) || misaligned(lens, 4) || misaligned(mask, 4) || misaligned(positions, 4))
        return TOPK_ERR_INVALID_ARG;
    if (lanes > TOPK_MAX_LANES || C > kMax32 || mask_ld > kMax32) return TOPK_ERR_UNSUPPORTED;
    topk::TreeArgs a = {};
    if (make_parts(&a.cols, col_start, C, lanes) != TOPK_OK) return TOPK_ERR_INVALID_ARG;
    a.lanes = (uint32_t)lanes;
    a.parents = parents;
    a.lens = lens;
    a.mask = mask;
    a.mask_ld = mask_ld;
    a.positions = positions;
    return answer(topk::launch_tree(a, stream));
}

int topk_cols_cache_write(const topk_cache* cache, const topk_cache_write_args* w, hipStream_t stream) {
    if (!w || w->C < 1 || !known_dtype(w->dtype) || !w->keys || !w->values || !w->slots) return TOPK_ERR_INVALID_ARG;
    if (const int bad = check_cache(cache)) return bad;
    if (w->layer < 0 || w->layer >= cache->layers) return TOPK_ERR_INVALID_ARG;
    const int64_t unit = w->dtype == TOPK_BF16 ? 8 : 4;
    if (misaligned(w->keys, 16) || misaligned(w->values, 16) || misaligned(w->slots, 8) || bad_stride(w->key_stride, unit) ||
        bad_stride(w->key_head_stride, unit) || bad_stride(w->value_stride, unit) || bad_stride(w->value_head_stride, unit))
        return TOPK_ERR_INVALID_ARG;
    if (w->C > kMaxRows / cache->heads) return TOPK_ERR_UNSUPPORTED;
    const topk::CacheWriteArgs a = {cache_at(*cache, w->layer), *w};
    return answer(topk::launch_cache_write(a, stream));
}

int topk_cols_cache_move(const topk_cache* cache, int64_t lanes, const int32_t* lens, const int32_t* table,
                         int64_t table_ld, const int32_t* columns, int64_t width, hipStream_t stream) {
    if (lanes < 1 || table_ld < 1 || width < 1 || !lens || !table || !columns) return TOPK_ERR_INVALID_ARG;
    if (const int bad = check_cache(cache)) return bad;
    if (misaligned(lens, 4) || misaligned(table, 4) || misaligned(columns, 4)) return TOPK_ERR_INVALID_ARG;
    if (lanes > TOPK_MAX_LANES || table_ld > kMax32 || width > kMax32) return TOPK_ERR_UNSUPPORTED;
    topk::CacheMoveArgs a = {};
    a.cache = cache_at(*cache, 0);
    a.lanes = (uint32_t)lanes;
    a.width = (uint32_t)width;
    a.lens = lens;
    a.table = table;
    a.columns = columns;
    a.table_ld = table_ld;
    return answer(topk::launch_cache_move(a, stream));
}

int topk_cols_attend_workspace(const topk_cache* cache, const topk_attend_args* args, int64_t* bytes) {
    if (!bytes) return TOPK_ERR_INVALID_ARG;
    *bytes = 0;
    topk::AttendArgs a = {};
    if (const int bad = make_attend(&a, cache, args, true)) return bad;
    *bytes = topk::attend_workspace(a);
    return TOPK_OK;
}

int topk_cols_attend(const topk_cache* cache, const topk_attend_args* args, hipStream_t stream) {
    topk::AttendArgs a = {};
    if (const int bad = make_attend(&a, cache, args, false)) return bad;
    const int64_t bytes = topk::attend_workspace(a);
    if (bytes > 0 && (!args->workspace || args->workspace_bytes < bytes)) return TOPK_ERR_INVALID_ARG;
    return answer(topk::launch_attend(a, stream));
}

int topk_cols_verify_tree(const topk_verify_tree_args* v, hipStream_t stream) {
    if (!v || v->lanes < 1 || v->C < 1 || v->max_tokens < 1 || !known_dtype(v->dtype)) return TOPK_ERR_INVALID_ARG;
    if (v->k < 1 || v->k > TOPK_MAX_K || !v->target_values || !v->target_ids || !v->tokens || !v->parents || !v->uniforms ||
        !v->out_tokens || !v->out_columns || !v->out_count)
        return TOPK_ERR_INVALID_ARG;
    if (!v->draft_values != !v->draft_ids) return TOPK_ERR_INVALID_ARG;
    if (v->draft_values && (v->kq < 1 || v->kq > TOPK_MAX_K)) return TOPK_ERR_INVALID_ARG;
    if (!(v->temperature >= 0.0) || v->temperature > 1.7976931348623157e308 || !(v->top_p > 0.0) || !(v->top_p <= 1.0))
        return TOPK_ERR_INVALID_ARG;
    const uintptr_t es = v->dtype == TOPK_BF16 ? 2 : 4;
    if (misaligned(v->target_values, es) || misaligned(v->draft_values, es) || misaligned(v->target_ids, 4) ||
        misaligned(v->draft_ids, 4) || misaligned(v->tokens, 4) || misaligned(v->parents, 4) || misaligned(v->uniforms, 4) ||
        misaligned(v->out_tokens, 4) || misaligned(v->out_columns, 4) || misaligned(v->out_count, 4))
        return TOPK_ERR_INVALID_ARG;
    if (v->lanes > TOPK_MAX_LANES || v->C > kMax32 || v->max_tokens > kMax32) return TOPK_ERR_UNSUPPORTED;
    topk::VerifyTreeArgs a = {};
    a.v = *v;
    if (make_parts(&a.cols, v->col_start, v->C, v->lanes) != TOPK_OK) return TOPK_ERR_INVALID_ARG;
    return answer(topk::launch_verify_tree(a, stream));
}

}  // extern "C"
