// C ABI of the steps around the top-k (declared in include/topk_cols.h):
// argument checks and dispatch to the kernels.  Nothing here allocates,
// synchronizes or aborts.
#include "topk_cols.h"

#include "topk_round.hpp"

namespace {

constexpr int64_t kMax32 = 0x7FFFFFFF;

bool misaligned(const void* p, uintptr_t bytes) { return (uintptr_t)p % bytes != 0; }
bool known_dtype(int32_t dtype) { return dtype == TOPK_BF16 || dtype == TOPK_F32; }
uintptr_t element_bytes(int32_t dtype) { return dtype == TOPK_BF16 ? 2 : 4; }

// [0, total) cut into lanes: by `start`, or evenly (then lanes must divide it).
int make_parts(topk::Parts* parts, const int32_t* start, int64_t total, int64_t lanes) {
    if (misaligned(start, 4) || (!start && total % lanes != 0)) return TOPK_ERR_INVALID_ARG;
    parts->start = start;
    parts->total = (uint32_t)total;
    parts->each = start ? 1u : (uint32_t)(total / lanes);
    return TOPK_OK;
}

}  // namespace

extern "C" {

int topk_cols_adjust(const topk_adjust_rules* r, const void* logits, void* out, hipStream_t stream) {
    if (!r || !logits || !out) return TOPK_ERR_INVALID_ARG;
    if (r->V < 1 || r->C < 1 || r->lanes < 1 || !known_dtype(r->dtype)) return TOPK_ERR_INVALID_ARG;
    if (r->layout != TOPK_COL_CONTIG && r->layout != TOPK_ROW_INTERLEAVED) return TOPK_ERR_INVALID_ARG;
    const int64_t least = r->layout == TOPK_COL_CONTIG ? r->V : r->C;
    if (r->ld < least || r->out_ld < least || (logits == out && r->ld != r->out_ld)) return TOPK_ERR_INVALID_ARG;
    const uintptr_t es = element_bytes(r->dtype);
    if (misaligned(logits, es) || misaligned(out, es)) return TOPK_ERR_INVALID_ARG;
    const int64_t words = (r->V + 31) / 32;
    if (!r->counts != !r->seen) return TOPK_ERR_INVALID_ARG;
    if (r->counts && (r->counts_ld < r->V || r->seen_ld < words)) return TOPK_ERR_INVALID_ARG;
    if (misaligned(r->counts, 4) || misaligned(r->seen, 4) || misaligned(r->repetition, 4) ||
        misaligned(r->presence, 4) || misaligned(r->frequency, 4))
        return TOPK_ERR_INVALID_ARG;
    if (r->n_drafts < 0 || (!r->drafts && (r->draft_start || r->n_drafts)) || misaligned(r->drafts, 4))
        return TOPK_ERR_INVALID_ARG;
    if (!r->bias_start != !r->bias_ids || !r->bias_start != !r->bias_values || r->n_bias < 0 ||
        (!r->bias_ids && r->n_bias) || misaligned(r->bias_ids, 4) || misaligned(r->bias_values, 4))
        return TOPK_ERR_INVALID_ARG;
    if (r->mask) {
        if (misaligned(r->mask, 4) || misaligned(r->mask_index, 4) || r->mask_ld < words || r->mask_count < 1 ||
            (!r->mask_index && r->mask_count < r->C))
            return TOPK_ERR_INVALID_ARG;
    } else if (r->mask_index) {
        return TOPK_ERR_INVALID_ARG;
    }
    if (r->V > TOPK_MAX_V || r->C > kMax32 || r->lanes > TOPK_MAX_LANES || r->n_drafts > kMax32 || r->n_bias > kMax32 ||
        (r->mask && r->mask_count > kMax32))
        return TOPK_ERR_UNSUPPORTED;
    topk::AdjustArgs a = {};
    if (make_parts(&a.cols, r->col_start, r->C, r->lanes) != TOPK_OK ||
        make_parts(&a.bias_parts, r->bias_start, r->bias_start ? r->n_bias : 0, r->lanes) != TOPK_OK ||
        make_parts(&a.draft_parts, r->draft_start, r->n_drafts, r->lanes) != TOPK_OK)
        return TOPK_ERR_INVALID_ARG;
    a.x = logits;
    a.out = out;
    a.ld = r->ld;
    a.out_ld = r->out_ld;
    a.V = (uint32_t)r->V;
    a.C = (uint32_t)r->C;
    a.lanes = (uint32_t)r->lanes;
    if (r->repetition || r->presence || r->frequency) {  // else the histories change nothing
        a.counts = r->counts;
        a.counts_ld = r->counts_ld;
        a.seen = r->seen;
        a.seen_ld = r->seen_ld;
        a.drafts = r->n_drafts ? r->drafts : nullptr;
    }
    a.repetition = r->repetition;
    a.presence = r->presence;
    a.frequency = r->frequency;
    a.bias_ids = r->n_bias ? r->bias_ids : nullptr;
    a.bias_values = r->bias_values;
    a.mask = r->mask;
    a.mask_ld = r->mask_ld;
    a.mask_count = (int32_t)r->mask_count;
    a.mask_index = r->mask_index;
    return topk::launch_adjust(r->dtype, r->layout, a, stream) == hipSuccess ? TOPK_OK : TOPK_ERR_HIP;
}

int topk_cols_count(int64_t V, int64_t lanes, const int32_t* ids, int64_t n_ids, const int32_t* start,
                    const int32_t* prompt_len, const int32_t* fresh, int32_t* counts, int64_t counts_ld,
                    uint32_t* seen, int64_t seen_ld, hipStream_t stream) {
    if (V < 1 || lanes < 1 || n_ids < 0 || !counts || !seen || (!ids && n_ids)) return TOPK_ERR_INVALID_ARG;
    if (counts_ld < V || seen_ld < (V + 31) / 32) return TOPK_ERR_INVALID_ARG;
    if (misaligned(ids, 4) || misaligned(prompt_len, 4) || misaligned(fresh, 4) || misaligned(counts, 4) ||
        misaligned(seen, 4))
        return TOPK_ERR_INVALID_ARG;
    if (V > TOPK_MAX_V || lanes > TOPK_MAX_LANES || n_ids > kMax32) return TOPK_ERR_UNSUPPORTED;
    topk::CountArgs a = {};
    if (make_parts(&a.parts, start, n_ids, lanes) != TOPK_OK) return TOPK_ERR_INVALID_ARG;
    a.V = (uint32_t)V;
    a.lanes = (uint32_t)lanes;
    a.ids = ids;
    a.prompt_len = prompt_len;
    a.fresh = fresh;
    a.counts = reinterpret_cast<uint32_t*>(counts);
    a.counts_ld = counts_ld;
    a.seen = seen;
    a.seen_ld = seen_ld;
    return topk::launch_count(a, stream) == hipSuccess ? TOPK_OK : TOPK_ERR_HIP;
}

int topk_cols_verify(const topk_verify_args* v, hipStream_t stream) {
    if (!v || v->lanes < 1 || v->C < 1 || v->n_drafts < 0 || v->max_tokens < 1 || !known_dtype(v->dtype))
        return TOPK_ERR_INVALID_ARG;
    if (v->k < 1 || v->k > TOPK_MAX_K || !v->target_values || !v->target_ids || !v->out_tokens || !v->out_count)
        return TOPK_ERR_INVALID_ARG;
    if (!v->drafts && v->n_drafts) return TOPK_ERR_INVALID_ARG;
    if (!v->draft_values != !v->draft_ids) return TOPK_ERR_INVALID_ARG;
    if (v->draft_values && (v->kq < 1 || v->kq > TOPK_MAX_K)) return TOPK_ERR_INVALID_ARG;
    if (!(v->temperature >= 0.0) || v->temperature > 1.7976931348623157e308 || !(v->top_p > 0.0) || !(v->top_p <= 1.0))
        return TOPK_ERR_INVALID_ARG;
    const uintptr_t es = element_bytes(v->dtype);
    if (misaligned(v->target_values, es) || misaligned(v->draft_values, es) || misaligned(v->target_ids, 4) ||
        misaligned(v->draft_ids, 4) || misaligned(v->drafts, 4) || misaligned(v->out_tokens, 4) ||
        misaligned(v->out_count, 4))
        return TOPK_ERR_INVALID_ARG;
    if (v->lanes > TOPK_MAX_LANES || v->C > kMax32 || v->n_drafts > kMax32 || v->max_tokens > kMax32) return TOPK_ERR_UNSUPPORTED;
    topk::VerifyArgs a = {};
    a.v = *v;
    if (make_parts(&a.cols, v->col_start, v->C, v->lanes) != TOPK_OK ||
        make_parts(&a.draft_parts, v->draft_start, v->n_drafts, v->lanes) != TOPK_OK)
        return TOPK_ERR_INVALID_ARG;
    return topk::launch_verify(a, stream) == hipSuccess ? TOPK_OK : TOPK_ERR_HIP;
}

int topk_cols_plan(const topk_plan_args* p, hipStream_t stream) {
    if (!p || p->lanes < 1 || p->capacity < 1 || p->block_size < 1 || p->table_ld < 1 || p->n_free_ids < 0)
        return TOPK_ERR_INVALID_ARG;
    if (!p->lens || !p->add || !p->held || !p->table || !p->free_count || (!p->free_ids && p->n_free_ids))
        return TOPK_ERR_INVALID_ARG;
    if (!p->out_held || !p->out_free_count || !p->out_refused || !p->out_col_start || !p->out_col_lane ||
        !p->out_col_pos || !p->out_slots)
        return TOPK_ERR_INVALID_ARG;
    if (p->out_held == p->held || p->out_free_count == p->free_count) return TOPK_ERR_INVALID_ARG;
    if (misaligned(p->lens, 4) || misaligned(p->add, 4) || misaligned(p->held, 4) || misaligned(p->table, 4) ||
        misaligned(p->free_ids, 4) || misaligned(p->free_count, 4) || misaligned(p->out_held, 4) ||
        misaligned(p->out_free_count, 4) || misaligned(p->out_refused, 4) || misaligned(p->out_col_start, 4) ||
        misaligned(p->out_col_lane, 4) || misaligned(p->out_col_pos, 4) || misaligned(p->out_slots, 8))
        return TOPK_ERR_INVALID_ARG;
    if (p->lanes > TOPK_MAX_LANES || p->capacity > kMax32 || p->table_ld > kMax32 || p->n_free_ids > kMax32)
        return TOPK_ERR_UNSUPPORTED;
    return topk::launch_plan_round(*p, stream) == hipSuccess ? TOPK_OK : TOPK_ERR_HIP;
}

}  // extern "C"
