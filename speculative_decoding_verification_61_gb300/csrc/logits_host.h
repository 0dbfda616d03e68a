// logits_host.h -- host-side argument checks of the logit operators.
#pragma once

#include "host_common.h"
#include "logits_common.cuh"

namespace speclog {

// The arguments every logit operator has: the logits, their rows, the output
// (the logits themselves, or a buffer that does not overlap them).
inline int check_rows_args(const void *logits, const spec_rows_t *rows, int V, int dtype, const void *out, Rows *rw) {
    if (!rows) return SPEC_ERR_INVALID_ARG;
    const int rc = specv::check_common(rows->B, V, dtype);
    if (rc != SPEC_OK) return rc;
    if (rows->rows < SPEC_ROWS_TARGET || rows->rows > SPEC_ROWS_TREE || rows->R < 0 || rows->n_tokens < 0)
        return SPEC_ERR_INVALID_ARG;
    *rw = Rows{rows->rows, rows->B, rows->R, rows->offsets, rows->parent, rows->draft_tokens, rows->n_tokens};
    if (rows->B == 0 || rows->R == 0) return SPEC_OK;
    if (!logits || !out || !rows->offsets) return SPEC_ERR_INVALID_ARG;
    if (!specv::aligned16(logits) || !specv::aligned16(out)) return SPEC_ERR_ALIGNMENT;
    if (logits != out) {
        const size_t bytes = static_cast<size_t>(rows->R) * V * (dtype == SPEC_F32 ? 4 : 2);
        const char *a = static_cast<const char *>(logits), *z = static_cast<const char *>(out);
        if (a < z + bytes && z < a + bytes) return SPEC_ERR_INVALID_ARG;
    }
    return SPEC_OK;
}

inline int check_process_args(const spec_rows_t *rows, const spec_logits_t *p, const Rows *rw, Process *ps) {
    if (!p) return SPEC_ERR_INVALID_ARG;
    *ps = Process{p->repetition, p->frequency,   p->presence,    p->counts, p->seen, p->slots,     p->S,
                  p->bias_offsets, p->bias_tokens, p->bias_values, p->n_bias, p->mask, p->mask_rows, p->M};
    if (rw->B == 0 || rw->R == 0) return SPEC_OK;
    if (p->counts) {
        if (!p->seen || p->S < 0 || (rw->n_tokens > 0 && !rw->tokens)) return SPEC_ERR_INVALID_ARG;
        if (rw->mode == SPEC_ROWS_TREE && !rows->parent) return SPEC_ERR_INVALID_ARG;
    } else if (p->repetition || p->frequency || p->presence || p->seen || p->slots) {
        return SPEC_ERR_INVALID_ARG;  // penalties without the counts they read
    }
    if (p->bias_offsets) {
        if (p->n_bias < 0 || (p->n_bias > 0 && (!p->bias_tokens || !p->bias_values))) return SPEC_ERR_INVALID_ARG;
    } else if (p->bias_tokens || p->bias_values) {
        return SPEC_ERR_INVALID_ARG;
    }
    if (p->mask) {
        if (p->M < 0 || (!p->mask_rows && p->M < rw->R)) return SPEC_ERR_INVALID_ARG;
    } else if (p->mask_rows) {
        return SPEC_ERR_INVALID_ARG;
    }
    return SPEC_OK;
}

}  // namespace speclog
