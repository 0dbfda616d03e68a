// logits_common.cuh -- device code shared by the logit operators (processing,
// truncation): which rows a sequence owns, the check of the offsets array,
// and the arithmetic of one logit's penalties, bias and mask.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "spec_verify.h"

namespace speclog {

using specv::Elem;

constexpr int kMaxPath = SPEC_MAX_TREE_NODES;  // drafted tokens (or tree nodes) of one sequence
static_assert(kMaxPath >= SPEC_MAX_K, "one word of 64 bits holds the tokens before a row");

// The rows of a call: sequence b owns first_row(b) .. first_row(b + 1) - 1.
struct Rows {
    int mode, B, R;
    const int32_t *offsets;
    const int32_t *parent;
    const int32_t *tokens;
    int n_tokens;

    __device__ __forceinline__ int first_row(int b, int off_b) const {
        return mode == SPEC_ROWS_TARGET ? off_b + b : mode == SPEC_ROWS_NEXT ? b : off_b;
    }
    __device__ __forceinline__ int first_row(int b) const { return first_row(b, __ldg(offsets + b)); }
};

// Whether the offsets are what the call's layout allows, found by the whole
// block.
__device__ __forceinline__ bool check_rows(const Rows &rw, bool need_tokens) {
    const int lo = rw.mode == SPEC_ROWS_TREE ? 1 : 0;
    const int hi = rw.mode == SPEC_ROWS_TREE ? SPEC_MAX_TREE_NODES : SPEC_MAX_K;
    const int o0 = __ldg(rw.offsets), oB = __ldg(rw.offsets + rw.B);
    bool bad = o0 != 0;
    for (int b = threadIdx.x; b < rw.B; b += blockDim.x) {
        const int n = __ldg(rw.offsets + b + 1) - __ldg(rw.offsets + b);
        bad |= n < lo || n > hi;
    }
    const int end = rw.first_row(rw.B, oB);
    bad |= end < 0 || end > rw.R || (need_tokens && oB > rw.n_tokens);
    return __syncthreads_or(bad) == 0;
}

// The same, and the sequence that holds row r into *s_seq (shared memory; -1:
// the row lies behind the last sequence's).
__device__ __forceinline__ bool check_rows(const Rows &rw, int64_t r, int *s_seq) {
    if (threadIdx.x == 0) *s_seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < rw.B; b += blockDim.x)
        if (r >= rw.first_row(b) && r < rw.first_row(b + 1)) *s_seq = b;
    return check_rows(rw, false);
}

// What the processing of logits reads beside them (spec_logits_t).
struct Process {
    const float *repetition, *frequency, *presence;
    const int32_t *counts, *seen, *slots;
    int S;
    const int32_t *bias_offsets, *bias_tokens;
    const float *bias_values;
    int n_bias;
    const int32_t *mask, *mask_rows;
    int M;
};

// One sequence's penalties.
struct Penalty {
    float rho, phi, pi;
};

// Reads them; false if one is not what the call allows.
__device__ __forceinline__ bool load_penalty(const Process &p, int b, Penalty *out) {
    out->rho = p.repetition ? __ldg(p.repetition + b) : 1.0f;
    out->phi = p.frequency ? __ldg(p.frequency + b) : 0.0f;
    out->pi = p.presence ? __ldg(p.presence + b) : 0.0f;
    return out->rho > 0.0f && isfinite(out->rho) && isfinite(out->phi) && isfinite(out->pi);
}

// A seen token's logit (c: how often it was emitted or drafted before the
// row).  Each step is one IEEE operation rounded to fp32, in the order of the
// definition, so that every kernel gives the same bits.
__device__ __forceinline__ float penalised(float z, int c, const Penalty &p) {
    float y = z > 0.0f ? __fdiv_rn(z, p.rho) : __fmul_rn(z, p.rho);
    y = __fsub_rn(y, __fmul_rn(p.phi, static_cast<float>(c)));
    return c > 0 ? __fsub_rn(y, p.pi) : y;
}

// The byte of a bit array (32-bit words, bit v % 32 of word v / 32) that
// holds columns col .. col + 7 (col a multiple of 8; little-endian words).
__device__ __forceinline__ uint32_t bit_byte(const int32_t *words, int64_t first_word, int col) {
    return __ldg(reinterpret_cast<const unsigned char *>(words + first_word) + (col >> 3));
}

}  // namespace speclog
