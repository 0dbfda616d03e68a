// logits_process.cu -- penalties for repeated tokens, per-token biases and
// grammar masks on packed logit rows, and the token counts that the penalties
// read, behind the C ABI of include/spec_verify.h.
//
// Row r of sequence b, token v (fp32, one rounding per step):
//   c    = output_counts[slot_b, v] + occurrences of v among the drafted
//          tokens before row r
//   seen = c > 0 or v in the prompt
//   y    = seen ? (z > 0 ? z / rho : z * rho) - phi c - pi [c > 0] : z
//   y    = y + bias_b(v);  y = allowed_r(v) ? y : -inf;  rounded once.
//
// The pass reads and writes every logit once and computes next to nothing, so
// memory bounds it.

#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "logits_host.h"

namespace speclog {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = kThreads * kCols;  // columns of one unit
template <int DT>
constexpr int kUnroll = DT == SPEC_BF16 ? 4 : 2;  // rows in flight per thread

template <int DT>
struct Vec {  // a thread's 8 columns of one row, as 32-bit words
    static constexpr int kWords = DT == SPEC_BF16 ? 4 : 8;
    uint32_t w[kWords];
};

template <int DT>
__device__ __forceinline__ void load_cols(Vec<DT> &v, const char *row, int col, int ncol) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row + static_cast<int64_t>(col) * Elem<DT>::kBytes);
    uint4 q = p[0];
    v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
    if constexpr (DT == SPEC_F32) {
        if (ncol > 4) q = p[1];
        v.w[4] = q.x, v.w[5] = q.y, v.w[6] = q.z, v.w[7] = q.w;
    }
}

template <int DT>
__device__ __forceinline__ void store_cols(const Vec<DT> &v, char *row, int col, int ncol) {
    uint4 *p = reinterpret_cast<uint4 *>(row + static_cast<int64_t>(col) * Elem<DT>::kBytes);
    p[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    if constexpr (DT == SPEC_F32) {
        if (ncol > 4) p[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
    }
}

template <int DT>
__device__ __forceinline__ void fill_cols(Vec<DT> &v, uint32_t word) {
#pragma unroll
    for (int i = 0; i < Vec<DT>::kWords; ++i) v.w[i] = word;
}

// Column c of the 8, read and written without indexing registers.
template <int DT>
__device__ __forceinline__ float get_col(const Vec<DT> &v, int c) {
    const int at = DT == SPEC_F32 ? c : c >> 1;
    uint32_t x = v.w[0];
#pragma unroll
    for (int i = 1; i < Vec<DT>::kWords; ++i) x = i == at ? v.w[i] : x;
    return __uint_as_float(DT == SPEC_F32 ? x : c & 1 ? x & 0xffff0000u : x << 16);
}
template <int DT>
__device__ __forceinline__ void set_col(Vec<DT> &v, int c, float z) {
    const int at = DT == SPEC_F32 ? c : c >> 1;
    const uint32_t h = DT == SPEC_F32 ? __float_as_uint(z) : __bfloat16_as_ushort(__float2bfloat16_rn(z));
    const uint32_t keep = DT == SPEC_F32 ? 0u : c & 1 ? 0xffffu : 0xffff0000u;
    const uint32_t put = DT == SPEC_BF16 && (c & 1) ? h << 16 : h;
#pragma unroll
    for (int i = 0; i < Vec<DT>::kWords; ++i) v.w[i] = i == at ? (v.w[i] & keep) | put : v.w[i];
}
// -inf in the columns whose bit is clear
template <int DT>
__device__ __forceinline__ void mask_cols(Vec<DT> &v, uint32_t allowed) {
#pragma unroll
    for (int i = 0; i < Vec<DT>::kWords; ++i) {
        uint32_t keep;
        if (DT == SPEC_F32) keep = (allowed >> i) & 1 ? 0xffffffffu : 0u;
        else keep = ((allowed >> (2 * i)) & 1 ? 0xffffu : 0u) | ((allowed >> (2 * i + 1)) & 1 ? 0xffff0000u : 0u);
        v.w[i] = (v.w[i] & keep) | (Elem<DT>::kNegInfWord & ~keep);
    }
}

template <int DT>
constexpr uint32_t kNanWord = DT == SPEC_BF16 ? 0x7fc07fc0u : 0x7fc00000u;

struct Shared {
    int seq;
    int mask_row[kMaxPath];
    int token[kMaxPath];
    uint64_t before[kMaxPath];      // by row: the tokens that precede it
    uint32_t drafted[kChunk / 32];  // columns that a drafted token names
    uint32_t biased[kChunk / 32];   // columns that a bias entry names
    int bias_token[kThreads];
    float bias_value[kThreads];
    int count[kCols][kThreads];   // by column of the thread: a seen token's count
    float bias[kCols][kThreads];  // and a biased token's bias
};

// A CTA takes an even share of the rows' chunks in the order (sequence,
// chunk, row), so that what depends on the sequence and the columns alone
// (its seen tokens, their counts, its biases) is read once for all its rows.
// A thread keeps the same 8 columns over the rows; its seen and biased columns
// are few, so they are taken one at a time.
template <int DT>
__global__ void __launch_bounds__(kThreads, 8)
    process_kernel(const char *logits, char *out, Rows rw, Process ps, int V, int chunks) {
    __shared__ Shared sm;
    const int tid = threadIdx.x;
    const bool inplace = logits == out;
    const int64_t row_bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    const int W = (V + 31) / 32;
    const bool pen = ps.counts != nullptr;

    int64_t total;
    const int64_t all = static_cast<int64_t>(__ldg(rw.offsets + rw.B));
    const int64_t rows_all = rw.mode == SPEC_ROWS_TARGET ? all + rw.B : rw.mode == SPEC_ROWS_NEXT ? rw.B : all;
    int64_t at = rows_all * chunks * blockIdx.x / gridDim.x;
    const int64_t end = rows_all * chunks * (blockIdx.x + 1) / gridDim.x;
    const bool ok = check_rows(rw, pen, at, chunks, &sm.seq, &total);
    if (!ok) {  // the call fails: every row is NaN
        Vec<DT> nan;
        fill_cols<DT>(nan, kNanWord<DT>);
        for (int64_t u = blockIdx.x; u < static_cast<int64_t>(rw.R) * chunks; u += gridDim.x) {
            const int col = static_cast<int>(u % chunks) * kChunk + tid * kCols;
            if (col < V) store_cols<DT>(nan, out + u / chunks * row_bytes, col, min(kCols, V - col));
        }
        return;
    }
    if (at >= end) return;
    int b = sm.seq;

    while (at < end) {
        const int o0 = __ldg(rw.offsets + b), o1 = __ldg(rw.offsets + b + 1);
        const int k = o1 - o0;  // drafted tokens, or tree nodes
        const int row0 = rw.first_row(b, o0), n = rw.first_row(b + 1, o1) - row0;
        const int64_t rel = at - static_cast<int64_t>(row0) * chunks;
        const int chunk = static_cast<int>(rel / n), i0 = static_cast<int>(rel % n);
        const int i1 = static_cast<int>(min(static_cast<int64_t>(n), i0 + (end - at)));
        const int c0 = chunk * kChunk, col = c0 + tid * kCols;
        const int ncol = max(0, min(kCols, V - col));

        // --- what the unit's rows share -----------------------------------
        __syncthreads();  // the last unit is done with the shared arrays
        if (tid < kChunk / 32) sm.drafted[tid] = sm.biased[tid] = 0;
        bool bad = false;
        if (tid < n) {
            int m = -1;
            if (ps.mask) {
                m = ps.mask_rows ? __ldg(ps.mask_rows + row0 + tid) : row0 + tid;
                if (m < -1 || m >= ps.M) m = -2;  // no such mask: the row is an error
            }
            sm.mask_row[tid] = m;
        }
        Penalty p;
        int64_t slot = b;
        uint32_t pbits = 0, obits = 0;
        if (pen) {
            bad |= !load_penalty(ps, b, &p);
            if (ps.slots) slot = __ldg(ps.slots + b);
            if (slot < 0 || slot >= ps.S) {
                bad = true;
            } else if (ncol > 0) {
                pbits = bit_byte(ps.seen, slot * 2 * W, col);
                obits = bit_byte(ps.seen, (slot * 2 + 1) * W, col);
            }
            if (tid < k) {
                const int t = __ldg(rw.tokens + o0 + tid);
                const bool root = rw.mode == SPEC_ROWS_TREE && tid == 0;
                sm.token[tid] = t;
                bad |= !root && (t < 0 || t >= V);
                if (rw.mode == SPEC_ROWS_TREE) {
                    const int up = __ldg(rw.parent + o0 + tid);
                    bad |= root ? up != -1 : (up < o0 || up >= o0 + tid);
                }
            }
        }
        __syncthreads();
        if (pen && tid < k && !(rw.mode == SPEC_ROWS_TREE && tid == 0)) {
            const int d = sm.token[tid] - c0;
            if (d >= 0 && d < kChunk) atomicOr(&sm.drafted[d >> 5], 1u << (d & 31));
        }
        if (pen && tid < n) {
            uint64_t m = 0;
            if (rw.mode == SPEC_ROWS_NEXT) {
                m = k == 64 ? ~0ull : (1ull << k) - 1;
            } else if (rw.mode == SPEC_ROWS_TREE) {
                // a bad parent ends the walk: it is reported above
                for (int g = tid, left = kMaxPath; g > 0 && left > 0; --left) {
                    m |= 1ull << g;
                    const int up = __ldg(rw.parent + o0 + g) - o0;
                    g = up < g ? up : 0;
                }
            } else {
                m = (1ull << tid) - 1;  // tid <= SPEC_MAX_K
            }
            sm.before[tid] = m;
        }
        uint32_t bbits = 0;
        if (ps.bias_offsets) {
            const int e0 = __ldg(ps.bias_offsets + b), e1 = __ldg(ps.bias_offsets + b + 1);
            const bool range = e0 >= 0 && e1 >= e0 && e1 <= ps.n_bias;
            bad |= !range;
            for (int e = e0; range && e < e1; e += kThreads) {
                const int len = min(kThreads, e1 - e);
                if (tid < len) {
                    const int t = __ldg(ps.bias_tokens + e + tid);
                    const float v = __ldg(ps.bias_values + e + tid);
                    bad |= t < 0 || t >= V || !(v < __int_as_float(0x7f800000));  // NaN and +inf
                    sm.bias_token[tid] = t - c0;
                    sm.bias_value[tid] = v;
                    const int d = t - c0;
                    if (d >= 0 && d < kChunk) atomicOr(&sm.biased[d >> 5], 1u << (d & 31));
                }
                __syncthreads();
                if (reinterpret_cast<const unsigned char *>(sm.biased)[tid]) {
                    // the same token twice: the entries add, in list order
                    for (int j = 0; j < len; ++j) {
                        const int d = sm.bias_token[j] - tid * kCols;
                        if (d < 0 || d >= kCols) continue;
                        sm.bias[d][tid] = (bbits >> d) & 1 ? __fadd_rn(sm.bias[d][tid], sm.bias_value[j]) : sm.bias_value[j];
                        bbits |= 1u << d;
                    }
                }
                __syncthreads();
            }
        }
        if (ncol < kCols) {  // bits behind the vocabulary say nothing
            pbits &= 0x0fu;
            obits &= 0x0fu;
        }
        for (uint32_t m = obits; m; m &= m - 1) {
            const int c = __ffs(m) - 1;
            sm.count[c][tid] = __ldg(ps.counts + slot * V + col + c);
        }
        bad = __syncthreads_or(bad);
        const uint32_t dbits = pen ? reinterpret_cast<const unsigned char *>(sm.drafted)[tid] : 0;
        const uint32_t touched = pbits | obits | dbits | bbits;

        // --- the rows -------------------------------------------------------
        for (int i = i0; i < i1 && ncol > 0; i += kUnroll<DT>) {
            Vec<DT> v[kUnroll<DT>];
            uint32_t allowed[kUnroll<DT>];
            bool write[kUnroll<DT>];
#pragma unroll
            for (int u = 0; u < kUnroll<DT>; ++u) {
                write[u] = i + u < i1;
                allowed[u] = 0xffu;
                if (!write[u]) continue;
                const int m = ps.mask ? sm.mask_row[i + u] : -1;
                if (m >= 0) allowed[u] = bit_byte(ps.mask, static_cast<int64_t>(m) * W, col);
                if (ncol < kCols) allowed[u] |= 0xf0u;
                if (bad || m == -2) {
                    fill_cols<DT>(v[u], kNanWord<DT>);
                    allowed[u] = 0x100u;
                    continue;
                }
                write[u] = !inplace || touched || allowed[u] != 0xffu;
                if ((allowed[u] & (ncol < kCols ? 0x0fu : 0xffu)) == 0) {
                    fill_cols<DT>(v[u], Elem<DT>::kNegInfWord);  // nothing of the input is needed
                    allowed[u] = 0x100u;
                } else if (write[u]) {
                    load_cols<DT>(v[u], logits + (row0 + i + u) * row_bytes, col, ncol);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll<DT>; ++u) {
                if (!write[u]) continue;
                if (allowed[u] != 0x100u) {
                    for (uint32_t m = touched & allowed[u]; m; m &= m - 1) {
                        const int c = __ffs(m) - 1;
                        float z = get_col<DT>(v[u], c);
                        int n_c = (obits >> c) & 1 ? sm.count[c][tid] : 0;
                        if ((dbits >> c) & 1) {
                            const int t = col + c;
                            for (uint64_t d = sm.before[i + u]; d; d &= d - 1) n_c += sm.token[__ffsll(d) - 1] == t;
                        }
                        if ((pbits >> c) & 1 || n_c > 0) z = penalised(z, n_c, p);
                        if ((bbits >> c) & 1) z = __fadd_rn(z, sm.bias[c][tid]);
                        set_col<DT>(v[u], c, z);
                    }
                    if (allowed[u] != 0xffu) mask_cols<DT>(v[u], allowed[u]);
                }
                store_cols<DT>(v[u], out + (row0 + i + u) * row_bytes, col, ncol);
            }
        }

        // --- the next unit ----------------------------------------------------
        at += i1 - i0;
        if (at < end && at == static_cast<int64_t>(row0 + n) * chunks) {
            ++b;
            if (rw.first_row(b + 1) == rw.first_row(b)) {  // a sequence without rows: look further
                for (int j = b + tid; j < rw.B; j += kThreads)
                    if (at >= static_cast<int64_t>(rw.first_row(j)) * chunks &&
                        at < static_cast<int64_t>(rw.first_row(j + 1)) * chunks)
                        sm.seq = j;
                __syncthreads();
                b = sm.seq;
            }
        }
    }
}

// ---------------------------------------------------------------- the counts
// A warp per sequence: the n_b + 1 tokens that the verify emitted are counted.
// Integer additions, so their order does not matter.
constexpr int kUpdateThreads = 256;

__global__ void __launch_bounds__(kUpdateThreads)
    update_kernel(int32_t *counts, int32_t *seen, int S, int V, const int32_t *__restrict__ slots, Rows rw,
                  const int32_t *__restrict__ out_tokens, const int32_t *__restrict__ num_accepted) {
    __shared__ int s_seq;
    int64_t total;
    if (!check_rows(rw, false, 0, 1, &s_seq, &total)) return;
    const int b = blockIdx.x * (kUpdateThreads / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (b >= rw.B) return;
    const int o0 = __ldg(rw.offsets + b), k = __ldg(rw.offsets + b + 1) - o0;
    const int n = __ldg(num_accepted + b);
    const int64_t slot = slots ? __ldg(slots + b) : b;
    const int most = rw.mode == SPEC_ROWS_TREE ? k - 1 : k;
    if (n < 0 || n > most || slot < 0 || slot >= S) return;
    const int64_t W = (V + 31) / 32;
    const int row0 = rw.first_row(b, o0);
    for (int i = lane; i <= n; i += 32) {
        const int t = __ldg(out_tokens + row0 + i);
        if (t < 0 || t >= V) continue;
        atomicAdd(counts + slot * V + t, 1);
        atomicOr(seen + (slot * 2 + 1) * W + (t >> 5), static_cast<int32_t>(1u << (t & 31)));
    }
}

// A CTA per (entry, chunk of columns): it builds the chunk's counts and bits
// in shared memory from the entry's tokens and writes them out whole, so the
// state is written once and needs no clearing before.
constexpr int kResetThreads = 256;
constexpr int kResetChunk = 4096;

__global__ void __launch_bounds__(kResetThreads)
    reset_kernel(int32_t *counts, int32_t *seen, int S, int V, const int32_t *__restrict__ slots, int n,
                 const int32_t *__restrict__ prompt_offsets, const int32_t *__restrict__ prompt_tokens, int n_prompt,
                 const int32_t *__restrict__ output_offsets, const int32_t *__restrict__ output_tokens, int n_output) {
    __shared__ int32_t s_count[kResetChunk];
    __shared__ uint32_t s_prompt[kResetChunk / 32];
    const int e = blockIdx.y, c0 = blockIdx.x * kResetChunk, tid = threadIdx.x;
    const int slot = __ldg(slots + e);
    bool skip = slot < 0 || slot >= S;
    for (int j = e + 1 + tid; j < n; j += kResetThreads) skip |= __ldg(slots + j) == slot;  // a later entry has it
    const int p0 = prompt_offsets ? __ldg(prompt_offsets + e) : 0, p1 = prompt_offsets ? __ldg(prompt_offsets + e + 1) : 0;
    const int q0 = output_offsets ? __ldg(output_offsets + e) : 0, q1 = output_offsets ? __ldg(output_offsets + e + 1) : 0;
    skip |= p0 < 0 || p1 < p0 || p1 > n_prompt || q0 < 0 || q1 < q0 || q1 > n_output;
    for (int i = tid; i < kResetChunk; i += kResetThreads) s_count[i] = 0;
    for (int i = tid; i < kResetChunk / 32; i += kResetThreads) s_prompt[i] = 0;
    if (__syncthreads_or(skip)) return;
    for (int i = p0 + tid; i < p1; i += kResetThreads) {
        const int t = __ldg(prompt_tokens + i);
        if (t >= c0 && t < c0 + kResetChunk && t < V) atomicOr(&s_prompt[(t - c0) >> 5], 1u << (t & 31));
    }
    for (int i = q0 + tid; i < q1; i += kResetThreads) {
        const int t = __ldg(output_tokens + i);
        if (t >= c0 && t < c0 + kResetChunk && t < V) atomicAdd(&s_count[t - c0], 1);
    }
    __syncthreads();
    const int64_t W = (V + 31) / 32;
    const int cols = min(kResetChunk, V - c0);
    int32_t *crow = counts + static_cast<int64_t>(slot) * V + c0;
    for (int i = tid; i < cols; i += kResetThreads) crow[i] = s_count[i];
    for (int w = tid; w < (cols + 31) / 32; w += kResetThreads) {
        uint32_t m = 0;
        for (int j = 0; j < 32; ++j) m |= (s_count[w * 32 + j] > 0 ? 1u : 0u) << j;
        seen[static_cast<int64_t>(slot) * 2 * W + c0 / 32 + w] = static_cast<int32_t>(s_prompt[w]);
        seen[(static_cast<int64_t>(slot) * 2 + 1) * W + c0 / 32 + w] = static_cast<int32_t>(m);
    }
}

template <int DT>
int launch_process(const void *logits, void *out, const Rows &rw, const Process &ps, int V, int sms,
                   cudaStream_t stream) {
    const int chunks = (V + kChunk - 1) / kChunk;
    const int64_t units = static_cast<int64_t>(rw.R) * chunks;
    const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(sms) * 8));
    process_kernel<DT><<<grid, kThreads, 0, stream>>>(static_cast<const char *>(logits), static_cast<char *>(out), rw,
                                                      ps, V, chunks);
    return specv::cuda_ok(cudaGetLastError(), "launch process_kernel") ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace speclog

using namespace speclog;

extern "C" {

int spec_logits_process(const void *logits, const spec_rows_t *rows, const spec_logits_t *process, int V, int dtype,
                        void *out, void *stream) {
    Rows rw;
    Process ps;
    int rc = check_rows_args(logits, rows, V, dtype, out, &rw);
    if (rc == SPEC_OK) rc = check_process_args(rows, process, &rw, &ps);
    if (rc != SPEC_OK || rw.B == 0 || rw.R == 0) return rc;
    int dev;
    specv::DeviceState *st = specv::device_state(&dev);
    if (!st) return SPEC_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_process<SPEC_F32>(logits, out, rw, ps, V, st->sms, s)
                             : launch_process<SPEC_BF16>(logits, out, rw, ps, V, st->sms, s);
}

int spec_penalty_update(int32_t *counts, int32_t *seen, int S, int V, const int32_t *slots, const spec_rows_t *rows,
                        const int32_t *out_tokens, const int32_t *num_accepted, void *stream) {
    if (!rows || S < 0 || V <= 0 || V > SPEC_MAX_V || rows->B < 0 || rows->B > SPEC_MAX_B) return SPEC_ERR_INVALID_ARG;
    if (rows->B == 0) return SPEC_OK;
    if (rows->rows != SPEC_ROWS_TARGET && rows->rows != SPEC_ROWS_TREE) return SPEC_ERR_INVALID_ARG;
    if (!counts || !seen || !rows->offsets || !out_tokens || !num_accepted || rows->R < 0) return SPEC_ERR_INVALID_ARG;
    const Rows rw{rows->rows, rows->B, rows->R, rows->offsets, nullptr, nullptr, 0};
    const int per = kUpdateThreads / 32;
    update_kernel<<<(rw.B + per - 1) / per, kUpdateThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        counts, seen, S, V, slots, rw, out_tokens, num_accepted);
    return specv::cuda_ok(cudaGetLastError(), "launch update_kernel") ? SPEC_OK : SPEC_ERR_CUDA;
}

int spec_penalty_reset(int32_t *counts, int32_t *seen, int S, int V, const int32_t *slots, int n,
                       const int32_t *prompt_offsets, const int32_t *prompt_tokens, int n_prompt,
                       const int32_t *output_offsets, const int32_t *output_tokens, int n_output, void *stream) {
    if (S < 0 || V <= 0 || V > SPEC_MAX_V || n < 0 || n > SPEC_MAX_B || n_prompt < 0 || n_output < 0)
        return SPEC_ERR_INVALID_ARG;
    if (n == 0) return SPEC_OK;
    if (!counts || !seen || !slots || (prompt_offsets && n_prompt > 0 && !prompt_tokens) ||
        (output_offsets && n_output > 0 && !output_tokens))
        return SPEC_ERR_INVALID_ARG;
    const dim3 grid((V + kResetChunk - 1) / kResetChunk, n);
    reset_kernel<<<grid, kResetThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        counts, seen, S, V, slots, n, prompt_offsets, prompt_tokens, n_prompt, output_offsets, output_tokens, n_output);
    return specv::cuda_ok(cudaGetLastError(), "launch reset_kernel") ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
