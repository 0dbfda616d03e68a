// beam_select.cu -- beam search's selection over beams and vocabulary behind the C ABI
// of include/spec_verify.h: the n best candidates (row, token) of each group by
//   s_r + z_{r,v} - ln sum_v exp z_{r,v}.
//
// Within a row the order is that of the logits, so the rows are streamed once
// without any selecting: a 2 KB piece of a row leaves its largest logit m and
// sum_v exp(z - m).  The best candidates are then found by narrowing down.  Of any
// cut of the candidates into pieces that are contiguous in (row, token), the n
// pieces that come first by (score of the piece's best descending, then
// position) hold the n best candidates: a candidate of any other piece has n
// others before it, the best of each of those pieces.  So
//   1. of all 2 KB pieces of the group, the first n;
//   2. of their cells of 64 bytes, the first n;
//   3. of the cells' candidates, the first n,
// and beyond the partial results only n pieces per group are read again.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "host_common.h"
#include "spec_verify.h"

namespace specbeam {
namespace {

using specv::Elem;

constexpr int kMaxBeams = SPEC_MAX_BEAMS;
constexpr int kMaxN = SPEC_MAX_CANDIDATES;
constexpr int kPieceBytes = 2048;
constexpr int kCellBytes = 64;
constexpr int kCells = kPieceBytes / kCellBytes;  // of a piece: one per lane
constexpr float kNegInf = -__builtin_huge_valf();

// ------------------------------------------------------------ rows, streamed
constexpr int kRowThreads = 256;
constexpr int kWarpPieces = 2;  // of a warp
constexpr int kBlockPieces = kRowThreads / 32 * kWarpPieces;

__device__ __forceinline__ float warp_max_nan(float m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = specv::fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

__device__ __forceinline__ uint4 load_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A row of the call is read if its hypothesis lives.
__device__ __forceinline__ bool row_is_read(const float *scores, const uint8_t *ended, int64_t r) {
    return __ldg(scores + r) != kNegInf && !(ended && __ldg(ended + r));
}

// part[r * n_pieces + p] = (largest logit, sum of exp(z - largest)) of piece p of row r.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const void *__restrict__ logits,
                                                           const float *__restrict__ scores,
                                                           const uint8_t *__restrict__ ended,
                                                           const int32_t *__restrict__ offsets, int B, int R, int V,
                                                           int n_pieces, int blocks_per_row, float2 *__restrict__ part) {
    const int r = blockIdx.x / blocks_per_row;
    const int lane = threadIdx.x & 31;
    const int p0 = (blockIdx.x - r * blocks_per_row) * kBlockPieces + (threadIdx.x >> 5) * kWarpPieces;
    if (r >= __ldg(offsets + B) || p0 >= n_pieces || !row_is_read(scores, ended, r)) return;
    const int n_vec = V / Elem<DT>::kPerVec;
    const uint4 *row = reinterpret_cast<const uint4 *>(logits) + static_cast<int64_t>(r) * n_vec;
    constexpr uint32_t ni = Elem<DT>::kNegInfWord;
    uint4 v[kWarpPieces][4];
#pragma unroll
    for (int k = 0; k < kWarpPieces; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (p0 + k) * 128 + j * 32 + lane;
            v[k][j] = at < n_vec ? load_stream(row + at) : make_uint4(ni, ni, ni, ni);
        }
#pragma unroll
    for (int k = 0; k < kWarpPieces; ++k) {
        if (p0 + k >= n_pieces) break;
        const float m = warp_max_nan(Elem<DT>::vmax4_nan(v[k]));
        float sum = 0.0f;
        if (m != kNegInf) {  // (of +inf or NaN: a NaN)
            const float2 nm = make_float2(-m, -m), c = make_float2(specv::kLog2e, specv::kLog2e);
            float2 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < Elem<DT>::kPairs; ++i) {
                    // z - m before the product: the lowest finite value does not overflow
                    const float2 d = specv::ffma2(specv::fadd2(Elem<DT>::pair(v[k][j], i), nm), c, make_float2(0.0f, 0.0f));
                    acc[j] = specv::fadd2(acc[j], make_float2(specv::ex2(d.x), specv::ex2(d.y)));
                }
            }
            const float2 t = specv::fadd2(specv::fadd2(acc[0], acc[1]), specv::fadd2(acc[2], acc[3]));
            sum = t.x + t.y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        }
        if (lane == 0) part[static_cast<int64_t>(r) * n_pieces + p0 + k] = make_float2(m, sum);
    }
}

// ------------------------------------------------------------ the n best
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;
constexpr float kBinsPerNat = 16.0f;
constexpr int kList = 512;        // what is put in order by counting
constexpr float kMagnitude = 1e4f;  // bases and scores up to here: an fp32 score is off by less than 2^-9

// The score in fp32; -inf for no candidate alone.
__device__ __forceinline__ float approx_score(float z, float top, float base) {
    return z == kNegInf ? z : fmaxf(base + (z - top), -3.402823466e38f);
}

struct Item {
    unsigned long long key;  // of the score: larger first
    int at;                  // then its position: smaller first
};

__device__ __forceinline__ unsigned long long key_of(double s) {
    const unsigned long long u = __double_as_longlong(s + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(unsigned long long k) {
    return __longlong_as_double(k >> 63 ? k & ~(1ull << 63) : ~k);
}

struct Shared {
    // a candidate's score is base + (z - top): top the row's largest logit, base the
    // row's score less ln sum exp(z - top).  An ended row: 0 and its score.
    double base[kMaxBeams];
    float base32[kMaxBeams], top[kMaxBeams];
    int live[kMaxBeams];      // 0: no candidates, 1: read, 2: ended
    float value[kMaxN * kCells];
    int first[kMaxN];         // the places chosen by the last narrowing
    unsigned long long key[kList];
    int at[kList];
    int bins[kBins];
    float red[kWarps];
    int count, bad, cut;
    float big;  // largest |base|
};

__device__ __forceinline__ float block_max(Shared &sh, float m) {
    m = warp_max_nan(m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = sh.red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = specv::fmax_nan(m, sh.red[w]);
    return m;
}

// The n first items of `count` in the order (score descending, then
// position) into sh.key / sh.at [0 .. result).  approx(i): the score in fp32, -inf for no item;
// item(i): exactly.
// Usually: a histogram of the fp32 scores gives a border that the n-th of
// them lies above; what lies above it (with twice the fp32 scores' error as a
// margin) is put in order by counting, for each, the ones before it.  Where scores are too
// large for that margin, or too many lie close together: digit by digit.
template <class Approx, class Exact>
__device__ int narrow(Shared &sh, int64_t count, int n, Approx approx, Exact item) {
    const int tid = threadIdx.x;
    float m = kNegInf;
    for (int64_t i = tid; i < count; i += kThreads) m = fmaxf(m, approx(i));
    for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
    if (tid == 0) sh.count = 0, sh.cut = kBins;
    m = block_max(sh, m);
    if (m == kNegInf) return 0;
    bool listed = fabsf(m) <= kMagnitude && sh.big <= kMagnitude;
    if (listed) {
        for (int64_t i = tid; i < count; i += kThreads) {
            const float a = approx(i);
            const float d = (m - a) * kBinsPerNat;
            if (d < static_cast<float>(kBins)) atomicAdd(&sh.bins[static_cast<int>(d)], 1);
        }
        __syncthreads();
        if (tid < 32) {
            constexpr int per = kBins / 32;
            int own = 0;
            for (int j = 0; j < per; ++j) own += sh.bins[tid * per + j];
            int incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, incl, off);
                if (tid >= off) incl += t;
            }
            if (incl >= n && incl - own < n) {
                int c = incl - own, j = 0;
                while ((c += sh.bins[tid * per + j]) < n) ++j;
                sh.cut = tid * per + j;
            }
        }
        __syncthreads();
        // a quarter of a bin: twice an fp32 score's error is a sixteenth
        const float border = sh.cut == kBins ? kNegInf : m - (sh.cut + 1.25f) / kBinsPerNat;
        for (int64_t i = tid; i < count; i += kThreads) {
            const float a = approx(i);
            if (a != kNegInf && a >= border) {
                const int p = atomicAdd(&sh.count, 1);
                if (p < kList) {
                    const Item x = item(i);
                    sh.key[p] = x.key, sh.at[p] = x.at;
                }
            }
        }
        __syncthreads();
        listed = sh.count <= kList;
    }
    if (!listed) {
        // the n-th key, eight bits at a time, then the n-th position of those that have it
        __syncthreads();
        unsigned long long key = 0;
        int at = -1, left = n;
        bool all = false;
        for (int digit = 0; digit < 12 && !all; ++digit) {
            const bool by_key = digit < 8;
            const int shift = by_key ? 56 - 8 * digit : 24 - 8 * (digit - 8);
            if (digit == 8) at = 0;
            for (int i = tid; i < 256; i += kThreads) sh.bins[i] = 0;
            __syncthreads();
            for (int64_t i = tid; i < count; i += kThreads) {
                if (approx(i) == kNegInf) continue;
                const Item x = item(i);
                if (by_key) {
                    if (digit == 0 || x.key >> (shift + 8) == key >> (shift + 8))
                        atomicAdd(&sh.bins[255 - static_cast<int>(x.key >> shift & 255)], 1);
                } else if (x.key == key && (digit == 8 || x.at >> (shift + 8) == at >> (shift + 8))) {
                    atomicAdd(&sh.bins[x.at >> shift & 255], 1);
                }
            }
            __syncthreads();
            int c = 0, j = 0;
            while (j < 256 && c + sh.bins[j] < left) c += sh.bins[j++];
            all = j == 256;  // fewer than n items
            if (!all) {
                left -= c;
                if (by_key) key |= static_cast<unsigned long long>(255 - j) << shift;
                else at |= j << shift;
            }
            __syncthreads();
        }
        if (tid == 0) sh.count = 0;
        __syncthreads();
        for (int64_t i = tid; i < count; i += kThreads) {
            if (approx(i) == kNegInf) continue;
            const Item x = item(i);
            if (all || x.key > key || (x.key == key && x.at <= at)) {
                const int p = atomicAdd(&sh.count, 1);
                if (p < kList) sh.key[p] = x.key, sh.at[p] = x.at;
            }
        }
        __syncthreads();
    }
    // in order: each goes to the place that the number of those before it says
    const int found = min(sh.count, kList);
    Item mine[kList / kThreads];
    int rank[kList / kThreads];
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
        const int p = tid + k * kThreads;
        rank[k] = kList;
        if (p < found) {
            mine[k] = Item{sh.key[p], sh.at[p]};
            int before = 0;
            for (int q = 0; q < found; ++q) {
                const unsigned long long kq = sh.key[q];
                before += kq > mine[k].key || (kq == mine[k].key && sh.at[q] < mine[k].at);
            }
            rank[k] = before;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k)
        if (rank[k] < n) sh.key[rank[k]] = mine[k].key, sh.at[rank[k]] = mine[k].at;
    __syncthreads();
    return min(found, n);
}

// A CTA per group.
template <int DT>
__global__ void __launch_bounds__(kThreads) select_kernel(const void *__restrict__ logits,
                                                          const float *__restrict__ scores,
                                                          const uint8_t *__restrict__ ended, int end_token,
                                                          const int32_t *__restrict__ offsets, int B, int R, int V,
                                                          int n_pieces, const float2 *__restrict__ part, int n,
                                                          float *__restrict__ out_scores,
                                                          int32_t *__restrict__ out_tokens,
                                                          int32_t *__restrict__ out_rows, float *__restrict__ out_lse) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    constexpr float nan = __builtin_nanf("");
    if (tid == 0) sh.bad = 0;
    bool bad = __ldg(offsets) != 0;
    for (int i = tid; i < B; i += kThreads) {
        const int w = __ldg(offsets + i + 1) - __ldg(offsets + i);
        bad |= w < 0 || w > kMaxBeams;
    }
    bad |= __ldg(offsets + B) > R;
    const bool invalid = __syncthreads_or(bad);
    const int r0 = __ldg(offsets + b), W = invalid ? 0 : __ldg(offsets + b + 1) - r0;
    // each row's sum, by a warp
    specv::grid_dependency_wait();
    if (invalid && out_lse) {
        for (int64_t i = static_cast<int64_t>(b) * kThreads + tid; i < R; i += static_cast<int64_t>(gridDim.x) * kThreads) out_lse[i] = nan;
    }
    for (int w = warp; w < W; w += kWarps) {
        const float s = __ldg(scores + r0 + w);
        const int live = s == kNegInf ? 0 : ended && __ldg(ended + r0 + w) ? 2 : 1;
        bool wrong = s != s || s == -kNegInf;
        double base = s, lse = nan;
        float top = 0.0f;
        if (live == 1) {
            const float2 *p = part + static_cast<int64_t>(r0 + w) * n_pieces;
            float m = kNegInf;
            for (int i = lane; i < n_pieces; i += 32) m = specv::fmax_nan(m, p[i].x);
            m = warp_max_nan(m);
            const bool finite = fabsf(m) < -kNegInf;
            double sum = 0.0;
            if (finite)
                for (int i = lane; i < n_pieces; i += 32) {
                    const float2 x = p[i];
                    sum += static_cast<double>(x.y * specv::ex2((x.x - m) * specv::kLog2e));
                }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (m == kNegInf) {
                base = 0.0, lse = m;
            } else if (!finite) {
                wrong = true;
            } else {
                const double log_sum = log(sum);
                top = m, base = static_cast<double>(s) - log_sum, lse = static_cast<double>(m) + log_sum;
            }
        }
        if (lane == 0) {
            sh.base[w] = base;
            sh.base32[w] = static_cast<float>(base);
            sh.top[w] = top;
            sh.live[w] = live;
            if (wrong) sh.bad = 1;
            if (out_lse) out_lse[r0 + w] = static_cast<float>(lse);
        }
    }
    __syncthreads();
    if (tid == 0) {
        float big = 0.0f;
        for (int w = 0; w < W; ++w)
            if (sh.live[w]) big = fmaxf(big, fabsf(sh.base32[w]));
        sh.big = big;
    }
    __syncthreads();
    const auto exact_score = [&](float z, int w) {
        return key_of(sh.base[w] + (static_cast<double>(z) - static_cast<double>(sh.top[w])));
    };
    int found = 0;
    if (!invalid && !sh.bad && W > 0) {
        // 1: pieces.  An ended row is a piece of its own.
        const auto piece = [&](int64_t i, int *w) -> float {  // its largest logit
            *w = static_cast<int>(i / n_pieces);
            const int p = static_cast<int>(i) - *w * n_pieces;
            const int live = sh.live[*w];
            return live == 1 ? part[static_cast<int64_t>(r0) * n_pieces + i].x : live == 2 && p == 0 ? 0.0f : kNegInf;
        };
        int chosen = narrow(
            sh, static_cast<int64_t>(W) * n_pieces, n,
            [&](int64_t i) {
                int w;
                const float z = piece(i, &w);
                return approx_score(z, sh.top[w], sh.base32[w]);
            },
            [&](int64_t i) {
                int w;
                const float z = piece(i, &w);
                return Item{exact_score(z, w), static_cast<int>(i)};
            });
        // 2: cells of the pieces
        if (tid < chosen) sh.first[tid] = sh.at[tid];
        __syncthreads();
        const int n_vec = V / Elem<DT>::kPerVec;
        constexpr int cell_vecs = kCellBytes / 16, per_cell = kCellBytes / Elem<DT>::kBytes;
        for (int c = warp; c < chosen; c += kWarps) {
            const int i = sh.first[c], w = i / n_pieces, p = i - w * n_pieces;
            float z = lane == 0 ? 0.0f : kNegInf;
            if (sh.live[w] == 1) {
                const uint4 *row = reinterpret_cast<const uint4 *>(logits) + static_cast<int64_t>(r0 + w) * n_vec;
                constexpr uint32_t ni = Elem<DT>::kNegInfWord;
                uint4 v[cell_vecs];
#pragma unroll
                for (int j = 0; j < cell_vecs; ++j) {
                    const int at = p * 128 + lane * cell_vecs + j;
                    v[j] = at < n_vec ? __ldg(row + at) : make_uint4(ni, ni, ni, ni);
                }
                z = Elem<DT>::vmax4_nan(v);
            }
            sh.value[c * kCells + lane] = z;
        }
        __syncthreads();
        const auto row_of = [&](int c) { return sh.first[c] / n_pieces; };
        chosen = narrow(
            sh, static_cast<int64_t>(chosen) * kCells, n,
            [&](int64_t i) {
                const int w = row_of(static_cast<int>(i) / kCells);
                return approx_score(sh.value[i], sh.top[w], sh.base32[w]);
            },
            [&](int64_t i) {
                const int c = static_cast<int>(i) / kCells;
                return Item{exact_score(sh.value[i], row_of(c)), sh.first[c] * kCells + static_cast<int>(i) % kCells};
            });
        // 3: the cells' candidates
        if (tid < chosen) sh.first[tid] = sh.at[tid];
        __syncthreads();
        const int row_cells = n_pieces * kCells;
        for (int i = tid; i < chosen * cell_vecs; i += kThreads) {
            const int cell = sh.first[i / cell_vecs], w = cell / row_cells;
            const int at = (cell - w * row_cells) * cell_vecs + i % cell_vecs;
            float x[Elem<DT>::kPerVec];
#pragma unroll
            for (int j = 0; j < Elem<DT>::kPerVec; ++j) x[j] = kNegInf;
            if (sh.live[w] == 2) {
                if (i % cell_vecs == 0) x[0] = 0.0f;
            } else if (at < n_vec) {
                Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4 *>(logits) + static_cast<int64_t>(r0 + w) * n_vec + at), x);
            }
#pragma unroll
            for (int j = 0; j < Elem<DT>::kPerVec; ++j) sh.value[i * Elem<DT>::kPerVec + j] = x[j];
        }
        __syncthreads();
        const auto row_at = [&](int64_t i) { return sh.first[static_cast<int>(i) / per_cell] / row_cells; };
        found = narrow(
            sh, static_cast<int64_t>(chosen) * per_cell, n,
            [&](int64_t i) {
                const int w = row_at(i);
                return approx_score(sh.value[i], sh.top[w], sh.base32[w]);
            },
            [&](int64_t i) {
                return Item{exact_score(sh.value[i], row_at(i)),
                            sh.first[static_cast<int>(i) / per_cell] * per_cell + static_cast<int>(i) % per_cell};
            });
    }
    if (tid < n) {
        const bool is_bad = invalid || sh.bad;
        float s = is_bad ? nan : kNegInf;
        int token = -1, row = -1;
        if (tid < found) {
            const int padded = n_pieces * (kPieceBytes / Elem<DT>::kBytes);  // a row's positions
            const int w = sh.at[tid] / padded;
            s = static_cast<float>(score_of(sh.key[tid]));
            token = sh.live[w] == 2 ? end_token : sh.at[tid] - w * padded;
            row = r0 + w;
        }
        const int64_t o = static_cast<int64_t>(b) * n + tid;
        out_scores[o] = s, out_tokens[o] = token, out_rows[o] = row;
    }
}

int pieces_of(int V, int dtype) {
    const int64_t bytes = static_cast<int64_t>(V) * (dtype == SPEC_F32 ? 4 : 2);
    return static_cast<int>((bytes + kPieceBytes - 1) / kPieceBytes);
}

template <int DT>
int launch(const void *logits, const float *scores, const uint8_t *ended, int32_t end_token, const int32_t *offsets,
           int B, int R, int V, int n, float *out_scores, int32_t *out_tokens, int32_t *out_rows, float *out_lse,
           float2 *part, cudaStream_t s) {
    const int n_pieces = pieces_of(V, DT);
    const int blocks = (n_pieces + kBlockPieces - 1) / kBlockPieces;
    const int rows = static_cast<int>(std::min<int64_t>(R, static_cast<int64_t>(B) * kMaxBeams));
    if (rows > 0 &&
        !specv::cuda_ok(specv::launch_k(false, rows_kernel<DT>, dim3(static_cast<unsigned>(rows) * blocks), dim3(kRowThreads),
                                        0, s, logits, scores, ended, offsets, B, R, V, n_pieces, blocks, part),
                        "rows_kernel"))
        return SPEC_ERR_CUDA;
    if (!specv::cuda_ok(specv::launch_k(rows > 0, select_kernel<DT>, dim3(B), dim3(kThreads), 0, s, logits, scores, ended,
                                        end_token, offsets, B, R, V, n_pieces, static_cast<const float2 *>(part), n,
                                        out_scores, out_tokens, out_rows, out_lse),
                        "select_kernel"))
        return SPEC_ERR_CUDA;
    return SPEC_OK;
}

}  // namespace
}  // namespace specbeam

extern "C" {

size_t spec_beam_workspace_bytes(int R, int V, int dtype) {
    if (R < 0 || specv::check_common(0, V, dtype) != SPEC_OK) return 0;
    const int64_t rows = std::min<int64_t>(R, static_cast<int64_t>(SPEC_MAX_B) * SPEC_MAX_BEAMS);
    return specv::align_up(static_cast<size_t>(std::max<int64_t>(rows, 1)) * specbeam::pieces_of(V, dtype) * sizeof(float2), 256);
}

int spec_beam_select(const void *logits, const float *scores, const uint8_t *ended, int32_t end_token,
                     const int32_t *offsets, int B, int R, int V, int dtype, int n, float *out_scores,
                     int32_t *out_tokens, int32_t *out_rows, float *out_lse, void *workspace, size_t workspace_bytes,
                     void *stream) {
    const int rc = specv::check_common(B, V, dtype);
    if (rc != SPEC_OK) return rc;
    if (R < 0 || n < 1 || n > SPEC_MAX_CANDIDATES || (ended && (end_token < 0 || end_token >= V))) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    if (!offsets || !out_scores || !out_tokens || !out_rows || (R > 0 && (!logits || !scores || !workspace)))
        return SPEC_ERR_INVALID_ARG;
    if (!specv::aligned16(logits) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SPEC_ERR_ALIGNMENT;
    if (R > 0 && workspace_bytes < spec_beam_workspace_bytes(std::min<int64_t>(R, static_cast<int64_t>(B) * SPEC_MAX_BEAMS), V, dtype))
        return SPEC_ERR_WORKSPACE;
    const auto run = dtype == SPEC_F32 ? specbeam::launch<SPEC_F32> : specbeam::launch<SPEC_BF16>;
    return run(logits, scores, ended, end_token, offsets, B, R, V, n, out_scores, out_tokens, out_rows, out_lse,
               static_cast<float2 *>(workspace), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
