// logits_process.cu -- penalties for repeated tokens, per-token biases and
// grammar masks on packed logit rows, and the token counts that the penalties
// read, behind the C ABI of include/spec_verify.h.
//
// Row r of sequence b, token v (fp32, one rounding per step):
//   c    = output_counts[slot_b, v] + occurrences of v among the drafted
//          tokens before row r
//   seen = c > 0 or v in the prompt
//   y    = seen ? (z > 0 ? z / rho : z * rho) - phi c - pi [c > 0] : z
//   y    = y + bias_b(v), v's entries of the list added up first;
//   y    = allowed_r(v) ? y : -inf;  rounded once.
//
// The pass reads and writes every logit once and computes next to nothing, so
// memory bounds it.  Few columns of a sequence are seen, drafted or biased
// (some hundreds of a vocabulary of 10^5), so the work is split in two: a
// stream that copies the rows and applies the masks, 16 bytes a lane, and a
// list of the few columns, whose logits are taken one a lane afterwards.  In
// place the stream touches only what a mask takes away.  Working the touched
// columns inside the stream instead took 830 us at B=512 (3267 rows of 128256
// bf16, a quarter of them under a grammar); this split takes 305 us, 5.6 TB/s of
// the bytes it has to move, 82 % of the copy rate.  What is left is latency: a
// CTA's set-up, its rows two at a time and its list are dependent loads, and
// 24 warps an SM do not cover all of it (30 % of the warps' slots, DRAM 75-80 %).
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "logits_host.h"

namespace speclog {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 256;    // columns listed at once
constexpr int kBias = 64;     // entries of the bias lists that are searched, in shared memory (see add_biases)
template <bool STREAM>
constexpr int kPerSm = STREAM ? 6 : 8;  // resident CTAs

template <int DT>
constexpr uint32_t kNanWord = DT == SPEC_BF16 ? 0x7fc07fc0u : 0x7fc00000u;

// How a group of threads takes a unit of 128 words of the bit arrays (4096
// columns): a CTA with the stream, a warp without it (in place, no masks).  A
// unit's words come in pieces of 2^piece words, spread over the vocabulary:
// ids are often ordered by frequency, and so every unit gets its share of the
// frequent ones, whose columns are the work beside the stream.
struct Units {
    int self, n, piece;
};

template <bool STREAM>
struct Group {
    static constexpr int kSize = STREAM ? kThreads : 32;
    static constexpr int kWords = 128;
    static constexpr int kWordsEach = kWords / kSize;
    static constexpr int kCount = kThreads / kSize;  // groups per CTA

    static __device__ __forceinline__ int self() { return threadIdx.x / kSize; }
    static __device__ __forceinline__ int thread() { return threadIdx.x % kSize; }
    static __device__ __forceinline__ void sync() {
        if (STREAM) __syncthreads();
        else __syncwarp();
    }
    static __device__ __forceinline__ bool any(bool x) {
        return STREAM ? __syncthreads_or(x) != 0 : __any_sync(0xffffffffu, x) != 0;
    }
    // the word that the unit's place i stands for, and back (-1: another unit's)
    static __device__ __forceinline__ int word(const Units &un, int i) {
        return (un.self + un.n * (i >> un.piece) << un.piece) + (i & ((1 << un.piece) - 1));
    }
    static __device__ __forceinline__ int place(const Units &un, int word) {
        const int piece = word >> un.piece, turn = piece / un.n;
        return piece - turn * un.n == un.self ? (turn << un.piece) + (word & ((1 << un.piece) - 1)) : -1;
    }
    static __host__ int units(int V, int piece) {
        const int pieces = (V + (32 << piece) - 1) / (32 << piece);
        return (pieces + (kWords >> piece) - 1) / (kWords >> piece);
    }
};

template <bool STREAM>
struct GroupShared {
    int mask[kMaxPath + 1];     // by row: its mask, -1: none, -2: none there is
    int token[kMaxPath];
    int up[kMaxPath];           // tree: parent within the sequence
    uint64_t before[kMaxPath];  // tree: the nodes whose tokens a row follows
    // by word of the unit; once a thread has read its own, with biases: the touched columns, and how many
    // of them are listed before the word's
    uint32_t drafted[Group<STREAM>::kWords], biased[Group<STREAM>::kWords];
    int warp_sum[kWarps];
    int column[kList];
    uint8_t flags[kList];
    float bias[kList];
    int bias_token[kBias];
    float bias_value[kBias];
};
enum { kPrompt = 1, kEmitted = 2, kDrafted = 4, kBiased = 8 };

template <int DT>
__device__ __forceinline__ float load_logit(const char *row, int col) {
    if (DT == SPEC_F32) return reinterpret_cast<const float *>(row)[col];
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[col]) << 16);
}
template <int DT>
__device__ __forceinline__ void store_logit(char *row, int col, float z) {
    if (DT == SPEC_F32) reinterpret_cast<float *>(row)[col] = z;
    else reinterpret_cast<uint16_t *>(row)[col] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
}

// -inf in the columns of a vector whose bit is clear.
template <int DT>
__device__ __forceinline__ void mask_vec(uint4 &q, uint32_t allowed) {
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t keep;
        if (DT == SPEC_F32) keep = 0u - ((allowed >> i) & 1u);
        else keep = (((allowed >> (2 * i)) & 1u) | ((allowed << (15 - 2 * i)) & 0x10000u)) * 0xffffu;  // a bit per half
        w[i] = (w[i] & keep) | (Elem<DT>::kNegInfWord & ~keep);
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
}

// The mask of a row: its number, -1 for none, -2 where it names none there is.
__device__ __forceinline__ int mask_of(const Process &ps, int row) {
    const int m = ps.mask_rows ? __ldg(ps.mask_rows + row) : row;
    return m < -1 || m >= ps.M ? -2 : m;
}

// The stream over rows row0 + i0 .. row0 + i1 - 1 of a CTA's columns: a copy with
// the masks applied; in place only what a mask takes away.
template <int DT>
__device__ __forceinline__ void stream_rows(const char *logits, char *out, const Process &ps, const int *mask_rows, int V, int row0,
                                            int i0, int i1, const Units &un, bool inplace) {
    using G = Group<true>;
    constexpr int kPer = Elem<DT>::kPerVec;
    constexpr int kVecs = 32 / kPer;                // a thread's vectors of one row
    constexpr int kRows = DT == SPEC_BF16 ? 2 : 1;  // rows in flight
    constexpr uint32_t kAll = (1u << kPer) - 1;
    const int64_t row_bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    int col[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int x = j * kThreads + static_cast<int>(threadIdx.x);
        col[j] = G::word(un, x / (32 / kPer)) * 32 + x % (32 / kPer) * kPer;
    }
    const char *src = logits + (static_cast<int64_t>(row0) + i0) * row_bytes;
    char *dst = out + (static_cast<int64_t>(row0) + i0) * row_bytes;
    if (!ps.mask) {
        for (int i = i0; i < i1; i += kRows, src += kRows * row_bytes, dst += kRows * row_bytes) {
            uint4 q[kRows][kVecs];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    if (col[j] < V && (u == 0 || i + u < i1))
                        q[u][j] = *reinterpret_cast<const uint4 *>(src + u * row_bytes + static_cast<int64_t>(col[j]) * Elem<DT>::kBytes);
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    if (col[j] < V && (u == 0 || i + u < i1))
                        *reinterpret_cast<uint4 *>(dst + u * row_bytes + static_cast<int64_t>(col[j]) * Elem<DT>::kBytes) = q[u][j];
        }
        return;
    }
    const int64_t mask_bytes = static_cast<int64_t>((V + 31) / 32) * 4;
    const char *masks = reinterpret_cast<const char *>(ps.mask);
    for (int i = i0; i < i1; i += kRows, src += kRows * row_bytes, dst += kRows * row_bytes) {
        uint32_t allowed[kRows][kVecs];
        uint4 q[kRows][kVecs];
        int m[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) m[u] = i + u < i1 ? mask_rows[i + u] : -3;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                allowed[u][j] = m[u] == -1 ? kAll : 0u;
                if (m[u] >= 0 && col[j] < V)
                    allowed[u][j] = static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned char *>(masks + m[u] * mask_bytes + (col[j] >> 3)))) >>
                                        (col[j] & 7) & kAll;
            }
#pragma unroll
        for (int u = 0; u < kRows; ++u)
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                // nothing of the input is needed where nothing is allowed
                constexpr uint32_t f = Elem<DT>::kNegInfWord, x = kNanWord<DT>;
                q[u][j] = m[u] == -2 ? make_uint4(x, x, x, x) : make_uint4(f, f, f, f);
                if (allowed[u][j] != 0 && !(inplace && allowed[u][j] == kAll) && col[j] < V)
                    q[u][j] = *reinterpret_cast<const uint4 *>(src + u * row_bytes + static_cast<int64_t>(col[j]) * Elem<DT>::kBytes);
            }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (m[u] == -3) continue;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (col[j] >= V || (inplace && allowed[u][j] == kAll)) continue;
                if (m[u] >= 0 && allowed[u][j] != kAll) mask_vec<DT>(q[u][j], allowed[u][j]);
                *reinterpret_cast<uint4 *>(dst + u * row_bytes + static_cast<int64_t>(col[j]) * Elem<DT>::kBytes) = q[u][j];
            }
        }
    }
}

// A unit's columns of some rows as NaN.
template <int DT, bool STREAM>
__device__ __forceinline__ void nan_rows(char *out, int V, int64_t row0, int i0, int i1, const Units &un) {
    using G = Group<STREAM>;
    const int64_t row_bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    constexpr uint32_t w = kNanWord<DT>;
    constexpr int kPer = Elem<DT>::kPerVec;
    for (int i = i0; i < i1; ++i)
        for (int x = G::thread(); x < G::kWords * 32 / kPer; x += G::kSize) {
            const int col = G::word(un, x / (32 / kPer)) * 32 + x % (32 / kPer) * kPer;
            if (col < V)
                *reinterpret_cast<uint4 *>(out + (row0 + i) * row_bytes + static_cast<int64_t>(col) * Elem<DT>::kBytes) =
                    make_uint4(w, w, w, w);
        }
}

// The entries of a bias list (all valid) added up per listed column, in list order,
// for the `len` columns listed from number `base` on: a warp takes a share of the
// columns and goes through the list once, the entries of one token by turns.  A search of the
// list by each biased column costs the square of its length: lists of 300 took 96 us
// for 384 rows of 128256, now 63, one of every token 265 ms a row, now 13.  Lists of up to
// kBias entries, which lie in shared memory, are searched all the same: B=512 with
// 32 entries each takes 321 us so and 331 by passes.
template <bool STREAM>
__device__ __forceinline__ void add_biases(GroupShared<STREAM> &sm, const Units &un, const int32_t *tokens, const float *values, uint32_t n,
                                           int base, int len) {
    using G = Group<STREAM>;
    constexpr int kShare = kList / (G::kSize / 32), kAhead = STREAM ? 8 : 4;
    const int me = G::thread(), lane = threadIdx.x & 31;
    for (int e = me; e < len; e += G::kSize) sm.bias[e] = -0.0f;  // (leaves every value as it is)
    G::sync();
#pragma unroll 1
    for (uint32_t x0 = 0; x0 < n; x0 += 32 * kAhead) {
        int t[kAhead], to[kAhead], most = -1;  // the entries' tokens, their places among the warp's columns
#pragma unroll
        for (int u = 0; u < kAhead; ++u) t[u] = x0 + u * 32 + lane < n ? __ldg(tokens + x0 + u * 32 + lane) : -1;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            to[u] = -1;
            if (t[u] >= 0) {
                const int d = G::place(un, t[u] >> 5);
                if (d >= 0) to[u] = static_cast<int>(sm.biased[d] + __popc(sm.drafted[d] & ((1u << (t[u] & 31)) - 1))) - base;
                if (to[u] < 0 || to[u] >= len || to[u] / kShare != me >> 5) to[u] = -1;
            }
            most = max(most, to[u]);
        }
        if (!__any_sync(0xffffffffu, most >= 0)) continue;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (!__any_sync(0xffffffffu, to[u] >= 0)) continue;
            const float v = to[u] >= 0 ? __ldg(values + x0 + u * 32 + lane) : 0.0f;
            const int turn = __popc(__match_any_sync(0xffffffffu, to[u]) & ((1u << lane) - 1));
            for (int i = 0; __any_sync(0xffffffffu, to[u] >= 0 && turn >= i); ++i) {
                if (to[u] >= 0 && turn == i) sm.bias[to[u]] = __fadd_rn(sm.bias[to[u]], v);
                __syncwarp();
            }
        }
    }
}

// A group takes one unit of one sequence's columns, for all its rows or an even
// part of them, so that what depends on the sequence and the columns alone
// (its seen tokens, their counts, its biases) is read once.  CTAs in the order
// (sequence, unit): the ones that run at a time stream through one window of
// memory.
template <int DT, bool STREAM, bool BIAS>
__global__ void __launch_bounds__(kThreads, kPerSm<STREAM>)
    process_kernel(const char *logits, char *out, Rows rw, Process ps, int V, int units, int piece, int parts) {
    using G = Group<STREAM>;
    __shared__ GroupShared<STREAM> s_group[G::kCount];
    const int me = G::thread(), lane = threadIdx.x & 31;
    GroupShared<STREAM> &sm = s_group[G::self()];
    const bool inplace = logits == out;
    const int64_t row_bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    const int W = (V + 31) / 32;
    const bool pen = ps.counts != nullptr, tree = rw.mode == SPEC_ROWS_TREE;

    // (32 bits hold the number of a group: it is at most 64 times the rows' units)
    const uint32_t self = blockIdx.x * G::kCount + G::self();
    specv::grid_launch_dependents();  // a truncation behind this may get ready while it drains
    if (!check_rows(rw, pen)) {
        // the call fails: every row is NaN
        for (int64_t u = self; u < static_cast<int64_t>(rw.R) * units; u += static_cast<int64_t>(gridDim.x) * G::kCount)
            nan_rows<DT, STREAM>(out, V, u / units, 0, 1, Units{static_cast<int>(u % units), units, piece});
        return;
    }
    const uint32_t pair = self / parts;
    const int part = static_cast<int>(self - pair * parts), b = static_cast<int>(pair / units);
    const Units un{static_cast<int>(pair - static_cast<uint32_t>(b) * units), units, piece};
    if (b >= rw.B) return;
    const int o0 = __ldg(rw.offsets + b), o1 = __ldg(rw.offsets + b + 1);
    const int k = o1 - o0;  // drafted tokens, or tree nodes
    const int row0 = rw.first_row(b, o0), n = rw.first_row(b + 1, o1) - row0;
    const int i0 = n * part / parts, i1 = n * (part + 1) / parts;
    if (i0 == i1) return;

    // --- what the sequence and the columns say: asked for before the stream, used after it
    Penalty p{1.0f, 0.0f, 0.0f};
    int64_t slot = b;
    uint32_t prompt[G::kWordsEach], emitted[G::kWordsEach];
    constexpr int kTokens = (kMaxPath + G::kSize - 1) / G::kSize;
    int token[kTokens], up[kTokens];
    bool bad = false;
    if (pen && ps.slots) slot = __ldg(ps.slots + b);
    const bool there = pen && slot >= 0 && slot < ps.S;
#pragma unroll
    for (int i = 0; i < G::kWordsEach; ++i) {
        const int word = G::word(un, i * G::kSize + me);
        prompt[i] = emitted[i] = 0;
        if (there && word < W) {
            prompt[i] = static_cast<uint32_t>(__ldg(ps.seen + slot * 2 * W + word));
            emitted[i] = static_cast<uint32_t>(__ldg(ps.seen + (slot * 2 + 1) * W + word));
        }
    }
    if (pen) {
        bad |= !there || !load_penalty(ps, b, &p);
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            token[t] = up[t] = 0;
            if (me + G::kSize * t < k) {
                token[t] = __ldg(rw.tokens + o0 + me + G::kSize * t);
                if (tree) up[t] = __ldg(rw.parent + o0 + me + G::kSize * t);
            }
        }
    }
    int e0 = 0, e1 = 0;
    if (BIAS) {
        e0 = __ldg(ps.bias_offsets + b), e1 = __ldg(ps.bias_offsets + b + 1);
        if (e0 < 0 || e1 < e0 || e1 > ps.n_bias) {
            bad = true;
            e1 = e0 = 0;
        }
    }
    if (ps.mask) {
        for (int i = i0 + me; i < i1; i += G::kSize) sm.mask[i] = mask_of(ps, row0 + i);
        G::sync();
    }
    if (STREAM) stream_rows<DT>(logits, out, ps, sm.mask, V, row0, i0, i1, un, inplace);

    // --- the unit's columns that anything applies to
#pragma unroll
    for (int i = 0; i < G::kWordsEach; ++i) sm.drafted[i * G::kSize + me] = sm.biased[i * G::kSize + me] = 0;
    G::sync();
    if (pen) {
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const int j = me + G::kSize * t;
            if (j >= k) continue;
            const bool root = tree && j == 0;
            sm.token[j] = token[t];
            if (!root) {
                const bool in = token[t] >= 0 && token[t] < V;
                bad |= !in;
                const int d = in ? G::place(un, token[t] >> 5) : -1;
                if (d >= 0) atomicOr(&sm.drafted[d], 1u << (token[t] & 31));
            }
            if (tree) {
                bad |= root ? up[t] != -1 : (up[t] < o0 || up[t] >= o0 + j);
                sm.up[j] = up[t] - o0;
            }
        }
    }
    for (uint32_t e = e0 + me; e < static_cast<uint32_t>(e1); e += G::kSize) {  // (the step behind the last may pass 31 bits)
        const int t = __ldg(ps.bias_tokens + e);
        const bool in = t >= 0 && t < V;
        const float v = __ldg(ps.bias_values + e);
        bad |= !in || !(v < __int_as_float(0x7f800000));  // NaN and +inf
        if (static_cast<int>(e - e0) < kBias) {
            sm.bias_token[e - e0] = t;
            sm.bias_value[e - e0] = v;
        }
        const int d = in ? G::place(un, t >> 5) : -1;
        if (d >= 0) atomicOr(&sm.biased[d], 1u << (t & 31));
    }
    bad = G::any(bad);
    G::sync();  // the shared arrays are whole, the stream's stores done
    if (bad) {
        nan_rows<DT, STREAM>(out, V, row0, i0, i1, un);
    } else {
        uint32_t touched[G::kWordsEach], drafted[G::kWordsEach], biased[G::kWordsEach];
        int rank = 0;
#pragma unroll
        for (int i = 0; i < G::kWordsEach; ++i) {
            const int word = G::word(un, i * G::kSize + me);
            // bits behind the vocabulary say nothing
            const uint32_t in_v = word >= W ? 0u : word == W - 1 && (V & 31) ? (1u << (V & 31)) - 1 : 0xffffffffu;
            drafted[i] = sm.drafted[i * G::kSize + me];
            biased[i] = BIAS ? sm.biased[i * G::kSize + me] : 0;
            touched[i] = (prompt[i] | emitted[i] | drafted[i] | biased[i]) & in_v;
            rank += __popc(touched[i]);
        }
        const int own = rank;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, rank, off);
            if (lane >= off) rank += x;
        }
        int listed = __shfl_sync(0xffffffffu, rank, 31);
        rank -= own;
        if (STREAM) {
            if (lane == 0) sm.warp_sum[threadIdx.x >> 5] = listed;
            __syncthreads();
            listed = 0;
            for (int i = 0; i < kWarps; ++i) {
                if (i == static_cast<int>(threadIdx.x >> 5)) rank += listed;
                listed += sm.warp_sum[i];
            }
        }
        // short lists are searched by each biased column
        const bool long_list = BIAS && e1 - e0 > kBias;
        if (long_list) {
            int at = rank;
#pragma unroll
            for (int i = 0; i < G::kWordsEach; ++i) {
                sm.drafted[i * G::kSize + me] = touched[i];
                sm.biased[i * G::kSize + me] = at;
                at += __popc(touched[i]);
            }
        }
        if (listed && tree && pen) {
            for (int j = me; j < n; j += G::kSize) {
                uint64_t m = 0;
                for (int g = j; g > 0; g = sm.up[g]) m |= 1ull << g;  // parents are earlier nodes
                sm.before[j] = m;
            }
        }
        for (int base = 0; base < listed; base += kList) {
            const int len = min(kList, listed - base);
            G::sync();
            int at = rank - base;  // the place of the thread's next column in the list
            auto put = [&](int to, int col, int bit, uint32_t p, uint32_t e, uint32_t d, uint32_t x) {
                if (to < 0 || to >= kList) return;
                sm.column[to] = col + bit;
                sm.flags[to] = static_cast<uint8_t>((p >> bit & 1) * kPrompt | (e >> bit & 1) * kEmitted | (d >> bit & 1) * kDrafted |
                                                    (x >> bit & 1) * kBiased);
            };
#pragma unroll
            for (int i = 0; i < G::kWordsEach; ++i) {
                // words with few columns by their threads, full ones (frequent ids) by the warp
                const int col = G::word(un, i * G::kSize + me) * 32, n_i = __popc(touched[i]);
                const bool full = n_i > 4;
                if (!full) {
                    int to = at;
                    for (uint32_t m = touched[i]; m; m &= m - 1) put(to++, col, __ffs(m) - 1, prompt[i], emitted[i], drafted[i], biased[i]);
                }
                for (uint32_t m = __ballot_sync(0xffffffffu, full); m; m &= m - 1) {
                    const int src = __ffs(m) - 1;
                    const uint32_t word = __shfl_sync(0xffffffffu, touched[i], src);
                    const int first = __shfl_sync(0xffffffffu, at, src), c = __shfl_sync(0xffffffffu, col, src);
                    const uint32_t p = __shfl_sync(0xffffffffu, prompt[i], src), e = __shfl_sync(0xffffffffu, emitted[i], src);
                    const uint32_t d = __shfl_sync(0xffffffffu, drafted[i], src), x = __shfl_sync(0xffffffffu, biased[i], src);
                    if (word >> lane & 1) put(first + __popc(word & ((1u << lane) - 1)), c, lane, p, e, d, x);
                }
                at += n_i;
            }
            if (long_list) add_biases<STREAM>(sm, un, ps.bias_tokens + e0, ps.bias_values + e0, e1 - e0, base, len);
            G::sync();
            // a thread takes a column, all its rows
            for (int e = me; e < len; e += G::kSize) {
                const int col = sm.column[e];
                const uint32_t f = sm.flags[e];
                const int count = f & kEmitted ? __ldg(ps.counts + slot * V + col) : 0;
                float bias = -0.0f;  // (leaves every value as it is)
                if (BIAS && f & kBiased) {
                    if (long_list)
                        bias = sm.bias[e];
                    else
                        for (int x = 0; x < e1 - e0; ++x)
                            if (sm.bias_token[x] == col) bias = __fadd_rn(bias, sm.bias_value[x]);
                }
                constexpr int kRows = 4;  // in flight
                for (int i = i0; i < i1; i += kRows) {
                    float z[kRows];
                    bool go[kRows];
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        go[u] = i + u < i1;
                        if (go[u] && ps.mask) {
                            const int m = sm.mask[i + u];
                            go[u] = m == -1 || (m >= 0 && ((bit_byte(ps.mask, static_cast<int64_t>(m) * W, col) >> (col & 7)) & 1));
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kRows; ++u)
                        z[u] = go[u] ? load_logit<DT>(logits + static_cast<int64_t>(row0 + i + u) * row_bytes, col) : 0.0f;
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        if (!go[u]) continue;
                        int c = count;
                        if (f & kDrafted) {
                            const uint64_t before = tree ? sm.before[i + u] : rw.mode == SPEC_ROWS_NEXT ? (1ull << k) - 1 : (1ull << (i + u)) - 1;
                            for (uint64_t d = before; d; d &= d - 1) c += sm.token[__ffsll(d) - 1] == col;
                        }
                        if ((f & kPrompt) || c > 0) z[u] = penalised(z[u], c, p);
                        if (BIAS && f & kBiased) z[u] = __fadd_rn(z[u], bias);
                        store_logit<DT>(out + static_cast<int64_t>(row0 + i + u) * row_bytes, col, z[u]);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- the counts
// A warp per sequence: the n_b + 1 tokens that the verify emitted are counted.
// Integer additions, so their order does not matter.  4.5 us at B=512, the
// latency of four dependent loads and an atomic; the host's call costs 7 us.
constexpr int kUpdateThreads = 256;

__global__ void __launch_bounds__(kUpdateThreads)
    update_kernel(int32_t *counts, int32_t *seen, int S, int V, const int32_t *__restrict__ slots, Rows rw,
                  const int32_t *__restrict__ out_tokens, const int32_t *__restrict__ num_accepted) {
    if (!check_rows(rw, false)) return;
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
// state is written once and needs no clearing before.  64 entries of 2000
// prompt tokens over 128256 columns (35 MB written): 12.3 us, 2.9 TB/s; chunks of
// 4096 and 16384 columns took 14 us.  The lists are read before anything is
// written, so half of the time is latency.
constexpr int kResetThreads = 256;
constexpr int kResetChunk = 8192;
constexpr int kResetAhead = 8;  // tokens in flight per thread

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
    const bool emitted = q1 > q0;  // (uniform) else the counts are zero
    if (emitted)
        for (int i = tid; i < kResetChunk; i += kResetThreads) s_count[i] = 0;
    for (int i = tid; i < kResetChunk / 32; i += kResetThreads) s_prompt[i] = 0;
    if (__syncthreads_or(skip)) return;
    // every chunk's CTA reads the whole lists (from L2), several tokens in flight a thread
    // (unsigned: the step behind the last may pass 31 bits)
    auto each = [&](const int32_t *tokens, uint32_t first, uint32_t end, auto &&f) {
        for (uint32_t i = first + tid; i < end; i += kResetThreads * kResetAhead) {
            int t[kResetAhead];
#pragma unroll
            for (int u = 0; u < kResetAhead; ++u) t[u] = i + u * kResetThreads < end ? __ldg(tokens + i + u * kResetThreads) : -1;
#pragma unroll
            for (int u = 0; u < kResetAhead; ++u)
                if (t[u] >= c0 && t[u] < c0 + kResetChunk && t[u] < V) f(t[u] - c0);
        }
    };
    each(prompt_tokens, p0, p1, [&](int c) { atomicOr(&s_prompt[c >> 5], 1u << (c & 31)); });
    each(output_tokens, q0, q1, [&](int c) { atomicAdd(&s_count[c], 1); });
    __syncthreads();
    const int64_t W = (V + 31) / 32;
    const int cols = min(kResetChunk, V - c0);
    int32_t *crow = counts + static_cast<int64_t>(slot) * V + c0;
    int32_t *srow = seen + static_cast<int64_t>(slot) * 2 * W + c0 / 32;
    if (!emitted) {
        if (V % 4 == 0 && reinterpret_cast<uintptr_t>(counts) % 16 == 0)
            for (int i = tid; i < cols / 4; i += kResetThreads) reinterpret_cast<int4 *>(crow)[i] = make_int4(0, 0, 0, 0);
        else
            for (int i = tid; i < cols; i += kResetThreads) crow[i] = 0;
        for (int i = tid; i < (cols + 31) / 32; i += kResetThreads) {
            srow[i] = static_cast<int32_t>(s_prompt[i]);
            srow[W + i] = 0;
        }
        return;
    }
    for (int i = tid; i < (cols + 31) / 32 * 32; i += kResetThreads) {
        const int n = s_count[i];
        if (i < cols) crow[i] = n;
        const uint32_t m = __ballot_sync(0xffffffffu, n > 0);
        if ((i & 31) == 0) {
            srow[i >> 5] = static_cast<int32_t>(s_prompt[i >> 5]);
            srow[W + (i >> 5)] = static_cast<int32_t>(m);
        }
    }
}

template <int DT, bool STREAM>
int launch_process(const void *logits, void *out, const Rows &rw, const Process &ps, int V, int sms,
                   cudaStream_t stream) {
    using G = Group<STREAM>;
    // Spread pieces even out the frequent ids, whole units keep the CTAs that run at a time
    // in one window of memory, which counts where many sequences run at a time. Spread and whole,
    // bf16: B=64 (384 rows of 128256) 48 and 62 us, B=512 (3267 rows) 304 and 331, B=1024 (2048
    // rows of 8000) 45 and 48, B=2048 (one row of 128256 each) 467 and 424, B=4096 (4 rows of 32000
    // each) 508 and 482, (one of 128256) 1238 and 992.
    const bool spread = !STREAM || rw.B < 2048;
    const int piece = !STREAM ? 0 : spread ? 1 : 7;
    const int units = G::units(V, piece);
    const int64_t pairs = static_cast<int64_t>(rw.B) * units;
    // few sequences: their rows are split until every SM has its CTAs; long ones into parts
    // of about 8 rows, so that the last CTAs are short (64 trees of 16 rows: 119 us whole,
    // 108 in halves; halves of 6 rows cost more set-up than they gain: 14 % at B=512)
    // (a buffer may have more rows than its sequences can own)
    const int64_t most = rw.mode == SPEC_ROWS_TREE ? SPEC_MAX_TREE_NODES : rw.mode == SPEC_ROWS_NEXT ? 1 : SPEC_MAX_K + 1;
    const int64_t room = static_cast<int64_t>(sms) * kPerSm<STREAM> * G::kCount, each = std::min<int64_t>(rw.R / rw.B, most);
    const int parts = static_cast<int>(std::max<int64_t>({1, std::min(room / pairs, each), each / 8}));
    const int64_t ctas = (pairs * parts + G::kCount - 1) / G::kCount;
    const auto kernel = ps.bias_offsets ? process_kernel<DT, STREAM, true> : process_kernel<DT, STREAM, false>;
    kernel<<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(
        static_cast<const char *>(logits), static_cast<char *>(out), rw, ps, V, units, piece, parts);
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
    const bool sparse = logits == out && !ps.mask;  // only the listed columns change
    if (dtype == SPEC_F32)
        return sparse ? launch_process<SPEC_F32, false>(logits, out, rw, ps, V, st->sms, s)
                      : launch_process<SPEC_F32, true>(logits, out, rw, ps, V, st->sms, s);
    return sparse ? launch_process<SPEC_BF16, false>(logits, out, rw, ps, V, st->sms, s)
                  : launch_process<SPEC_BF16, true>(logits, out, rw, ps, V, st->sms, s);
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
