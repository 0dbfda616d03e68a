// beam_select.cu -- beam search's selection over beams and vocabulary behind the C ABI
// of include/spec_verify.h: the n best candidates (row, token) of each group by
//   s_r + z_{r,v} - ln sum_v exp z_{r,v}.
//
// Within a row the order is that of the logits, so the rows are streamed once
// without any selecting: a 2 KB piece of a row leaves its largest logit, and
// a unit of four pieces its largest, m, with sum_v exp(z - m).  The best candidates are then found by
// narrowing down.  Of any cut of the candidates into pieces that are contiguous in (row, token),
// the n pieces that come first by (score of the piece's best descending, then
// position) hold the n best candidates: a candidate of any other piece has n
// others before it, the best of each of those pieces.  So beyond the partial results only
// about n pieces per group are read again.
//
// Times (GB300, events over captured calls): 64 groups of 8 rows of 128256 bf16, 26.6 us, of which the rows are 20
// (118 MB; 17.8 us at the copy rate) and the selection behind them 6.5: a chain of eight
// block-wide steps on 64 SMs, bound by latency.  128 groups of 16 rows of 152064, 93.8 us: 84 (7.0 TB/s of
// reads) and 9.  One group of 4 rows of 32000 fp32, 7.7 us, all latency.
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
constexpr int kRowThreads = 128;  // (256: 104 us for the 128 groups)
constexpr int kUnitPieces = 4;  // of a warp: 8 KB under way each, 192 KB per SM
constexpr int kBlockUnits = kRowThreads / 32;

// What a row leaves, and where.
struct Partial {
    float2 *unit;  // [R, n_units] (largest logit, sum of exp(z - largest))
    float *piece;  // [R, n_pieces] largest logits
    int n_units, n_pieces;
};

// The largest of a warp's values; NaN if one is NaN.
__device__ __forceinline__ float warp_max_nan(float m) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}

__device__ __forceinline__ uint4 load_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The arguments of a call.
struct Call {
    const void *logits;
    const float *scores;
    const uint8_t *ended;
    const int32_t *offsets;
    int end_token, B, R, V, n;
    Partial part;
    float *out_scores;
    int32_t *out_tokens, *out_rows;
    float *out_lse;
};

// Unit u of row r, by a warp.
template <int DT>
__device__ __forceinline__ void stream_unit(const Call &call, int r, int u) {
    const Partial &part = call.part;
    const int lane = threadIdx.x & 31;
    const int n_vec = call.V / Elem<DT>::kPerVec;
    const uint4 *row = reinterpret_cast<const uint4 *>(call.logits) + static_cast<int64_t>(r) * n_vec;
    constexpr uint32_t ni = Elem<DT>::kNegInfWord;
    uint4 v[kUnitPieces][4];
    const int first = u * kUnitPieces * 128 + lane;
    if ((u + 1) * kUnitPieces * 128 <= n_vec) {
#pragma unroll
        for (int k = 0; k < kUnitPieces; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k][j] = load_stream(row + first + (k * 4 + j) * 32);
    } else {
#pragma unroll
        for (int k = 0; k < kUnitPieces; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = first + (k * 4 + j) * 32;
                v[k][j] = at < n_vec ? load_stream(row + at) : make_uint4(ni, ni, ni, ni);
            }
    }
    float m = kNegInf, own = 0.0f;  // own: of the lane's piece
#pragma unroll
    for (int k = 0; k < kUnitPieces; ++k) {
        const float x = warp_max_nan(Elem<DT>::vmax4_nan(v[k]));
        m = specv::fmax_nan(m, x);
        if (lane == k) own = x;
    }
    float sum = 0.0f;
    if (m != kNegInf) {  // (of +inf or NaN: a NaN)
        const float2 nm = make_float2(-m, -m), c = make_float2(specv::kLog2e, specv::kLog2e);
        float2 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kUnitPieces; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < Elem<DT>::kPairs; ++i) {
                    // z - m before the product: the lowest finite value does not overflow
                    const float2 d = specv::ffma2(specv::fadd2(Elem<DT>::pair(v[k][j], i), nm), c, make_float2(0.0f, 0.0f));
                    acc[j] = specv::fadd2(acc[j], make_float2(specv::ex2(d.x), specv::ex2(d.y)));
                }
        const float2 t = specv::fadd2(specv::fadd2(acc[0], acc[1]), specv::fadd2(acc[2], acc[3]));
        sum = t.x + t.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    if (lane == 0) part.unit[static_cast<int64_t>(r) * part.n_units + u] = make_float2(m, sum);
    const int p = u * kUnitPieces + lane;
    if (lane < kUnitPieces && p < part.n_pieces) part.piece[static_cast<int64_t>(r) * part.n_pieces + p] = own;
}

// A row that is not a group's, or whose hypothesis has ended or does not live, is not read.
__device__ __forceinline__ bool row_is_read(const Call &call, int r) {
    return __ldg(call.scores + r) != kNegInf && !(call.ended && __ldg(call.ended + r));
}

// A warp per unit; CTAs blocks_per_row * r .. of row r.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ Call call, int blocks_per_row) {
    specv::grid_launch_dependents();
    const int r = blockIdx.x / blocks_per_row;
    const int u = (blockIdx.x - r * blocks_per_row) * kBlockUnits + (threadIdx.x >> 5);
    if (u < call.part.n_units && r < __ldg(call.offsets + call.B) && row_is_read(call, r)) stream_unit<DT>(call, r, u);
}

// ------------------------------------------------------------ the n best
constexpr int kThreads = 512;  // (256: 28.7 us for the 64 groups, 101 for the 128)
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kSms = 152;
constexpr int kBins = 256;
constexpr int kList = 512;          // candidates that are put in order by counting
constexpr int kChosen = 256;        // pieces that are read again
constexpr int kValues = kMaxN * kCells;
constexpr int kTaken = kValues * 4 / kCellBytes;  // cells that are looked at one candidate a thread
constexpr float kMagnitude = 1e4f;  // bases up to here: an fp32 score is off by less than 2^-9
constexpr int kHeld = 4;            // pieces whose scores a lane holds

// The score in fp32; -inf for no candidate alone.
__device__ __forceinline__ float approx_score(float z, float top, float base) {
    return z == kNegInf ? z : fmaxf(base + (z - top), -3.402823466e38f);
}

// Exact scores are kept in two fp32 terms, x the value rounded and y the rest (48 bits): a step of
// 64-bit arithmetic takes 65 cycles on this GPU.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
// a + b, a in two terms
__device__ __forceinline__ float2 add_to(float2 a, float b) {
    const float2 s = two_sum(a.x, b);
    return make_float2(s.x, __fadd_rn(a.y, s.y));
}
__device__ __forceinline__ float2 rounded(float2 a) {
    const float s = __fadd_rn(a.x, a.y);
    return make_float2(s, __fsub_rn(a.y, __fsub_rn(s, a.x)));
}

struct Item {
    unsigned long long key;  // of the score: larger first
    int at;                  // then its position: smaller first
};

// A position: row, then token (up to 2^24 of them).
constexpr int kRowShift = 25;
static_assert(SPEC_MAX_V <= 1 << (kRowShift - 1) && kMaxBeams <= 1 << (31 - kRowShift), "a position in 31 bits");

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float score_of(unsigned long long key) {
    const uint32_t u = max(static_cast<uint32_t>(key >> 32), 0x00800000u);  // ordered(the lowest value)
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}
// The key of base + (z - top).  A place without a candidate has the score -inf, so a score below the lowest value is
// written as that value; such scores have the codes below the lowest value's, of which the upper word
// has 2^23.
__device__ __forceinline__ unsigned long long key_of(float z, float top, float2 base) {
    if (__fsub_rn(z, top) > -0x1p33f) {  // no sum passes the largest value: far less than half a step of it is added
        const float2 d = two_sum(z, -top);
        float2 s = add_to(base, d.x);
        s = rounded(make_float2(s.x, s.y + d.y));
        return static_cast<unsigned long long>(ordered(s.x)) << 32 | ordered(s.y);
    }
    // beside a mask, ordinary numbers are nothing (what follows gives the same; all but one token of 8 groups of 64 rows at the
    // lowest value: 268 -> 250 us)
    if (fmaxf(fabsf(base.x), fabsf(top)) < z * -0x1p-55f) return static_cast<unsigned long long>(ordered(z)) << 32 | ordered(0.0f);
    // of far distances a 16th, which is exact: three of the largest values stay below 2^126
    constexpr float part = 0.0625f;
    const float2 d = two_sum(z * part, -top * part);
    float2 s = add_to(make_float2(base.x * part, base.y * part), d.x);
    s = rounded(make_float2(s.x, s.y + d.y));
    // the second term to 2^-52 of the distance: tokens that are masked by one value tie between rows, as they do in
    // 64 bits, and go by row
    const float grid = __uint_as_float(__float_as_uint(d.x) & 0x7f800000u) * 0x3p-30f;
    s.y = __fsub_rn(__fadd_rn(s.y, grid), grid);
    const float x = s.x * 16.0f;
    if (x != kNegInf) return static_cast<unsigned long long>(ordered(x)) << 32 | ordered(s.y * 16.0f);
    // s.x is in [-3 * 2^124, -2^124]: 3 * 2^22 codes, so that with half of the lower word's they are fewer than 2^55
    constexpr uint32_t least = 0x01bfffffu;  // ordered(-3 * 2^124)
    return (static_cast<unsigned long long>(ordered(s.x) - least) << 32 | ordered(s.y)) >> 1;
}

struct Shared {
    // a candidate's score is base + (z - top): top the row's largest logit, base the
    // row's score less ln sum exp(z - top).  An ended row: 0 and its score.
    float2 base[kMaxBeams];
    float top[kMaxBeams];
    int live[kMaxBeams];      // 0: no candidates, 1: read, 2: ended
    float2 sum[kMaxBeams];    // of exp(z - top), in two terms
    int first[kChosen];       // the pieces chosen
    unsigned long long key[kList];
    int at[kList];
    int bins[2][kBins];       // of the pieces, of the candidates
    int n_pieces, n_cells, count;  // chosen, taken, listed
    int cell[kTaken];         // row << 20 | cell
    float best[kMaxBeams / 32];
    int bad, large;           // a data error; a base that fp32 scores are too coarse for
    alignas(16) float value[kValues];  // the cells taken; where digits decide, cells' or candidates' logits
};
static_assert(kChosen >= kMaxN && kList >= kMaxN, "what the digits' path keeps");
static_assert(SPEC_MAX_V * 4ll / kCellBytes <= 1 << 20 && kMaxBeams <= 1 << 11, "a row and a cell in 31 bits");

// Bins by how far a score lies below the best one: 32 to each doubling of
// 1 + d, so a thirty-second of a nat wide at the best score and an eighth at three nats below it; up to 255 nats.
constexpr int kBinShift = 18, kBinBase = 0x3f800000 >> kBinShift;
__device__ __forceinline__ void count_in_bins(int *bins, float most, float a) {
    const int bin = (__float_as_int(1.0f + (most - a)) >> kBinShift) - kBinBase;  // (a <= most but for rounding)
    if (bin < kBins) atomicAdd(&bins[max(bin, 0)], 1);
}

// The bin that the n-th counted item lies in, and how many are in those before it; -1: fewer than n are in
// the bins.  By each warp for itself.
__device__ __forceinline__ int nth_bin(const int *bins, int n, int *before) {
    const int lane = threadIdx.x & 31;
    int own[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int4 v = reinterpret_cast<const int4 *>(bins)[lane * 2 + k];
        own[4 * k] = v.x, own[4 * k + 1] = v.y, own[4 * k + 2] = v.z, own[4 * k + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += own[k], own[k] = sum;
    int below = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, below, off);
        if (lane >= off) below += t;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, below >= n);
    if (!reach) return -1;
    below -= sum;
    int bin = lane * 8, count = below;
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (below + own[k] < n) ++bin, count = below + own[k];
    *before = __shfl_sync(0xffffffffu, count, __ffs(reach) - 1);
    return __shfl_sync(0xffffffffu, bin, __ffs(reach) - 1);
}

// A border that the n-th counted score lies above: the lower end of its bin, less a sixty-fourth (twice an
// fp32 score's error is 2^-8).  -inf: fewer than n are in the bins.
__device__ __forceinline__ float border_of(const int *bins, float most, int n) {
    int before;
    const int bin = nth_bin(bins, n, &before);
    return bin < 0 ? kNegInf : most - (__int_as_float((bin + 1 + kBinBase) << kBinShift) - 1.0f) - 0.015625f;
}

// The place of each listed item: the number of those before it, counted by eight
// lanes.  put(item, place) is called once for each, by one thread.
template <class Put>
__device__ __forceinline__ void by_rank(const Shared &sh, int found, Put put) {
    const int part = threadIdx.x & 7;
#pragma unroll 1
    for (int p0 = 0; p0 < found; p0 += kThreads / 8) {
        const int p = p0 + (threadIdx.x >> 3);
        const Item x = p < found ? Item{sh.key[p], sh.at[p]} : Item{0, 0};
        int before = 0;
        if (p < found)
#pragma unroll 4
            for (int q = part; q < found; q += 8) {
                const unsigned long long k = sh.key[q];
                before += k > x.key || (k == x.key && sh.at[q] < x.at);
            }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
        if (p < found && part == 0) put(x, before);
    }
}

template <int DT>
struct Group {
    const uint4 *logits;  // of its first row
    const float *piece;   // its pieces' largest logits
    int W, V, n_vec, n_pieces;

    // Lane's cell of piece p of row w, which is read.
    __device__ __forceinline__ void load_cell(int w, int p, int lane, uint4 (&v)[kCellBytes / 16]) const {
        const uint4 *row = logits + static_cast<int64_t>(w) * n_vec;
        constexpr uint32_t ni = Elem<DT>::kNegInfWord;
#pragma unroll
        for (int j = 0; j < kCellBytes / 16; ++j) {
            const int at = p * 128 + lane * (kCellBytes / 16) + j;
            v[j] = at < n_vec ? __ldg(row + at) : make_uint4(ni, ni, ni, ni);
        }
    }
};

// The usual way: a histogram of the pieces' fp32 scores gives a border that
// the n-th best of them lies above; of the pieces above it, the candidates above
// it are listed, by way of the cells above it.  If the cells or the candidates are too many (tokens in
// order of their frequency: the best ones lie in a few pieces; or short rows), a histogram of theirs gives a
// nearer border.  Returns how many are listed, -1 if they are too many still.
template <int DT, int kFlight>
__device__ __forceinline__ int list_candidates(Shared &sh, const Group<DT> &g, const float (&mine)[kHeld], int share, float most, int n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float border = 0.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // counted, then chosen
#pragma unroll 1
        for (int w = warp >> share; w < g.W; w += kWarps >> share) {
            const int live = sh.live[w];
            if (live == 0) continue;
            const float top = sh.top[w], base = sh.base[w].x;
            const int first = ((warp & ((1 << share) - 1)) << 5) + lane;
            const auto see = [&](float z, int p) {
                const float a = approx_score(z, top, base);
                if (a == kNegInf) return;
                if (pass == 0) {
                    count_in_bins(sh.bins[0], most, a);
                } else if (a >= border) {
                    const int i = atomicAdd(&sh.n_pieces, 1);
                    if (i < kChosen) sh.first[i] = w << 16 | p;  // (at most 2^15 pieces)
                }
            };
            if (live == 2) {
                if (first == 0) see(0.0f, 0);
                continue;
            }
            const float *piece = g.piece + static_cast<int64_t>(w) * g.n_pieces;
#pragma unroll 1
            for (int p0 = first; p0 < g.n_pieces; p0 += kHeld * 32 << share) {
                float z[kHeld];
                const bool held = w < kWarps && p0 == first;  // the first of them
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int p = p0 + (k * 32 << share);
                    z[k] = held ? mine[k] : p < g.n_pieces ? piece[p] : kNegInf;
                }
#pragma unroll
                for (int k = 0; k < kHeld; ++k) see(z[k], p0 + (k * 32 << share));
            }
        }
        __syncthreads();
        if (pass == 0) border = border_of(sh.bins[0], most, n);
    }
    const int chosen = sh.n_pieces;
    if (chosen > kChosen) return -1;
    constexpr int cell_vecs = kCellBytes / 16, per_cell = kCellBytes / Elem<DT>::kBytes;
    sh.bins[0][threadIdx.x & (kBins - 1)] = 0;
    // the chosen pieces' cells that reach above the border
    int taken;
#pragma unroll 1
    for (int round = 0;; ++round) {
#pragma unroll 1
        for (int c0 = warp; c0 < chosen; c0 += kFlight * kWarps) {
            // some pieces of a warp under way before the first is looked at
            uint4 v[kFlight][cell_vecs];
            int f[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                f[k] = c0 + k * kWarps < chosen ? sh.first[c0 + k * kWarps] : -1;
                if (f[k] >= 0 && sh.live[f[k] >> 16] == 1) g.load_cell(f[k] >> 16, f[k] & 0xffff, lane, v[k]);
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                if (f[k] < 0) break;
                const int w = f[k] >> 16;
                float z = lane == 0 ? 0.0f : kNegInf;  // of an ended row
                if (sh.live[w] == 1) z = Elem<DT>::vmax4_nan(v[k]);
                const float a = approx_score(z, sh.top[w], sh.base[w].x);
                if (a == kNegInf || a < border) continue;
                if (round == 0) count_in_bins(sh.bins[1], most, a);
                const int i = atomicAdd(&sh.n_cells, 1);
                if (i >= kTaken) continue;
                sh.cell[i] = w << 20 | ((f[k] & 0xffff) * kCells + lane);
#pragma unroll
                for (int j = 0; j < cell_vecs; ++j) reinterpret_cast<uint4 *>(sh.value)[i * cell_vecs + j] = v[k][j];
            }
        }
        __syncthreads();
        taken = sh.n_cells;
        if (taken <= kTaken) break;
        if (round == 1) return -1;
        border = border_of(sh.bins[1], most, n);
        __syncthreads();
        if (threadIdx.x == 0) sh.n_cells = 0;
        __syncthreads();
    }
    // of those, a candidate per thread
#pragma unroll 1
    for (int round = 0;; ++round) {
#pragma unroll 1
        for (int i = threadIdx.x; i < taken * per_cell; i += kThreads) {
            const int c = sh.cell[i / per_cell], w = c >> 20, in_cell = i % per_cell;
            float z = DT == SPEC_F32 ? sh.value[i] : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(sh.value)[i]) << 16);
            if (sh.live[w] == 2) z = in_cell == 0 ? 0.0f : kNegInf;
            const float2 base = sh.base[w];
            const float a = approx_score(z, sh.top[w], base.x);
            if (a == kNegInf || a < border) continue;
            if (round == 0) count_in_bins(sh.bins[0], most, a);
            const int k = atomicAdd(&sh.count, 1);
            if (k < kList) {
                sh.key[k] = key_of(z, sh.top[w], base);
                sh.at[k] = w << kRowShift | ((c & 0xfffff) * per_cell + in_cell);
            }
        }
        __syncthreads();
        const int found = sh.count;
        // (putting them in order takes the square of their number)
        if (found <= (round == 0 ? n + 64 : kList)) return found;
        if (round == 1) return -1;
        border = border_of(sh.bins[0], most, n);
        __syncthreads();
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
    }
}

// Any scores and any number of equal ones: the first n pieces, of their cells the first n, of those the
// first n candidates, each by digits.  Rare, so it is kept small: the code of a
// kernel that runs each instruction once is fetched from memory.
template <int DT>
struct Digits {
    static constexpr int kCellVecs = kCellBytes / 16, kPerCell = kCellBytes / Elem<DT>::kBytes;

    // Whether there is an item i of a level (0: pieces, 1: cells of sh.first's pieces, 2: candidates of sh.first's
    // cells), and it.  An ended row is a piece, a cell, a candidate of its own.
    __device__ static __noinline__ bool item(const Shared &sh, const Group<DT> &g, int level, int i, Item *x) {
        const int from = level == 0 ? i : sh.first[i / (level == 1 ? kCells : kPerCell)];
        const int w = from / (level == 2 ? g.n_pieces * kCells : g.n_pieces);
        float z;
        if (level > 0) z = sh.value[i];
        else z = sh.live[w] == 1 ? g.piece[i] : sh.live[w] == 2 && i == w * g.n_pieces ? 0.0f : kNegInf;
        x->key = key_of(z, sh.top[w], sh.base[w]);
        x->at = level == 0 ? i : level == 1 ? from * kCells + i % kCells : w << kRowShift | ((from - w * g.n_pieces * kCells) * kPerCell + i % kPerCell);
        return z != kNegInf;
    }

    // The n first of a level's items in the order (score descending, then position) into sh.key / sh.at
    // [0 .. result), in no order: the n-th key, eight bits at a time, then the n-th position of
    // those that have it.
    __device__ static __noinline__ int first(Shared &sh, const Group<DT> &g, int level, int count, int n) {
        const int tid = threadIdx.x;
        unsigned long long key = 0;
        int at = -1, left = n;
        bool all = false;
        Item x;
        __syncthreads();
#pragma unroll 1
        for (int digit = 0; digit < 12 && !all; ++digit) {
            const bool by_key = digit < 8;
            const int shift = by_key ? 56 - 8 * digit : 24 - 8 * (digit - 8);
            if (digit == 8) at = 0;
            if (tid < 256) sh.bins[0][tid] = 0;
            __syncthreads();
#pragma unroll 1
            for (int i = tid; i < count; i += kThreads) {
                if (!item(sh, g, level, i, &x)) continue;
                if (by_key) {
                    if (digit == 0 || x.key >> (shift + 8) == key >> (shift + 8))
                        atomicAdd(&sh.bins[0][255 - static_cast<int>(x.key >> shift & 255)], 1);
                } else if (x.key == key && (digit == 8 || x.at >> (shift + 8) == at >> (shift + 8))) {
                    atomicAdd(&sh.bins[0][x.at >> shift & 255], 1);
                }
            }
            __syncthreads();
            int c = 0;
            const int j = nth_bin(sh.bins[0], left, &c);
            all = j < 0;  // fewer than n items
            if (!all) {
                left -= c;
                if (by_key) key |= static_cast<unsigned long long>(255 - j) << shift;
                else at |= j << shift;
            }
            __syncthreads();
        }
        if (tid == 0) sh.count = 0;
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < count; i += kThreads)
            if (item(sh, g, level, i, &x) && (all || x.key > key || (x.key == key && x.at <= at))) {
                const int p = atomicAdd(&sh.count, 1);
                if (p < kList) sh.key[p] = x.key, sh.at[p] = x.at;
            }
        __syncthreads();
        const int found = min(sh.count, n);
        if (level < 2 && tid < found) sh.first[tid] = sh.at[tid];
        __syncthreads();
        return found;
    }

    __device__ static __noinline__ int narrow(Shared &sh, const Group<DT> &g, int n) {
        const int tid = threadIdx.x, lane = tid & 31;
        int chosen = first(sh, g, 0, g.W * g.n_pieces, n);
#pragma unroll 1
        for (int c = tid >> 5; c < chosen; c += kWarps) {
            const int w = sh.first[c] / g.n_pieces, p = sh.first[c] - w * g.n_pieces;
            float z = lane == 0 ? 0.0f : kNegInf;
            if (sh.live[w] == 1) {
                uint4 v[kCellVecs];
                g.load_cell(w, p, lane, v);
                z = Elem<DT>::vmax4_nan(v);
            }
            sh.value[c * kCells + lane] = z;
        }
        chosen = first(sh, g, 1, chosen * kCells, n);
        const int row_cells = g.n_pieces * kCells;
#pragma unroll 1
        for (int i = tid; i < chosen * kPerCell; i += kThreads) {
            const int cell = sh.first[i / kPerCell], w = cell / row_cells, place = (cell - w * row_cells) * kPerCell + i % kPerCell;
            float z = kNegInf;
            if (sh.live[w] == 2) z = i % kPerCell == 0 ? 0.0f : kNegInf;
            else if (place < g.V) z = Elem<DT>::load1(g.logits + static_cast<int64_t>(w) * g.n_vec, place);
            sh.value[i] = z;
        }
        return first(sh, g, 2, chosen * kPerCell, n);
    }
};

// ln(s.x + s.y), s.x >= 1, to 5e-9, in two terms: with s.x = 2^k m, 0.75 <= m < 1.5, and t = (m - 1) / (m + 1),
// ln m = 2 (t + t^3 / 3 + t^5 / 5 + ..).  t is wanted in two terms, the others are below 2^-7 of one.
__device__ __forceinline__ float2 log_of(float2 s) {
    const uint32_t u = __float_as_uint(s.x);
    const int k = static_cast<int>((u - 0x3f400000u) >> 23);
    const float m = __uint_as_float(u - (static_cast<uint32_t>(k) << 23));
    const float a = __fsub_rn(m, 1.0f);  // exact
    const float d = __fadd_rn(m, 1.0f), dl = __fsub_rn(m, __fsub_rn(d, 1.0f));  // m + 1 in two terms
    const float t = __fdividef(a, d);
    const float r = __fmaf_rn(-t, dl, __fmaf_rn(-t, d, a));  // what t leaves of the quotient, times d
    const float q = t * t;
    float y = 1.0f / 13;
    y = __fmaf_rn(y, q, 1.0f / 11);
    y = __fmaf_rn(y, q, 1.0f / 9);
    y = __fmaf_rn(y, q, 1.0f / 7);
    y = __fmaf_rn(y, q, 1.0f / 5);
    y = __fmaf_rn(y, q, 1.0f / 3);
    // the smaller terms: t^3 y, t's second term, and s.y / s.x
    const float small = 2.0f * __fmaf_rn(t * q, y, __fdividef(r, d)) + __fdividef(s.y, s.x);
    constexpr float ln2_hi = 0x1.62e400p-1f;  // 15 bits: k times it is exact
    constexpr float ln2_lo = static_cast<float>(specv::kLn2D - static_cast<double>(ln2_hi));
    const float2 h = two_sum(k * ln2_hi, 2.0f * t);
    return rounded(make_float2(h.x, h.y + __fmaf_rn(static_cast<float>(k), ln2_lo, small)));
}

// Group b's rows, and whether the call's offsets are valid (else W = 0).  The whole block.
__device__ __forceinline__ bool find_group(Shared &sh, const Call &call, int b, int *first, int *width) {
    const int tid = threadIdx.x;
    bool bad = __ldg(call.offsets) != 0;
#pragma unroll 1
    for (int i = tid; i < call.B; i += kThreads) {
        const int w = __ldg(call.offsets + i + 1) - __ldg(call.offsets + i);
        bad |= w < 0 || w > kMaxBeams;
    }
    bad |= __ldg(call.offsets + call.B) > call.R;
    const bool valid = !__syncthreads_or(bad);
    const int r0 = __ldg(call.offsets + b), W = valid ? __ldg(call.offsets + b + 1) - r0 : 0;
    if (tid < W) sh.live[tid] = __ldg(call.scores + r0 + tid) == kNegInf ? 0 : call.ended && __ldg(call.ended + r0 + tid) ? 2 : 1;
    if (tid == 0) sh.bad = 0, sh.large = 0, sh.count = 0, sh.n_pieces = 0, sh.n_cells = 0;
    static_assert(sizeof(sh.bins) == kThreads * sizeof(int), "a thread clears one");
    (&sh.bins[0][0])[tid] = 0;
    __syncthreads();
    *first = r0, *width = W;
    return valid;
}

// The candidates of group b, by a CTA, from what its rows have left.
template <int DT, int kFlight>
__device__ __forceinline__ void select_group(Shared &sh, const Call &call, int b, bool valid, int r0, int W) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Partial &part = call.part;
    const int n = call.n;
    constexpr float nan = __builtin_nanf("");
    const float score = tid < W ? __ldg(call.scores + r0 + tid) : kNegInf;
    // where there are fewer rows than warps, 2^share warps take a row's pieces
    const int share = W == 0 || W > kWarps ? 0 : 31 - __clz(kWarps / W);
    const int n_vec = call.V / Elem<DT>::kPerVec;
    const Group<DT> g{static_cast<const uint4 *>(call.logits) + static_cast<int64_t>(r0) * n_vec,
                      part.piece + static_cast<int64_t>(r0) * part.n_pieces, W, call.V, n_vec, part.n_pieces};
    if (!valid && call.out_lse) {
#pragma unroll 1
        for (int64_t i = static_cast<int64_t>(b) * kThreads + tid; i < call.R; i += static_cast<int64_t>(call.B) * kThreads) call.out_lse[i] = nan;
    }
    // the largest logits of the pieces that this lane is to look at, and each row's sum, a warp a row
    float mine[kHeld];
    if ((warp >> share) < W) {
        const float *piece = g.piece + static_cast<int64_t>(warp >> share) * g.n_pieces;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int p = ((warp & ((1 << share) - 1)) << 5) + lane + (k * 32 << share);
            mine[k] = p < g.n_pieces ? piece[p] : kNegInf;
        }
    }
#pragma unroll 1
    for (int w = warp; w < W; w += kWarps) {
        if (sh.live[w] != 1) continue;
        const float2 *unit = part.unit + static_cast<int64_t>(r0 + w) * part.n_units;
        float top = kNegInf, from = 0.0f;  // from: what the lane's sum is relative to
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int u = lane; u < part.n_units; u += 32) {
            const float2 x = unit[u];
            const float now = specv::fmax_nan(top, x.x), to = now == kNegInf ? 0.0f : now;
            const float old = top == kNegInf ? 0.0f : specv::ex2((from - to) * specv::kLog2e);
            sum = add_to(make_float2(sum.x * old, sum.y * old), x.y * specv::ex2((x.x - to) * specv::kLog2e));
            top = now, from = to;
        }
        const float all = warp_max_nan(top);
        const float old = specv::ex2((top - (all == kNegInf ? 0.0f : all)) * specv::kLog2e);
        sum.x *= old, sum.y *= old;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, sum.x, off), lo = __shfl_xor_sync(0xffffffffu, sum.y, off);
            sum = add_to(make_float2(sum.x, sum.y + lo), hi);
        }
        if (lane == 0) sh.top[w] = all, sh.sum[w] = sum;
    }
    __syncthreads();
    if (tid < kMaxBeams) {
        float best = kNegInf;
        if (tid < W) {
            const int live = sh.live[tid];
            float2 base = make_float2(score, 0.0f);
            float lse = nan, top = 0.0f;
            bool wrong = score != score || score == -kNegInf;
            if (live == 1) {
                top = sh.top[tid];
                if (top == kNegInf) {
                    lse = top;
                } else if (!(fabsf(top) < -kNegInf)) {
                    wrong = true;
                } else {
                    const float2 log_sum = log_of(sh.sum[tid]);
                    base = add_to(make_float2(-log_sum.x, -log_sum.y), score);
                    base = rounded(base);
                    const float2 sum = add_to(log_sum, top);
                    lse = sum.x + sum.y;
                }
            }
            if (call.out_lse) call.out_lse[r0 + tid] = lse;
            if (wrong) sh.bad = 1;
            sh.base[tid] = base, sh.top[tid] = top;
            if (live && top != kNegInf) {
                best = base.x;  // of a row's best candidate
                if (!(fabsf(best) <= kMagnitude)) sh.large = 1;
            }
        }
        best = warp_max_nan(best);
        if (lane == 0) sh.best[warp] = best;
    }
    __syncthreads();
    const float most = fmaxf(sh.best[0], sh.best[1]);
    const bool fine = valid && !sh.bad;
    int found = 0;
    if (fine && most != kNegInf) {
        found = sh.large ? -1 : list_candidates<DT, kFlight>(sh, g, mine, share, most, n);
        if (found < 0) found = Digits<DT>::narrow(sh, g, n);
        by_rank(sh, found, [&](const Item &x, int place) {
            if (place >= n) return;
            const int w = x.at >> kRowShift;
            const int64_t o = static_cast<int64_t>(b) * n + place;
            call.out_scores[o] = score_of(x.key);
            call.out_tokens[o] = sh.live[w] == 2 ? call.end_token : x.at & ((1 << kRowShift) - 1);
            call.out_rows[o] = r0 + w;
        });
    }
    if (tid < n && tid >= found) {
        const int64_t o = static_cast<int64_t>(b) * n + tid;
        call.out_scores[o] = fine ? kNegInf : nan, call.out_tokens[o] = -1, call.out_rows[o] = -1;
    }
}

// Behind rows_kernel: a CTA per group.  One per SM where there are no more groups than SMs, with three pieces of a warp
// under way; else two, with the registers for two (400 groups of 8 rows of 8000: 35.4 -> 30 us; 64 groups of 8 rows of 128256
// 26.7 -> 27.8, 128 of 16 rows of 152064 94 -> 96.5.  Four and five pieces are as three).
template <int DT, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) select_kernel(const __grid_constant__ Call call) {
    __shared__ __align__(16) Shared sh;
    int r0, W;
    const bool valid = find_group(sh, call, blockIdx.x, &r0, &W);
    specv::grid_dependency_wait();
    select_group<DT, kPerSm == 1 ? 3 : 2>(sh, call, blockIdx.x, valid, r0, W);
}

// Few and small groups, in one launch: of a cluster, the first CTA finds out about the group while the others stream its
// rows (those without a candidate too: whether one has them is not waited for), and then selects.
template <int DT>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) group_kernel(const __grid_constant__ Call call, int rows) {
    __shared__ __align__(16) Shared sh;
    const int b = blockIdx.x / kCluster, rank = blockIdx.x - b * kCluster;
    int r0 = 0, W = 0;
    bool valid = false;
    if (rank == 0) {
        valid = find_group(sh, call, b, &r0, &W);
    } else {
        r0 = __ldg(call.offsets + b);
        const int end = __ldg(call.offsets + b + 1);
        const int units = r0 >= 0 && end > r0 && end <= rows && end - r0 <= kMaxBeams ? (end - r0) * call.part.n_units : 0;
#pragma unroll 1
        for (int i = (rank - 1) * kWarps + (threadIdx.x >> 5); i < units; i += (kCluster - 1) * kWarps) {
            const int w = i / call.part.n_units;
            stream_unit<DT>(call, r0 + w, i - w * call.part.n_units);
        }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0) select_group<DT, 3>(sh, call, b, valid, r0, W);
}

// The partial results of R rows, from `base` on; their bytes.
size_t partial_of(void *base, int64_t R, int V, int dtype, Partial *part) {
    const int64_t bytes = static_cast<int64_t>(V) * (dtype == SPEC_F32 ? 4 : 2);
    part->n_pieces = static_cast<int>((bytes + kPieceBytes - 1) / kPieceBytes);
    part->n_units = (part->n_pieces + kUnitPieces - 1) / kUnitPieces;
    const size_t units = static_cast<size_t>(R) * part->n_units * sizeof(float2);
    part->unit = static_cast<float2 *>(base);
    part->piece = reinterpret_cast<float *>(static_cast<char *>(base) + units);
    return specv::align_up(units + static_cast<size_t>(R) * part->n_pieces * sizeof(float), 256);
}

template <int DT>
int launch(const Call &call, int rows, cudaStream_t s) {
    const Partial &part = call.part;
    // A cluster per group where they fill no more than the GPU's SMs and a warp has two units at most on average: the
    // host's part of a second launch costs more than the SMs that stay idle.  One group of 4 rows of 32000 in fp32: 6 us less a
    // call than in two launches (25.5 against 31.8 at the time), on the device 7.7 us against 6.9.
    if (rows > 0 && call.B * kCluster <= kSms && static_cast<int64_t>(rows) * part.n_units <= int64_t{2} * call.B * kCluster * kWarps)
        return specv::cuda_ok(specv::launch_k(false, group_kernel<DT>, dim3(call.B * kCluster), dim3(kThreads), 0, s, call, rows), "group_kernel")
                   ? SPEC_OK
                   : SPEC_ERR_CUDA;
    const int blocks = (part.n_units + kBlockUnits - 1) / kBlockUnits;
    if (rows > 0 && !specv::cuda_ok(specv::launch_k(false, rows_kernel<DT>, dim3(static_cast<unsigned>(rows) * blocks), dim3(kRowThreads), 0, s, call, blocks),
                                    "rows_kernel"))
        return SPEC_ERR_CUDA;
    const auto select = call.B <= kSms ? select_kernel<DT, 1> : select_kernel<DT, 2>;
    return specv::cuda_ok(specv::launch_k(rows > 0, select, dim3(call.B), dim3(kThreads), 0, s, call), "select_kernel") ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace specbeam

extern "C" {

size_t spec_beam_workspace_bytes(int R, int V, int dtype) {
    if (R < 0 || specv::check_common(0, V, dtype) != SPEC_OK) return 0;
    const int64_t rows = std::min<int64_t>(R, static_cast<int64_t>(SPEC_MAX_B) * SPEC_MAX_BEAMS);
    specbeam::Partial part;
    return specbeam::partial_of(nullptr, std::max<int64_t>(rows, 1), V, dtype, &part);
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
    // rows of no group are not read
    const int rows = static_cast<int>(std::min<int64_t>(R, static_cast<int64_t>(B) * SPEC_MAX_BEAMS));
    specbeam::Partial part;
    if (specbeam::partial_of(workspace, rows, V, dtype, &part) > workspace_bytes && rows > 0) return SPEC_ERR_WORKSPACE;
    const specbeam::Call call{logits, scores, ended, offsets, end_token, B, R, V, n, part, out_scores, out_tokens, out_rows, out_lse};
    const auto run = dtype == SPEC_F32 ? specbeam::launch<SPEC_F32> : specbeam::launch<SPEC_BF16>;
    return run(call, rows, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
