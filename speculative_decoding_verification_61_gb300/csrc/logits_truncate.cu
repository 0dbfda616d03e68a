// logits_truncate.cu -- top-k, top-p and min-p truncation of packed logit
// rows behind the C ABI of include/spec_verify.h: tokens outside the kept set
// become -inf.
//
// All three keep a prefix of one order, z descending and then index
// ascending, so a row's result is one cut: the last kept (z, index).  With
// w = exp((z - zmax) / T):
//   top-k   the first k tokens;
//   top-p   the tokens whose mass before them is < p Z, Z the mass of the
//           first k tokens;
//   min-p   the tokens with (z - zmax) / T >= ln(min_p).
// A token on the wrong side of the top-p border is a wrong answer, however
// small its mass, so masses are exact far below one token's mass: weights
// come from a two-term fp32 exponential (relative error below 2^-42 down to e^-20), and
// are summed as integers of up to 125 bits, whose sum does not depend on its order and
// keeps a small weight's bits beside a large one.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "logits_host.h"

namespace speclog {
namespace {

constexpr int kThreads = 512;
constexpr int kPerSm = 2;  // resident CTAs
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;        // elements of one bin that are sorted in shared memory
constexpr int kAnyGroups = 2048;   // groups of 32 vectors whose largest values are kept
constexpr int kBinsPerOctave = 32;  // first-level bins per halving of the weight

using Mass = unsigned __int128;  // a fixed-point sum of weights

struct Truncate {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
};

// ------------------------------------------------------------- order of keys
// Unsigned key in the order of the values (-0 and +0 alike).
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t u = __float_as_uint(__fadd_rn(z, 0.0f));
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
// Position in the order: a larger one comes first.
__device__ __forceinline__ uint64_t place_of(uint32_t key, int index) {
    return static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(index);
}

// ------------------------------------------------------------------- weights
// 2^(j/64) in two fp32 terms, j = 0..63, rounded from 60 digits.
__constant__ float2 kExp2Table[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},
};

// exp((z - zmax) / T).  2^x, x = (z - zmax) log2(e) / T, by the split x = n + j / 64 + r,
// |r| <= 1/128: a table of 2^(j/64) in two fp32 terms, and the Taylor
// polynomial of e^(r ln 2) whose leading terms are carried in two fp32 terms
// as well (error-free sums and products).  Relative error below 2^-46 + x 2^-47,
// x = (zmax - z) / T, of 1.5 million weights (2^-42.6 up to x = 20); the
// second part is x's own, a product of two fp32 terms.
struct Weights {
    float zmax, ch, cl;  // log2(e) / T in two terms
    int frac;            // of cut_of_row's bins
    const float2 *table;  // shared memory: 2^(j/64), j = 0..63
};

// s + e = a + b exactly (|a| >= |b| or a = 0)
__device__ __forceinline__ float fast_two_sum(float a, float b, float *e) {
    const float s = __fadd_rn(a, b);
    *e = __fsub_rn(b, __fsub_rn(s, a));
    return s;
}
__device__ __forceinline__ float two_sum(float a, float b, float *e) {
    const float s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    *e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// The weight as mantissa * 2^exponent: mantissa in (0.99 2^48, 2^49), exponent <= -48;
// mantissa 0 where the weight is below 2^-120.
__device__ __forceinline__ uint64_t weight_mantissa(const Weights &w, float z, int *exponent) {
    float dl;
    const float dh = two_sum(z, -w.zmax, &dl);
    const float xh = __fmul_rn(dh, w.ch);
    if (!(xh > -120.0f)) {
        *exponent = 0;
        return 0;
    }
    float xl = __fmaf_rn(dh, w.ch, -xh);
    xl = __fmaf_rn(dh, w.cl, xl);
    xl = __fmaf_rn(dl, w.ch, xl);
    const int m = __float2int_rn(xh * 64.0f);
    const float r0 = __fsub_rn(xh, static_cast<float>(m) * 0.015625f);  // exact
    float rl;
    const float rh = two_sum(r0, xl, &rl);
    // t = r ln 2
    constexpr float kLn2Hi = 0.693147180559945309417f;
    constexpr float kLn2Lo = static_cast<float>(0.69314718055994530941723212145818 - static_cast<double>(kLn2Hi));
    const float th = __fmul_rn(rh, kLn2Hi);
    float tl = __fmaf_rn(rh, kLn2Hi, -th);
    tl = __fmaf_rn(rh, kLn2Lo, tl);
    tl = __fmaf_rn(rl, kLn2Hi, tl);
    // e^t - 1 = t + t^2 / 2 + t^3 (1/6 + t / 24 + t^2 / 120)
    const float sq = __fmul_rn(th, th);
    float sql = __fmaf_rn(th, th, -sq);
    sql = __fmaf_rn(2.0f * th, tl, sql);
    const float q = __fmul_rn(__fmul_rn(sq, th), __fmaf_rn(th, __fmaf_rn(th, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f));
    float el;
    const float eh = two_sum(th, 0.5f * sq, &el);
    el = __fadd_rn(el, __fadd_rn(__fadd_rn(tl, 0.5f * sql), q));
    // 2^(j/64) (1 + e)
    const float2 tj = w.table[m & 63];
    const float ph = __fmul_rn(tj.x, eh);
    float pl = __fmaf_rn(tj.x, eh, -ph);
    pl = __fmaf_rn(tj.x, el, pl);
    pl = __fmaf_rn(tj.y, eh, pl);
    float ul;
    const float uh = fast_two_sum(tj.x, ph, &ul);
    ul = __fadd_rn(ul, __fadd_rn(tj.y, pl));
    *exponent = (m >> 6) - 48;
    // (uh is a whole number of 2^-24: below 1 where j = 0 and t < 0, whose steps are half of those from 1 on)
    return (static_cast<uint64_t>(__float2uint_rn(uh * 16777216.0f)) << 24) +
           static_cast<int64_t>(__float2int_rn(ul * 281474976710656.0f));
}

// A token's weight in the sums of cut_of_row, in units of 2^-(frac + octave).
// `octave` is the one of its first-level bin, which it is at most a hair above,
// so V of them fit 64 bits, and a tail of V tokens however small is summed to
// a relative error of 2^-frac (2^-45 below 2^17 columns, 2^-37 at 2^24).  With the one
// unit of the largest weights for all, a flat tail's tokens are all rounded the same way,
// by up to V 2^-(frac + 1) of the largest weight together.
__device__ __forceinline__ uint64_t bin_weight(const Weights &w, float z, int octave) {
    int e;
    const uint64_t m = weight_mantissa(w, z, &e);
    const int shift = -(e + w.frac + octave);  // at least 1: frac <= 47
    return shift > 63 ? 0 : (m + (1ull << (shift - 1))) >> shift;
}
// The same in units of 2^-(frac + kMostOctave), in which sums over several octaves
// are kept: no bit is lost, 125 of them are used at most.
constexpr int kMostOctave = kBins / kBinsPerOctave - 1;
__device__ __forceinline__ Mass wide_mass(uint64_t units, int octave) { return static_cast<Mass>(units) << (kMostOctave - octave); }

__device__ __forceinline__ Mass shfl(Mass m, int src) {
    const uint64_t hi = __shfl_sync(0xffffffffu, static_cast<uint64_t>(m >> 64), src);
    return static_cast<Mass>(hi) << 64 | __shfl_sync(0xffffffffu, static_cast<uint64_t>(m), src);
}
__device__ __forceinline__ Mass shfl_up(Mass m, int off) {
    const uint64_t hi = __shfl_up_sync(0xffffffffu, static_cast<uint64_t>(m >> 64), off);
    return static_cast<Mass>(hi) << 64 | __shfl_up_sync(0xffffffffu, static_cast<uint64_t>(m), off);
}

// ------------------------------------------------------------ block helpers
// What one thread finds for the row (fp64 runs at a small fraction of fp32's
// rate, so no thread does it twice).
struct RowConstants {
    float ch, cl;  // log2(e) / T
    uint32_t min_p_key;
};

struct Shared {
    int seq;
    float2 table[64];
    uint32_t count[kBins], lo[kBins], hi[kBins];
    uint64_t list[kList];
    uint32_t group_max[kAnyGroups];  // of rows with at most so many groups
    Mass warp_mass[32];
    uint32_t warp_count[32];
    uint32_t red[32];
    uint32_t n_list, key_lo, key_hi;
    // where the scan of the bins stopped
    int bin;
    uint32_t above_count, bin_count;
    Mass above_mass, total_mass;
    // what lies above the first bin or the list
    uint32_t base_count;
    Mass base_mass;
    Mass target;  // of a search by mass
    uint64_t cut;
    Mass mass;    // up to the cut
    RowConstants row;
};

// What a search looks for: the first place in the order where the tokens up to and
// with it number `need`, without or with their mass, or weigh sm.target.
enum Search { kCount, kCountMass, kMass };

template <Search S>
__device__ __forceinline__ bool reached(uint32_t need, Mass target, uint32_t c, Mass m) {
    return S == kMass ? m >= target : c >= need;
}

// Sums over the block of the threads before of a count and (not in a search by count
// alone) a mass per thread.
template <Search S>
__device__ __forceinline__ void block_scan(Shared &sm, uint32_t &c, Mass &m) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t c0 = c;
    const Mass m0 = m;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t cc = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += cc;
        if (S != kCount) {
            const Mass mm = shfl_up(m, off);
            if (lane >= off) m += mm;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sm.warp_count[warp] = c;
        if (S != kCount) sm.warp_mass[warp] = m;
    }
    __syncthreads();
    // the sums of the warps before: every warp scans them for itself
    const int warps = static_cast<int>(blockDim.x) >> 5;
    uint32_t bc = lane < warps ? sm.warp_count[lane] : 0;
    Mass bm = 0;
    if (S != kCount && lane < warps) bm = sm.warp_mass[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t cc = __shfl_up_sync(0xffffffffu, bc, off);
        if (lane >= off) bc += cc;
        if (S != kCount) {
            const Mass mm = shfl_up(bm, off);
            if (lane >= off) bm += mm;
        }
    }
    bc = __shfl_sync(0xffffffffu, bc, (warp + 31) & 31);
    c += (warp ? bc : 0) - c0;
    if (S != kCount) {
        bm = shfl(bm, (warp + 31) & 31);
        m += (warp ? bm : 0) - m0;
    }
}

__device__ __forceinline__ uint64_t bin_mass(const Shared &sm, int bin) { return static_cast<uint64_t>(sm.hi[bin]) << 32 | sm.lo[bin]; }

// Finds the search's bin in the histogram, given what lies above the first bin
// (sm.base_*); leaves it with what lies above it in sm.bin, sm.above_*, sm.bin_count,
// and the mass of everything in sm.total_mass; sm.bin is -1 if none reaches it.
// The bins are of one octave, or (-1) the first-level ones, each of its own.
template <int T, Search S>
__device__ __noinline__ void find_bin(Shared &sm, uint32_t need, int octave) {
    constexpr int kPer = kBins / T;
    static_assert(kBinsPerOctave % kPer == 0, "a thread's bins are of one octave");
    const int first = threadIdx.x * kPer, oct = octave < 0 ? first / kBinsPerOctave : octave;
    if (threadIdx.x == 0) sm.bin = -1;
    uint32_t c = 0;
    uint64_t units = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        c += sm.count[first + i];
        if (S != kCount) units += bin_mass(sm, first + i);
    }
    const uint32_t own_c = c;
    const Mass own_m = wide_mass(units, oct);
    Mass m = own_m, target = 0;
    block_scan<S>(sm, c, m);
    c += sm.base_count;
    if (S != kCount) {
        m += sm.base_mass;
        if (S == kMass) target = sm.target;
        if (threadIdx.x == T - 1) sm.total_mass = m + own_m;
    }
    if (reached<S>(need, target, c + own_c, m + own_m) && !reached<S>(need, target, c, m)) {
#pragma unroll 1
        for (int i = first;; ++i) {  // (in one of the thread's)
            const uint32_t n = sm.count[i];
            const Mass here = S != kCount ? wide_mass(bin_mass(sm, i), oct) : 0;
            if (reached<S>(need, target, c + n, m + here)) {
                sm.bin = i;
                sm.above_count = c;
                if (S != kCount) sm.above_mass = m;
                sm.bin_count = n;
                break;
            }
            c += n;
            m += here;
        }
    }
    __syncthreads();
}

// f(value, index) for a row's elements, several vectors of a thread in flight;
// groups (a warp's 32 vectors) whose largest key is below `low` are passed over.
// (bf16 rows come here rarely: small code, beside the pass that they usually take)
template <int DT>
constexpr int kFlight = DT == SPEC_F32 ? 4 : 1;
template <int DT, int T, int FLIGHT, typename F>
__device__ __forceinline__ void for_each(const Shared &sm, const char *row, int V, uint32_t low, F &&f) {
    constexpr int kPer = Elem<DT>::kPerVec;
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
    const int vecs = V / kPer;
    const auto wanted = [&](int v) { return v < vecs && (low == 0 || sm.group_max[v >> 5] >= low); };
    if (FLIGHT == 1) {  // much work per vector: the next one comes meanwhile
        int v = threadIdx.x;
        bool in = wanted(v);
        uint4 q = make_uint4(0, 0, 0, 0);
        if (in) q = p[v];
#pragma unroll 1
        for (; v < vecs; v += T) {
            const bool in_next = wanted(v + T);
            uint4 next = make_uint4(0, 0, 0, 0);
            if (in_next) next = p[v + T];
            if (in) {
                float x[kPer];
                Elem<DT>::unpack(q, x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) f(x[i], v * kPer + i);
            }
            q = next;
            in = in_next;
        }
        return;
    }
    for (int v0 = threadIdx.x; v0 < vecs; v0 += T * FLIGHT) {
        uint4 q[FLIGHT];
        bool in[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int v = v0 + u * T;
            in[u] = wanted(v);
            if (in[u]) q[u] = p[v];
        }
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            if (!in[u]) continue;
            float x[kPer];
            Elem<DT>::unpack(q[u], x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) f(x[i], (v0 + u * T) * kPer + i);
        }
    }
}
// The largest value (NaN if there is one) and the groups' largest keys; the row
// into `hold` on the way, if given.
template <int DT, int T>
__device__ __forceinline__ float largest(Shared &sm, const char *row, int V, bool grouped, uint4 *hold) {
    constexpr int kPer = Elem<DT>::kPerVec, FLIGHT = kFlight<DT>;
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
    const int vecs = V / kPer, lane = threadIdx.x & 31;
    float top = __int_as_float(0xff800000);
    for (int v0 = threadIdx.x; v0 - lane < vecs; v0 += T * FLIGHT) {
        uint4 q[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u)
            if (v0 + u * T < vecs) q[u] = p[v0 + u * T];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int v = v0 + u * T;
            if (v - lane >= vecs) break;
            const float m = v < vecs ? Elem<DT>::vmax_nan(q[u]) : __int_as_float(0xff800000);
            if (DT == SPEC_F32 && hold && v < vecs) hold[v] = q[u];
            top = specv::fmax_nan(top, m);
            const uint32_t key = __reduce_max_sync(0xffffffffu, key_of(m));
            if (grouped && lane == 0) sm.group_max[v >> 5] = key;
        }
    }
    return top;
}

// (scale is finite, so the largest value is in bin 0)
__device__ __forceinline__ int first_bin(float z, float zmax, float scale) {
    // to the nearest whole number, by the bits of 2^23 + x (a conversion is slower)
    return __float_as_int(__fadd_rn(fminf(__fmul_rn(__fsub_rn(zmax, z), scale), static_cast<float>(kBins - 1)), 8388608.0f)) & (kBins - 1);
}

// A key that no element of the bins up to `bin` is below (0 where groups are not kept).
__device__ __forceinline__ uint32_t bin_low(int bin, float zmax, float scale, bool grouped) {
    if (!grouped || bin >= kBins - 1) return 0;
    const float z = zmax - (static_cast<float>(bin) + 1.0f) / scale;  // half a bin lower than need be
    return isfinite(z) ? key_of(z - fabsf(z) * 1e-6f) : 0;
}

__device__ __forceinline__ void add_to_bin(Shared &sm, int bin, bool mass, uint64_t w) {
    atomicAdd(&sm.count[bin], 1u);
    if (mass) {
        const uint32_t lo = static_cast<uint32_t>(w);
        const uint32_t old = atomicAdd(&sm.lo[bin], lo);
        const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi) atomicAdd(&sm.hi[bin], hi);  // (one 64-bit atomic for both: 378 -> 515 us)
    }
}

template <int T>
__device__ __forceinline__ void clear_bins(Shared &sm) {
    for (int i = threadIdx.x; i < kBins; i += T) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
    __syncthreads();
}

// The list's n elements in the order, largest first (bitonic).
template <int T>
__device__ __noinline__ void sort_list(Shared &sm, uint32_t n) {
    for (int i = n + threadIdx.x; i < kList; i += T) sm.list[i] = 0;
    int size = 2;
    while (size < static_cast<int>(n)) size <<= 1;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1) {  // bitonic, largest first
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = threadIdx.x; t < size / 2; t += T) {
                const int a = 2 * t - (t & (j - 1)), b = a + j;
                const uint64_t x = sm.list[a], y = sm.list[b];
                if ((x < y) == ((a & k) == 0)) {
                    sm.list[a] = y;
                    sm.list[b] = x;
                }
            }
            __syncthreads();
        }
    }
}

// The search's place in the sorted list, given what lies above it (sm.base_*): sm.cut,
// and the mass up to it in sm.mass.
template <int T, Search S>
__device__ __noinline__ void place_in_list(Shared &sm, uint32_t n, const Weights w, float scale, uint32_t need) {
    constexpr int kPer = kList / T;
    const auto mass_at = [&](int t) {  // as the bins have it
        const float z = value_of(static_cast<uint32_t>(sm.list[t] >> 32));
        const int octave = first_bin(z, w.zmax, scale) / kBinsPerOctave;
        return wide_mass(bin_weight(w, z, octave), octave);
    };
    const int first = threadIdx.x * kPer, end = min(first + kPer, static_cast<int>(n));
    uint32_t c = max(end - first, 0);
    Mass m = 0, target = 0;
    if (S != kCount)
        for (int t = first; t < end; ++t) m += mass_at(t);
    const uint32_t own_c = c;
    const Mass own_m = m;
    block_scan<S>(sm, c, m);
    c += sm.base_count;
    if (S != kCount) m += sm.base_mass;
    if (S == kMass) target = sm.target;
    if (reached<S>(need, target, c + own_c, m + own_m) && !reached<S>(need, target, c, m)) {
#pragma unroll 1
        for (int t = first; t < end; ++t) {
            ++c;
            if (S != kCount) m += mass_at(t);
            if (reached<S>(need, target, c, m)) {
                sm.cut = sm.list[t];
                sm.mass = m;
                break;
            }
        }
    }
    __syncthreads();
}

// The search's place inside the bin that find_bin left: the bin's elements are
// sorted if they fit the list, else the bin is split by key until they do or
// one value is left, whose ties go by index.  Leaves the place in sm.cut, and
// the mass of the tokens up to it in sm.mass.
template <int DT, int T, Search S>
__device__ __noinline__ void find_place(Shared &sm, const char *row, int V, const Weights w, float scale, uint32_t need, bool grouped) {
    constexpr bool mass = S != kCount;
    const int bin = sm.bin, octave = bin / kBinsPerOctave;
    uint32_t n = sm.bin_count;
    __syncthreads();
    const auto step_down = [&] {  // into the bin found
        sm.base_count = sm.above_count;
        if (mass) sm.base_mass = sm.above_mass;
        sm.n_list = 0;
    };
    if (threadIdx.x == 0) {
        step_down();
        sm.key_lo = 0xffffffffu;
        sm.key_hi = 0;
    }
    __syncthreads();
    uint32_t klo = 0xffffffffu, khi = 0;
    for_each<DT, T, kFlight<DT>>(sm, row, V, bin_low(bin, w.zmax, scale, grouped), [&](float z, int i) {
        if (first_bin(z, w.zmax, scale) != bin) return;
        const uint32_t key = key_of(z);
        klo = min(klo, key);
        khi = max(khi, key);
        if (n <= kList) sm.list[atomicAdd(&sm.n_list, 1u)] = place_of(key, i);
    });
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if ((threadIdx.x & 31) == 0) {
        atomicMin(&sm.key_lo, klo);
        atomicMax(&sm.key_hi, khi);
    }
    __syncthreads();
    klo = sm.key_lo;
    khi = sm.key_hi;
    bool listed = n <= kList;
    while (!listed && klo < khi) {
        // 2048 equal parts of the keys khi .. klo
        const int shift = max(0, 32 - __clz(khi - klo) - 11);
        clear_bins<T>(sm);
        for_each<DT, T, 1>(sm, row, V, grouped ? klo : 0, [&](float z, int) {
            const uint32_t key = key_of(z);
            if (key < klo || key > khi) return;
            add_to_bin(sm, static_cast<int>((khi - key) >> shift), mass, mass ? bin_weight(w, z, octave) : 0);
        });
        __syncthreads();
        find_bin<T, S>(sm, need, octave);
        const uint32_t j = static_cast<uint32_t>(sm.bin);
        const uint32_t top = khi - (j << shift);
        const uint32_t width = (1u << shift) - 1;
        klo = top - klo > width ? top - width : klo;
        khi = top;
        n = sm.bin_count;
        __syncthreads();
        if (threadIdx.x == 0) step_down();
        __syncthreads();
        if (n <= kList) {
            for_each<DT, T, 1>(sm, row, V, grouped ? klo : 0, [&](float z, int i) {
                const uint32_t key = key_of(z);
                if (key >= klo && key <= khi) sm.list[atomicAdd(&sm.n_list, 1u)] = place_of(key, i);
            });
            __syncthreads();
            listed = true;
        }
    }
    if (listed) {
        sort_list<T>(sm, n);
        place_in_list<T, S>(sm, n, w, scale, need);
        return;
    }
    // one value: how many of its ties the search takes, and the last one's index
    const uint64_t wt = mass ? bin_weight(w, value_of(khi), octave) : 0;
    uint32_t take = n;
    if (S != kMass) {
        take = need - sm.base_count;
    } else {
        const Mass base = sm.base_mass, target = sm.target;
        uint32_t lo = 1, hi = n;  // the fewest whose mass reaches the target
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (base + wide_mass(mid * wt, octave) >= target) hi = mid;
            else lo = mid + 1;
        }
        take = lo;
    }
    uint32_t last = 0xffffffffu;
    if (take < n) {
        // a thread owns a run of vectors: count its ties, then find the one
        constexpr int kPer = Elem<DT>::kPerVec;
        const int vecs = V / kPer, per = (vecs + T - 1) / T;
        const int v0 = min(vecs, static_cast<int>(threadIdx.x) * per), v1 = min(vecs, v0 + per);
        const uint4 *p = reinterpret_cast<const uint4 *>(row);
        uint32_t c = 0;
        Mass none = 0;
        for (int v = v0; v < v1; ++v) {
            float x[kPer];
            Elem<DT>::unpack(p[v], x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) c += key_of(x[i]) == khi;
        }
        const uint32_t own = c;
        block_scan<kCount>(sm, c, none);
        if (c < take && c + own >= take) {
            for (int v = v0; v < v1; ++v) {
                float x[kPer];
                Elem<DT>::unpack(p[v], x);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (key_of(x[i]) == khi && ++c == take) sm.red[0] = v * kPer + i;
            }
        }
        __syncthreads();
        last = sm.red[0];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sm.cut = place_of(khi, static_cast<int>(last));
        if (mass) sm.mass = sm.base_mass + wide_mass(take * wt, octave);
    }
    __syncthreads();
}

// The lowest key whose value passes min-p, by the definition's test in fp64:
// the border's own value is at most a few keys off (one thread's work).
__device__ __noinline__ uint32_t min_p_key(float zmax, float T, float min_p) {
    const double border = log(static_cast<double>(min_p));
    const uint32_t last = key_of(__int_as_float(0xff800000)), first = key_of(zmax);
    const double shift = static_cast<double>(T) * border;
    auto passes = [&](uint32_t key) {
        const double d = static_cast<double>(value_of(key)) - static_cast<double>(zmax), gap = d - shift;
        if (fabs(gap) > 1e-12 * fabs(shift)) return gap > 0.0;  // the division would say the same
        return d / static_cast<double>(T) >= border;
    };
    uint32_t key = key_of(static_cast<float>(static_cast<double>(zmax) + shift));
    key = min(max(key, last), first);
    while (key < first && !passes(key)) ++key;
    while (key > last && passes(key - 1)) --key;
    return key;
}

// One row's settings.
struct Settings {
    float T;
    int k;
    float p, m;
    bool valid, active;
};

__device__ __forceinline__ Settings load_settings(const Truncate &tr, int b, int V) {
    Settings s;
    s.T = __ldg(tr.temperature + b);
    s.k = tr.top_k ? __ldg(tr.top_k + b) : 0;
    s.p = tr.top_p ? __ldg(tr.top_p + b) : 1.0f;
    s.m = tr.min_p ? __ldg(tr.min_p + b) : 0.0f;
    const float c = specv::temp_scale(s.T);
    s.valid = c == c && s.k >= 0 && s.p > 0.0f && s.p <= 1.0f && s.m >= 0.0f && s.m <= 1.0f;
    if (s.k >= V) s.k = 0;
    s.active = s.T != 0.0f && (s.k > 0 || s.p < 1.0f || s.m > 0.0f);
    return s;
}

__device__ __forceinline__ void set_scale(RowConstants &rc, const Settings &s) {
    const double c = specv::kLog2eD / static_cast<double>(s.T);
    rc.ch = static_cast<float>(c);
    rc.cl = static_cast<float>(c - static_cast<double>(rc.ch));
}
__device__ __forceinline__ Weights row_weights(const RowConstants &rc, float zmax, int V, const float2 *table) {
    // V weights of at most 1.02 sum to less than 2^63
    return Weights{zmax, rc.ch, rc.cl, min(47, 30 + __clz(V)), table};
}
// The least mass that is not below p Z, exactly: p = mantissa 2^-q, 24 <= q <= 149.
__device__ __forceinline__ Mass mass_target(float p, Mass Z) {
    const uint32_t u = __float_as_uint(p), ex = u >> 23;  // (0 < p < 1)
    const uint32_t mantissa = ex ? (u & 0x7fffffu) | 0x800000u : u;
    const int q = ex ? 150 - static_cast<int>(ex) : 149;
    const Mass lo = static_cast<Mass>(static_cast<uint64_t>(Z)) * mantissa;
    const Mass hi = static_cast<Mass>(static_cast<uint64_t>(Z >> 64)) * mantissa + (lo >> 64);  // the product: hi 2^64 + l
    const uint64_t l = static_cast<uint64_t>(lo);
    if (q < 64) return (hi << (64 - q) | l >> q) + (l << (64 - q) != 0);
    return (hi >> (q - 64)) + (l != 0 || (hi & ((static_cast<Mass>(1) << (q - 64)) - 1)) != 0);
}
__device__ __forceinline__ void fill_table(float2 *table) {
    if (threadIdx.x < 64) table[threadIdx.x] = kExp2Table[threadIdx.x];
}

// The cut of one row in memory, for rows of any kind: every token whose place is
// below it goes; 0: the row stays as it is.  Passes over the row: its largest
// value (and its copy in `hold`, if given, which the others then read), a histogram
// over 32 bins per halving of the weight, the border bin's elements, sorted.  fp32 logits have no few values, so top-p computes a weight
// per token (about 45 instructions): 384 rows of 128256 take 139 us with top-k
// (2.8 TB/s), 340 with top-p alone (1.2 TB/s), where those instructions bound it:
// exact masses for the bins around the border alone, the rest summed in
// registers, took 427.
template <int DT, int T>
__device__ __noinline__ uint64_t cut_of_row(Shared &sm, const char *row, int V, const Settings &s, char *hold) {
    const int tid = threadIdx.x;
    const bool grouped = V <= kAnyGroups * 32 * Elem<DT>::kPerVec;
    float top = largest<DT, T>(sm, row, V, grouped, reinterpret_cast<uint4 *>(hold));
    if (hold) row = hold;  // (the block meets below before it is read)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = specv::fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    __syncthreads();
    if ((tid & 31) == 0) sm.red[tid >> 5] = __float_as_uint(top);
    __syncthreads();
    top = __uint_as_float(sm.red[tid & (T / 32 - 1)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = specv::fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float zmax = value_of(key_of(top));  // (+0 for -0)
    if (!isfinite(top)) return 0;  // NaN, +inf, or nothing but -inf
    if (tid == 0) {
        set_scale(sm.row, s);
        if (s.m > 0.0f) sm.row.min_p_key = min_p_key(zmax, s.T, s.m);
    }
    __syncthreads();
    const Weights w = row_weights(sm.row, zmax, V, sm.table);
    const float scale = fminf(w.ch * kBinsPerOctave, 3.0e38f);
    const bool mass = s.p < 1.0f;
    uint64_t cut = 0;
    if (s.k > 0 || mass) {
        const uint32_t k = s.k;
        auto fill = [&](bool mass) {
            clear_bins<T>(sm);
            if (mass)
                for_each<DT, T, 1>(sm, row, V, 0, [&](float z, int) {
                    const int bin = first_bin(z, zmax, scale);
                    add_to_bin(sm, bin, true, bin_weight(w, z, bin / kBinsPerOctave));
                });
            else
                for_each<DT, T, kFlight<DT>>(sm, row, V, 0, [&](float z, int) { atomicAdd(&sm.count[first_bin(z, zmax, scale)], 1u); });
            __syncthreads();
        };
        auto from_top = [&] {  // nothing above the first bin
            if (tid == 0) {
                sm.base_count = 0;
                sm.base_mass = 0;
            }
        };
        bool done = false;
        from_top();
        if (s.k > 0 && s.k <= kList) {
            // few tokens: they are listed and sorted, and only theirs are the weights that matter
            fill(false);
            find_bin<T, kCount>(sm, k, -1);
            const int bin = sm.bin;
            const uint32_t n = sm.above_count + sm.bin_count;
            __syncthreads();
            done = n <= kList;
            if (done) {
                if (tid == 0) sm.n_list = 0;
                __syncthreads();
                for_each<DT, T, kFlight<DT>>(sm, row, V, bin_low(bin, zmax, scale, grouped), [&](float z, int i) {
                    if (first_bin(z, zmax, scale) <= bin) sm.list[atomicAdd(&sm.n_list, 1u)] = place_of(key_of(z), i);
                });
                __syncthreads();
                sort_list<T>(sm, n);
                if (mass) {
                    place_in_list<T, kCountMass>(sm, n, w, scale, k);
                    if (tid == 0) sm.target = mass_target(s.p, sm.mass);
                    __syncthreads();
                    place_in_list<T, kMass>(sm, k, w, scale, 0);
                    cut = sm.cut;
                } else {
                    cut = sm.list[k - 1];
                }
                __syncthreads();
            }
        }
        if (!done) fill(mass);
        if (s.k > 0 && !done) {
            if (mass) {
                find_bin<T, kCountMass>(sm, k, -1);
                const bool splits = sm.bin_count > kList;  // find_place then uses the bins itself
                find_place<DT, T, kCountMass>(sm, row, V, w, scale, k, grouped);
                cut = sm.cut;
                __syncthreads();
                from_top();
                if (splits) fill(true);
            } else {
                find_bin<T, kCount>(sm, k, -1);
                find_place<DT, T, kCount>(sm, row, V, w, scale, k, grouped);
                cut = sm.cut;
            }
        }
        if (mass && !done) {
            if (s.k == 0) find_bin<T, kCountMass>(sm, 0xffffffffu, -1);  // (none reaches it) the mass of everything
            if (tid == 0) sm.target = mass_target(s.p, s.k > 0 ? sm.mass : sm.total_mass);
            __syncthreads();
            find_bin<T, kMass>(sm, 0, -1);
            find_place<DT, T, kMass>(sm, row, V, w, scale, 0, grouped);
            cut = max(cut, sm.cut);
        }
    }
    if (s.m > 0.0f) cut = max(cut, place_of(sm.row.min_p_key, -1));
    __syncthreads();
    return cut;
}

// The row with -inf below the cut.
template <int DT, int T>
__device__ __forceinline__ void write_cut(const Shared &sm, const char *row, uint4 *dst, int V, uint64_t cut) {
    constexpr int kPer = Elem<DT>::kPerVec, FLIGHT = kFlight<DT>;
    const uint32_t ckey = static_cast<uint32_t>(cut >> 32), cidx = ~static_cast<uint32_t>(cut);
    const uint32_t low = V <= kAnyGroups * 32 * kPer ? ckey : 0;  // (0: all groups)
    constexpr uint32_t kNone = Elem<DT>::kNegInfWord;
    const int vecs = V / kPer;
    for (int v0 = threadIdx.x; v0 < vecs; v0 += T * FLIGHT) {
        uint4 q[FLIGHT];
        bool in[FLIGHT];
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int v = v0 + u * T;
            q[u] = make_uint4(kNone, kNone, kNone, kNone);
            in[u] = v < vecs && (low == 0 || sm.group_max[v >> 5] >= low);
            if (in[u]) q[u] = reinterpret_cast<const uint4 *>(row)[v];
        }
#pragma unroll
        for (int u = 0; u < FLIGHT; ++u) {
            const int v = v0 + u * T;
            if (v >= vecs) break;
            if (in[u]) {
                float x[kPer];
                Elem<DT>::unpack(q[u], x);
                uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const uint32_t key = key_of(x[i]);
                    const bool keep = cut == 0 || key > ckey || (key == ckey && static_cast<uint32_t>(v * kPer + i) <= cidx);
                    if (keep) continue;
                    if (DT == SPEC_F32) w[i % 4] = 0xff800000u;
                    else w[i / 2 % 4] = i & 1 ? (w[i / 2 % 4] & 0xffffu) | 0xff800000u : (w[i / 2 % 4] & 0xffff0000u) | 0xff80u;
                }
                q[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            dst[v] = q[u];
        }
    }
}

template <int DT>
__device__ __forceinline__ void fill_nan(uint4 *dst, int64_t vecs, int64_t first, int64_t step) {
    constexpr uint32_t kNan = DT == SPEC_BF16 ? 0x7fc07fc0u : 0x7fc00000u;
    for (int64_t v = first; v < vecs; v += step) dst[v] = make_uint4(kNan, kNan, kNan, kNan);
}

// Rows of any kind, a CTA per row: neighbouring rows at a time, whatever each takes.
// A row that fits stays in shared memory from the first pass on (`held`).
template <int DT, int T>
__global__ void __launch_bounds__(T, 1024 / T)
    truncate_kernel(const char *logits, char *out, Rows rw, Truncate tr, int V, bool held) {
    extern __shared__ __align__(16) char smem[];
    Shared &sm = *reinterpret_cast<Shared *>(smem);
    char *hold = smem + (sizeof(Shared) + 15) / 16 * 16;
    const int tid = threadIdx.x;
    const int64_t row_bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    const int vecs = V / Elem<DT>::kPerVec;
    fill_table(sm.table);
    const int64_t r = blockIdx.x;
    const bool rows_ok = check_rows(rw, r, &sm.seq);
    specv::grid_dependency_wait();  // behind the processing: its rows are there from here on
    if (!rows_ok) {
        fill_nan<DT>(reinterpret_cast<uint4 *>(out), static_cast<int64_t>(rw.R) * vecs, r * T + tid,
                     static_cast<int64_t>(gridDim.x) * T);
        return;
    }
    const int b = sm.seq;
    if (b < 0) return;  // behind the last sequence's rows
    const char *row = logits + r * row_bytes;
    uint4 *dst = reinterpret_cast<uint4 *>(out + r * row_bytes);
    const Settings s = load_settings(tr, b, V);
    if (!s.valid) {
        fill_nan<DT>(dst, vecs, tid, T);
        return;
    }
    const uint64_t cut = s.active ? cut_of_row<DT, T>(sm, row, V, s, held ? hold : nullptr) : 0;
    if (s.active && held) row = hold;
    if (cut != 0 || logits != out) write_cut<DT, T>(sm, row, dst, V, cut);
}

// ------------------------------------------------------------ bf16, in two passes
// bf16 rows have few values, so a histogram with one bin per value settles
// everything: counts are exact, and a weight is computed once per value
// instead of once per token.  A bin per value of magnitude 2^-32 .. 2^16, 6144
// a side, 48 KB; zeros have a counter of their own.  Values at or below -2^16
// (masked logits) have no weight and are not counted.  Rows with other values
// outside the bins, with NaN or +inf, or whose border is not in the bins, take
// cut_of_row: 3200 rows of 128256 then cost 2150 us with top-p (480 by the bins), 1310
// where top-k asks for more tokens than a mask of the type's lowest value left (325 us
// with -inf), one row 131 (22) and 81 us: such rows are rare, their path is small.
constexpr int kTiny = (127 - 32) << 7;   // magnitude bits of 2^-32
constexpr int kHuge = (127 + 16) << 7;   // of 2^16
constexpr int kSide = kHuge - kTiny;     // values a side
// The order: positive values falling, zero, negative values falling, in
// segments of 128 places (an octave), 4 a lane.
constexpr int kSegPlaces = 128;
constexpr int kSideSegs = kSide / kSegPlaces;
constexpr int kSegs = 2 * kSideSegs + 1;
constexpr int kSegsPerLane = (kSegs + 31) / 32;
constexpr int kPlaces = kSegs * kSegPlaces;
constexpr int kGroupCols = 256;           // a warp's 32 vectors
constexpr int kMaxGroups = 1024;
constexpr int kMaxFastV = kGroupCols * kMaxGroups;
constexpr int kAhead = 4;  // vectors in flight per thread, beside the ones at work

struct FastShared {
    alignas(16) uint32_t hist[2 * kSide];  // bin: magnitude - kTiny, + kSide if negative
    uint32_t zeros;
    // of each segment, then (by the warp that finds the border) of it and those before
    uint32_t seg_count[32 * kSegsPerLane];
    alignas(16) Mass seg_mass[32 * kSegsPerLane];
    uint16_t group_max[kMaxGroups];  // order key of each group's largest value
    int first;                       // the largest value's place
    // the border: tokens above its value stay, `take` of its ties do
    int place, take, ties;
    int cut_group, cut_index;
    bool elsewhere;  // not in the bins

    // how often each group holds the border value: written once the bins are done with
    __device__ uint16_t *group_ties() { return reinterpret_cast<uint16_t *>(hist); }
    // the tokens at a lane's 4 places of a segment
    __device__ __forceinline__ void counts(int seg, uint32_t (&n)[4]) const {
        const int lane = threadIdx.x & 31;
        if (seg == kSideSegs) {
            n[0] = lane == 0 ? zeros : 0;
            n[1] = n[2] = n[3] = 0;
            return;
        }
        const bool up = seg < kSideSegs;  // positive values lie in rising order
        const int at = up ? kSide - 4 - (seg * kSegPlaces + lane * 4) : kSide + (seg - kSideSegs - 1) * kSegPlaces + lane * 4;
        const uint4 q = *reinterpret_cast<const uint4 *>(hist + at);
        n[0] = up ? q.w : q.x;
        n[1] = up ? q.z : q.y;
        n[2] = up ? q.y : q.z;
        n[3] = up ? q.x : q.w;
    }
};

struct BothShared {
    union {
        Shared any;
        FastShared fast;
    };
    // apart from the union: both paths'
    float2 table[64];
    RowConstants row;
    int seq;
    // in a cluster, CTA 0's: what the CTAs' shares of a row hold, what it found, each CTA's ties
    uint32_t odd;
    int place, take, ties;
    bool slow;
    uint32_t rank_ties[8];
};

// The cluster's barrier, this CTA's number in it, another CTA's copy of a shared object.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
template <typename X>
__device__ __forceinline__ X *cluster_map(X *p, uint32_t rank) {
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(p), "r"(rank));
    return reinterpret_cast<X *>(a);
}

__device__ __forceinline__ float place_value(int place) {
    const int neg = place - (kSideSegs + 1) * kSegPlaces;
    const uint32_t u = place < kSide ? kHuge - 1 - place : neg < 0 ? 0 : 0x8000 | (neg + kTiny);
    return __uint_as_float(u << 16);
}
// Unsigned 16-bit key in the order of the values (-0 below +0).
__device__ __forceinline__ uint32_t key16(uint32_t u) { return u ^ (u & 0x8000u ? 0xffffu : 0x8000u); }

// t tokens' weight in units of 2^-100: no bit of a weight above 2^-52 is lost, and
// 2^18 of the largest fit.  (In 64 bits the values' sums are rounded at 2^-46 at 128256
// columns: thousands of small values around zero, a token each, lose the same way,
// 2^-33 of the largest weight together.)
struct TokenWeight {
    uint64_t mantissa;
    int up;
    __device__ __forceinline__ TokenWeight(const Weights &w, float z) {
        int e;
        mantissa = weight_mantissa(w, z, &e);
        up = e + 100;  // -68 .. 52
        if (up < 0) {
            mantissa = up > -64 ? mantissa >> -up : 0;
            up = 0;
        }
    }
    __device__ __forceinline__ Mass times(uint32_t t) const {
        const uint64_t lo = mantissa * t, hi = __umul64hi(mantissa, t);
        return static_cast<Mass>(hi << up | lo >> 1 >> (63 - up)) << 64 | lo << up;
    }
};

// The sum over the lanes of masses below 2^120: 27 bits at a time, so that 32 of them fit 32 bits.
__device__ __forceinline__ Mass warp_sum(Mass m) {
    Mass sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        sum += static_cast<Mass>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(m >> (27 * i)) & 0x7ffffffu)) << (27 * i);
    return sum;
}

// 0xffff in the halves of a that are greater than (or equal to) b's
__device__ __forceinline__ uint32_t above_mask(uint32_t a, uint32_t b, bool equal) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&a), y = *reinterpret_cast<const __nv_bfloat162 *>(&b);
    return equal ? __hge2_mask(x, y) : __hgt2_mask(x, y);
}
__device__ __forceinline__ uint32_t equal_mask(uint32_t a, uint32_t b) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&a), y = *reinterpret_cast<const __nv_bfloat162 *>(&b);
    return __heq2_mask(x, y);
}
__device__ __forceinline__ uint32_t below_mask(uint32_t a, uint32_t b) {  // or equal
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&a), y = *reinterpret_cast<const __nv_bfloat162 *>(&b);
    return __hle2_mask(x, y);
}

// What a row holds beside the values of the bins and -inf.
enum { kOdd = 1, kFiniteLow = 2 };

// A vector with values outside the bins.
__device__ __noinline__ uint32_t count_rare(FastShared &sm, uint4 q) {
    uint32_t odd = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = q.x & 0xffffu, m = u & 0x7fffu;
        if (m - kTiny < static_cast<uint32_t>(kSide)) atomicAdd(&sm.hist[m - kTiny + (u >> 15) * kSide], 1u);
        else if (m == 0) atomicAdd(&sm.zeros, 1u);
        else if (u < (0x8000u | kHuge) || u > 0xff80u) odd |= kOdd;
        else if (u != 0xff80u) odd |= kFiniteLow;
        q.x >>= 16;
        if (i & 1) q.x = q.y, q.y = q.z, q.z = q.w;
    }
    return odd;
}

// A vector's 8 values into the histogram.
__device__ __forceinline__ void count_values(FastShared &sm, const uint4 &q, uint32_t *odd) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t t[4], outside = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // both halves at once; a half below kTiny borrows from its neighbour, and is seen to be outside itself
        t[i] = (w[i] & 0x7fff7fffu) - kTiny * 0x10001u;
        outside |= t[i] | (t[i] + (0x8000 - kSide) * 0x10001u);
    }
    if ((outside & 0x80008000u) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // bins as byte offsets
            static_assert(8 * kSide < 1 << 16, "a byte offset in 16 bits");
            const uint32_t c = t[i] * 4 + ((w[i] >> 15) & 0x10001u) * (4 * kSide);
            atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(sm.hist) + (c & 0xffffu)), 1u);
            atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(sm.hist) + (c >> 16)), 1u);
        }
        return;
    }
    // values at or below -2^16, as masks leave them, are passed over
    uint32_t low[4], none = ~0u, finite = 0;
    outside = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        low[i] = below_mask(w[i], (0x8000u | kHuge) * 0x10001u);
        outside |= (t[i] | (t[i] + (0x8000 - kSide) * 0x10001u)) & ~low[i];
        none &= low[i];
        finite |= low[i] & ~equal_mask(w[i], 0xff80ff80u);
    }
    if (finite) *odd |= kFiniteLow;
    if (none == ~0u) return;
    if (outside & 0x80008000u) {
        *odd |= count_rare(sm, q);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (without the halves passed over, whose offsets would carry into their neighbours)
        const uint32_t c = (t[i] & ~low[i]) * 4 + ((w[i] >> 15) & 0x10001u) * (4 * kSide);
        if (!(low[i] & 0xffffu)) atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(sm.hist) + (c & 0xffffu)), 1u);
        if (!(low[i] >> 16)) atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(sm.hist) + (c >> 16)), 1u);
    }
}

// Inclusive sums over the lanes of a count and, if wanted, a mass.
template <bool MASS>
__device__ __forceinline__ void warp_scan(uint32_t &c, Mass &m) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t cc = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += cc;
        if (MASS) {
            const Mass mm = shfl_up(m, off);
            if (lane >= off) m += mm;
        }
    }
}

// The segments' sums into running sums, by one warp.
template <bool MASS>
__device__ __forceinline__ void scan_segments(FastShared &sm) {
    const int s0 = (threadIdx.x & 31) * kSegsPerLane;
    uint32_t n[kSegsPerLane], c = 0;
    Mass nm[kSegsPerLane], m = 0;
#pragma unroll
    for (int i = 0; i < kSegsPerLane; ++i) {
        n[i] = sm.seg_count[s0 + i];
        nm[i] = MASS ? sm.seg_mass[s0 + i] : 0;
        c += n[i];
        m += nm[i];
    }
    const uint32_t own_c = c;
    const Mass own_m = m;
    warp_scan<MASS>(c, m);
    c -= own_c;
    m -= own_m;
#pragma unroll
    for (int i = 0; i < kSegsPerLane; ++i) {
        sm.seg_count[s0 + i] = c += n[i];
        if (MASS) sm.seg_mass[s0 + i] = m += nm[i];
    }
    __syncwarp();
}

// A place in the order: what lies above it, and the tokens there.
struct Border {
    int place;
    uint32_t above_count, n;
    Mass above_mass;
};

// Where the search ends in the histogram, by one warp, from the running
// sums; place -1 if the bins end before.  (Shared-memory round trips are what
// this costs beside another CTA's histogram, so it makes few.)
template <Search S>
__device__ __forceinline__ Border locate(const FastShared &sm, const Weights &w, uint32_t need, Mass target) {
    constexpr bool mass = S != kCount;
    const int lane = threadIdx.x & 31, s0 = lane * kSegsPerLane;
    uint32_t c = lane ? sm.seg_count[s0 - 1] : 0;
    Mass m = mass && lane ? sm.seg_mass[s0 - 1] : 0;
    int seg = -1;
#pragma unroll
    for (int i = 0; i < kSegsPerLane; ++i) {
        const uint32_t c1 = sm.seg_count[s0 + i];
        const Mass m1 = mass ? sm.seg_mass[s0 + i] : 0;
        if (seg < 0) {
            if (reached<S>(need, target, c1, m1)) {
                seg = s0 + i;
            } else {
                c = c1;
                m = m1;
            }
        }
    }
    uint32_t hit = __ballot_sync(0xffffffffu, seg >= 0);
    if (!hit) return Border{-1, 0, 0, 0};
    int at = __ffs(hit) - 1;
    seg = __shfl_sync(0xffffffffu, seg, at);
    c = __shfl_sync(0xffffffffu, c, at);
    if (mass) m = shfl(m, at);
    uint32_t n[4];
    Mass nm[4];
    sm.counts(seg, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) nm[i] = mass ? TokenWeight(w, place_value(seg * kSegPlaces + lane * 4 + i)).times(n[i]) : 0;
    uint32_t cs = n[0] + n[1] + n[2] + n[3];
    Mass ms = nm[0] + nm[1] + nm[2] + nm[3];
    const uint32_t own_c = cs;
    const Mass own_m = ms;
    warp_scan<mass>(cs, ms);
    cs += c;
    ms += m;
    at = __ffs(__ballot_sync(0xffffffffu, reached<S>(need, target, cs, ms))) - 1;
    cs -= own_c;
    ms -= own_m;
    int place = seg * kSegPlaces + lane * 4;
    uint32_t here = n[0];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (place != seg * kSegPlaces + lane * 4 + i || reached<S>(need, target, cs + n[i], ms + nm[i])) continue;
        cs += n[i];
        ms += nm[i];
        here = n[i + 1];
        ++place;
    }
    return Border{__shfl_sync(0xffffffffu, place, at), __shfl_sync(0xffffffffu, cs, at), __shfl_sync(0xffffffffu, here, at),
                  mass ? shfl(ms, at) : 0};
}

// The fewest of n ties whose weight reaches the target, by one warp.
__device__ __forceinline__ uint32_t ties_for(const TokenWeight &w, uint32_t n, Mass above, Mass target) {
    uint32_t lo = 1, hi = n;  // the answer lies in [lo, hi]
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32;
        const uint32_t t = min(lo + step * (threadIdx.x & 31), hi);
        const uint32_t hit = __ballot_sync(0xffffffffu, above + w.times(t) >= target);
        if (!hit) {
            lo = min(lo + step * 31, hi) + 1;  // (hi reaches it)
            continue;
        }
        const int at = __ffs(hit) - 1;
        hi = min(lo + step * at, hi);
        if (at > 0) lo = min(lo + step * (at - 1) + 1, hi);
        else break;
    }
    return hi;
}

// Order key of a vector's largest value.
__device__ __forceinline__ uint32_t max_key(const uint4 &q) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&q);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return key16(__bfloat16_as_ushort(__hmax(__low2bfloat16(m), __high2bfloat16(m))));
}

// One row per CTA: a pass that builds the histogram and the groups' largest
// values (13 of a row's 28 us at two CTAs per SM), the segments' sums and weights
// (3 us), the border by one warp (4 us), its ties (2 us), and the row out (5 us),
// which reads again only the groups that hold a kept token.  3267 rows of 128256:
// 340 us, 4.9 TB/s of the 256.5 KB in and out per row, 73 % of the copy rate, DRAM
// traffic 1.0 x.  One shared-memory atomic per token (2.4 cycles with its bank
// conflicts) and about 18 instructions per 32 tokens bound it with the border's
// latency; three CTAs of 384 threads or four of 256 measured the same, evenly
// spaced runs of rows per CTA 20 % slower (neighbouring rows share address
// translations), the hardware's scheduling of a CTA per row 7 % faster than a
// fixed share each.
// CL CTAs of a cluster share a row, each a run of its groups: CTA 0 adds up the
// histograms and finds the border for all.  One row: 25 us alone, 18 by eight.
template <int CL>
__global__ void __launch_bounds__(kThreads, kPerSm)
    truncate_bf16_kernel(const char *logits, char *out, Rows rw, Truncate tr, int V) {
    extern __shared__ __align__(16) char smem[];
    BothShared &all = *reinterpret_cast<BothShared *>(smem);
    FastShared &sm = all.fast;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row_bytes = static_cast<int64_t>(V) * 2;
    const int vecs = V / 8, groups = (vecs + 31) / 32;
    // this CTA's groups, and CTA 0's shared memory
    const int rank = CL > 1 ? static_cast<int>(cluster_rank()) : 0, part = (groups + CL - 1) / CL;
    const int gb = min(groups, rank * part), ge = min(groups, gb + part), vb = gb * 32, ve = min(vecs, ge * 32);
    BothShared &lead = CL > 1 ? *cluster_map(&all, 0) : all;
    fill_table(all.table);
    const int64_t r = blockIdx.x / CL;
    if (tid == 0) all.odd = 0;
    const bool rows_ok = check_rows(rw, r, &all.seq);
    specv::grid_dependency_wait();  // behind the processing: its rows are there from here on
    if (!rows_ok) {
        fill_nan<SPEC_BF16>(reinterpret_cast<uint4 *>(out), static_cast<int64_t>(rw.R) * vecs,
                            static_cast<int64_t>(blockIdx.x) * kThreads + tid, static_cast<int64_t>(gridDim.x) * kThreads);
        return;
    }
    const int b = all.seq;
    if (b < 0) return;  // behind the last sequence's rows
    const uint4 *row = reinterpret_cast<const uint4 *>(logits + r * row_bytes);
    uint4 *dst = reinterpret_cast<uint4 *>(out + r * row_bytes);
    const Settings s = load_settings(tr, b, V);
    if (!s.valid) {
        fill_nan<SPEC_BF16>(dst, ve, vb + tid, kThreads);
        return;
    }
    if (!s.active) {
        if (logits != out)
            for (int v = vb + tid; v < ve; v += kThreads) dst[v] = row[v];
        return;
    }
    const bool mass = s.p < 1.0f, counted = mass || s.k > 0;
    // --- one pass over the row: the histogram, the groups' largest values
    __syncthreads();  // the last row is done with the shared arrays
    for (int i = tid; i < 2 * kSide / 4; i += kThreads) reinterpret_cast<uint4 *>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
    if (tid < 32 * kSegsPerLane - kSegs) {
        sm.seg_count[kSegs + tid] = 0;
        sm.seg_mass[kSegs + tid] = 0;
    }
    if (tid == kThreads - 1) set_scale(all.row, s);
    if (tid == 0) {
        sm.zeros = 0;
        sm.first = kPlaces;
        sm.elsewhere = false;
    }
    __syncthreads();
    uint32_t odd = 0;
    {
        uint4 q[kAhead], next[kAhead];
        auto load = [&](uint4 (&to)[kAhead], int g0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int v = (g0 + u * kWarps) * 32 + lane;
                to[u] = v < ve ? row[v] : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
            }
        };
        load(q, gb + warp);
        for (int g0 = gb + warp; g0 < ge; g0 += kWarps * kAhead) {
            load(next, g0 + kWarps * kAhead);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (g0 + u * kWarps >= ge) break;
                count_values(sm, q[u], &odd);
                const uint32_t key = __reduce_max_sync(0xffffffffu, max_key(q[u]));
                if (lane == 0) sm.group_max[g0 + u * kWarps - gb] = static_cast<uint16_t>(key);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) q[u] = next[u];
        }
    }
    const uint32_t odd_all = (__syncthreads_or(odd & kOdd) ? kOdd : 0) | (__syncthreads_or(odd & kFiniteLow) ? kFiniteLow : 0);
    bool slow = (odd_all & kOdd) != 0;
    if (CL > 1) {
        cluster_sync();  // CTA 0's sums are there to be added to
        if (tid == 0 && odd_all) atomicOr(&lead.odd, odd_all);
        if (rank > 0) {
            for (int i = tid; i < 2 * kSide; i += kThreads)
                if (const uint32_t n = sm.hist[i]) atomicAdd(&lead.fast.hist[i], n);
            if (tid == 0 && sm.zeros) atomicAdd(&lead.fast.zeros, sm.zeros);
        }
        cluster_sync();
        slow = (lead.odd & kOdd) != 0;
    }
    const bool finite_low = ((CL > 1 ? all.odd : odd_all) & kFiniteLow) != 0;  // (CTA 0's is meant)
    float zmax = 0.0f;
    if (!slow && rank == 0) {
        // --- the bins' sums by segments
        int first = kPlaces;
        for (int g = warp; g < kSegs; g += kWarps) {
            uint32_t n[4];
            sm.counts(g, n);
            const uint32_t own = n[0] + n[1] + n[2] + n[3];
            const uint32_t any = __ballot_sync(0xffffffffu, own > 0);
            uint32_t sum = 0;
            if (any) {
                if (first == kPlaces) {
                    const int i = n[0] ? 0 : n[1] ? 1 : n[2] ? 2 : 3, at = __ffs(any) - 1;
                    first = g * kSegPlaces + at * 4 + __shfl_sync(0xffffffffu, i, at);
                }
                sum = __reduce_add_sync(0xffffffffu, own);
            }
            if (lane == 0) sm.seg_count[g] = sum;
        }
        if (lane == 0) atomicMin(&sm.first, first);
        __syncthreads();
        first = sm.first;
        slow = first == kPlaces;
        if (!slow) zmax = place_value(first);
    }
    // (values at or below -2^16 have no weight, and min-p excludes them)
    if (rank == 0 && !slow && !((-65536.0f - zmax) * specv::temp_scale(s.T) < -150.0f)) slow = true;
    Weights w{};
    if (!slow && rank == 0) {
        w = row_weights(all.row, zmax, V, all.table);
        if (mass) {
            for (int g = warp; g < kSegs; g += kWarps) {
                Mass m = 0;
                if (sm.seg_count[g]) {
                    uint32_t n[4];
                    sm.counts(g, n);
#pragma unroll
                    for (int i = 0; i < 4; ++i) m += TokenWeight(w, place_value(g * kSegPlaces + lane * 4 + i)).times(n[i]);
                    m = warp_sum(m);
                }
                if (lane == 0) sm.seg_mass[g] = m;
            }
            __syncthreads();
        }
        // --- the border, by one warp
        if (warp == 0 && counted) {
            Border k{kPlaces, 0, 0, 0};
            uint32_t take = 0;
            Mass Z = 0;
            if (mass) {
                scan_segments<true>(sm);
                Z = sm.seg_mass[kSegs - 1];
            } else {
                scan_segments<false>(sm);
            }
            if (s.k > 0) {
                const uint32_t need = s.k;
                k = mass ? locate<kCountMass>(sm, w, need, 0) : locate<kCount>(sm, w, need, 0);
                if (k.place >= 0) {
                    take = need - k.above_count;
                    if (mass) Z = k.above_mass + TokenWeight(w, place_value(k.place)).times(take);
                } else if (!finite_low) {
                    k = Border{kPlaces, 0, 0, 0};  // fewer than k tokens are not -inf: all of them
                }
            }
            if (mass && k.place >= 0) {
                const Mass target = mass_target(s.p, Z);
                const Border p = locate<kMass>(sm, w, 0, target);
                if (p.place >= 0) {
                    const uint32_t t = ties_for(TokenWeight(w, place_value(p.place)), p.n, p.above_mass, target);
                    take = p.place < k.place ? t : min(t, take);
                }
                k = p;
            }
            if (lane == 0) {
                sm.elsewhere = k.place < 0;
                sm.place = k.place;
                sm.take = static_cast<int>(take);
                sm.ties = static_cast<int>(k.n);
            }
        } else if (tid == 32 && s.m > 0.0f) {
            all.row.min_p_key = min_p_key(zmax, s.T, s.m);
        }
        __syncthreads();
        slow = sm.elsewhere;
    }
    if (CL > 1) {
        __syncthreads();  // every thread of CTA 0 has read `odd`
        if (rank == 0 && tid == 0) {
            all.place = sm.place;
            all.take = sm.take;
            all.ties = sm.ties;
            all.slow = slow;
        }
        cluster_sync();
        slow = lead.slow;
    }
    if (slow) {
        if (CL > 1) cluster_sync();  // CTA 0's shared memory has been read
        if (rank > 0) return;
        __syncthreads();
        if (tid < 64) all.any.table[tid] = all.table[tid];
        __syncthreads();
        const uint64_t cut = cut_of_row<SPEC_BF16, kThreads>(all.any, reinterpret_cast<const char *>(row), V, s, nullptr);
        if (cut != 0 || logits != out) write_cut<SPEC_BF16, kThreads>(all.any, reinterpret_cast<const char *>(row), dst, V, cut);
        return;
    }
    // --- the border value: the lowest one kept, and how its ties go
    uint32_t border = 0xff80u;  // -inf: everything
    bool split = false;
    if (counted) {
        const int place = CL > 1 ? lead.place : sm.place;
        if (place < kPlaces) border = __float_as_uint(place_value(place)) >> 16;
        split = CL > 1 ? lead.take < lead.ties : sm.take < sm.ties;
    }
    if (s.m > 0.0f) {
        // the lowest bf16 value at or above min-p's border
        const float f = value_of(lead.row.min_p_key);
        uint32_t h = __bfloat16_as_ushort(__float2bfloat16_ru(f));
        if ((h & 0x7fffu) == 0) h = 0;
        if (!counted || __uint_as_float(h << 16) > __uint_as_float(border << 16)) {
            border = h;
            split = false;
        }
    }
    const uint32_t pair = border | border << 16;
    // groups below the border (as keys; a zero border takes -0 too)
    const uint32_t low = key16(border == 0 ? 0x8000u : border);
    int cut_group = ge, cut_index = -1;
    if (split) {
        int take = CL > 1 ? lead.take : sm.take;
        for (int g0 = gb + warp; g0 < ge; g0 += kWarps * kAhead) {
            uint4 q[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int g = g0 + u * kWarps, v = g * 32 + lane;
                q[u] = make_uint4(~pair, ~pair, ~pair, ~pair);
                if (g < ge && sm.group_max[g - gb] >= low && v < ve) q[u] = row[v];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int g = g0 + u * kWarps;
                if (g >= ge) break;
                uint32_t n = __popc(equal_mask(q[u].x, pair)) + __popc(equal_mask(q[u].y, pair)) +
                             __popc(equal_mask(q[u].z, pair)) + __popc(equal_mask(q[u].w, pair));
                n = __reduce_add_sync(0xffffffffu, n >> 4);
                if (lane == 0) sm.group_ties()[g - gb] = static_cast<uint16_t>(n);
            }
        }
        __syncthreads();
        // a warp's running sums of the groups' ties
        constexpr int kRun = kMaxGroups / 32;
        uint32_t n = 0, c = 0;
        const int g0 = lane * kRun, g1 = min(ge - gb, g0 + kRun);
        if (warp == 0) {
            for (int g = g0; g < g1; ++g) n += sm.group_ties()[g];
            c = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t cc = __shfl_up_sync(0xffffffffu, c, off);
                if (lane >= off) c += cc;
            }
        }
        bool here = true;  // the ties run out in this CTA's groups
        if (CL > 1) {
            if (tid == 31) lead.rank_ties[rank] = c;
            cluster_sync();
            for (int i = 0; i < rank; ++i) take -= lead.rank_ties[i];
            here = take > 0 && take < static_cast<int>(lead.rank_ties[rank]);
            if (take <= 0) cut_group = gb;
        }
        if (here && warp == 0) {
            // the group where they do, then the token
            const int owner = __ffs(__ballot_sync(0xffffffffu, c >= static_cast<uint32_t>(take))) - 1;
            c -= n;
            int g = g0;
            if (lane == owner)
                while (c + sm.group_ties()[g] < static_cast<uint32_t>(take)) c += sm.group_ties()[g++];
            g = __shfl_sync(0xffffffffu, g, owner);
            c = __shfl_sync(0xffffffffu, c, owner);
            const int v = (gb + g) * 32 + lane;
            uint32_t bits = 0;  // a bit per tie of this lane's vector
            if (v < ve) {
                const uint4 q = row[v];
                const uint32_t e[4] = {equal_mask(q.x, pair), equal_mask(q.y, pair), equal_mask(q.z, pair), equal_mask(q.w, pair)};
#pragma unroll
                for (int i = 0; i < 4; ++i) bits |= (e[i] & 1u) << (2 * i) | (e[i] >> 31) << (2 * i + 1);
            }
            uint32_t before = __popc(bits);
            const uint32_t own = before;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t cc = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += cc;
            }
            before += c - own;
            if (before < static_cast<uint32_t>(take) && before + own >= static_cast<uint32_t>(take)) {
                for (int left = take - before; left > 1; --left) bits &= bits - 1;
                sm.cut_group = gb + g;
                sm.cut_index = v * 8 + __ffs(bits) - 1;
            }
        }
        __syncthreads();
        if (here) {
            cut_group = sm.cut_group;
            cut_index = sm.cut_index;
        }
    }
    // --- the row out: groups below the border need not be read again
    for (int g0 = gb + warp; g0 < ge; g0 += kWarps * kAhead) {
        uint4 q[kAhead];
        bool kept[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = g0 + u * kWarps;
            kept[u] = g < ge && sm.group_max[g - gb] >= low;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int v = (g0 + u * kWarps) * 32 + lane;
            q[u] = kept[u] && v < ve ? row[v] : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = g0 + u * kWarps, v = g * 32 + lane;
            if (v >= ve) continue;
            if (kept[u]) {
                uint32_t x[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                const bool equal = g < cut_group;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t keep = above_mask(x[i], pair, equal);
                    if (g == cut_group) {
                        const uint32_t e = equal_mask(x[i], pair);
                        if (v * 8 + 2 * i <= cut_index) keep |= e & 0xffffu;
                        if (v * 8 + 2 * i + 1 <= cut_index) keep |= e & 0xffff0000u;
                    }
                    x[i] = (x[i] & keep) | (0xff80ff80u & ~keep);
                }
                q[u] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            __stcs(dst + v, q[u]);  // (not read again here: 346 -> 340 us at B=512)
        }
    }
    if (CL > 1) cluster_sync();  // CTA 0's shared memory is read until here
}

// `behind`: launched to start while the processing before it on the stream drains
// (it reads the call's inputs, which were there before that, and then waits).
template <typename K, typename... Args>
cudaError_t launch_rows(K kernel, int grid, int threads, size_t smem, int cluster, bool behind, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (behind) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMostHeld = 180 * 1024;  // bytes of a row kept in shared memory
constexpr int kAnyShared = (sizeof(Shared) + 15) / 16 * 16;

template <int DT, int T>
cudaError_t launch_any(const char *in, char *to, const Rows &rw, const Truncate &tr, int V, bool behind, cudaStream_t stream) {
    const int64_t bytes = static_cast<int64_t>(V) * Elem<DT>::kBytes;
    const bool held = DT == SPEC_F32 && bytes <= kMostHeld;
    return launch_rows(truncate_kernel<DT, T>, rw.R, T, kAnyShared + (held ? bytes : 0), 1, behind, stream, in, to, rw, tr, V, held);
}

template <int DT>
int launch_truncate(const void *logits, void *out, const Rows &rw, const Truncate &tr, int V, int sms, bool behind,
                    cudaStream_t stream) {
    const char *in = static_cast<const char *>(logits);
    char *to = static_cast<char *>(out);
    cudaError_t e;
    if (DT == SPEC_BF16 && V <= kMaxFastV) {
        // few rows: clusters of CTAs share them, while every warp has groups of its own
        int cl = 1;
        while (cl < 8 && static_cast<int64_t>(rw.R) * cl * 2 <= static_cast<int64_t>(sms) * kPerSm && V >= cl * 2 * kWarps * kGroupCols) cl *= 2;
        const auto kernel = cl == 8   ? truncate_bf16_kernel<8>
                            : cl == 4 ? truncate_bf16_kernel<4>
                            : cl == 2 ? truncate_bf16_kernel<2>
                                      : truncate_bf16_kernel<1>;
        e = launch_rows(kernel, rw.R * cl, kThreads, sizeof(BothShared), cl, behind, stream, in, to, rw, tr, V);
    } else if constexpr (DT == SPEC_F32) {
        // short rows: small CTAs, several to an SM
        e = V <= 8192    ? launch_any<DT, 256>(in, to, rw, tr, V, behind, stream)
            : V <= 16384 ? launch_any<DT, 512>(in, to, rw, tr, V, behind, stream)
                         : launch_any<DT, 1024>(in, to, rw, tr, V, behind, stream);
    } else {
        e = launch_any<DT, 1024>(in, to, rw, tr, V, behind, stream);  // longer rows than the kernel above takes
    }
    return specv::cuda_ok(e, "launch truncate_kernel") ? SPEC_OK : SPEC_ERR_CUDA;
}

inline int check_truncate_args(const spec_truncate_t *t, const Rows &rw, Truncate *tr) {
    if (!t) return SPEC_ERR_INVALID_ARG;
    *tr = Truncate{t->temperature, t->top_k, t->top_p, t->min_p};
    return rw.B > 0 && rw.R > 0 && !t->temperature ? SPEC_ERR_INVALID_ARG : SPEC_OK;
}

}  // namespace
}  // namespace speclog

namespace specv {
bool set_logits_attrs() {
    const auto bf16 = [](auto kernel) {
        return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(speclog::BothShared)),
                       "cudaFuncSetAttribute(truncate_bf16_kernel)");
    };
    const auto any = [](auto kernel) {
        return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            speclog::kAnyShared + speclog::kMostHeld),
                       "cudaFuncSetAttribute(truncate_kernel)");
    };
    return bf16(speclog::truncate_bf16_kernel<1>) && bf16(speclog::truncate_bf16_kernel<2>) &&
           bf16(speclog::truncate_bf16_kernel<4>) && bf16(speclog::truncate_bf16_kernel<8>) &&
           any(speclog::truncate_kernel<SPEC_F32, 256>) && any(speclog::truncate_kernel<SPEC_F32, 512>) &&
           any(speclog::truncate_kernel<SPEC_F32, 1024>);
}
}  // namespace specv

using namespace speclog;

namespace {
int truncate_call(const void *logits, const spec_rows_t *rows, const spec_truncate_t *truncate, int V, int dtype, void *out,
                  bool behind, void *stream) {
    Rows rw;
    Truncate tr;
    int rc = check_rows_args(logits, rows, V, dtype, out, &rw);
    if (rc == SPEC_OK) rc = check_truncate_args(truncate, rw, &tr);
    if (rc != SPEC_OK || rw.B == 0 || rw.R == 0) return rc;
    int dev;
    specv::DeviceState *st = specv::device_state(&dev);
    if (!st) return SPEC_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_truncate<SPEC_F32>(logits, out, rw, tr, V, st->sms, behind, s)
                             : launch_truncate<SPEC_BF16>(logits, out, rw, tr, V, st->sms, behind, s);
}
}  // namespace

extern "C" {

int spec_logits_truncate(const void *logits, const spec_rows_t *rows, const spec_truncate_t *truncate, int V,
                         int dtype, void *out, void *stream) {
    return truncate_call(logits, rows, truncate, V, dtype, out, false, stream);
}

int spec_logits_process_truncate(const void *logits, const spec_rows_t *rows, const spec_logits_t *process,
                                 const spec_truncate_t *truncate, int V, int dtype, void *out, void *stream) {
    Rows rw;
    Truncate tr;
    int rc = check_rows_args(logits, rows, V, dtype, out, &rw);
    if (rc == SPEC_OK) rc = check_truncate_args(truncate, rw, &tr);
    if (rc == SPEC_OK) rc = spec_logits_process(logits, rows, process, V, dtype, out, stream);
    if (rc != SPEC_OK) return rc;
    return truncate_call(out, rows, truncate, V, dtype, out, true, stream);
}

}  // extern "C"
