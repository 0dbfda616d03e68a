// cache.cu -- a cache of keys and values in 8 bits: the rows that a round kept
// written, positions read back, behind the C ABI of include/spec_verify.h.
//
// A block of 32 elements shares the scale 2^e, e the least integer >= -127
// with max |x| <= 448 * 2^e.  With max |x| = f * 2^p, 1 <= f < 2, and 448 = 1.75 * 2^8,
// e = p - 8 + (f > 1.75): an addition to the float's bits, whose carry out of the
// mantissa is that comparison.  x * 2^-e is exact, so that rounding to e4m3 is the
// only one, and reading back multiplies exactly.
//
// Both ways are bound by memory: a thread takes a block of 32 (64 bytes of bf16 in, 32 out and a byte), so that it needs no
// other thread's values and the arithmetic of addresses is shared by as many as share a scale; half a block per thread came to
// 287 instructions per 16 elements and 218 us for the prompts below.  A CTA takes several rows, for the dependent loads that find
// a row's place (offsets; length; page) to be waited for once.
//
// Times (GB300, events over captured calls): 9676 rows of 8 prompts, 16 layers of 8 heads of 128, 142 us (6.75 TB/s, 101 % of the copy
// rate); what 64 verifies kept, 32 layers, 14 us (7.2 at the copy rate: launch, three dependent loads, one wave); 16 sequences of
// 1000 to 8192 tokens read back, 274 us (101 %); the smallest calls 3.6 us.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "host_common.h"
#include "spec_verify.h"

namespace speccache {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;    // elements that share a scale: a thread's
constexpr int kGranule = 16;  // heads are multiples of it
constexpr int64_t kMaxCtas = 0x7ffffff0;
constexpr int kMaxRows = 128;  // of a CTA

// Division of n < 2^31 by d < 2^31, by a product: floor(n * m / 2^(32 + s)), m = ceil(2^(32 + s) / d), 2^s >= d
// (m < 2^33, its upper bit apart).
struct Divide {
    uint32_t m, d;
    int s;
    __device__ __forceinline__ int operator()(int n) const {
        const uint32_t u = static_cast<uint32_t>(n);
        return static_cast<int>((__umulhi(u, m) + u) >> s);
    }
};
Divide divide_by(int d) {
    Divide r;
    r.d = static_cast<uint32_t>(d);
    r.s = 0;
    while ((int64_t{1} << r.s) < d) ++r.s;
    r.m = static_cast<uint32_t>((((uint64_t{1} << 32) * ((uint64_t{1} << r.s) - r.d)) + r.d - 1) / r.d);
    return r;
}

struct Cache {
    unsigned char *data[2], *scale[2];  // keys, values
    int n;                              // of them: 1 or 2
    bool wide;                          // blocks lie at multiples of 32 bytes
    int L, P, T, D, blocks;             // blocks: of a head
    int row_blocks, row_elements;       // of a position: H * blocks, H * D
    int S, M;
    const int32_t *pages, *lengths;
    // A line is one layer's and tensor's part of a position: row_blocks blocks, in chunks of `width` that a CTA's threads
    // take `abreast` at a time.  Parts of a position: lines * chunks.
    int width, chunks, abreast, parts;
    Divide by_parts, by_chunks, by_blocks, by_width;

    // Where position p of a slot lies: page * T + place in it; -1: nowhere.
    __device__ __forceinline__ int64_t entry(int slot, int64_t p) const {
        if (p >= static_cast<int64_t>(M) * T) return -1;
        if (!pages) return static_cast<int64_t>(slot) * T + p;
        const int page = __ldg(pages + static_cast<int64_t>(slot) * M + p / T);
        return page < 0 || page >= P ? -1 : static_cast<int64_t>(page) * T + p % T;
    }
};

__device__ __forceinline__ float nan32() { return __int_as_float(0x7fffffff); }

// 32 bytes at a time
struct Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ Words8 load32(const void *p) {
    Words8 v;
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                   "=r"(v.w[7])
                 : "l"(p));
    return v;
}
__device__ __forceinline__ Words8 load16(const void *p) {
    Words8 v{};
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
    return v;
}
__device__ __forceinline__ void store16(void *p, const Words8 &v) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]) : "memory");
}
__device__ __forceinline__ void store32(void *p, const Words8 &v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
                 "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
}

// A block of the pool, the upper half of it only if it has one.
__device__ __forceinline__ Words8 load_pool(const Cache &c, const unsigned char *p, bool half) {
    if (c.wide) return load32(p);
    Words8 v = load16(p);
    if (!half) {
        const Words8 u = load16(p + 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) v.w[4 + k] = u.w[k];
    }
    return v;
}
__device__ __forceinline__ void store_pool(const Cache &c, unsigned char *p, const Words8 &v, bool half) {
    if (c.wide) return store32(p, v);
    store16(p, v);
    if (!half) store16(p + 16, Words8{{v.w[4], v.w[5], v.w[6], v.w[7]}});
}

// 32 elements in their type; the upper 16 are 0 where a head ends.
template <int DT>
struct Block;
template <>
struct Block<SPEC_BF16> {
    static constexpr int kBytes = 2;
    Words8 v[2];
    __device__ __forceinline__ void load(const void *p, bool half) {
        v[0] = load32(p);
        v[1] = half ? Words8{} : load32(static_cast<const char *>(p) + 32);
    }
    __device__ __forceinline__ __nv_bfloat162 pair(int i) const { return *reinterpret_cast<const __nv_bfloat162 *>(&v[i / 8].w[i % 8]); }
    // the largest |x|, NaN passed over
    __device__ __forceinline__ float largest() const {
        __nv_bfloat162 m[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) m[j] = __habs2(pair(j));
#pragma unroll
        for (int j = 8; j > 0; j /= 2)
#pragma unroll
            for (int k = 0; k < j; ++k) m[k] = __hmax2(m[k], m[k + j]);
        return fmaxf(__bfloat162float(__hmax(__low2bfloat16(m[0]), __high2bfloat16(m[0]))), 0.0f);
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? __high2float(pair(i / 2)) : __low2float(pair(i / 2)); }
    // pair i times a power of two; exact
    __device__ __forceinline__ float2 scaled(int i, float up) const {
        return __bfloat1622float2(__hmul2(pair(i), __float2bfloat162_rn(up)));
    }
    __device__ __forceinline__ void set2(int i, float a, float b) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
        v[i / 16].w[i % 16 / 2] = *reinterpret_cast<const uint32_t *>(&t);
    }
    __device__ __forceinline__ void store(void *p, bool half) const {
        store32(p, v[0]);
        if (!half) store32(static_cast<char *>(p) + 32, v[1]);
    }
};
template <>
struct Block<SPEC_F32> {
    static constexpr int kBytes = 4;
    Words8 v[4];
    __device__ __forceinline__ void load(const void *p, bool half) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = half && k >= 2 ? Words8{} : load32(static_cast<const char *>(p) + 32 * k);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i / 8].w[i % 8]); }
    __device__ __forceinline__ float largest() const {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < kBlock; ++j) m = fmaxf(m, fabsf(get(j)));
        return m;
    }
    __device__ __forceinline__ float2 scaled(int i, float up) const { return make_float2(get(2 * i) * up, get(2 * i + 1) * up); }
    __device__ __forceinline__ void set2(int i, float a, float b) {
        v[i / 8].w[i % 8] = __float_as_uint(a);
        v[i / 8].w[i % 8 + 1] = __float_as_uint(b);
    }
    __device__ __forceinline__ void store(void *p, bool half) const {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!half || k < 2) store32(static_cast<char *>(p) + 32 * k, v[k]);
    }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// ------------------------------------------------------------------- writing
struct Write {
    Cache c;
    const char *in[2];
    int64_t layer_stride, row_stride;  // bytes
    int mode, B, R;
    const int32_t *offsets, *parent, *num_accepted, *last_node, *slots;
    int32_t *out_lengths;
};

// How many rows of sequence b, which has the tokens (or nodes, or rows) o .. e - 1, are kept, and the slot they go to;
// 0: it is skipped.
__device__ __forceinline__ int kept_rows(const Write &w, int b, int64_t o, int64_t e, int *slot) {
    *slot = w.slots ? __ldg(w.slots + b) : b;
    const int n = w.num_accepted ? __ldg(w.num_accepted + b) : 0;
    if (*slot < 0 || *slot >= w.c.S) return 0;
    if (w.mode == SPEC_ROWS_NEXT) return 1;
    if (w.mode == SPEC_ROWS_PROMPT) return static_cast<int>(e - o);
    return n < 0 || n >= e - o + (w.mode == SPEC_ROWS_TARGET ? 1 : 0) ? 0 : n + 1;
}

// The rows of a CTA, as they are found: the sequence (-1: none), which of its rows it is, how many of them are kept,
// the slot.
struct Found {
    int seq[kMaxRows], at[kMaxRows], kept[kMaxRows], slot[kMaxRows];
};

// Whether the offsets are valid; the rows r0 .. r0 + rows - 1 into *f.  The whole block.
__device__ __forceinline__ bool find_rows(const Write &w, int r0, int rows, Found *f) {
    const int tid = threadIdx.x;
    if (w.mode == SPEC_ROWS_NEXT) {
        if (tid < rows) {
            const int r = r0 + tid;
            f->seq[tid] = r < w.B ? r : -1, f->at[tid] = 0;
            f->kept[tid] = r < w.B ? kept_rows(w, r, 0, 0, &f->slot[tid]) : 0;
        }
        __syncthreads();
        return w.B <= w.R;
    }
    if (tid < rows) f->seq[tid] = -1;
    __syncthreads();
    const int lo = w.mode == SPEC_ROWS_TREE ? 1 : 0;
    const int hi = w.mode == SPEC_ROWS_TREE ? SPEC_MAX_TREE_NODES : w.mode == SPEC_ROWS_TARGET ? SPEC_MAX_K : 0x7fffffff;
    const int one = w.mode == SPEC_ROWS_TARGET ? 1 : 0;
    bool bad = __ldg(w.offsets) != 0;
    for (int b = tid; b < w.B; b += kThreads) {
        const int64_t o = __ldg(w.offsets + b), e = __ldg(w.offsets + b + 1);
        int slot;
        const int kept = kept_rows(w, b, o, e, &slot);  // (fetched with the offsets, whether they are wanted or not)
        bad |= e - o < lo || e - o > hi;
        const int64_t first = o + one * b, end = min(e + one * (b + 1), int64_t{r0} + rows);
        for (int64_t r = max(first, int64_t{r0}); r < end; ++r) {
            const int k = static_cast<int>(r - r0);
            f->seq[k] = b, f->at[k] = static_cast<int>(r - first), f->kept[k] = kept, f->slot[k] = slot;
        }
    }
    bad |= static_cast<int64_t>(__ldg(w.offsets + w.B)) + one * w.B > w.R;
    return __syncthreads_or(bad) == 0;
}

// The place of node r (-1: any) on the path of n nodes from the root o to
// last, or -1; and whether that is a path.
__device__ int place_on_path(const int32_t *parent, int o, int last, int nodes, int n, int r, bool *valid) {
    int node = last, place = -1;
    *valid = false;
    if (last < o || last >= o + nodes) return -1;
    for (int i = n - 1; i > 0; --i) {
        if (node == r) place = i;
        const int up = __ldg(parent + node);
        if (up < o || up >= node) return -1;
        node = up;
    }
    if (node == r) place = 0;
    *valid = node == o;
    return node == o ? place : -1;
}

// out_lengths, by one CTA (in place: after the rows are written).
__device__ __noinline__ void write_lengths(const Write &w) {
    const bool valid = find_rows(w, 0, 0, nullptr);
    if (w.out_lengths != w.c.lengths)
        for (int i = threadIdx.x; i < w.c.S; i += kThreads) w.out_lengths[i] = w.c.lengths[i];
    __syncthreads();
    if (!valid) return;
    // a sequence per lane; the pages that a long one needs are looked at by the whole warp
    const int lane = threadIdx.x & 31;
    for (int b0 = threadIdx.x & ~31; b0 < w.B; b0 += kThreads) {
        const int b = b0 + lane;
        int slot = 0, n = 0;
        int64_t length = -1;
        if (b < w.B) {
            const bool any = w.mode != SPEC_ROWS_NEXT;
            n = kept_rows(w, b, any ? __ldg(w.offsets + b) : 0, any ? __ldg(w.offsets + b + 1) : 0, &slot);
            if (n > 0) length = w.c.lengths[slot];
            if (length >= 0 && w.mode == SPEC_ROWS_TREE) {
                const int o = __ldg(w.offsets + b);
                bool is_path;
                place_on_path(w.parent, o, __ldg(w.last_node + b), __ldg(w.offsets + b + 1) - o, n, -1, &is_path);
                if (!is_path) length = -1;
            }
        }
        const int64_t end = length + n;
        bool room = end <= static_cast<int64_t>(w.c.M) * w.c.T && end <= 0x7fffffff;
        const bool look = length >= 0 && room && w.c.pages;
        const int first = look ? static_cast<int>(length / w.c.T) : 0, pages = look ? static_cast<int>((end - 1) / w.c.T) + 1 - first : 0;
        const auto is_page = [&](int64_t at) {
            const int page = __ldg(w.c.pages + at);
            return page >= 0 && page < w.c.P;
        };
        const int64_t at = static_cast<int64_t>(slot) * w.c.M + first;
        constexpr int few = 4;
        if (pages <= few) {
            for (int p = 0; p < pages; ++p) room &= is_page(at + p);
        }
        for (unsigned left = __ballot_sync(0xffffffffu, pages > few); left; left &= left - 1) {
            const int from = __ffs(left) - 1, count = __shfl_sync(0xffffffffu, pages, from);
            const int64_t start = __shfl_sync(0xffffffffu, at, from);
            bool all = true;
            for (int p = lane; p < count; p += 32) all &= is_page(start + p);
            all = __all_sync(0xffffffffu, all);
            if (lane == from) room &= all;
        }
        if (length >= 0) w.out_lengths[slot] = room ? static_cast<int>(end) : -1;
    }
}

// The rows of a CTA that are kept: which they are, and their entries in the pool.
struct Rows {
    int count;
    int warp[kMaxRows / 32];  // kept by each of the first warps
    int row[kMaxRows];
    int64_t entry[kMaxRows];
};
// By the whole block: the row of each of the first threads is kept (or not) at `entry`.
__device__ __forceinline__ void keep_rows(Rows &rows, int row, bool kept, int64_t entry) {
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned all = __ballot_sync(0xffffffffu, kept);
    if (lane == 0 && tid < kMaxRows) rows.warp[tid >> 5] = __popc(all);
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kMaxRows / 32; ++w) {
        if (w < tid >> 5) before += rows.warp[w];
        sum += rows.warp[w];
    }
    if (kept) {
        const int at = before + __popc(all & ((1u << lane) - 1));
        rows.row[at] = row, rows.entry[at] = entry;
    }
    if (tid == 0) rows.count = sum;
    __syncthreads();
}

// A thread's way through the blocks of a CTA's kept rows: a block of one chunk, line and row at a time.
struct Walk {
    int k, part;            // row and part of it
    int step_k, step_part;  // from one to the next
    int in_chunk;           // the thread's block of a chunk; -1: the thread has none
    __device__ __forceinline__ Walk(const Cache &c, int split, int splits) {
        const int first = c.by_width(threadIdx.x);
        in_chunk = first < c.abreast ? static_cast<int>(threadIdx.x) - first * c.width : -1;
        const int start = split * c.abreast + first, step = c.abreast * splits;
        k = c.by_parts(start), part = start - k * c.parts;
        step_k = c.by_parts(step), step_part = step - step_k * c.parts;
    }
    __device__ __forceinline__ void next(const Cache &c) {
        k += step_k, part += step_part;
        if (part >= c.parts) part -= c.parts, ++k;
    }
};

// One block: where it lies.
struct Place {
    bool mine, half;
    int row, tensor, layer, element, block;  // element, block: of a position
    int64_t position;                        // in the pool, of all layers; -1: nowhere
    __device__ __forceinline__ Place(const Cache &c, const Rows &rows, const Walk &w) {
        mine = w.k < rows.count && w.in_chunk >= 0;
        const int k = mine ? w.k : 0, line = c.chunks == 1 ? w.part : c.by_chunks(w.part);
        block = w.in_chunk + (c.chunks == 1 ? 0 : (w.part - line * c.chunks) * c.width);
        mine = mine && block < c.row_blocks;
        const int h = c.by_blocks(block), in_head = block - h * c.blocks;
        element = h * c.D + in_head * kBlock;
        half = in_head * kBlock + kGranule == c.D;
        tensor = c.n == 2 ? line & 1 : 0, layer = c.n == 2 ? line >> 1 : line;
        row = rows.row[k];
        const int64_t entry = rows.entry[k];
        position = entry < 0 ? -1 : static_cast<int64_t>(layer) * c.P * c.T + entry;
    }
    __device__ __forceinline__ unsigned char *data(const Cache &c) const {
        return (tensor ? c.data[1] : c.data[0]) + position * c.row_elements + element;
    }
    __device__ __forceinline__ unsigned char *scale(const Cache &c) const {
        return (tensor ? c.scale[1] : c.scale[0]) + position * c.row_blocks + block;
    }
};

// CTAs splits * k .. of the rows per_cta * k ..; one more at the end for the lengths.
template <int DT>
__global__ void __launch_bounds__(kThreads, 4) write_kernel(const __grid_constant__ Write w, int per_cta, int splits) {
    constexpr int U = DT == SPEC_BF16 ? 2 : 1;  // blocks of a thread under way
    __shared__ Found found;
    __shared__ Rows rows;
    const int k = blockIdx.x / splits;
    const int64_t r64 = static_cast<int64_t>(k) * per_cta;
    if (r64 >= w.R) {
        write_lengths(w);
        return;
    }
    const int r0 = static_cast<int>(r64), tid = threadIdx.x;
    if (!find_rows(w, r0, per_cta, &found)) return;
    const Cache &c = w.c;
    const int b = tid < per_cta ? found.seq[tid] : -1, r = r0 + tid;
    int64_t entry = -1;
    if (b >= 0 && found.kept[tid] > 0) {
        const int n = found.kept[tid], slot = found.slot[tid];
        int i = found.at[tid];
        if (w.mode == SPEC_ROWS_TREE || i < n) {
            const int length = __ldg(c.lengths + slot);
            if (w.mode == SPEC_ROWS_TREE) {
                const int o = __ldg(w.offsets + b);
                bool is_path;
                i = place_on_path(w.parent, o, __ldg(w.last_node + b), __ldg(w.offsets + b + 1) - o, n, r, &is_path);
            }
            if (i >= 0 && length >= 0) entry = c.entry(slot, static_cast<int64_t>(length) + i);
        }
    }
    keep_rows(rows, r, entry >= 0, entry);
    for (Walk at(c, blockIdx.x - k * splits, splits); at.k < rows.count;) {
        Walk from = at;
        Block<DT> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u, at.next(c)) {
            const Place a(c, rows, at);
            if (a.mine)
                x[u].load((a.tensor ? w.in[1] : w.in[0]) + a.layer * w.layer_stride + a.row * w.row_stride + a.element * Block<DT>::kBytes, a.half);
        }
#pragma unroll
        for (int u = 0; u < U; ++u, from.next(c)) {
            const Place a(c, rows, from);
            if (!a.mine) continue;
            float big = x[u].largest();
            const bool infinite = __float_as_uint(big) == 0x7f800000u;
            if (infinite) {
                big = 0.0f;
#pragma unroll
                for (int j = 0; j < kBlock; ++j) {
                    const float y = fabsf(x[u].get(j));
                    if (y < __int_as_float(0x7f800000)) big = fmaxf(big, y);
                }
            }
            const int e = max(0, static_cast<int>((__float_as_uint(big) + 0x1fffffu) >> 23) - 8);  // e + 127
            const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
            Words8 q;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 y = x[u].scaled(2 * j, up), z = x[u].scaled(2 * j + 1, up);
                q.w[j] = e4m3x2(y.x, y.y) | e4m3x2(z.x, z.y) << 16;
            }
            if (infinite) {  // (converted, they are the largest values)
#pragma unroll
                for (int j = 0; j < kBlock; ++j)
                    if (fabsf(x[u].get(j)) == __int_as_float(0x7f800000)) q.w[j / 4] |= 0x7fu << 8 * (j % 4);
            }
            store_pool(c, a.data(c), q, a.half);
            *a.scale(c) = static_cast<unsigned char>(e);
        }
    }
}

__global__ void __launch_bounds__(kThreads) lengths_kernel(const __grid_constant__ Write w) {
    specv::grid_dependency_wait();
    write_lengths(w);
}

// ------------------------------------------------------------------- reading
struct Read {
    Cache c;
    char *out[2];
    int B, R;
    const int32_t *offsets, *first, *slots;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Read w, int per_cta, int splits) {
    constexpr int U = 2;  // blocks of a thread under way
    __shared__ int s_seq[kMaxRows];
    __shared__ Rows rows;
    const int tid = threadIdx.x;
    const int k = blockIdx.x / splits, r0 = k * per_cta;
    if (tid < kMaxRows) s_seq[tid] = -1;
    __syncthreads();
    bool bad = __ldg(w.offsets) != 0 || __ldg(w.offsets + w.B) > w.R;
    for (int b = tid; b < w.B; b += kThreads) {
        const int64_t o = __ldg(w.offsets + b), e = __ldg(w.offsets + b + 1);
        bad |= e < o;
        for (int64_t r = max(o, int64_t{r0}); r < min(e, int64_t{r0} + per_cta); ++r) s_seq[r - r0] = b;
    }
    if (__syncthreads_or(bad)) return;
    const Cache &c = w.c;
    const int b = tid < kMaxRows ? s_seq[tid] : -1, r = r0 + tid;
    int64_t entry = -1;
    if (b >= 0) {
        const int slot = w.slots ? __ldg(w.slots + b) : b;
        const int64_t p = static_cast<int64_t>(r) - __ldg(w.offsets + b) + (w.first ? __ldg(w.first + b) : 0);
        if (slot >= 0 && slot < c.S && p >= 0 && p < __ldg(c.lengths + slot)) entry = c.entry(slot, p);
    }
    keep_rows(rows, r, b >= 0, entry);
    for (Walk at(c, blockIdx.x - k * splits, splits); at.k < rows.count;) {
        Walk from = at;
        Words8 q[U];
        uint32_t e[U];
#pragma unroll
        for (int u = 0; u < U; ++u, at.next(c)) {
            const Place a(c, rows, at);
            if (a.mine && a.position >= 0) {
                q[u] = load_pool(c, a.data(c), a.half);
                e[u] = __ldg(a.scale(c));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u, from.next(c)) {
            const Place a(c, rows, from);
            if (!a.mine) continue;
            // 2^(e - 127); a byte of 255 is not written: NaN
            float scale = e[u] == 0 ? __uint_as_float(0x00400000u) : e[u] == 255 ? nan32() : __uint_as_float(e[u] << 23);
            if (a.position < 0) scale = nan32(), q[u] = Words8{};
            Block<DT> x;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 y = from_e4m3x2(q[u].w[j / 2] >> (j & 1 ? 16 : 0));
                x.set2(2 * j, y.x * scale, y.y * scale);
            }
            x.store((a.tensor ? w.out[1] : w.out[0]) +
                        ((static_cast<int64_t>(a.layer) * w.R + a.row) * c.row_elements + a.element) * Block<DT>::kBytes,
                    a.half);
        }
    }
}

// ---------------------------------------------------------------------- host
bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

int check_cache(const spec_cache_t *in, Cache *c) {
    if (!in) return SPEC_ERR_INVALID_ARG;
    if (in->L < 0 || in->P < 0 || in->T <= 0 || in->H <= 0 || in->D <= 0 || in->S < 0 || in->M < 0) return SPEC_ERR_INVALID_ARG;
    if (in->D % kGranule != 0 || in->D > 1024 || static_cast<int64_t>(in->H) * in->D > 65536) return SPEC_ERR_INVALID_ARG;
    if (!in->pages && in->S != in->P) return SPEC_ERR_INVALID_ARG;
    if (!in->k || !in->k_scale || !in->lengths || !in->v != !in->v_scale) return SPEC_ERR_INVALID_ARG;
    if (!specv::aligned16(in->k) || !specv::aligned16(in->v)) return SPEC_ERR_ALIGNMENT;
    c->data[0] = static_cast<unsigned char *>(in->k), c->data[1] = static_cast<unsigned char *>(in->v);
    c->scale[0] = in->k_scale, c->scale[1] = in->v_scale;
    c->n = in->v ? 2 : 1;
    c->wide = in->D % kBlock == 0 && aligned32(in->k) && aligned32(in->v);
    c->L = in->L, c->P = in->P, c->T = in->T, c->D = in->D, c->S = in->S, c->M = in->pages ? in->M : 1;
    c->blocks = (in->D + 31) / 32, c->row_blocks = in->H * c->blocks, c->row_elements = in->H * in->D;
    c->pages = in->pages, c->lengths = in->lengths;
    if (static_cast<int64_t>(c->L) * c->n * c->row_blocks * kMaxRows > 0x3fffffff) return SPEC_ERR_INVALID_ARG;
    c->width = std::min(c->row_blocks, kThreads), c->chunks = (c->row_blocks + c->width - 1) / c->width, c->abreast = kThreads / c->width;
    c->parts = c->L * c->n * c->chunks;
    c->by_parts = divide_by(std::max(c->parts, 1)), c->by_chunks = divide_by(c->chunks);
    c->by_blocks = divide_by(c->blocks), c->by_width = divide_by(c->width);
    return SPEC_OK;
}

// How the rows are shared out: rows of a CTA, and CTAs of these rows, so that a thread has up to
// 8 blocks, for the CTA to set out on once, but fewer where the GPU would not be full.  `together`: rows that a CTA takes
// at least, where some of them are dropped, so that the CTAs are left with about as much.
struct Shares {
    int per_cta, splits;
    int64_t ctas;
};
Shares share_rows(const Cache &c, int R, int together) {
    Shares s{1, 1, 0};
    if (c.parts == 0 || R == 0) return s;
    for (int each = 8; each >= 1; each /= 2) {
        const int64_t parts = static_cast<int64_t>(each) * c.abreast;  // of a CTA
        s.per_cta = static_cast<int>(std::min<int64_t>({std::max<int64_t>(parts / c.parts, together), kMaxRows, R}));
        s.splits = static_cast<int>(std::min((static_cast<int64_t>(s.per_cta) * c.parts + parts - 1) / parts, std::max<int64_t>(kMaxCtas / (int64_t{R} + 1), 1)));
        s.ctas = (int64_t{R} + s.per_cta - 1) / s.per_cta * s.splits;
        if (s.ctas >= 152 * 2) break;
    }
    return s;
}

}  // namespace
}  // namespace speccache

extern "C" {

int spec_cache_write(const spec_cache_t *cache, const void *keys, const void *values, int64_t layer_stride,
                     int64_t row_stride, int dtype, const spec_rows_t *rows, const int32_t *num_accepted,
                     const int32_t *last_node, const int32_t *slots, int32_t *out_lengths, void *stream) {
    using namespace speccache;
    Write w{};
    const int rc = check_cache(cache, &w.c);
    if (rc != SPEC_OK) return rc;
    if (!rows || rows->B < 0 || rows->B > SPEC_MAX_B || rows->R < 0) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
    const int mode = rows->rows;
    if (mode != SPEC_ROWS_TARGET && mode != SPEC_ROWS_TREE && mode != SPEC_ROWS_NEXT && mode != SPEC_ROWS_PROMPT)
        return SPEC_ERR_INVALID_ARG;
    const bool verified = mode == SPEC_ROWS_TARGET || mode == SPEC_ROWS_TREE;
    if (verified != (num_accepted != nullptr) || (mode == SPEC_ROWS_TREE) != (last_node != nullptr)) return SPEC_ERR_INVALID_ARG;
    if (mode == SPEC_ROWS_TREE && !rows->parent) return SPEC_ERR_INVALID_ARG;
    if (mode != SPEC_ROWS_NEXT && !rows->offsets) return SPEC_ERR_INVALID_ARG;
    if (rows->R > 0 && (!keys || (w.c.n == 2) != (values != nullptr))) return SPEC_ERR_INVALID_ARG;
    const int size = dtype == SPEC_F32 ? 4 : 2;
    if (!aligned32(keys) || !aligned32(values) || layer_stride % kGranule != 0 || row_stride % kGranule != 0) return SPEC_ERR_ALIGNMENT;
    if (row_stride < static_cast<int64_t>(cache->H) * cache->D || layer_stride < 0) return SPEC_ERR_INVALID_ARG;
    if (rows->R >= kMaxCtas) return SPEC_ERR_INVALID_ARG;
    // the lengths themselves, or clear of them: written while they are still read
    if (out_lengths && out_lengths != cache->lengths && out_lengths < cache->lengths + cache->S && cache->lengths < out_lengths + cache->S)
        return SPEC_ERR_INVALID_ARG;
    if (rows->B == 0 && (!out_lengths || out_lengths == cache->lengths)) return SPEC_OK;
    w.in[0] = static_cast<const char *>(keys), w.in[1] = static_cast<const char *>(values);
    w.layer_stride = layer_stride * size, w.row_stride = row_stride * size;
    w.mode = mode, w.B = rows->B, w.R = rows->R;
    w.offsets = rows->offsets, w.parent = rows->parent, w.num_accepted = num_accepted, w.last_node = last_node, w.slots = slots;
    w.out_lengths = out_lengths;
    const Shares shares = share_rows(w.c, w.R, verified ? 16 : 1);
    const int64_t ctas = shares.ctas;
    // in place, the lengths are read by every CTA before one may write them
    const bool apart = out_lengths && (out_lengths == cache->lengths || ctas == 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ctas > 0) {
        const auto kernel = dtype == SPEC_F32 ? write_kernel<SPEC_F32> : write_kernel<SPEC_BF16>;
        if (!specv::cuda_ok(specv::launch_k(false, kernel, dim3(static_cast<unsigned>(ctas + (out_lengths && !apart))), dim3(kThreads), 0, s, w, shares.per_cta, shares.splits),
                            "write_kernel"))
            return SPEC_ERR_CUDA;
    }
    if (apart && !specv::cuda_ok(specv::launch_k(ctas > 0, lengths_kernel, dim3(1), dim3(kThreads), 0, s, w), "lengths_kernel"))
        return SPEC_ERR_CUDA;
    return SPEC_OK;
}

int spec_cache_read(const spec_cache_t *cache, const int32_t *offsets, int B, int R, const int32_t *first,
                    const int32_t *slots, int dtype, void *out_keys, void *out_values, void *stream) {
    using namespace speccache;
    Read w{};
    const int rc = check_cache(cache, &w.c);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || B > SPEC_MAX_B || R < 0 || R >= kMaxCtas || (dtype != SPEC_F32 && dtype != SPEC_BF16)) return SPEC_ERR_INVALID_ARG;
    if (B == 0 || R == 0 || w.c.L == 0) return SPEC_OK;
    if (!offsets || !out_keys || (w.c.n == 2) != (out_values != nullptr)) return SPEC_ERR_INVALID_ARG;
    if (!aligned32(out_keys) || !aligned32(out_values)) return SPEC_ERR_ALIGNMENT;
    w.out[0] = static_cast<char *>(out_keys), w.out[1] = static_cast<char *>(out_values);
    w.B = B, w.R = R, w.offsets = offsets, w.first = first, w.slots = slots;
    const Shares shares = share_rows(w.c, R, 1);
    const auto kernel = dtype == SPEC_F32 ? read_kernel<SPEC_F32> : read_kernel<SPEC_BF16>;
    return specv::cuda_ok(specv::launch_k(false, kernel, dim3(static_cast<unsigned>(shares.ctas)), dim3(kThreads), 0,
                                          static_cast<cudaStream_t>(stream), w, shares.per_cta, shares.splits),
                          "read_kernel")
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // extern "C"
