// cache.cu -- a cache of keys and values in 8 bits: the rows that a round kept
// written, positions read back, behind the C ABI of include/spec_verify.h.
//
// A block of 32 elements shares the scale 2^e, e the least integer >= -127
// with max |x| <= 448 * 2^e.  With max |x| = f * 2^p, 1 <= f < 2, and 448 = 1.75 * 2^8,
// e = p - 8 + (f > 1.75): an addition to the float's bits, whose carry out of the
// mantissa is that comparison.  x * 2^-e is exact, so that rounding to e4m3 is the
// only one, and reading back multiplies exactly.
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
constexpr int kGranule = 16;  // elements of a thread's access: half a block
constexpr int64_t kMaxCtas = 0x7ffffff0;

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
    int L, P, T, D, blocks;             // blocks: of a head
    int row_blocks;                     // of a position: H * blocks
    int S, M;
    const int32_t *pages, *lengths;
    int work;            // threads' accesses of one layer's and tensor's position, two per block
    Divide by_work, by_head;  // by_head: by the accesses of a head

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
__device__ __forceinline__ void store32(void *p, const Words8 &v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
                 "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
}

template <int DT>
struct Granule;  // 16 elements in their type
template <>
struct Granule<SPEC_BF16> {
    static constexpr int kBytes = 32;
    Words8 v;
    __device__ __forceinline__ void load(const void *p) { v = load32(p); }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? v.w[i / 2] & 0xffff0000u : v.w[i / 2] << 16);
    }
    __device__ __forceinline__ void set2(int i, float a, float b) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
        v.w[i / 2] = *reinterpret_cast<const uint32_t *>(&t);
    }
    __device__ __forceinline__ void store(void *p) const { store32(p, v); }
};
template <>
struct Granule<SPEC_F32> {
    static constexpr int kBytes = 64;
    Words8 v[2];
    __device__ __forceinline__ void load(const void *p) {
        v[0] = load32(p);
        v[1] = load32(static_cast<const char *>(p) + 32);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i / 8].w[i % 8]); }
    __device__ __forceinline__ void set2(int i, float a, float b) {
        v[i / 8].w[i % 8] = __float_as_uint(a);
        v[i / 8].w[i % 8 + 1] = __float_as_uint(b);
    }
    __device__ __forceinline__ void store(void *p) const {
        store32(p, v[0]);
        store32(static_cast<char *>(p) + 32, v[1]);
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

__device__ __forceinline__ int first_row(const Write &w, int b) {
    return w.mode == SPEC_ROWS_NEXT ? b : __ldg(w.offsets + b) + (w.mode == SPEC_ROWS_TARGET ? b : 0);
}

// Whether the offsets are valid; the sequence of row r into *s_seq (-1: none).  The whole block.
__device__ bool check_offsets(const Write &w, int r, int *s_seq) {
    if (w.mode == SPEC_ROWS_NEXT) {
        if (threadIdx.x == 0) *s_seq = r < w.B ? r : -1;
        __syncthreads();
        return w.B <= w.R;
    }
    if (threadIdx.x == 0) *s_seq = -1;
    __syncthreads();
    const int lo = w.mode == SPEC_ROWS_TREE ? 1 : 0;
    const int hi = w.mode == SPEC_ROWS_TREE ? SPEC_MAX_TREE_NODES : w.mode == SPEC_ROWS_TARGET ? SPEC_MAX_K : 0x7fffffff;
    bool bad = __ldg(w.offsets) != 0;
    for (int b = threadIdx.x; b < w.B; b += blockDim.x) {
        const int64_t o = __ldg(w.offsets + b), e = __ldg(w.offsets + b + 1);
        bad |= e - o < lo || e - o > hi;
        const int64_t shift = w.mode == SPEC_ROWS_TARGET ? b : 0, one = w.mode == SPEC_ROWS_TARGET ? 1 : 0;
        if (r >= o + shift && r < e + shift + one) *s_seq = b;
    }
    bad |= static_cast<int64_t>(__ldg(w.offsets + w.B)) + (w.mode == SPEC_ROWS_TARGET ? w.B : 0) > w.R;
    return __syncthreads_or(bad) == 0;
}

// How many rows of sequence b are kept and the slot they go to; 0: it is skipped.
__device__ int kept_rows(const Write &w, int b, int *slot) {
    *slot = w.slots ? __ldg(w.slots + b) : b;
    if (*slot < 0 || *slot >= w.c.S) return 0;
    if (w.mode == SPEC_ROWS_NEXT) return 1;
    const int rows = __ldg(w.offsets + b + 1) - __ldg(w.offsets + b) + (w.mode == SPEC_ROWS_TARGET ? 1 : 0);
    if (w.mode == SPEC_ROWS_PROMPT) return rows;
    const int n = __ldg(w.num_accepted + b);
    return n < 0 || n >= rows ? 0 : n + 1;
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
__device__ void write_lengths(const Write &w, int *s_seq) {
    const bool valid = check_offsets(w, -1, s_seq);
    if (w.out_lengths != w.c.lengths)
        for (int i = threadIdx.x; i < w.c.S; i += kThreads) w.out_lengths[i] = w.c.lengths[i];
    __syncthreads();
    if (!valid) return;
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < w.B; b += kThreads / 32) {
        int slot;
        int n = kept_rows(w, b, &slot);
        if (n == 0) continue;
        const int64_t length = w.c.lengths[slot];
        if (length < 0) continue;
        if (w.mode == SPEC_ROWS_TREE) {
            const int o = __ldg(w.offsets + b);
            bool is_path;
            place_on_path(w.parent, o, __ldg(w.last_node + b), __ldg(w.offsets + b + 1) - o, n, -1, &is_path);
            if (!is_path) continue;
        }
        const int64_t end = length + n;
        bool room = end <= static_cast<int64_t>(w.c.M) * w.c.T && end <= 0x7fffffff;
        if (room && w.c.pages)
            for (int64_t p = length / w.c.T + lane; p * w.c.T < end; p += 32) {
                const int page = __ldg(w.c.pages + static_cast<int64_t>(slot) * w.c.M + p);
                room &= page >= 0 && page < w.c.P;
            }
        room = __all_sync(0xffffffffu, room);
        if (lane == 0) w.out_lengths[slot] = room ? static_cast<int>(end) : -1;
    }
}

// CTAs of row r: splits * r ..; one more at the end for the lengths.
template <int DT>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ Write w, int splits) {
    __shared__ int s_seq;
    __shared__ int64_t s_entry;
    const int r = blockIdx.x / splits;
    if (r >= w.R) {
        write_lengths(w, &s_seq);
        return;
    }
    const bool valid = check_offsets(w, r, &s_seq);
    const int b = s_seq;
    if (!valid || b < 0) return;
    if (threadIdx.x == 0) {
        int slot;
        const int n = kept_rows(w, b, &slot);
        int64_t entry = -1;
        if (n > 0) {
            int i = r - first_row(w, b);
            if (w.mode == SPEC_ROWS_TREE) {
                const int o = __ldg(w.offsets + b);
                bool is_path;
                i = place_on_path(w.parent, o, __ldg(w.last_node + b), __ldg(w.offsets + b + 1) - o, n, r, &is_path);
            }
            const int length = __ldg(w.c.lengths + slot);
            if (i >= 0 && i < n && length >= 0) entry = w.c.entry(slot, static_cast<int64_t>(length) + i);
        }
        s_entry = entry;
    }
    __syncthreads();
    const int64_t entry = s_entry;
    if (entry < 0) return;
    const Cache &c = w.c;
    const int total = c.L * c.n * c.work;
    const int head = 2 * c.blocks;  // accesses of a head; the last one is empty where D is an odd number of them
    const int split = blockIdx.x - r * splits;
    // whole warps, so that both threads of a block are there
    for (int at = split * kThreads + threadIdx.x; at < (total + 31 & ~31); at += splits * kThreads) {
        const int line = c.by_work(at), in_row = at - line * c.work;
        const int h = c.by_head(in_row), g = in_row - h * head;
        const int tensor = c.n == 2 ? line & 1 : 0, layer = c.n == 2 ? line >> 1 : line;
        const bool mine = at < total && g * kGranule < c.D;
        Granule<DT> x;
        float big = 0.0f;
        if (mine) {
            x.load(w.in[tensor] + layer * w.layer_stride + r * w.row_stride + (static_cast<int64_t>(h) * c.D + g * kGranule) * (Granule<DT>::kBytes / kGranule));
#pragma unroll
            for (int i = 0; i < kGranule; ++i) big = fmaxf(big, fabsf(x.get(i)));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        const bool infinite = __float_as_uint(big) == 0x7f800000u;  // (fmaxf passes over NaN)
        if (__any_sync(0xffffffffu, infinite)) {
            float finite = 0.0f;
            if (mine)
#pragma unroll
                for (int i = 0; i < kGranule; ++i) {
                    const float a = fabsf(x.get(i));
                    if (a < __int_as_float(0x7f800000)) finite = fmaxf(finite, a);
                }
            big = fmaxf(finite, __shfl_xor_sync(0xffffffffu, finite, 1));
        }
        if (!mine) continue;
        const int e = max(0, static_cast<int>((__float_as_uint(big) + 0x1fffffu) >> 23) - 8);  // e + 127
        const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = x.get(4 * i + j) * up;
            if (infinite)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (fabsf(x.get(4 * i + j)) == __int_as_float(0x7f800000)) y[j] = nan32();
            q[i] = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
        }
        const int64_t place = (static_cast<int64_t>(layer) * c.P * c.T + entry);
        const int64_t H_D = static_cast<int64_t>(c.row_blocks / c.blocks) * c.D;
        *reinterpret_cast<uint4 *>(c.data[tensor] + place * H_D + h * c.D + g * kGranule) = make_uint4(q[0], q[1], q[2], q[3]);
        if ((g & 1) == 0) c.scale[tensor][place * c.row_blocks + h * c.blocks + g / 2] = static_cast<unsigned char>(e);
    }
}

__global__ void __launch_bounds__(kThreads) lengths_kernel(const __grid_constant__ Write w) {
    __shared__ int s_seq;
    specv::grid_dependency_wait();
    write_lengths(w, &s_seq);
}

// ------------------------------------------------------------------- reading
struct Read {
    Cache c;
    char *out[2];
    int B, R;
    const int32_t *offsets, *first, *slots;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Read w, int splits) {
    __shared__ int s_seq;
    __shared__ int64_t s_entry;
    const int r = blockIdx.x / splits;
    if (threadIdx.x == 0) s_seq = -1;
    __syncthreads();
    bool bad = __ldg(w.offsets) != 0 || __ldg(w.offsets + w.B) > w.R;
    for (int b = threadIdx.x; b < w.B; b += kThreads) {
        const int o = __ldg(w.offsets + b), e = __ldg(w.offsets + b + 1);
        bad |= e < o;
        if (r >= o && r < e) s_seq = b;
    }
    if (__syncthreads_or(bad) || s_seq < 0) return;
    const Cache &c = w.c;
    if (threadIdx.x == 0) {
        const int b = s_seq, slot = w.slots ? __ldg(w.slots + b) : b;
        int64_t entry = -1;
        if (slot >= 0 && slot < c.S) {
            const int64_t p = static_cast<int64_t>(r) - __ldg(w.offsets + b) + (w.first ? __ldg(w.first + b) : 0);
            if (p >= 0 && p < __ldg(c.lengths + slot)) entry = c.entry(slot, p);
        }
        s_entry = entry;
    }
    __syncthreads();
    const int64_t entry = s_entry;
    const int total = c.L * c.n * c.work, head = 2 * c.blocks;
    const int split = blockIdx.x - r * splits;
    const int64_t H_D = static_cast<int64_t>(c.row_blocks / c.blocks) * c.D;
    for (int at = split * kThreads + threadIdx.x; at < total; at += splits * kThreads) {
        const int line = c.by_work(at), in_row = at - line * c.work;
        const int h = c.by_head(in_row), g = in_row - h * head;
        const int tensor = c.n == 2 ? line & 1 : 0, layer = c.n == 2 ? line >> 1 : line;
        if (g * kGranule >= c.D) continue;
        Granule<DT> x;
        uint4 q = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        uint32_t e = 127;
        const int64_t place = static_cast<int64_t>(layer) * c.P * c.T + entry;
        if (entry >= 0) {
            q = __ldg(reinterpret_cast<const uint4 *>(c.data[tensor] + place * H_D + h * c.D + g * kGranule));
            e = __ldg(c.scale[tensor] + place * c.row_blocks + h * c.blocks + g / 2);
        }
        // 2^(e - 127); a byte of 255 is not written: NaN
        const float scale = e == 0 ? __uint_as_float(0x00400000u) : e == 255 ? nan32() : __uint_as_float(e << 23);
        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 y = from_e4m3x2(words[i / 2] >> (i & 1 ? 16 : 0));
            x.set2(2 * i, y.x * scale, y.y * scale);
        }
        x.store(w.out[tensor] + ((static_cast<int64_t>(layer) * w.R + r) * H_D + h * c.D + g * kGranule) * (Granule<DT>::kBytes / kGranule));
    }
}

// ---------------------------------------------------------------------- host
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
    c->L = in->L, c->P = in->P, c->T = in->T, c->D = in->D, c->S = in->S, c->M = in->pages ? in->M : 1;
    c->blocks = (in->D + 31) / 32, c->row_blocks = in->H * c->blocks;
    c->pages = in->pages, c->lengths = in->lengths;
    c->work = 2 * c->row_blocks;
    if (static_cast<int64_t>(c->L) * c->n * c->work > (1 << 30)) return SPEC_ERR_INVALID_ARG;
    c->by_work = divide_by(c->work), c->by_head = divide_by(2 * c->blocks);
    return SPEC_OK;
}

// CTAs of a row: enough of them to fill the GPU, none with less than an access per thread.
int splits_of(const Cache &c, int R) {
    const int64_t total = static_cast<int64_t>(c.L) * c.n * c.work;
    const int64_t most = (total + kThreads - 1) / kThreads;
    const int64_t wanted = std::max<int64_t>((total + 4 * kThreads - 1) / (4 * kThreads), 152 * 8 / std::max(R, 1));
    return static_cast<int>(std::min({most, std::max<int64_t>(wanted, 1), kMaxCtas / (int64_t{R} + 1)}));
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

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
    if (rows->B == 0 && (!out_lengths || out_lengths == cache->lengths)) return SPEC_OK;
    w.in[0] = static_cast<const char *>(keys), w.in[1] = static_cast<const char *>(values);
    w.layer_stride = layer_stride * size, w.row_stride = row_stride * size;
    w.mode = mode, w.B = rows->B, w.R = rows->R;
    w.offsets = rows->offsets, w.parent = rows->parent, w.num_accepted = num_accepted, w.last_node = last_node, w.slots = slots;
    w.out_lengths = out_lengths;
    const int splits = splits_of(w.c, w.R);
    const int64_t ctas = static_cast<int64_t>(w.R) * splits;
    // in place, the lengths are read by every CTA before one may write them
    const bool apart = out_lengths && (out_lengths == cache->lengths || ctas == 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ctas > 0) {
        const auto kernel = dtype == SPEC_F32 ? write_kernel<SPEC_F32> : write_kernel<SPEC_BF16>;
        if (!specv::cuda_ok(specv::launch_k(false, kernel, dim3(static_cast<unsigned>(ctas + (out_lengths && !apart))), dim3(kThreads), 0, s, w, splits),
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
    const int splits = splits_of(w.c, R);
    const auto kernel = dtype == SPEC_F32 ? read_kernel<SPEC_F32> : read_kernel<SPEC_BF16>;
    return specv::cuda_ok(specv::launch_k(false, kernel, dim3(static_cast<unsigned>(R) * splits), dim3(kThreads), 0,
                                          static_cast<cudaStream_t>(stream), w, splits),
                          "read_kernel")
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // extern "C"
