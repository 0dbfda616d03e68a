// state_reorder.cu -- the states that belong to hypotheses (a cache, token
// counts) put into the order of what a beam kept, in place, behind the C ABI of
// include/spec_verify.h.
//
// A move copies slot s(rows[i]) to slot s(i), for every entry i of a group whose two
// slots differ, as if all moves of the group were made at once.  A CTA takes some
// bytes of one run, the same of all the group's slots: it has read them of every source
// before it writes any, so that no CTA waits on another and nothing is kept
// outside of it.  Where runs are multiples of 16 bytes the copy engine moves the
// bytes, by way of shared memory: each distinct source once in, and out to every
// destination of it; a warp does no more than to start the copies and to wait for them.
//
// Times (GB300, events over captured calls): 8 groups of 8 ragged 8-bit caches, 3.9 GB read and written, 600 us (6.5 TB/s,
// 97 % of the copy rate; by columns in registers it took 1400); the token counts of 64 groups of
// 4, 134 MB, 28.3 us (20.1 at the copy rate: the three dependent loads of finding the moves, and the
// first copies); one group's short cache 6.4 us, latency.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "host_common.h"
#include "spec_verify.h"
#include "state_bytes.h"

namespace specstate {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxGroup = SPEC_MAX_BEAMS;
constexpr int kMaxStates = SPEC_MAX_STATES;
constexpr int kStages = 4;           // chunks of a CTA under way
constexpr int kRing = 44 * 1024;     // bytes of them: 4 CTAs and 176 KB to an SM (32 KB: 611 us for the caches)
constexpr int kMinSpan = 16 * 1024;  // of a group of up to 4; of more, so that a CTA has as much to move
constexpr int kMaxSpan = 128 * 1024;
constexpr int kNarrow = 8;           // spans of narrow columns are shorter by this
constexpr int kCtas = 152 * 8;       // a span is made shorter until there are so many (152 * 2: 39 us for the counts)

struct State {
    unsigned char *data;
    int64_t plane, slot, run, unit;  // bytes from one to the next; run holds run / unit positions
    int planes, runs;
    int T;                           // positions of a run
    int spans, span;                 // CTAs of a run, bytes of one (of each slot)
    int width;                       // bytes of a column; 16: moved by the copy engine
    int first;                       // its first CTA of a group
};

struct Map {
    int S, B, R;
    int ctas;      // of a group
    int arrivals;  // that a stage's barrier waits for: 1; 2, of which one never comes, in the self-check
    const int32_t *rows, *offsets, *slots, *lengths;
};
// A call's arguments, with room for N states: a launch copies them.
template <int N>
struct Job {
    Map map;
    int n_states;
    State state[N];
};
constexpr int kFewStates = 8;

// The moves of a group.
struct Moves {
    int count, n_sources;
    // of each distinct source: its slot and the positions that are moved, at least one (past T: all)
    int source[kMaxGroup], length[kMaxGroup];
    // of each move: its destination and which source it has
    int to[kMaxGroup], from[kMaxGroup];
};

struct Scratch {
    int slot[kMaxGroup];
    int index[kMaxGroup];  // entries that are sources: which one; else -1
    unsigned sources[2], moves[2];
};

// SPEC_ERR_TIMEOUT from when a wait has run out on this device; there is no workspace to hold it.
__device__ int g_status;

// Leaves mv.count = 0 for a group that stays as it is.
__device__ void find_moves(const Map &job, int b, Moves &mv, Scratch &sc) {
    const int tid = threadIdx.x;
    bool bad = __ldg(job.offsets) != 0 || __ldg(job.offsets + job.B) > job.R;
    for (int i = tid; i < job.B; i += kThreads) {
        const int w = __ldg(job.offsets + i + 1) - __ldg(job.offsets + i);
        bad |= w < 0 || w > kMaxGroup;
    }
    if (tid == 0) mv.count = 0;
    const int r0 = __ldg(job.offsets + b);
    if (__syncthreads_or(bad)) return;
    const int W = __ldg(job.offsets + b + 1) - r0;
    int slot = -1, source = -1;
    if (tid < W) {
        slot = job.slots ? __ldg(job.slots + r0 + tid) : r0 + tid;
        const int row = __ldg(job.rows + r0 + tid);
        bad = slot < 0 || slot >= job.S || row < -1 || (row >= 0 && (row < r0 || row >= r0 + W));
        source = row < 0 ? tid : row - r0;
        sc.slot[tid] = slot;
    }
    if (__syncthreads_or(bad)) return;
    int length = 0x7fffffff;
    if (tid < kMaxGroup) sc.index[tid] = -1;
    __syncthreads();
    if (tid < W) {
        for (int i = 0; i < W; ++i) bad |= i != tid && sc.slot[i] == slot;
        if (source != tid && job.lengths) length = __ldg(job.lengths + sc.slot[source]);
        if (length <= 0) source = tid;
        if (source != tid) sc.index[source] = 0;
    }
    if (__syncthreads_or(bad)) return;
    const bool moves = tid < W && source != tid, is_source = tid < kMaxGroup && sc.index[tid] == 0;
    const unsigned with_move = __ballot_sync(0xffffffffu, moves), with_source = __ballot_sync(0xffffffffu, is_source);
    if ((tid & 31) == 0 && tid < kMaxGroup) sc.moves[tid >> 5] = with_move, sc.sources[tid >> 5] = with_source;
    __syncthreads();
    const unsigned below = (1u << (tid & 31)) - 1;
    if (is_source) {
        const int at = __popc(with_source & below) + (tid >= 32 ? __popc(sc.sources[0]) : 0);
        sc.index[tid] = at;
        mv.source[at] = slot;
    }
    __syncthreads();
    if (moves) {
        const int at = __popc(with_move & below) + (tid >= 32 ? __popc(sc.moves[0]) : 0);
        mv.to[at] = slot, mv.from[at] = sc.index[source];
        mv.length[sc.index[source]] = length;  // (the same of all moves of a source)
    }
    if (tid == 0) mv.count = __popc(sc.moves[0]) + __popc(sc.moves[1]), mv.n_sources = __popc(sc.sources[0]) + __popc(sc.sources[1]);
    __syncthreads();
}

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src_smem, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(specv::smem_u32(src_smem)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// What is moved of source k of a run, in bytes.
__device__ __forceinline__ int64_t limit_of(const State &st, const Moves &mv, int k) {
    return moved_bytes(st.run, st.unit, st.T, mv.length[k]);
}

// Bytes [begin, end) of a run, each source's as far as a multiple of 16, in chunks through a ring, by one warp.  A wait
// that runs out (2 s; a copy that never comes) leaves the rest as it was and is recorded: false.
__device__ bool move_bulk(const State &st, unsigned char *base, const Moves &mv, int64_t begin, int64_t end, unsigned char *ring, uint64_t *full) {
    const int lane = threadIdx.x, D = mv.n_sources, n = mv.count;
    const int stages = D > 8 ? 2 : kStages;  // (copies of a few hundred bytes are slow)
    const int chunk = static_cast<int>(min(int64_t{kRing} / (stages * D), int64_t{16384})) & ~63;  // at least 320 bytes
    const int chunks = static_cast<int>((end - begin + chunk - 1) / chunk);
    // what is moved of source k in chunk c
    const auto bytes_of = [&](int k, int c) {
        const int64_t most = (min(end, limit_of(st, mv, k)) & ~int64_t{15}) - (begin + static_cast<int64_t>(c) * chunk);
        return static_cast<uint32_t>(max(int64_t{0}, min(most, static_cast<int64_t>(chunk))));
    };
    const auto load = [&](int c) {
        unsigned char *stage = ring + (c % stages) * D * chunk;
        uint64_t *bar = full + c % stages;
        uint32_t sum = 0;
        for (int k = lane; k < D; k += 32) sum += bytes_of(k, c);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) specv::mbar_arrive_expect_tx(bar, sum);
        __syncwarp();
        for (int k = lane; k < D; k += 32) {
            const uint32_t bytes = bytes_of(k, c);
            if (bytes) specv::bulk_g2s(stage + k * chunk, base + mv.source[k] * st.slot + begin + static_cast<int64_t>(c) * chunk, bytes, bar);
        }
    };
    for (int c = 0; c < min(chunks, stages - 1); ++c) load(c);
    int c = 0;
    for (; c < chunks; ++c) {
        if (!__all_sync(0xffffffffu, specv::mbar_wait_bounded(full + c % stages, (c / stages) & 1))) break;
        const unsigned char *stage = ring + (c % stages) * D * chunk;
        for (int i = lane; i < n; i += 32) {
            const uint32_t bytes = bytes_of(mv.from[i], c);
            if (bytes) bulk_s2g(base + mv.to[i] * st.slot + begin + static_cast<int64_t>(c) * chunk, stage + mv.from[i] * chunk, bytes);
        }
        bulk_commit();
        if (c + stages - 1 < chunks) {  // into the stage whose chunk was written the turn before
            bulk_wait_read<1>();
            __syncwarp();
            load(c + stages - 1);
        }
    }
    const bool ok = c == chunks;
    if (!ok && lane == 0) specv::set_status(&g_status, SPEC_ERR_TIMEOUT);
    for (int k = c + 1; !ok && k < min(chunks, c + stages - 1); ++k) specv::mbar_wait_bounded(full + k % stages, (k / stages) & 1);
    bulk_wait_read<0>();
    return ok;
}

// The same by columns, a thread a column, for states of any alignment.  The thread has read its column of all
// sources, into places of its own in the ring, before it writes one.
template <class Vec>
__device__ __forceinline__ void move_columns(const State &st, unsigned char *base, const Moves &mv, int64_t begin, int64_t end, unsigned char *ring) {
    constexpr int w = sizeof(Vec), batch = 4;
    static_assert(kMaxGroup * kThreads * w <= kRing || w == 8, "a column of each source per thread");
    const int threads = min(kThreads, kRing / (w * mv.n_sources));  // (8 bytes of 64 sources are more than the ring holds of 128)
    if (static_cast<int>(threadIdx.x) >= threads) return;
    Vec *mine = reinterpret_cast<Vec *>(ring) + threadIdx.x;  // source k at k * threads
    for (int64_t byte = begin + threadIdx.x * w; byte < end; byte += threads * w) {
        for (int k0 = 0; k0 < mv.n_sources; k0 += batch) {
            Vec v[batch];
#pragma unroll
            for (int k = 0; k < batch; ++k)
                if (k0 + k < mv.n_sources && byte + w <= limit_of(st, mv, k0 + k))
                    v[k] = *reinterpret_cast<const Vec *>(base + mv.source[k0 + k] * st.slot + byte);
#pragma unroll
            for (int k = 0; k < batch; ++k)
                if (k0 + k < mv.n_sources) {
                    if (byte + w <= limit_of(st, mv, k0 + k)) {
                        mine[(k0 + k) * threads] = v[k];
                    } else {  // a column that ends inside
                        unsigned char *to = reinterpret_cast<unsigned char *>(mine + (k0 + k) * threads);
                        for (int64_t j = byte; j < limit_of(st, mv, k0 + k); ++j) to[j - byte] = base[mv.source[k0 + k] * st.slot + j];
                    }
                }
        }
        for (int i = 0; i < mv.count; ++i) {
            const int k = mv.from[i];
            if (byte + w <= limit_of(st, mv, k)) {
                *reinterpret_cast<Vec *>(base + mv.to[i] * st.slot + byte) = mine[k * threads];
            } else {
                const unsigned char *from = reinterpret_cast<const unsigned char *>(mine + k * threads);
                for (int64_t j = byte; j < limit_of(st, mv, k); ++j) base[mv.to[i] * st.slot + j] = from[j - byte];
            }
        }
    }
}

// CTAs ctas * b .. of group b: each takes a span of one run of one plane of one state.
template <int N>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ Job<N> job) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ Moves mv;
    __shared__ Scratch sc;
    __shared__ uint64_t full[kStages];
    __shared__ unsigned char tail[kMaxGroup][16];
    const int b = blockIdx.x / job.map.ctas;
    int at = blockIdx.x - b * job.map.ctas;
    int k = 0;
    while (k + 1 < job.n_states && at >= job.state[k + 1].first) ++k;
    const State &st = job.state[k];
    at -= st.first;
    const int line = at / st.spans, plane = line / st.runs;
    const int64_t begin = static_cast<int64_t>(at - line * st.spans) * st.span;
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) specv::mbar_init(full + i, job.map.arrivals);
        specv::fence_barrier_init();
    }
    find_moves(job.map, b, mv, sc);
    if (mv.count == 0) return;
    // the span ends where the longest source does
    int64_t end = 0;
    for (int i = 0; i < mv.n_sources; ++i) end = max(end, limit_of(st, mv, i));
    end = min(begin + st.span, end);
    if (begin >= end) return;
    unsigned char *base = st.data + plane * st.plane + (line - plane * st.runs) * st.run;
    if (st.width == 16) {
        // bytes behind a source's last multiple of 16: read before anything is written, written when all is read
        const auto tail_of = [&](int k, int64_t *from) {
            const int64_t limit = limit_of(st, mv, k);
            *from = limit & ~int64_t{15};
            return *from >= begin && *from < begin + st.span ? static_cast<int>(limit - *from) : 0;
        };
        int64_t from;
        if (tid < mv.n_sources)
            for (int j = 0, n = tail_of(tid, &from); j < n; ++j) tail[tid][j] = base[mv.source[tid] * st.slot + from + j];
        __syncthreads();
        const bool ok = tid >= 32 || begin >= (end & ~int64_t{15}) || move_bulk(st, base, mv, begin, end, ring, full);
        if (!__syncthreads_and(ok)) return;
        if (tid < mv.count)
            for (int j = 0, n = tail_of(mv.from[tid], &from); j < n; ++j) base[mv.to[tid] * st.slot + from + j] = tail[mv.from[tid]][j];
    } else if (st.width == 8) {
        move_columns<uint2>(st, base, mv, begin, end, ring);
    } else if (st.width == 4) {
        move_columns<uint32_t>(st, base, mv, begin, end, ring);
    } else {
        move_columns<unsigned char>(st, base, mv, begin, end, ring);
    }
}

template <int N>
int launch(const Map &map, const State *states, int n, cudaStream_t s) {
    Job<N> job;
    job.map = map, job.n_states = n;
    std::copy(states, states + n, job.state);
    return specv::cuda_ok(specv::launch_k(false, reorder_kernel<N>, dim3(static_cast<unsigned>(map.ctas) * map.B), dim3(kThreads), kRing, s, job), "reorder_kernel")
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

int reorder(const spec_state_t *states, int n_states, int S, const int32_t *rows, const int32_t *offsets, int B, int R,
            const int32_t *slots, const int32_t *lengths, void *stream, int arrivals) {
    if (n_states < 0 || n_states > kMaxStates || S < 0 || B < 0 || B > SPEC_MAX_B || R < 0) return SPEC_ERR_INVALID_ARG;
    if (B == 0 || R == 0 || n_states == 0) return SPEC_OK;
    if (!states || !rows || !offsets) return SPEC_ERR_INVALID_ARG;
    Map map{S, B, R, 0, arrivals, rows, offsets, slots, lengths};
    State state[kMaxStates];
    int n = 0;
    int64_t bytes[kMaxStates];
    for (int k = 0; k < n_states; ++k) {
        const spec_state_t &in = states[k];
        if (in.planes < 0 || in.runs < 0 || in.T < 0 || in.unit < 0 || in.T > 0x7fffffff) return SPEC_ERR_INVALID_ARG;
        State &st = state[n];
        int64_t all;
        if (__builtin_mul_overflow(in.T, in.unit, &st.run) || __builtin_mul_overflow(st.run, in.runs, &st.slot) ||
            __builtin_mul_overflow(st.slot, static_cast<int64_t>(S), &st.plane) ||
            __builtin_mul_overflow(st.plane, in.planes, &all))
            return SPEC_ERR_INVALID_ARG;
        if (all == 0) continue;
        if (!in.data) return SPEC_ERR_INVALID_ARG;
        if (in.planes > 0x7fffffff || in.runs > 0x7fffffff) return SPEC_ERR_INVALID_ARG;
        st.data = static_cast<unsigned char *>(in.data), st.unit = in.unit, st.T = static_cast<int>(in.T);
        for (int i = 0; i < n; ++i)
            if (st.data < state[i].data + bytes[i] && state[i].data < st.data + all) return SPEC_ERR_INVALID_ARG;
        // nor one that overlaps what says how it is moved: other CTAs still read that
        const auto overlaps = [&](const int32_t *p, int64_t entries) {
            const unsigned char *l = reinterpret_cast<const unsigned char *>(p);
            return l && st.data < l + entries * 4 && l < st.data + all;
        };
        if (overlaps(lengths, S) || overlaps(rows, R) || overlaps(slots, R) || overlaps(offsets, int64_t{B} + 1)) return SPEC_ERR_INVALID_ARG;
        st.planes = static_cast<int>(in.planes), st.runs = static_cast<int>(in.runs);
        const uintptr_t low = reinterpret_cast<uintptr_t>(st.data) | static_cast<uintptr_t>(st.run);
        st.width = (low & 15) == 0 ? 16 : (low & 7) == 0 ? 8 : (low & 3) == 0 ? 4 : 1;
        bytes[n++] = all;
    }
    if (n == 0) return SPEC_OK;
    // spans as long as leave enough CTAs; longer where there would be too many for a launch
    const auto ctas_of = [&](int64_t span) {
        int64_t ctas = 0;
        for (int k = 0; k < n; ++k) {
            State &st = state[k];
            st.span = static_cast<int>(st.width == 16 ? span : std::max<int64_t>(span / kNarrow, 1024));
            const int64_t spans = (st.run + st.span - 1) / st.span;
            int64_t all;
            if (spans > 0x7fffffff || __builtin_mul_overflow(spans, static_cast<int64_t>(st.planes), &all) ||
                __builtin_mul_overflow(all, static_cast<int64_t>(st.runs), &all) || all > 0x7fffffff)
                return int64_t{1} << 40;
            st.spans = static_cast<int>(spans), st.first = static_cast<int>(std::min<int64_t>(ctas, 0x7fffffff));
            ctas += all;
        }
        return ctas * B;
    };
    int64_t span = kMaxSpan, least = kMinSpan;
    for (int64_t w = 4; w < R / B && least > 2048; w *= 2) least /= 2;
    while (span > least && ctas_of(span) < kCtas) span /= 2;
    while (ctas_of(span) > 0x7fffffff) {
        if (span >= int64_t{1} << 30) return SPEC_ERR_INVALID_ARG;  // more planes and runs than CTAs can be
        span *= 2;
    }
    map.ctas = static_cast<int>(ctas_of(span) / B);
    const auto run = n <= kFewStates ? launch<kFewStates> : launch<kMaxStates>;
    return run(map, state, n, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace specstate

extern "C" {

int spec_state_reorder(const spec_state_t *states, int n_states, int S, const int32_t *rows, const int32_t *offsets,
                       int B, int R, const int32_t *slots, const int32_t *lengths, void *stream) {
    return specstate::reorder(states, n_states, S, rows, offsets, B, R, slots, lengths, stream, 1);
}

int spec_state_reorder_status(int *status_out, int clear) {
    if (!status_out) return SPEC_ERR_INVALID_ARG;
    int v = 0;
    if (!specv::cuda_ok(cudaDeviceSynchronize(), "cudaDeviceSynchronize(reorder status)") ||
        !specv::cuda_ok(cudaMemcpyFromSymbol(&v, specstate::g_status, sizeof v), "cudaMemcpyFromSymbol(reorder status)"))
        return SPEC_ERR_CUDA;
    *status_out = v;
    const int ok = SPEC_OK;
    if (clear && !specv::cuda_ok(cudaMemcpyToSymbol(specstate::g_status, &ok, sizeof ok), "cudaMemcpyToSymbol(reorder status)")) return SPEC_ERR_CUDA;
    return SPEC_OK;
}

int spec_selfcheck_reorder_timeout(const spec_state_t *states, int n_states, int S, const int32_t *rows,
                                   const int32_t *offsets, int B, int R, const int32_t *slots, const int32_t *lengths,
                                   void *stream) {
    return specstate::reorder(states, n_states, S, rows, offsets, B, R, slots, lengths, stream, 2);
}

}  // extern "C"
