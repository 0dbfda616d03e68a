// state_reorder.cu -- the states that belong to hypotheses (a cache, token
// counts) put into the order of what a beam kept, in place, behind the C ABI of
// include/spec_verify.h.
//
// A move copies slot s(rows[i]) to slot s(i), for every entry i of a group whose two
// slots differ, as if all moves of the group were made at once.  A thread
// takes one column (the same 16 bytes or fewer of every slot) of a whole
// group, so that threads never wait on one another.  It loads the column of up to
// kBatch moves' sources before it stores any; with more moves they are put in
// an order in which none reads what an earlier one wrote, except that of each cycle
// the first destination is kept in a register for the cycle's last move.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "host_common.h"
#include "spec_verify.h"

namespace specstate {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroup = SPEC_MAX_BEAMS;
constexpr int kMaxStates = SPEC_MAX_STATES;
constexpr int kBatch = 8;       // moves whose columns a thread holds at once
constexpr int kColumns = 4096;  // of a CTA: 64 KB of a slot in columns of 16 bytes

struct State {
    unsigned char *data;
    int64_t plane, slot, run, unit;  // bytes from one to the next; run holds run / unit positions
    int planes, runs, chunks;        // chunks: CTAs of a run
    int width;                       // bytes of a column
    int first;                       // its first CTA of a group
};

struct Job {
    State state[kMaxStates];
    int n_states, S, B, R;
    int ctas, columns;  // CTAs of a group, columns of a CTA
    const int32_t *rows, *offsets, *slots, *lengths;
};

// The moves of a group in their order.
struct Moves {
    int count;
    int from[kMaxGroup], to[kMaxGroup], length[kMaxGroup];
    int keep[kMaxGroup];  // positions of its destination to keep before it is overwritten; 0: none
    bool kept[kMaxGroup];  // takes what was kept instead of its source
};

struct Scratch {
    int slot[kMaxGroup], source[kMaxGroup], length[kMaxGroup];
    int readers[kMaxGroup];  // moves to come that read the slot; a move made: -1
};

// Leaves mv.count = 0 for a group that stays as it is.
__device__ void find_moves(const Job &job, int b, Moves &mv, Scratch &sc) {
    const int tid = threadIdx.x;
    bool bad = __ldg(job.offsets) != 0 || __ldg(job.offsets + job.B) > job.R;
    for (int i = tid; i < job.B; i += kThreads) {
        const int w = __ldg(job.offsets + i + 1) - __ldg(job.offsets + i);
        bad |= w < 0 || w > kMaxGroup;
    }
    if (tid == 0) mv.count = 0;
    if (tid < kMaxGroup) sc.readers[tid] = 0;
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
    if (tid < W) {
        for (int i = 0; i < W; ++i) bad |= i != tid && sc.slot[i] == slot;
        if (source != tid && job.lengths) length = __ldg(job.lengths + sc.slot[source]);
        if (length <= 0) source = tid;
        sc.source[tid] = source, sc.length[tid] = length;
        if (source != tid) atomicAdd(&sc.readers[source], 1);
    }
    if (__syncthreads_or(bad)) return;
    if (tid == 0) {
        int n = 0;
        const auto make = [&](int e) {
            mv.from[n] = sc.slot[sc.source[e]], mv.to[n] = sc.slot[e], mv.length[n] = sc.length[e];
            mv.keep[n] = 0, mv.kept[n] = false;
            sc.readers[e] = -1;
            ++n;
        };
        // moves into slots that nothing reads any more; each may free its source's slot
        for (int i = 0; i < W; ++i)
            for (int e = i; sc.readers[e] == 0 && sc.source[e] != e; e = sc.source[e]) {
                make(e);
                if (--sc.readers[sc.source[e]] != 0) break;
            }
        // what is left are cycles
        for (int i = 0; i < W; ++i) {
            if (sc.readers[i] < 0 || sc.source[i] == i) continue;
            const int first = n;
            int e = i;
            do {
                const int next = sc.source[e];
                make(e);
                e = next;
            } while (e != i);
            mv.keep[first] = mv.length[n - 1], mv.kept[n - 1] = true;
        }
        mv.count = n;
    }
    __syncthreads();
}

template <class Vec>
__device__ __forceinline__ void move_columns(const State &st, unsigned char *base, const Moves &mv, int64_t c0,
                                             int columns) {
    const int n = mv.count;
    for (int k = threadIdx.x; k < columns; k += kThreads) {
        const int64_t byte = (c0 + k) * static_cast<int64_t>(sizeof(Vec));
        if (byte >= st.run) break;
        const int position = static_cast<int>(byte / st.unit);
        Vec kept{};
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            Vec v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j;
                if (i < n) {
                    if (mv.kept[i]) v[j] = kept;
                    else if (position < mv.length[i]) v[j] = *reinterpret_cast<const Vec *>(base + mv.from[i] * st.slot + byte);
                    if (position < mv.keep[i]) kept = *reinterpret_cast<const Vec *>(base + mv.to[i] * st.slot + byte);
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j;
                if (i < n && position < mv.length[i]) *reinterpret_cast<Vec *>(base + mv.to[i] * st.slot + byte) = v[j];
            }
        }
    }
}

// CTAs ctas * b .. of group b: each takes some columns of one run of one plane of one state.
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ Job job) {
    __shared__ Moves mv;
    __shared__ Scratch sc;
    const int b = blockIdx.x / job.ctas;
    int at = blockIdx.x - b * job.ctas;
    int k = 0;
    while (k + 1 < job.n_states && at >= job.state[k + 1].first) ++k;
    const State &st = job.state[k];
    at -= st.first;
    const int line = at / st.chunks, chunk = at - line * st.chunks;
    const int plane = line / st.runs, run = line - plane * st.runs;
    find_moves(job, b, mv, sc);
    if (mv.count == 0) return;
    unsigned char *base = st.data + plane * st.plane + run * st.run;
    const int64_t c0 = static_cast<int64_t>(chunk) * job.columns;
    if (st.width == 16) move_columns<uint4>(st, base, mv, c0, job.columns);
    else if (st.width == 4) move_columns<uint32_t>(st, base, mv, c0, job.columns);
    else move_columns<unsigned char>(st, base, mv, c0, job.columns);
}

}  // namespace
}  // namespace specstate

extern "C" int spec_state_reorder(const spec_state_t *states, int n_states, int S, const int32_t *rows,
                                  const int32_t *offsets, int B, int R, const int32_t *slots, const int32_t *lengths,
                                  void *stream) {
    using namespace specstate;
    if (n_states < 0 || n_states > kMaxStates || S < 0 || B < 0 || B > SPEC_MAX_B || R < 0) return SPEC_ERR_INVALID_ARG;
    if (B == 0 || R == 0 || n_states == 0) return SPEC_OK;
    if (!states || !rows || !offsets) return SPEC_ERR_INVALID_ARG;
    Job job;
    job.S = S, job.B = B, job.R = R;
    job.rows = rows, job.offsets = offsets, job.slots = slots, job.lengths = lengths;
    int n = 0;
    int64_t bytes[kMaxStates];
    for (int k = 0; k < n_states; ++k) {
        const spec_state_t &in = states[k];
        if (in.planes < 0 || in.runs < 0 || in.T < 0 || in.unit < 0 || in.T > 0x7fffffff) return SPEC_ERR_INVALID_ARG;
        State &st = job.state[n];
        int64_t all;
        if (__builtin_mul_overflow(in.T, in.unit, &st.run) || __builtin_mul_overflow(st.run, in.runs, &st.slot) ||
            __builtin_mul_overflow(st.slot, static_cast<int64_t>(S), &st.plane) ||
            __builtin_mul_overflow(st.plane, in.planes, &all))
            return SPEC_ERR_INVALID_ARG;
        if (all == 0) continue;
        if (!in.data) return SPEC_ERR_INVALID_ARG;
        if (in.planes > 0x7fffffff || in.runs > 0x7fffffff) return SPEC_ERR_INVALID_ARG;
        st.data = static_cast<unsigned char *>(in.data), st.unit = in.unit;
        for (int i = 0; i < n; ++i)
            if (st.data < job.state[i].data + bytes[i] && job.state[i].data < st.data + all) return SPEC_ERR_INVALID_ARG;
        const unsigned char *l = reinterpret_cast<const unsigned char *>(lengths);
        if (l && st.data < l + static_cast<int64_t>(S) * 4 && l < st.data + all) return SPEC_ERR_INVALID_ARG;
        st.planes = static_cast<int>(in.planes), st.runs = static_cast<int>(in.runs);
        // a column lies in one position, so that a length cuts none
        const uintptr_t low = reinterpret_cast<uintptr_t>(st.data) | static_cast<uintptr_t>(in.unit);
        st.width = (low & 15) == 0 ? 16 : (low & 3) == 0 ? 4 : 1;
        bytes[n++] = all;
    }
    if (n == 0) return SPEC_OK;
    job.n_states = n;
    for (job.columns = kColumns;; job.columns *= 2) {
        int64_t ctas = 0;
        for (int k = 0; k < n; ++k) {
            State &st = job.state[k];
            const int64_t chunks = (st.run / st.width + job.columns - 1) / job.columns;
            int64_t all;
            if (chunks > 0x7fffffff || __builtin_mul_overflow(chunks, static_cast<int64_t>(st.planes), &all) ||
                __builtin_mul_overflow(all, static_cast<int64_t>(st.runs), &all) || all > 0x7fffffff) {
                ctas = int64_t{1} << 40;
                break;
            }
            st.chunks = static_cast<int>(chunks), st.first = static_cast<int>(std::min<int64_t>(ctas, 0x7fffffff));
            ctas += all;
        }
        if (ctas * B <= 0x7fffffff) {
            job.ctas = static_cast<int>(ctas);
            break;
        }
        if (job.columns > 0x20000000) return SPEC_ERR_INVALID_ARG;  // more planes and runs than CTAs can be
    }
    return specv::cuda_ok(specv::launch_k(false, reorder_kernel, dim3(static_cast<unsigned>(job.ctas) * B), dim3(kThreads), 0,
                                          static_cast<cudaStream_t>(stream), job),
                          "reorder_kernel")
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
