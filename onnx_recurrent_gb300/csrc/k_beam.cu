// A step of beam search (what it computes stands in include/onnx_recurrent.h):
// the selection among the rows' best, and the reordering of states.
//
// The B best of an item's beams are among the B best of each beam, which the scores' kernel has
// found (k_scores.cu: the rows are read once, there) and sorted, ties to the lowest token.  So a
// warp holds an item's beams, lane b the next candidate of beam b, and takes the largest B
// times.  Totals are formed in 64 bits, from the logit itself and lse with what its rounding left
// off: fp32 totals of an item's beams come as close as 10^-6, and would tie.
#include <math_constants.h>

#include "norm_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) beam_select_kernel(const BeamSelectParams p)
{
    const int64_t item = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (item >= p.items) return;
    const int b = threadIdx.x % 32, B = p.B;
    const bool mine = b < B;
    const int64_t rows = p.shared ? p.items : p.items * B, row = p.shared ? item : item * B + (mine ? b : 0);
    const double none = -CUDART_INF;
    const float s = mine ? p.scores[item * B + b] : 0.f;
    const bool done = mine && p.finished && p.finished[item * B + b];
    const double lse = (double)p.lse[row] + (double)p.lse[rows + row];
    // a beam without a finite score, or whose row has no finite lse, has candidates of -inf alone
    const bool dead = !(fabsf(s) < CUDART_INF_F) || (!done && !(fabs(lse) < CUDART_INF));
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    // Candidates of -inf alone come by token; a finished beam's first is its end, then the others.
    auto at = [&](int i, double& total, int& id) {
        total = none;
        id = i;
        if (i >= p.V) {
            id = -1;        // none left: behind every candidate
        } else if (dead) {
        } else if (done) {
            id = i == 0 ? (int)p.end : i <= p.end ? i - 1 : i;
            if (i == 0) total = (double)s;
        } else if (i < p.top) {
            id = p.top_ids[row * p.top + i];
            const double logit = (double)to_f(x[id]);
            total = (double)s + (logit - lse);
            if (!(total == total)) total = none;
        }
    };
    int next = 0, id = -1;
    double total = none;
    if (mine) at(0, total, id);
    int parent = 0, token = 0;
    double score = none;
    for (int k = 0; k < B; ++k) {
        // the largest total; ties to the lowest beam; a beam without a candidate is never taken
        double best = total;
        int who = id >= 0 ? b : 64 + b;
        for (int o = 16; o; o /= 2) {
            const double t = __shfl_xor_sync(0xffffffffu, best, o);
            const int w = __shfl_xor_sync(0xffffffffu, who, o);
            const bool other = (w < 64) != (who < 64) ? w < 64 : t != best ? t > best : w < who;
            if (other) {
                best = t;
                who = w;
            }
        }
        const int from = who & 31, took = __shfl_sync(0xffffffffu, id, from);
        if (b == k) {
            parent = from;
            token = took;
            score = best;
        }
        if (b == from && mine) at(++next, total, id);
    }
    const bool ended = __shfl_sync(0xffffffffu, (int)done, parent) != 0;
    if (mine) {
        p.parents[item * B + b] = parent;
        p.ids[item * B + b] = token;
        p.new_scores[item * B + b] = (float)score;
        if (p.new_finished) p.new_finished[item * B + b] = ended || (p.end >= 0 && token == p.end);
    }
}

constexpr int kThreads = 128;

// A thread has one unit of a row's bytes of all B rows of an item: it has read them all before it
// writes, so a tensor may be reordered in place.
template <typename U>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const ReorderParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    U* held = reinterpret_cast<U*>(raw) + threadIdx.x;      // [B][kThreads]
    __shared__ int64_t from[kMaxBeams], to[kMaxBeams];
    const ReorderTensor& t = p.t[blockIdx.z];
    const int64_t item = blockIdx.y, units = t.bytes / (int64_t)sizeof(U);
    const int B = p.B;
    if (threadIdx.x < B) {
        const int64_t row = item * B + threadIdx.x;
        const int parent = p.parents[row];
        bool good = parent >= 0 && parent < B;
        int64_t to_ = row, from_ = item * B + (good ? parent : 0);
        if (p.slots) {
            to_ = p.slots[row];
            const bool none = to_ == -1;
            if (good && !none) from_ = p.slots[from_];
            if (!none && (to_ < 0 || to_ >= p.n_slots || from_ < 0 || from_ >= p.n_slots)) good = false;
            if (!good && !none) *p.status = 2;       // RNN_ERR_INVALID_INPUT
            if (none) good = false;
        } else if (!good) {
            *p.status = 2;
        }
        from[threadIdx.x] = good ? from_ : -1;
        to[threadIdx.x] = to_;
    }
    __syncthreads();
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kThreads) {
        for (int b = 0; b < B; ++b)
            if (from[b] >= 0) held[b * kThreads] = static_cast<const U*>(t.in)[from[b] * units + u];
        for (int b = 0; b < B; ++b)
            if (from[b] >= 0) static_cast<U*>(t.out)[to[b] * units + u] = held[b * kThreads];
    }
}

template <typename U>
cudaError_t reorder(const ReorderParams& p, cudaStream_t s, int* launches)
{
    static std::atomic<uint64_t> done{0};
    const size_t bytes = sizeof(U) * kThreads * (size_t)p.B;
    cudaError_t e = allow_shared(beam_reorder_kernel<U>, sizeof(U) * kThreads * (size_t)kMaxBeams, done);
    if (e != cudaSuccess) return e;
    int64_t most = 1;
    for (int i = 0; i < p.n; ++i) most = p.t[i].bytes / (int64_t)sizeof(U) > most ? p.t[i].bytes / (int64_t)sizeof(U) : most;
    const int64_t want = (most + kThreads - 1) / kThreads;
    for (int64_t at = 0; at < p.items; at += 65535) {
        ReorderParams q = p;
        q.items = p.items - at < 65535 ? p.items - at : 65535;
        q.parents += at * p.B;
        if (q.slots) q.slots += at * p.B;
        else
            for (int i = 0; i < p.n; ++i) {
                q.t[i].in = static_cast<const char*>(p.t[i].in) + at * p.B * p.t[i].bytes;
                q.t[i].out = static_cast<char*>(p.t[i].out) + at * p.B * p.t[i].bytes;
            }
        beam_reorder_kernel<U><<<dim3((unsigned)(want < 4096 ? want : 4096), (unsigned)q.items, (unsigned)p.n), kThreads, bytes, s>>>(q);
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectParams& p, cudaStream_t s, int* launches)
{
    const unsigned blocks = (unsigned)((p.items + kWarps - 1) / kWarps);
    if (p.io == 0) beam_select_kernel<float><<<blocks, 32 * kWarps, 0, s>>>(p);
    else if (p.io == 1) beam_select_kernel<__half><<<blocks, 32 * kWarps, 0, s>>>(p);
    else beam_select_kernel<__nv_bfloat16><<<blocks, 32 * kWarps, 0, s>>>(p);
    ++*launches;
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderParams& p, cudaStream_t s, int* launches)
{
    uintptr_t all = 0;
    for (int i = 0; i < p.n; ++i) all |= (uintptr_t)p.t[i].in | (uintptr_t)p.t[i].out | (uintptr_t)p.t[i].bytes;
    return all % 16 == 0 ? reorder<uint4>(p, s, launches) : all % 4 == 0 ? reorder<uint32_t>(p, s, launches) : reorder<uint8_t>(p, s, launches);
}

}  // namespace rnngb
