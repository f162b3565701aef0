// A step of beam search (what it computes stands in include/onnx_recurrent.h):
// the selection over beams and vocabulary, and the reordering of states.
//
// The B best of an item's beams are among the B best of each beam.  A first launch finds those, and the sum of the row's
// exponentials: a block has a part of a row and holds it in shared memory, so a logit is read once.  Of the eight warps'
// four largest threads' largest logits, the B-th is a bound that at least B logits reach; what reaches it (few) goes to a list that
// is sorted.  Keys
// are whole numbers that sort like (logit, lowest place first).  Where too many reach the bound (equal logits, or a thread
// with many of the largest), warps keep sorted lists of 32 and insert what is above their last; a part of nothing but -inf is
// its first places.  A beam at its end, or without a finite score, has no row to be read.
// 512 rows of 50001 bf16 logits, top 8, take 26 us, 1.9 TB/s: instructions and the steps of a block one after another (by the
// scores' kernel 39 us).
//
// The second launch has a block an item: warps join their beams' parts, totals are formed in 64 bits (fp32 totals of
// an item's beams come as close as 10^-6, and would tie), and every candidate finds its rank: its place in its beam's list, and by
// bisection how many of each other beam's list come before it.
#include <math_constants.h>

#include <type_traits>

#include "norm_internal.h"
#include "ssm_tile.cuh"

namespace rnngb {
namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32, kPieces = 2048, kList = 512;

// Whole numbers that sort like the logits (no NaN among them: a row with one is out), +0 like -0.
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float x, unsigned i) { return (Key)order_of(x) << 32 | (unsigned)~i; }
__device__ __forceinline__ float logit_of(Key key)
{
    const unsigned o = (unsigned)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// The 32 largest of two sorted lists (largest in lane 0), sorted.
template <typename T>
__device__ __forceinline__ void join(T& list, T other)
{
    const int lane = threadIdx.x % 32;
    const T back = __shfl_sync(~0u, other, 31 - lane);
    list = list > back ? list : back;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const T far = __shfl_xor_sync(~0u, list, o);
        list = (lane & o) == 0 ? (list > far ? list : far) : (list > far ? far : list);
    }
}
// The warp's values, sorted, largest in lane 0.
template <typename T>
__device__ __forceinline__ T sorted(T v)
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int o = k / 2; o > 0; o /= 2) {
            const T far = __shfl_xor_sync(~0u, v, o);
            const bool larger = ((lane & k) == 0) == ((lane & o) == 0);
            v = larger ? (v > far ? v : far) : (v > far ? far : v);
        }
    return v;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float v;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
    return v;
}
// The largest of 16 bytes of logits; a NaN counts as that.
template <typename T>
__device__ __forceinline__ float most_of_piece(const uint4& raw)
{
    if constexpr (sizeof(T) == 4) {
        return max_nan(max_nan(__uint_as_float(raw.x), __uint_as_float(raw.y)), max_nan(__uint_as_float(raw.z), __uint_as_float(raw.w)));
    } else {
        using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
        __align__(16) T2 v[4];
        *reinterpret_cast<uint4*>(v) = raw;
        const T2 m = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
        return max_nan(to_f(m.x), to_f(m.y));
    }
}

// What a part leaves: its largest logit and the sum of 2^((x - largest) log2 e) (NaN if it has a NaN or +inf), and its `top`
// largest keys.
struct Part {
    float most, sum;
    Key keys[kMaxBeams];
};
template <typename T>
constexpr int kPartLength = kPieces * 16 / (int)sizeof(T);

// (Its loops are short ones, over shared memory: with the part in registers and all unrolled, the first block of a
// multiprocessor waited longer for its instructions than for its logits, 30 us of a launch.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads) beam_rows_kernel(const BeamSelectParams p)
{
    constexpr int N = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) unsigned char raw[];
    uint4* held = reinterpret_cast<uint4*>(raw);        // the part's pieces
    __shared__ float warp_most[kRowWarps], warp_sum[kRowWarps];
    __shared__ unsigned lists[kRowWarps][32], bound_, count_;
    __shared__ Key found[kList];
    __shared__ Key warp_list[kRowWarps][32];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, top = p.top;
    const int64_t row = blockIdx.x / p.parts, lo = (int64_t)(blockIdx.x % p.parts) * p.length;
    if (!p.shared) {        // (of a shared row, some beam may go on)
        const float s = p.scores[row];
        if (!(fabsf(s) < CUDART_INF_F) || (p.finished && p.finished[row])) return;
    }
    Part* out = reinterpret_cast<Part*>(p.scratch) + blockIdx.x;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride + lo;
    const int n = (int)(p.V - lo < p.length ? p.V - lo : p.length);
    // Pieces of 16 bytes from the first boundary on; the few logits before it and after the last piece are one thread's each.
    int head = (int)((16 - (uintptr_t)x % 16) % 16 / sizeof(T));
    head = head < n ? head : n;
    const int pieces = (n - head) / N, tail = head + pieces * N;
    const int single = tid < head ? tid : tail + tid - head < n && tid >= head && tid < 2 * N ? tail + tid - head : -1;
    const uint4* body = reinterpret_cast<const uint4*>(x + head);
    const float alone = single >= 0 ? to_f(x[single]) : -CUDART_INF_F;
    auto values = [](const uint4& q, float (&v)[N]) {
        __align__(16) T e[N];
        *reinterpret_cast<uint4*>(e) = q;
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = to_f(e[k]);
    };
    float most = alone;
    constexpr int kAhead = 8;
#pragma unroll 1
    for (int i0 = tid; i0 < pieces; i0 += kRowThreads * kAhead) {
        uint4 q[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (i0 + a * kRowThreads < pieces) q[a] = body[i0 + a * kRowThreads];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (i0 + a * kRowThreads < pieces) held[i0 + a * kRowThreads] = q[a];
    }
    // (a thread has its own pieces back: no barrier)
#pragma unroll 1
    for (int i = tid; i < pieces; i += kRowThreads) most = max_nan(most, most_of_piece<T>(held[i]));
    const bool bad = !(most < CUDART_INF_F);        // a NaN or +inf
    // the part's largest
    float m = most;
#pragma unroll
    for (int o = 16; o; o /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (lane == 0) warp_most[warp] = m;
    lists[warp][lane] = sorted(order_of(most));
    if (tid == 0) count_ = 0;
    if (__syncthreads_or(bad)) {
        if (tid == 0) out->most = CUDART_INF_F, out->sum = CUDART_NAN_F;
        return;
    }
    m = warp_most[0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) m = fmaxf(m, warp_most[w]);
    if (m == -CUDART_INF_F) {
        if (tid == 0) out->most = m, out->sum = 0.f;
        if (tid < top) out->keys[tid] = tid < n ? key_of(m, (unsigned)(lo + tid)) : 0;
        return;
    }
    if (warp == 0) {
        const int whole = pieces / 32;          // warps all of whose threads have logits; with fewer than eight, what all of them reach
        unsigned v = lists[lane / 4][lane % 4];
        if (whole >= kRowWarps) {
            v = sorted(v);
        } else {
            v = 0;
            if (whole > 0) v = lists[lane < whole ? lane : 0][(top + whole - 1) / whole - 1];
            v = __reduce_min_sync(~0u, v);
        }
        if (lane == top - 1) bound_ = v;
    }
    // the sum, from the part's largest
    float sum = single >= 0 ? ex2((alone - m) * kLog2e) : 0.f;
    {
        const f2 minus = dup2(-m), scale = dup2(kLog2e);
        f2 sums = dup2(0.f);
#pragma unroll 2
        for (int i = tid; i < pieces; i += kRowThreads) {
            float v[N];
            values(held[i], v);
#pragma unroll
            for (int k = 0; k < N; k += 2) sums = add2(sums, ex2_2(mul2(add2(pack2(v[k], v[k + 1]), minus), scale)));
        }
        float a, b;
        unpack2(sums, a, b);
        sum += a + b;
    }
#pragma unroll
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    const unsigned bound = bound_;
    if (order_of(most) >= bound) {
        auto put = [&](float v, int i) {
            if (order_of(v) < bound) return;
            const unsigned c = atomicAdd(&count_, 1u);
            if (c < kList) found[c] = key_of(v, (unsigned)(lo + i));
        };
        if (single >= 0) put(alone, single);
#pragma unroll 1
        for (int i = tid; i < pieces; i += kRowThreads) {
            if (order_of(most_of_piece<T>(held[i])) < bound) continue;
#pragma unroll 1
            for (int k = 0; k < N; ++k) put(to_f(reinterpret_cast<const T*>(held + i)[k]), head + i * N + k);
        }
    }
    __syncthreads();
    const unsigned count = count_;
    Key list = 0;
    if (count <= kList) {
        // (their order in the list is the atomics', their sorted order is not)
#pragma unroll 1
        for (unsigned i = warp * 32; i < count; i += kRowThreads) found[i + lane] = sorted(i + lane < count ? found[i + lane] : 0);
        __syncthreads();
        if (warp == 0 && count) {
            list = found[lane];
#pragma unroll 1
            for (unsigned i = 32; i < count; i += 32) join(list, found[i + lane]);
        }
    } else {
        auto insert = [&](float v, int i) {
            const Key key = i >= 0 ? key_of(v, (unsigned)(lo + i)) : 0;
            unsigned todo = __ballot_sync(~0u, key > __shfl_sync(~0u, list, 31));
            while (todo) {
                const Key c = __shfl_sync(~0u, key, __ffs(todo) - 1);
                if (c > __shfl_sync(~0u, list, 31)) {
                    const int to = __popc(__ballot_sync(~0u, list > c));
                    const Key up = __shfl_up_sync(~0u, list, 1);
                    list = lane < to ? list : lane == to ? c : up;
                }
                todo &= todo - 1;
            }
        };
        insert(alone, single);
        const T* elements = reinterpret_cast<const T*>(held);
#pragma unroll 1
        for (int i = warp * 32; i < pieces * N; i += kRowThreads) insert(i + lane < pieces * N ? to_f(elements[i + lane]) : 0.f, i + lane < pieces * N ? head + i + lane : -1);
        warp_list[warp][lane] = list;
        __syncthreads();
        if (warp == 0)
#pragma unroll 1
            for (int w = 1; w < kRowWarps; ++w) join(list, warp_list[w][lane]);
    }
    if (warp == 0) {
        if (lane < top) out->keys[lane] = list;
        if (lane == 0) {
            float s = warp_sum[0];
#pragma unroll 1
            for (int w = 1; w < kRowWarps; ++w) s += warp_sum[w];
            out->most = m;
            out->sum = s;
        }
    }
}

constexpr int kItemThreads = 256;

__global__ void __launch_bounds__(kItemThreads) beam_select_kernel(const BeamSelectParams p)
{
    __shared__ Key order[kMaxBeams][kMaxBeams];         // totals, as whole numbers that sort like them
    __shared__ int places[kMaxBeams][kMaxBeams];
    __shared__ double totals[kMaxBeams][kMaxBeams];
    __shared__ bool ended[kMaxBeams];
    const int64_t item = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, B = p.B;
    const double none = -CUDART_INF;
#pragma unroll 1
    for (int b = warp; b < B; b += kItemThreads / 32) {
        const float s = p.scores[item * B + b];
        const bool done = p.finished && p.finished[item * B + b];
        const Part* parts = reinterpret_cast<const Part*>(p.scratch) + (p.shared ? item : item * B + b) * p.parts;
        bool dead = !(fabsf(s) < CUDART_INF_F);
        double most = 0.0, rest = 0.0;      // lse = most + rest, apart: of a row of nothing but a mask's lowest value, 3e38, the sum would be `most` again
        Key list = 0;
        if (!dead && !done) {
            float m = -CUDART_INF_F, sum = 0.f;
            for (int i = lane; i < p.parts; i += 32) m = fmaxf(m, parts[i].most);
#pragma unroll
            for (int o = 16; o; o /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            dead = !(fabsf(m) < CUDART_INF_F);
            if (!dead) {
                for (int i = lane; i < p.parts; i += 32) sum += parts[i].sum * ex2((parts[i].most - m) * kLog2e);
#pragma unroll
                for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
#pragma unroll 1
                for (int i = 0; i < p.parts * p.top; i += 32) {
                    const int c = i + lane;
                    const Key some = sorted(c < p.parts * p.top ? parts[c / p.top].keys[c % p.top] : 0);
                    if (i == 0) list = some;
                    else join(list, some);
                }
                most = (double)m;
                rest = log((double)sum);
            }
        }
        // Candidates of -inf alone come by token; a finished beam's first is its end, then the others.
        double total = none;
        int id = lane;
        if (done && !dead) {
            id = lane == 0 ? (int)p.end : lane <= p.end ? lane - 1 : lane;
            if (lane == 0) total = (double)s;
        } else if (!dead) {
            id = (int)~(unsigned)list;
            total = (double)s + (((double)logit_of(list) - most) - rest);
            if (!(total == total)) total = none;
        }
        const long long bits = __double_as_longlong(total + 0.0);
        order[b][lane] = (Key)bits ^ ((Key)(bits >> 63) | 0x8000000000000000ull);
        totals[b][lane] = total;
        places[b][lane] = id;
        if (lane == 0) ended[b] = done;
    }
    __syncthreads();
    const int top = p.top;
#pragma unroll 1
    for (int c = threadIdx.x; c < B * top; c += kItemThreads) {
        const int b = c / top, i = c - b * top;
        const Key key = order[b][i];
        int rank = i;
#pragma unroll 1
        for (int other = 0; other < B && rank < B; ++other) {
            if (other == b) continue;
            int lo = 0, hi = top;       // how many come first: larger, or as large and of a lower beam
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                const Key k = order[other][mid];
                if (k > key || (k == key && other < b)) lo = mid + 1;
                else hi = mid;
            }
            rank += lo;
        }
        if (rank >= B) continue;
        p.parents[item * B + rank] = b;
        p.ids[item * B + rank] = places[b][i];
        p.new_scores[item * B + rank] = (float)totals[b][i];
        if (p.new_finished) p.new_finished[item * B + rank] = ended[b] || (p.end >= 0 && places[b][i] == p.end);
    }
}

constexpr int kThreads = 128;

// A thread has one unit of a row's bytes of all B rows of an item: it has read them all before it
// writes, so a tensor may be reordered in place.  Eight rows' loads are in flight together; more rows wait in shared memory.
// (A row that is to become itself is left.)  Bytes bound it: 134 MB of states of 64 x 8 beams take 29.5 us, 9 TB/s of reads
// and writes, of which the second-level cache serves some (parents' rows are read by several beams).
constexpr int kAtOnce = 8;
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
        from[threadIdx.x] = good && !(t.in == t.out && from_ == to_) ? from_ : -1;
        to[threadIdx.x] = to_;
    }
    __syncthreads();
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kThreads) {
        U v[kAtOnce] = {};
        for (int b0 = 0; b0 < B; b0 += kAtOnce) {
#pragma unroll
            for (int b = 0; b < kAtOnce; ++b)
                if (b0 + b < B && from[b0 + b] >= 0) v[b] = static_cast<const U*>(t.in)[from[b0 + b] * units + u];
            if (B > kAtOnce)
#pragma unroll
                for (int b = 0; b < kAtOnce; ++b)
                    if (b0 + b < B) held[(b0 + b) * kThreads] = v[b];
        }
        if (B > kAtOnce) {
            for (int b = 0; b < B; ++b)
                if (from[b] >= 0) static_cast<U*>(t.out)[to[b] * units + u] = held[b * kThreads];
        } else {
#pragma unroll
            for (int b = 0; b < kAtOnce; ++b)
                if (b < B && from[b] >= 0) static_cast<U*>(t.out)[to[b] * units + u] = v[b];
        }
    }
}

template <typename U>
cudaError_t reorder(const ReorderParams& p, cudaStream_t s, int* launches)
{
    static std::atomic<uint64_t> done{0};
    const size_t bytes = p.B > kAtOnce ? sizeof(U) * kThreads * (size_t)p.B : 0;
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

// As many parts of a row as fill the multiprocessors three times, of 2048 logits at least and of what a block holds at most.
void beam_plan(BeamSelectParams& p)
{
    const int64_t rows = p.shared ? p.items : p.items * p.B, most = p.io == 0 ? kPartLength<float> : kPartLength<__half>;
    int64_t parts = (p.V + most - 1) / most;
    const int64_t wanted = (p.sms * 3 + rows - 1) / rows, useful = (p.V + 2047) / 2048;
    if (parts < wanted) parts = wanted < useful ? wanted : useful;
    p.length = (p.V + parts - 1) / parts;
    p.length = (p.length + 7) / 8 * 8;
    p.parts = (int)((p.V + p.length - 1) / p.length);
}

size_t beam_scratch_bytes(const BeamSelectParams& p)
{
    return sizeof(Part) * (size_t)((p.shared ? p.items : p.items * p.B) * p.parts);
}

cudaError_t launch_beam_select(const BeamSelectParams& p, cudaStream_t s, int* launches)
{
    const int64_t rows = (p.shared ? p.items : p.items * p.B), blocks = rows * p.parts;
    if (blocks > 0x7fffffffLL || p.items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaSuccess;
    auto go = [&](auto one) {
        using T = decltype(one);
        static std::atomic<uint64_t> done{0};
        e = allow_shared(beam_rows_kernel<T>, 16 * kPieces, done);
        if (e != cudaSuccess) return;
        beam_rows_kernel<T><<<(unsigned)blocks, kRowThreads, (size_t)((p.length * (int)sizeof(T) + 15) / 16 * 16), s>>>(p);
        beam_select_kernel<<<(unsigned)p.items, kItemThreads, 0, s>>>(p);
    };
    if (p.io == 0) go(0.f);
    else if (p.io == 1) go(__half());
    else go(__nv_bfloat16());
    if (e != cudaSuccess) return e;
    *launches += 2;
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderParams& p, cudaStream_t s, int* launches)
{
    uintptr_t all = 0;
    for (int i = 0; i < p.n; ++i) all |= (uintptr_t)p.t[i].in | (uintptr_t)p.t[i].out | (uintptr_t)p.t[i].bytes;
    return all % 16 == 0 ? reorder<uint4>(p, s, launches) : all % 4 == 0 ? reorder<uint32_t>(p, s, launches) : reorder<uint8_t>(p, s, launches);
}

}  // namespace rnngb
