// Scores of rows of logits and their gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// One pass over a row keeps, per thread, a whole number R and, with
// d_i = x_i log2 e - R, none so far larger than kSlack,
//     s = sum_i 2^d_i,   u = sum_i d_i 2^d_i
// (when R grows by g: u = (u - g s) 2^-g, s = s 2^-g), from which
//     logp_i = d_i log 2 - log s,   entropy = log s - u / s log 2.
// d_i is one fused operation, rounded once; R is exact, and so is g, whatever a
// row's offset from zero: sums of different R are joined without an error of their
// own.  (A logit m times log2 e, rounded to fp32, is off by half a unit in its
// last place, by another in each thread: 4 % of a row's weights around 10^6.)  And
// logp does not go through lse, which at an offset of 30 is rounded by 10^-6.
// With kSlack = 0 both parts of the entropy are >= 0 and nothing cancels; the
// slack of 6 lets at most 6 units of them cancel (an error of 4 * 2^-24 in units of log 2,
// kept from making an entropy negative), and spares a warp, one of whose 32 threads finds
// a larger logit nearly every time, the growing (8192 rows of 32000 bf16 logits took 107 us
// without a slack and 101 us with one, before R was a whole number).  A -inf adds 0 to both sums (u takes d no
// lower than -150, where 2^d is 0).
//
// R begins at that of -2^21, which logits of a mask's -10^38 leave where it is, and
// is a NaN, as s then is, past 2^21, where whole numbers in fp32 would give out soon.  So
// a row whose largest logit is a NaN, infinite or not within 2^21 of zero ends with s
// = 0 or a NaN, and is read again with that logit taken from the others: d_i = (x_i - m) log2 e.
//
// Alternatives: the pass leaves every thread its largest logit.  The `top`-th
// largest of these is a bound that at least `top` logits reach, and logits that reach it
// are few: they belong to threads whose own largest does.  Warps read such threads'
// logits again, all lanes one thread's, and put those that reach the bound in a
// list, which is sorted: keys are whole numbers that sort like (logit, lowest place
// first).  If many logits equal the bound (a masked row, say), only those above it and the
// first equal ones are taken; if even those above it are too many, each warp
// keeps a sorted list of the 32 largest keys, one per lane, and inserts what is above the
// last one wanted (done for every row, that took 677 us for 8192 rows of
// 32000 bf16 logits, top 20, against 137 us this way).  Sorted lists are joined by
// taking the larger of one and the other reversed, and sorting that.
//
// A logit is read once (once more by the gradient, which writes it once).  At 16
// bits the SMs' issue slots weigh as much as the bytes: about 10 instructions a
// logit (conversion, d, 2^d, two sums, the extremes), 72 % of the slots.
// The rows above take 88 us (6.0 TB/s; a copy's rate is 6.8 TB/s), their gradient 178 us
// (5.9 TB/s), and as many bytes of 32-bit logits, top 8, 102 us (5.1 TB/s).  Tried and
// no faster: one, three or four 16-byte loads ahead instead of two, copies to a
// ring in shared memory.  A row is a block's; with fewer rows than fill the SMs it is
// a cluster's, whose blocks' results the first joins through distributed
// shared memory, so no launch and no memory is needed for that.
#include <type_traits>

#include "ssm_tile.cuh"
#include "tma.cuh"

namespace rnngb {
namespace {

constexpr int kMaxCluster = 8;
constexpr float kSlack = 6.0f;
constexpr float kNear = 2097152.0f;                     // 2^21
constexpr float kLn2 = 0.6931471805599453f, kLn2Rest = 7.348693209507928e-09f;      // 1 / kLog2e = kLn2 + kLn2Rest

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float a_nan() { return __int_as_float(0x7fc00000); }

// Whole numbers that sort like the logits: NaN above +inf, +0 like -0.
__device__ __forceinline__ unsigned order_of(float x)
{
    if (x != x) return 0xffffffffu;
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

// Insert key c (the same in all lanes) into the warp's sorted list.
__device__ __forceinline__ void insert(Key& list, Key c)
{
    const int lane = threadIdx.x % 32;
    const int at = __popc(__ballot_sync(~0u, list > c));
    const Key up = __shfl_up_sync(~0u, list, 1);
    list = lane < at ? list : lane == at ? c : up;
}
// The 32 largest of two sorted lists, sorted.
template <typename T>
__device__ __forceinline__ void merge(T& list, T other)
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
// R of a near logit: v log2 e, rounded to a whole number where 1.5 * 2^23 has its last place.
__device__ __forceinline__ float whole(float v) { return fmaf(v, kLog2e, 12582912.0f) - 12582912.0f; }
struct Sums {
    float r, s, u;
};
// The sums of groups of `width` lanes, in every lane.
__device__ __forceinline__ Sums join(Sums a, int width)
{
    float r = a.r;
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        if (o < width) r = max_nan(r, __shfl_xor_sync(~0u, r, o));
    const float g = r - a.r, f = ex2(-g);
    a.u = fmaf(-g, a.s, a.u) * f;
    a.s *= f;
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        if (o < width) {
            a.s += __shfl_xor_sync(~0u, a.s, o);
            a.u += __shfl_xor_sync(~0u, a.u, o);
        }
    return Sums{r, a.s, a.u};
}

// The elements of [lo, hi) of a row before its first 16-byte boundary.
template <typename V>
__device__ __forceinline__ int64_t to_boundary(const V* x, int64_t lo, int64_t hi)
{
    const int64_t n = (16 - (int64_t)((uintptr_t)(x + lo) % 16)) % 16 / (int64_t)sizeof(V);
    return n < hi - lo ? n : hi - lo;
}
template <typename V, int N>
__device__ __forceinline__ void unpack_vec(const uint4& raw, float (&v)[N])
{
    __align__(16) V e[N];
    *reinterpret_cast<uint4*>(e) = raw;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f(e[i]);
}

// A thread's sums, in two halves; minus_r is -R.
struct Running {
    float minus_r;
    f2 s, u;
};
// N neighbouring logits, of which the largest and the smallest are given.
// Ordinary ones (none of a d below -92, so no -inf) need no lower bound on d.
template <int N>
__device__ __forceinline__ void take(Running& run, const float (&x)[N], float most, float least)
{
    if (!(fmaf(most, kLog2e, run.minus_r) <= kSlack)) {
        const float r = most < kNear ? whole(most) : a_nan(), g = r + run.minus_r;
        const f2 f = dup2(ex2(-g));
        run.u = mul2(fma2(run.s, dup2(-g), run.u), f);
        run.s = mul2(run.s, f);
        run.minus_r = -r;
    }
    const f2 scale = dup2(kLog2e), minus = dup2(run.minus_r);
    if (fmaf(least, kLog2e, run.minus_r) > -92.0f) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const f2 d = fma2(pack2(x[e], x[e + 1]), scale, minus), p = ex2_2(d);
            run.s = add2(run.s, p);
            run.u = fma2(p, d, run.u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const f2 d = fma2(pack2(x[e], x[e + 1]), scale, minus), p = ex2_2(d);
            float d0, d1;
            unpack2(d, d0, d1);
            run.s = add2(run.s, p);
            run.u = fma2(p, pack2(fmaxf(d0, -150.0f), fmaxf(d1, -150.0f)), run.u);
        }
    }
}
// The largest (a NaN counts as one) and smallest of 16 bytes of logits.
__device__ __forceinline__ void extremes(const uint4& raw, const float (&x)[4], float& most, float& least, float)
{
    most = max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
    least = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
}
template <typename V>
__device__ __forceinline__ void extremes(const uint4& raw, const float (&x)[8], float& most, float& least, V)
{
    using V2 = std::conditional_t<std::is_same_v<V, __half>, __half2, __nv_bfloat162>;
    __align__(16) V2 v[4];
    *reinterpret_cast<uint4*>(v) = raw;
    const V2 hi = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
    const V2 lo = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
    most = max_nan(to_f(hi.x), to_f(hi.y));
    least = fminf(to_f(lo.x), to_f(lo.y));
}

// A row's part [lo, hi): single logits at its ends, 16 bytes at a time between.
template <typename V>
struct Part {
    static constexpr int N = 16 / (int)sizeof(V);
    const V* x;
    int64_t lo, hi, first;      // first: where the 16-byte pieces begin
    int vecs;

    __device__ __forceinline__ Part(const V* row, int64_t V_, int part, int blocks) : x(row)
    {
        const int64_t per = ((V_ + blocks - 1) / blocks + N - 1) / N * N;
        lo = part * per < V_ ? part * per : V_;
        hi = lo + per < V_ ? lo + per : V_;
        first = lo + to_boundary(x, lo, hi);
        vecs = (int)((hi - first) / N);
    }
    // The place of thread t's single logit, or -1: at most 14 threads have one.
    __device__ __forceinline__ int64_t single(int t) const
    {
        const int64_t i = lo + t;
        const int64_t at = i < first ? i : i + (int64_t)vecs * N;      // the tail's threads come after the head's
        return at < hi && t < 2 * N ? at : -1;
    }
    __device__ __forceinline__ const uint4* body() const { return reinterpret_cast<const uint4*>(x + first); }
};

constexpr int kCandidates = 512;
struct Found {
    Sums sums;
    Key list[32];
};
// Shared memory of a row's alternatives.
template <int WARPS>
struct Shared {
    Found found[WARPS];
    Found mine;
    unsigned most[WARPS][32], bound, threads, count;
    unsigned short again[32 * WARPS];
    Key candidates[kCandidates];
};

// The part's 32 largest keys (at least its `top` largest), sorted over the lanes of warp 0.
// `most`: this thread's largest logit.
template <typename V, int THREADS>
__device__ __forceinline__ Key largest(const Part<V>& r, float most, int top, Shared<THREADS / 32>& sh)
{
    constexpr int N = Part<V>::N, WARPS = THREADS / 32;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const unsigned own = order_of(most);
    sh.most[warp][lane] = sorted(own);
    if (threadIdx.x == 0) sh.count = sh.threads = 0;
    __syncthreads();
    if (warp == 0) {
        unsigned v = sh.most[0][lane];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) merge(v, sh.most[w][lane]);
        if (lane == top - 1) sh.bound = v;
    }
    __syncthreads();
    const unsigned bound = sh.bound;
    if (own >= bound) sh.again[atomicAdd(&sh.threads, 1u)] = threadIdx.x;
    __syncthreads();
    // Logits of at least `from` go into the list (their order there does not matter).
    auto put = [&](float v, int64_t i, unsigned long long from) {
        if (order_of(v) < from) return;
        const unsigned at = atomicAdd(&sh.count, 1u);
        if (at < kCandidates) sh.candidates[at] = key_of(v, (unsigned)i);
    };
    auto look = [&](int v, unsigned long long from) {
        float e[N];
        unpack_vec<V, N>(r.body()[v], e);
        float of = e[0];
#pragma unroll
        for (int i = 1; i < N; ++i) of = max_nan(of, e[i]);
        if (order_of(of) < from) return;
#pragma unroll
        for (int i = 0; i < N; ++i) put(e[i], r.first + (int64_t)v * N + i, from);
    };
    const unsigned threads = sh.threads;
    auto again = [&](unsigned long long from) {
        if (threads <= THREADS / 4) {
            for (unsigned k = warp; k < threads; k += WARPS) {
                const int t = sh.again[k];
                const int64_t one = r.single(t);
                if (lane == 0 && one >= 0) put(to_f(r.x[one]), one, from);
                for (int v = t + lane * THREADS; v < r.vecs; v += 32 * THREADS) look(v, from);
            }
        } else if (own >= bound) {
            const int64_t one = r.single(threadIdx.x);
            if (one >= 0) put(to_f(r.x[one]), one, from);
#pragma unroll 2
            for (int v = threadIdx.x; v < r.vecs; v += THREADS) look(v, from);
        }
    };
    again(bound);
    __syncthreads();
    unsigned count = sh.count;
    __syncthreads();
    if (count > kCandidates) {
        // Many logits equal the bound: those above it, and the first `top` equal ones.
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
        again((unsigned long long)bound + 1);
        __syncthreads();
        count = sh.count;
        __syncthreads();
        if (count <= kCandidates - 32 * 4 && warp == 0) {
            unsigned found = 0;
            for (int64_t i0 = r.lo; i0 < r.hi && found < top; i0 += 32 * 4) {
                bool same[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t i = i0 + k * 32 + lane;
                    same[k] = i < r.hi && order_of(to_f(r.x[i])) == bound;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned hits = __ballot_sync(~0u, same[k]);
                    const unsigned at = count + found + __popc(hits & ((1u << lane) - 1));
                    const int64_t i = i0 + k * 32 + lane;
                    // (a NaN's key says so whatever the NaN, and -0's is +0's)
                    if (same[k] && at < kCandidates) sh.candidates[at] = (Key)bound << 32 | (unsigned)~(unsigned)i;
                    found += __popc(hits);
                }
            }
            if (lane == 0) sh.count = count + found < kCandidates ? count + found : kCandidates;
        } else if (count > kCandidates - 32 * 4 && threadIdx.x == 0) {
            sh.count = kCandidates + 1;
        }
        __syncthreads();
        count = sh.count;
    }
    Key list = 0;
    if (count <= kCandidates) {
        for (unsigned i = warp * 32; i < count; i += THREADS)
            sh.candidates[i + lane] = sorted(i + lane < count ? sh.candidates[i + lane] : 0);
        __syncthreads();
        if (warp == 0 && count > 0) {
            list = sh.candidates[lane];
            for (unsigned i = 32; i < count; i += 32) merge(list, sh.candidates[i + lane]);
        }
        return list;
    }
    // too many: sorted lists of the warps' own
    for (int64_t i0 = r.lo; i0 < r.hi; i0 += THREADS) {
        const int64_t i = i0 + threadIdx.x;
        const Key key = i < r.hi ? key_of(to_f(r.x[i]), (unsigned)i) : 0;
        unsigned todo = __ballot_sync(~0u, key > __shfl_sync(~0u, list, top - 1));
        while (todo) {
            const Key c = __shfl_sync(~0u, key, __ffs(todo) - 1);
            if (c > __shfl_sync(~0u, list, top - 1)) insert(list, c);
            todo &= todo - 1;
        }
    }
    sh.found[warp].list[lane] = list;
    __syncthreads();
    if (warp == 0)
        for (int w = 1; w < WARPS; ++w) merge(list, sh.found[w].list[lane]);
    return list;
}

// f(logits, their number) of this thread's pieces of the part.
template <typename V, int THREADS, typename F>
__device__ __forceinline__ void each(const Part<V>& r, F f)
{
    const int64_t one = r.single(threadIdx.x);
    if (one >= 0) {
        const float v = to_f(r.x[one]);
        f(&v, 1);
    }
    for (int v = threadIdx.x; v < r.vecs; v += THREADS) {
        float e[Part<V>::N];
        unpack_vec<V, Part<V>::N>(r.body()[v], e);
        f(e, Part<V>::N);
    }
}

// What another block of the cluster has at an address of this one's.
__device__ __forceinline__ float remote(const float* mine, int block)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(smem_addr(mine), block)) : "memory");
    return v;
}
__device__ __forceinline__ Key remote(const Key* mine, int block)
{
    Key v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_map(smem_addr(mine), block)) : "memory");
    return v;
}

// The largest logit m of a row read before (as r), and its sums with d_i = (x_i - m) log2 e:
// in all threads of warp 0 of the row's first block.  `most`: this thread's largest, if KNOWN.
template <typename V, int THREADS, bool KNOWN>
__device__ __noinline__ Sums read_again(const V* x, int64_t V_, int part, int blocks, float most, Found* found, Found* mine)
{
    constexpr int WARPS = THREADS / 32;
    const Part<V> r(x, V_, part, blocks);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (!KNOWN) {
        most = neg_inf();
        each<V, THREADS>(r, [&](const float* x, int n) {
            for (int i = 0; i < n; ++i) most = max_nan(most, x[i]);
        });
    }
    for (int o = 16; o > 0; o /= 2) most = max_nan(most, __shfl_xor_sync(~0u, most, o));
    __syncthreads();                     // all have read the first sums
    if (blocks > 1) cluster_sync_all();
    if (lane == 0) found[warp].sums.r = most;
    __syncthreads();
    float m = found[0].sums.r;
    for (int w = 1; w < WARPS; ++w) m = max_nan(m, found[w].sums.r);
    if (blocks > 1) {
        if (threadIdx.x == 0) mine->sums.r = m;
        cluster_sync_all();
        m = remote(&mine->sums.r, lane % blocks);
        for (int o = blocks / 2; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    }
    float s = 0.0f, u = 0.0f;
    if (m == neg_inf()) return Sums{m, s, u};
    each<V, THREADS>(r, [&](const float* x, int n) {
        for (int i = 0; i < n; ++i) {
            const float d = (x[i] - m) * kLog2e, p = ex2(d);
            s += p;
            u = fmaf(p, fmaxf(d, -150.0f), u);
        }
    });
    for (int o = 16; o > 0; o /= 2) {
        s += __shfl_xor_sync(~0u, s, o);
        u += __shfl_xor_sync(~0u, u, o);
    }
    if (lane == 0) found[warp].sums.s = s, found[warp].sums.u = u;
    __syncthreads();
    s = u = 0.0f;
    for (int w = 0; w < WARPS; ++w) s += found[w].sums.s, u += found[w].sums.u;
    if (blocks > 1) {
        if (threadIdx.x == 0) mine->sums.s = s, mine->sums.u = u;
        cluster_sync_all();
        s = remote(&mine->sums.s, lane % blocks);
        u = remote(&mine->sums.u, lane % blocks);
        for (int o = blocks / 2; o > 0; o /= 2) {
            s += __shfl_xor_sync(~0u, s, o);
            u += __shfl_xor_sync(~0u, u, o);
        }
    }
    return Sums{m, s, u};
}

template <typename V, int THREADS, bool TOP>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) scores_kernel(const ScoreParams p, int blocks)
{
    constexpr int N = Part<V>::N, AHEAD = 2, WARPS = THREADS / 32;
    __shared__ std::conditional_t<TOP, Shared<WARPS>, Found[WARPS + 1]> shared;
    const int part = blockIdx.x % blocks, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Found *found, *mine;
    if constexpr (TOP) found = shared.found, mine = &shared.mine;
    else found = shared, mine = shared + WARPS;
    const int64_t row = blockIdx.x / blocks;
    const V* x = static_cast<const V*>(p.x) + row * p.stride;
    const Part<V> r(x, p.V, part, blocks);
    Running run{-whole(-kNear), 0, 0};
    const int64_t one = r.single(threadIdx.x);
    if (one >= 0) {
        const float v = to_f(x[one]), two[2] = {v, neg_inf()};
        take<2>(run, two, v, neg_inf());
    }
    float most_here = one >= 0 ? to_f(x[one]) : neg_inf();       // this thread's largest
    for (int v = threadIdx.x; v < r.vecs; v += AHEAD * THREADS) {
        uint4 raw[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (v + k * THREADS < r.vecs) raw[k] = r.body()[v + k * THREADS];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (v + k * THREADS < r.vecs) {
                float e[N], most, least;
                unpack_vec<V, N>(raw[k], e);
                extremes(raw[k], e, most, least, V{});
                if (TOP) most_here = max_nan(most_here, most);
                take<N>(run, e, most, least);
            }
    }
    Sums a;
    {
        float v0, v1, w0, w1;
        unpack2(run.s, v0, v1);
        unpack2(run.u, w0, w1);
        a = join(Sums{-run.minus_r, v0 + v1, w0 + w1}, 32);
    }
    if (lane == 0) found[warp].sums = a;
    Key list = 0;
    if constexpr (TOP) list = largest<V, THREADS>(r, most_here, p.top, shared);
    __syncthreads();
    Key next = 0;
    a = found[lane % WARPS].sums;        // over the lanes: of the block's warps,
    if (blocks > 1) {                    // then of the row's blocks
        if (warp == 0) {
            a = join(a, WARPS);
            if (lane == 0) mine->sums = a;
            if (TOP) mine->list[lane] = list;
        }
        cluster_sync_all();
        const int k = lane % blocks;
        const bool joins = part == 0 && warp == 0;       // the others look at s alone
        if (TOP && joins) next = remote(&mine->list[lane], 1);
        a = Sums{joins ? remote(&mine->sums.r, k) : 0.0f, remote(&mine->sums.s, k), joins ? remote(&mine->sums.u, k) : 0.0f};
    }
    // (where R is a logit's, that one's 2^d is above 0.7); the same in all threads
    const bool near = !__any_sync(~0u, a.s != a.s) && __any_sync(~0u, a.s > 0.5f);
    if (!near) a = read_again<V, THREADS, TOP>(x, p.V, part, blocks, most_here, found, mine);
    else if (warp == 0 && part == 0) a = join(a, blocks == 1 ? WARPS : blocks);
    if (blocks > 1) {
        if (TOP && part == 0 && warp == 0) {
            for (int k = 1; k < blocks; ++k) {
                const Key other = next;
                if (k + 1 < blocks) next = remote(&mine->list[lane], k + 1);
                merge(list, other);
            }
        }
        cluster_sync_all();      // no block leaves before its results are read
        if (part != 0) return;
    }
    if (warp != 0) return;
    // a.r is R, or the row's largest logit
    const bool bad = a.s != a.s, empty = a.s == 0.0f;
    const float total = empty ? 0.0f : logf(a.s);
    const float small = near ? fmaf(a.r, kLn2Rest, total) : total;         // lse without the large part
    const float lse = bad ? a_nan() : empty ? neg_inf() : near ? fmaf(a.r, kLn2, small) : a.r + small;
    auto log_p = [&](float v) {
        if (bad || empty) return bad ? a_nan() : neg_inf();
        // (past 10^30, a mask's value, the product would leave fp32's range)
        const float lp = !near ? v - a.r - total : fabsf(v) < 1e30f ? fmaf(fmaf(v, kLog2e, -a.r), kLn2, -total) : v - lse;
        return lp > 0.0f ? 0.0f : lp;          // a certain token's, rounded up
    };
    if (lane == 0) {
        if (p.lse) p.lse[row] = lse;
        if (p.lse_rest) p.lse_rest[row] = bad || empty ? 0.0f : (near ? fmaf(a.r, kLn2, -lse) : a.r - lse) + small;
        if (p.entropy) p.entropy[row] = bad ? a_nan() : empty ? 0.0f : fmaxf(total - a.u * kLn2 / a.s, 0.0f);
        if (p.logp) {
            const int id = p.ids[row];
            p.logp[row] = id < 0 ? 0.0f : id >= p.V ? a_nan() : log_p(to_f(x[id]));
        }
    }
    if (TOP && lane < p.top) {
        if (p.top_ids) p.top_ids[row * p.top + lane] = (int)~(unsigned)list;
        if (p.top_logp) p.top_logp[row * p.top + lane] = log_p(logit_of(list));
    }
}

// dlogits of a row, with d_i = (x_i - lse) log2 e and p_i = 2^d_i (lse in two parts where
// the caller has the second: rounded to fp32 alone, it is off by 10^-6 at 30, and by all of
// log V in an even row of a mask's -10^38, whose p_i would each be 1):
//     g_i = p_i (k0 + k1 d_i),  k0 = -(d_logp + sum d_top + d_entropy entropy),
//                               k1 = -d_entropy log 2,
// plus a term of its own at the given token and at each alternative.  Those
// places are taken out before the block writes and put in after it: the
// gradient may overwrite the logits.
template <typename V, int THREADS>
__global__ void __launch_bounds__(THREADS) scores_grad_kernel(const ScoreGradParams p, int blocks)
{
    constexpr int N = 16 / (int)sizeof(V);
    __shared__ int at[kMaxTop + 1];
    __shared__ float extra[kMaxTop + 1];
    const int64_t row = blockIdx.x / blocks;
    const int part = blockIdx.x % blocks;
    const V* x = static_cast<const V*>(p.x) + row * p.stride;
    V* dx = static_cast<V*>(p.dx) + row * p.d_stride;
    const int64_t per = ((p.V + blocks - 1) / blocks + N - 1) / N * N;
    const int64_t lo = part * per < p.V ? part * per : p.V, hi = lo + per < p.V ? lo + per : p.V;
    const float lse = p.lse[row], minus_rest = p.lse_rest ? -p.lse_rest[row] * kLog2e : 0.0f;
    const float dh = p.d_entropy ? p.d_entropy[row] : 0.0f, h = p.d_entropy ? p.entropy[row] : 0.0f;
    const int id = p.ids ? p.ids[row] : -1;
    const float dl = p.d_logp && id >= 0 ? p.d_logp[row] : 0.0f;
    const bool empty = lse == neg_inf();
    float all = dl;
    for (int j = 0; j < p.top; ++j) all += p.d_top[row * p.top + j];
    const float k0 = empty ? 0.0f : -fmaf(dh, h, all), k1 = empty ? 0.0f : -dh * kLn2;
    auto slope = [&](float v) {
        const float d = empty ? neg_inf() : fmaf(v - lse, kLog2e, minus_rest);
        return ex2(d) * fmaf(k1, fmaxf(d, -150.0f), k0);
    };
    float special = 0.0f;
    int64_t place = -1;
    if (p.top > 0) {
        if (threadIdx.x <= p.top) {
            const int j = threadIdx.x;
            at[j] = j < p.top ? p.top_ids[row * p.top + j] : id;
            extra[j] = j < p.top ? p.d_top[row * p.top + j] : dl;
        }
        __syncthreads();
        if (threadIdx.x <= p.top) place = at[threadIdx.x];
    } else if (threadIdx.x == 0) {
        place = id;
    }
    if (place >= lo && place < hi) {
        special = slope(to_f(x[place]));
        if (!empty) {
            if (p.top > 0) {
                for (int j = 0; j <= p.top; ++j)
                    if (at[j] == place) special += extra[j];
            } else {
                special += dl;
            }
        }
    } else {
        place = -1;
    }
    __syncthreads();

    const int64_t head = to_boundary(dx, lo, hi), vecs = (hi - lo - head) / N, tail = lo + head + vecs * N;
    const bool same = (uintptr_t)(x + lo + head) % 16 == 0;      // 16-byte loads as well as stores
    {
        const int64_t i = threadIdx.x < head ? lo + threadIdx.x : tail + threadIdx.x - head;
        if (threadIdx.x < head || i < hi) dx[i] = from_f<V>(slope(to_f(x[i])));
    }
    const f2 scale = dup2(kLog2e), k0_2 = dup2(k0), k1_2 = dup2(k1), minus = dup2(-lse), rest2 = dup2(minus_rest);
    auto body = [&](const uint4& raw, int64_t v) {
        float e[N];
        unpack_vec<V, N>(raw, e);
        __align__(16) V out[N];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const f2 d = fma2(add2(pack2(e[i], e[i + 1]), minus), scale, rest2);
            float d0, d1;
            unpack2(d, d0, d1);
            const f2 g = mul2(ex2_2(d), fma2(k1_2, pack2(fmaxf(d0, -150.0f), fmaxf(d1, -150.0f)), k0_2));
            unpack2(g, d0, d1);
            out[i] = from_f<V>(d0);
            out[i + 1] = from_f<V>(d1);
        }
        __stcs(reinterpret_cast<uint4*>(dx + lo + head) + v, *reinterpret_cast<uint4*>(out));
    };
    auto load = [&](int64_t v) {
        const V* from = x + lo + head + v * N;
        if (same) return __ldcs(reinterpret_cast<const uint4*>(from));
        __align__(16) V e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from[i];
        return *reinterpret_cast<uint4*>(e);
    };
    if (empty) {
        for (int64_t v = threadIdx.x; v < vecs; v += THREADS)
            reinterpret_cast<uint4*>(dx + lo + head)[v] = make_uint4(0, 0, 0, 0);
    } else {
        for (int64_t v = threadIdx.x; v < vecs; v += 2 * THREADS) {
            const bool two = v + THREADS < vecs;
            const uint4 a = load(v);
            uint4 b = a;
            if (two) b = load(v + THREADS);
            body(a, v);
            if (two) body(b, v + THREADS);
        }
    }
    __syncthreads();
    if (place >= 0) dx[place] = from_f<V>(special);
}

// Blocks of a row.  One while the rows give every SM four blocks (2048
// threads hold enough loads in flight); fewer rows are split, down to 2048
// logits a block.
int blocks_of(int64_t rows, int64_t V, int sms, int most)
{
    int b = 1;
    while (b < most && rows * b < 4 * (int64_t)sms && V / (2 * b) >= 2048) b *= 2;
    return b;
}

// Threads of a block with `per` logits: enough 16-byte pieces for each.
int threads_of(int64_t per) { return per < 4096 ? 64 : 256; }

template <typename V, int THREADS, bool TOP>
cudaError_t run(const ScoreParams& p, int blocks, cudaStream_t s)
{
    if (blocks == 1) {
        scores_kernel<V, THREADS, TOP><<<(unsigned)p.rows, THREADS, 0, s>>>(p, 1);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(p.rows * blocks));
    c.blockDim = dim3(THREADS);
    c.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, scores_kernel<V, THREADS, TOP>, p, blocks);
}
template <typename V>
cudaError_t run(const ScoreParams& p, int blocks, cudaStream_t s)
{
    const bool few = threads_of(p.V / blocks) == 64;
    if (p.top) return few ? run<V, 64, true>(p, blocks, s) : run<V, 256, true>(p, blocks, s);
    return few ? run<V, 64, false>(p, blocks, s) : run<V, 256, false>(p, blocks, s);
}
template <typename V>
cudaError_t run_grad(const ScoreGradParams& p, int blocks, cudaStream_t s)
{
    const unsigned grid = (unsigned)(p.rows * blocks);
    if (threads_of(p.V / blocks) == 64) scores_grad_kernel<V, 64><<<grid, 64, 0, s>>>(p, blocks);
    else scores_grad_kernel<V, 256><<<grid, 256, 0, s>>>(p, blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scores(const ScoreParams& p, cudaStream_t s, int* launches)
{
    int sms = 0;
    cudaError_t e = ssm_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int blocks = blocks_of(p.rows, p.V, sms, kMaxCluster);
    ++*launches;
    return p.io == 1 ? run<__half>(p, blocks, s) : p.io == 2 ? run<__nv_bfloat16>(p, blocks, s) : run<float>(p, blocks, s);
}

cudaError_t launch_scores_grad(const ScoreGradParams& p, cudaStream_t s, int* launches)
{
    int sms = 0;
    cudaError_t e = ssm_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int blocks = blocks_of(p.rows, p.V, sms, 64);
    ++*launches;
    return p.io == 1   ? run_grad<__half>(p, blocks, s)
           : p.io == 2 ? run_grad<__nv_bfloat16>(p, blocks, s)
                       : run_grad<float>(p, blocks, s);
}

}  // namespace rnngb
