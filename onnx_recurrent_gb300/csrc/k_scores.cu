// Scores of rows of logits and their gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// One pass over a row keeps, per thread, the largest logit m so far and, with
// d_i = x_i - m <= 0,
//     s = sum_i exp(d_i),   u = sum_i d_i exp(d_i)
// (when m grows by g: u = (u - g s) exp(-g), s = s exp(-g)), from which
//     lse = m + log s,      entropy = log s - u / s:
// both parts of the entropy are >= 0, so nothing cancels.
//
// Alternatives: each warp keeps the 32 largest logits it has seen, one per
// lane and sorted, as whole numbers that sort like (logit, lowest place
// first); a logit is compared with the last one wanted and inserted if it is
// above it, which after the first few hundred is rare.
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Whole numbers that sort like the logits: NaN above +inf, +0 like -0.
__device__ __forceinline__ unsigned order_of(float x)
{
    if (x != x) return 0xffffffffu;
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(float x, unsigned i)
{
    return (unsigned long long)order_of(x) << 32 | (unsigned)~i;
}
__device__ __forceinline__ float logit_of(unsigned long long key)
{
    const unsigned o = (unsigned)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// Insert key c (the same in all lanes) into the warp's sorted list.
__device__ __forceinline__ void insert(unsigned long long& list, unsigned long long c)
{
    const int lane = threadIdx.x % 32;
    const int at = __popc(__ballot_sync(~0u, list > c));
    const unsigned long long up = __shfl_up_sync(~0u, list, 1);
    list = lane < at ? list : lane == at ? c : up;
}

struct Sums {
    float m, s, u;
};
__device__ __forceinline__ void add_logit(Sums& a, float x)
{
    if (x > a.m) {
        const float g = x - a.m, f = expf(-g);   // the first one: f = 0
        a.u = a.s > 0.0f ? (a.u - g * a.s) * f : 0.0f;
        a.s *= f;
        a.m = x;
    }
    const float d = x - a.m, e = expf(d);
    if (e > 0.0f) {                               // so -inf adds nothing
        a.s += e;
        a.u = fmaf(d, e, a.u);
    }
}
__device__ __forceinline__ void join(Sums& a, const Sums& b)
{
    if (b.s == 0.0f) return;
    if (a.s == 0.0f) {
        a = b;
        return;
    }
    const float m = fmaxf(a.m, b.m), ga = m - a.m, gb = m - b.m, fa = expf(-ga), fb = expf(-gb);
    const float ua = fa > 0.0f ? (a.u - ga * a.s) * fa : 0.0f, ub = fb > 0.0f ? (b.u - gb * b.s) * fb : 0.0f;
    a.m = m;
    a.s = a.s * fa + b.s * fb;
    a.u = ua + ub;
}

template <typename V>
__global__ void __launch_bounds__(kThreads) scores_kernel(const ScoreParams p)
{
    __shared__ Sums sums[kWarps];
    __shared__ unsigned long long lists[kWarps][32];
    __shared__ int bad;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const V* x = static_cast<const V*>(p.x) + row * p.stride;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    Sums a{neg_inf(), 0.0f, 0.0f};
    unsigned long long list = 0;
    bool odd = false;
    for (int64_t i0 = 0; i0 < p.V; i0 += kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const float v = i < p.V ? to_f(x[i]) : neg_inf();
        odd |= v != v || v == -neg_inf();
        add_logit(a, v);
        if (p.top) {
            const unsigned long long key = i < p.V ? key_of(v, (unsigned)i) : 0;
            unsigned todo = __ballot_sync(~0u, key > __shfl_sync(~0u, list, p.top - 1));
            while (todo) {
                insert(list, __shfl_sync(~0u, key, __ffs(todo) - 1));
                todo &= todo - 1;
            }
        }
    }
    if (odd) bad = 1;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const Sums b{__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.s, o), __shfl_xor_sync(~0u, a.u, o)};
        join(a, b);
    }
    if (lane == 0) sums[warp] = a;
    lists[warp][lane] = list;
    __syncthreads();
    if (warp != 0) return;
    a = sums[0];
    for (int w = 1; w < kWarps; ++w) join(a, sums[w]);
    const float nan = __int_as_float(0x7fc00000);
    const float total = a.s > 0.0f ? logf(a.s) : 0.0f;
    const float lse = bad ? nan : a.s > 0.0f ? a.m + total : neg_inf();
    const bool empty = !bad && a.s == 0.0f;
    if (lane == 0) {
        if (p.lse) p.lse[row] = lse;
        if (p.entropy) p.entropy[row] = bad ? nan : empty ? 0.0f : total - a.u / a.s;
        if (p.logp) {
            const int id = p.ids[row];
            p.logp[row] = id < 0 ? 0.0f : id >= p.V ? nan : empty ? neg_inf() : to_f(x[id]) - lse;
        }
    }
    if (!p.top) return;
    list = lists[0][lane];
    for (int w = 1; w < kWarps; ++w)
        for (int j = 0; j < p.top; ++j) insert(list, lists[w][j]);
    if (lane < p.top) {
        if (p.top_ids) p.top_ids[row * p.top + lane] = (int)~(unsigned)list;
        if (p.top_logp) p.top_logp[row * p.top + lane] = empty ? neg_inf() : logit_of(list) - lse;
    }
}

// dlogits of one row.  Places that are the given token or an alternative get
// a term of their own; the row's other places share
//     -(d_logp + sum d_top) p - d_entropy p (log p + entropy).
template <typename V>
__global__ void __launch_bounds__(kThreads) scores_grad_kernel(const ScoreGradParams p)
{
    __shared__ int at[kMaxTop + 1];
    __shared__ float extra[kMaxTop + 1];
    const int64_t row = blockIdx.x;
    const V* x = static_cast<const V*>(p.x) + row * p.stride;
    V* dx = static_cast<V*>(p.dx) + row * p.d_stride;
    const float lse = p.lse[row];
    const float h = p.d_entropy ? p.entropy[row] : 0.0f, dh = p.d_entropy ? p.d_entropy[row] : 0.0f;
    const int id = p.ids ? p.ids[row] : -1;
    const float dl = p.d_logp && id >= 0 ? p.d_logp[row] : 0.0f;
    const int terms = p.top + 1;
    if (threadIdx.x < terms) {
        const int j = threadIdx.x;
        at[j] = j < p.top ? p.top_ids[row * p.top + j] : id;
        extra[j] = j < p.top ? p.d_top[row * p.top + j] : dl;
    }
    __syncthreads();
    float all = 0.0f;
    for (int j = 0; j < terms; ++j) all += extra[j];
    const bool empty = lse == neg_inf();
    for (int64_t i = threadIdx.x; i < p.V; i += kThreads) {
        float g = 0.0f;
        if (!empty) {
            const float l = to_f(x[i]) - lse, pr = expf(l);
            g = -all * pr;
            if (pr > 0.0f) g -= dh * pr * (l + h);
            if (pr != pr) g = pr;
            for (int j = 0; j < terms; ++j)
                if (at[j] == i) g += extra[j];
        }
        dx[i] = from_f<V>(g);
    }
}

}  // namespace

cudaError_t launch_scores(const ScoreParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    const unsigned grid = (unsigned)p.rows;
    if (p.io == 1) scores_kernel<__half><<<grid, kThreads, 0, s>>>(p);
    else if (p.io == 2) scores_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else scores_kernel<float><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_scores_grad(const ScoreGradParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    const unsigned grid = (unsigned)p.rows;
    if (p.io == 1) scores_grad_kernel<__half><<<grid, kThreads, 0, s>>>(p);
    else if (p.io == 2) scores_grad_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else scores_grad_kernel<float><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rnngb
