// Short causal convolution over time for each channel (the formulas stand in
// include/onnx_recurrent.h), its gradients and its single-token form.
//
// Little is computed for an element's bytes (2 values, 3 with the gradient), but
// at 16 bits the instructions weigh as much.  A thread takes NV neighbouring
// channels of one row (four where the tensors allow it), whose sums it forms in
// packed pairs, and walks along a run of steps with the next K sums in
// registers, so each input is read once (and K - 1 again at the start of a run).
// The thread's inputs of the next kRing steps are on their way to its own places
// in shared memory, so no barrier is needed and loads in flight cost no registers.
// 8 rows of 2048 steps x 2048 bf16 channels, 4 taps, take 29 us (4.6 TB/s; 5.6 TB/s
// with 32-bit values) and their gradient 66 us; with single arithmetic 32 us and
// 79 us, with the next four steps' inputs in registers 51 to 76 us.
// The gradient's walk keeps the last K inputs and slopes of the sums: with
// pre[t] = bias + sum_j W[j] X[t-K+1+j] and e[t] = dY[t] f'(pre[t]),
//     dX[u] = sum_j W[j] e[u+K-1-j],   dW[j] = sum_t e[t] X[t-K+1+j],
// so after step t the walk can write dX[t-K+1].  dW and dbias are summed over
// a run in registers, then over runs and rows in order by a kernel of their own.
#include <initializer_list>
#include <type_traits>

#include "ssm_tile.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 128;
constexpr int kRing = 8;          // steps whose inputs are in flight
constexpr int kUnroll = 4;        // steps of a loop's body: the K values in registers then rotate without moves

template <typename T, int NV>
struct __align__(sizeof(T) * NV) Vec {
    T v[NV];
};

// The NV channels from d on of step t (a carried one for t < 0), or zeros.
template <typename T, int K, int NV>
__device__ __forceinline__ Vec<T, NV> conv_input(const ConvParams& p, int64_t n, int64_t t, int64_t d)
{
    const T* from;
    if (t >= 0) from = static_cast<const T*>(p.X.data) + t * p.X.ss + n * p.X.bs + d;
    else from = p.h0 ? static_cast<const T*>(p.h0) + (n * (K - 1) + (t + K - 1)) * p.D + d : nullptr;
    Vec<T, NV> r;
    if (from) {
        r = *reinterpret_cast<const Vec<T, NV>*>(from);
    } else {
#pragma unroll
        for (int e = 0; e < NV; ++e) r.v[e] = from_f<T>(0.0f);
    }
    return r;
}

// N floats, in 16-byte pieces where they allow it.
template <int N>
__device__ __forceinline__ void load_floats(const float* from, float (&to)[N])
{
    if (N % 4 == 0 && (uintptr_t)from % 16 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(from)[i];
            to[4 * i] = v.x, to[4 * i + 1] = v.y, to[4 * i + 2] = v.z, to[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = from[i];
    }
}
// A thread's own ring of inputs.
template <typename T, int NV>
struct Ring {
    using V = Vec<T, NV>;
    static constexpr bool ASYNC = sizeof(V) >= 4;      // a single 16-bit value is too small to copy
    V* at;                                             // this thread's place in each slot, kThreads apart

    // Step's values to the slot, or zeros.
    __device__ __forceinline__ void start(int slot, const T* from, bool on, const void* valid) const
    {
        if constexpr (ASYNC) {
            const unsigned d = (unsigned)__cvta_generic_to_shared(at + slot * kThreads);
            const void* src = on ? from : valid;
            const int bytes = on ? (int)sizeof(V) : 0;
            if constexpr (sizeof(V) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(src), "r"(bytes) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;\n" ::"r"(d), "l"(src), "r"(bytes), "n"((int)sizeof(V)) : "memory");
        } else {
            at[slot * kThreads].v[0] = on ? *from : from_f<T>(0.0f);
        }
    }
    // Without asynchronous copies: a body's steps at once, so that their loads overlap.
    __device__ __forceinline__ void refill(int slot, const T* from, int64_t ss, int left) const
    {
        T v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) v[i] = i < left ? from[i * ss] : from_f<T>(0.0f);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) at[(slot + i) % kRing * kThreads].v[0] = v[i];
    }
    __device__ __forceinline__ V get(int slot) const { return at[slot * kThreads]; }
};

// NV channels' values: packed pairs, or the one channel's (packed arithmetic with
// a half idle takes 156 us for the gradient of 8 rows of 2048 steps x 2047
// bf16 channels, single arithmetic 110 us).
template <int NV>
struct Pairs {
    using V = std::conditional_t<NV == 1, float, f2>;
    static constexpr int N = (NV + 1) / 2;
    V v[N];
};
__device__ __forceinline__ f2 plus(f2 a, f2 b) { return add2(a, b); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ f2 times_plus(f2 a, f2 b, f2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float times_plus(float a, float b, float c) { return fmaf(a, b, c); }
// x f'(v) of silu
__device__ __forceinline__ f2 silu_slope(f2 x, f2 v)
{
    const f2 o = sigmoid_fast2(v), one = dup2(1.0f);
    return mul2(x, mul2(o, fma2(v, fma2(o, dup2(-1.0f), one), one)));
}
__device__ __forceinline__ float silu_slope(float x, float v)
{
    const float o = sigmoid_fast(v);
    return x * (o * fmaf(v, 1.0f - o, 1.0f));
}
template <int NV>
__device__ __forceinline__ Pairs<NV> make_pairs(const float (&x)[NV])
{
    Pairs<NV> r;
    if constexpr (NV == 1) {
        r.v[0] = x[0];
    } else {
#pragma unroll
        for (int e = 0; e < NV / 2; ++e) r.v[e] = pack2(x[2 * e], x[2 * e + 1]);
    }
    return r;
}
template <typename T, int NV>
__device__ __forceinline__ Pairs<NV> pairs_of(const Vec<T, NV>& x)
{
    float f[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) f[e] = to_f(x.v[e]);
    return make_pairs<NV>(f);
}
template <int NV>
__device__ __forceinline__ void floats_of(const Pairs<NV>& x, float (&f)[NV])
{
    if constexpr (NV == 1) {
        f[0] = x.v[0];
    } else {
#pragma unroll
        for (int e = 0; e < NV / 2; ++e) unpack2(x.v[e], f[2 * e], f[2 * e + 1]);
    }
}
template <typename T, int NV>
__device__ __forceinline__ Vec<T, NV> vec_of(const Pairs<NV>& x)
{
    Vec<T, NV> r;
    float f[NV];
    floats_of(x, f);
#pragma unroll
    for (int e = 0; e < NV; ++e) r.v[e] = from_f<T>(f[e]);
    return r;
}
template <int NV>
__device__ __forceinline__ Pairs<NV> fma_pairs(const Pairs<NV>& a, const Pairs<NV>& b, const Pairs<NV>& c)
{
    Pairs<NV> r;
#pragma unroll
    for (int e = 0; e < Pairs<NV>::N; ++e) r.v[e] = times_plus(a.v[e], b.v[e], c.v[e]);
    return r;
}
template <int NV>
__device__ __forceinline__ Pairs<NV> silu_pairs(const Pairs<NV>& v)
{
    Pairs<NV> r;
#pragma unroll
    for (int e = 0; e < Pairs<NV>::N; ++e)
        if constexpr (NV == 1) r.v[e] = silu_fast(v.v[e]);
        else r.v[e] = silu_fast2(v.v[e]);
    return r;
}

template <int K, int NV>
struct Weights {
    Pairs<NV> w[K], bias;
    __device__ __forceinline__ Weights(const ConvParams& p, int64_t d)
    {
        float all[NV * K], b[NV];
        load_floats(p.W + d * K, all);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float tap[NV];
#pragma unroll
            for (int e = 0; e < NV; ++e) tap[e] = all[e * K + j];
            w[j] = make_pairs<NV>(tap);
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) b[e] = 0.0f;
        if (p.bias) load_floats(p.bias + d, b);
        bias = make_pairs<NV>(b);
    }
};

// What a thread has: channels d .., row n, steps t0 .. t1-1; false: nothing.
template <int NV>
__device__ __forceinline__ bool find(const ConvParams& p, unsigned dblocks, unsigned runs, int run, int64_t& d, int64_t& n,
                                     int64_t& t0, int64_t& t1)
{
    d = ((int64_t)(blockIdx.x % dblocks) * kThreads + threadIdx.x) * NV;
    t0 = (int64_t)(blockIdx.x / dblocks % runs) * run;
    n = blockIdx.x / dblocks / runs;
    t1 = t0 + run < p.S ? t0 + run : p.S;
    return d < p.D;
}

template <typename T, int K, int NV>
__global__ void __launch_bounds__(kThreads, K <= 4 ? 8 : 4) ssm_conv_kernel(const ConvParams p, unsigned dblocks, unsigned runs, int run)
{
    __shared__ Vec<T, NV> ring_mem[kRing][kThreads];
    int64_t d, n, t0, t1;
    if (!find<NV>(p, dblocks, runs, run, d, n, t0, t1)) return;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t live = len < t1 ? len : t1;
    T* y = static_cast<T*>(p.Y.data) + n * p.Y.bs + d;
    if (t0 < live) {
        const Weights<K, NV> w(p, d);
        // sums[i]: what the inputs so far give to the sum i steps ahead, taps in order from the bias
        Pairs<NV> sums[K];
#pragma unroll
        for (int j = 0; j < K; ++j) sums[j] = w.bias;
        // takes the next input, returns the sum that it completes
        auto next = [&](const Pairs<NV>& x) {
            const Pairs<NV> done = fma_pairs(w.w[K - 1], x, sums[0]);
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) sums[j] = fma_pairs(w.w[K - 2 - j], x, j + 2 < K ? sums[j + 1] : w.bias);
            return done;
        };
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) next(pairs_of(conv_input<T, K, NV>(p, n, t0 - K + 1 + j, d)));
        const Ring<T, NV> ring{ring_mem[0] + threadIdx.x};
        const int steps = (int)(live - t0);
        const T* x = static_cast<const T*>(p.X.data) + n * p.X.bs + d + t0 * p.X.ss;      // the next input to start
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            ring.start(i, x, i < steps, p.X.data);
            cp_async_commit();
            x += p.X.ss;
        }
        T* to = y + t0 * p.Y.ss;
        for (int i0 = 0; i0 < steps; i0 += kUnroll) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int slot = (i0 + i) % kRing;
                cp_async_wait<kRing - 1>();
                Pairs<NV> v = next(pairs_of(ring.get(slot)));
                if (p.silu) v = silu_pairs(v);
                if (i0 + i < steps) *reinterpret_cast<Vec<T, NV>*>(to) = vec_of<T>(v);
                to += p.Y.ss;
                if (ring.ASYNC) {
                    ring.start(slot, x, i0 + i + kRing < steps, p.X.data);
                    x += p.X.ss;
                }
                cp_async_commit();
            }
            if (!ring.ASYNC) {
                ring.refill(i0, x, p.X.ss, steps - i0 - kRing);
                x += kUnroll * p.X.ss;
            }
        }
        cp_async_wait<0>();
    }
    Vec<T, NV> zero;
#pragma unroll
    for (int e = 0; e < NV; ++e) zero.v[e] = from_f<T>(0.0f);
    for (int64_t t = live > t0 ? live : t0; t < t1; ++t) *reinterpret_cast<Vec<T, NV>*>(y + t * p.Y.ss) = zero;
    if (t0 == 0 && p.hT) {   // the last K-1 inputs, reaching back into the carried ones
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
            *reinterpret_cast<Vec<T, NV>*>(static_cast<T*>(p.hT) + (n * (K - 1) + j) * p.D + d) =
                conv_input<T, K, NV>(p, n, len - K + 1 + j, d);
    }
}

template <typename T, int K, int NV>
__global__ void __launch_bounds__(kThreads, K <= 4 ? 5 : 3) ssm_conv_grad_kernel(const ConvGradParams q, unsigned dblocks, unsigned runs, int run)
{
    const ConvParams& p = q.f;
    __shared__ Vec<T, NV> ring_mem[2][kRing][kThreads];
    int64_t d, n, t0, t1;
    if (!find<NV>(p, dblocks, runs, run, d, n, t0, t1)) return;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const Weights<K, NV> w(p, d);
    Pairs<NV> zeros;
#pragma unroll
    for (int e = 0; e < Pairs<NV>::N; ++e) zeros.v[e] = 0;
    Pairs<NV> x[K], s[K], dw[K], db = zeros;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        x[j] = j > 0 && t0 < len ? pairs_of(conv_input<T, K, NV>(p, n, t0 - K + j, d)) : zeros;
        s[j] = dw[j] = zeros;
    }
    const T* dhT = static_cast<const T*>(q.dhT);
    const Ring<T, NV> ring_x{ring_mem[0][0] + threadIdx.x}, ring_y{ring_mem[1][0] + threadIdx.x};
    // slopes of the run's steps, and of the K-1 after it that its inputs reach
    const int owned = (int)(t1 - t0), steps = owned + K - 1, known = len - t0 < steps ? (int)(len > t0 ? len - t0 : 0) : steps;
    const T* xs = static_cast<const T*>(p.X.data) + n * p.X.bs + d + t0 * p.X.ss;         // the next ones to start
    const T* ys = static_cast<const T*>(q.dY.data) + n * q.dY.bs + d + t0 * q.dY.ss;
    auto start = [&](int i) {
        ring_x.start(i % kRing, xs, i < known, p.X.data);
        ring_y.start(i % kRing, ys, i < known, p.X.data);
        xs += p.X.ss;
        ys += q.dY.ss;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
        start(i);
        cp_async_commit();
    }
    T* to = static_cast<T*>(q.dX.data) + n * q.dX.bs + d + (t0 - K + 1) * q.dX.ss;       // of step u below
    const int last = dhT && len - (K - 1) - t0 < steps ? (int)(len - (K - 1) - t0) : steps;      // u - t0 from which dhT reaches
    for (int i0 = 0; i0 < steps; i0 += kUnroll) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int k = i0 + i, u = k - K + 1;     // the input whose slopes are complete, from t0
            cp_async_wait<kRing - 1>();
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) {
                x[j] = x[j + 1];
                s[j] = s[j + 1];
            }
            x[K - 1] = pairs_of(ring_x.get(k % kRing));          // zero past the row's end, as is dY
            Pairs<NV> g = pairs_of(ring_y.get(k % kRing));
            if (p.silu) {
                Pairs<NV> v = w.bias;
#pragma unroll
                for (int j = 0; j < K; ++j) v = fma_pairs(w.w[j], x[j], v);
#pragma unroll
                for (int e = 0; e < Pairs<NV>::N; ++e) g.v[e] = silu_slope(g.v[e], v.v[e]);
            }
            s[K - 1] = k < known ? g : zeros;
            if (k < known && k < owned) {
#pragma unroll
                for (int e = 0; e < Pairs<NV>::N; ++e) db.v[e] = plus(db.v[e], g.v[e]);
#pragma unroll
                for (int j = 0; j < K; ++j) dw[j] = fma_pairs(g, x[j], dw[j]);
            }
            if (k < steps && (u >= 0 || t0 == 0)) {
                Pairs<NV> sum = zeros;
#pragma unroll
                for (int j = 0; j < K; ++j) sum = fma_pairs(w.w[K - 1 - j], s[j], sum);
                if (u >= last && u < known && t0 + u < len) {
                    const int64_t at = (n * (K - 1) + (t0 + u - len + K - 1)) * p.D + d;
                    const Pairs<NV> more = pairs_of(*reinterpret_cast<const Vec<T, NV>*>(dhT + at));
#pragma unroll
                    for (int e = 0; e < Pairs<NV>::N; ++e) sum.v[e] = plus(sum.v[e], more.v[e]);
                }
                if (u >= 0) {
                    if (q.dX.data) *reinterpret_cast<Vec<T, NV>*>(to) = vec_of<T>(sum);
                } else if (q.dh0) {
                    *reinterpret_cast<Vec<T, NV>*>(static_cast<T*>(q.dh0) + (n * (K - 1) + (u + K - 1)) * p.D + d) = vec_of<T>(sum);
                }
            }
            to += q.dX.ss;
            if (ring_x.ASYNC) start(k + kRing);
            cp_async_commit();
        }
        if (!ring_x.ASYNC) {
            ring_x.refill(i0, xs, p.X.ss, known - i0 - kRing);
            ring_y.refill(i0, ys, q.dY.ss, known - i0 - kRing);
            xs += kUnroll * p.X.ss;
            ys += kUnroll * q.dY.ss;
        }
    }
    cp_async_wait<0>();
    if (q.part) {
        float* part = q.part + (n * runs + t0 / run) * p.D * (K + 1);
#pragma unroll
        for (int j = 0; j <= K; ++j) {
            float v[NV];
            floats_of(j < K ? dw[j < K ? j : 0] : db, v);
#pragma unroll
            for (int e = 0; e < NV; ++e) part[j < K ? (d + e) * K + j : p.D * K + d + e] = v[e];
        }
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) ssm_conv_step_kernel(const ConvStepParams p, int dblocks)
{
    const int64_t d = (int64_t)(blockIdx.x % dblocks) * kThreads + threadIdx.x;
    const int64_t n = blockIdx.x / dblocks;
    if (d >= p.D) return;
    T* y = static_cast<T*>(p.Y.data) + n * p.Y.bs + d;
    int64_t slot = n;
    if (p.slots) {
        slot = p.slots[n];
        if (slot < 0 || slot >= p.slots_n) {
            if (slot != -1) *p.status = 2;   // RNN_ERR_INVALID_INPUT
            *y = from_f<T>(0.0f);
            return;
        }
    }
    const T* st = static_cast<const T*>(p.state) + slot * (K - 1) * p.D + d;
    T* so = static_cast<T*>(p.state_out) + slot * (K - 1) * p.D + d;
    T x[K];
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) x[j] = st[j * p.D];
    x[K - 1] = static_cast<const T*>(p.X.data)[n * p.X.bs + d];
    float v = p.bias ? p.bias[d] : 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) v = fmaf(p.W[d * K + j], to_f(x[j]), v);
    *y = from_f<T>(p.silu ? silu_fast(v) : v);
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) so[j * p.D] = x[j + 1];
}

// One partial result per blockDim.y row and pass, added in the order of the
// rows and then of the passes.
__global__ void __launch_bounds__(512) sum_parts_kernel(const float* part, int64_t parts, float* out0, int64_t n0,
                                                        float* out1, int64_t n1, float* out2, int64_t n2)
{
    __shared__ float sums[16][33];
    const int64_t n = n0 + n1 + n2;
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (i < n) {
#pragma unroll 8
        for (int64_t r = threadIdx.y; r < parts; r += 16) s += part[r * n + i];
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || i >= n) return;
    s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += sums[r][threadIdx.x];
    if (i < n0) {
        if (out0) out0[i] = s;
    } else if (i < n0 + n1) {
        if (out1) out1[i - n0] = s;
    } else if (out2) {
        out2[i - n0 - n1] = s;
    }
}

// f(element type, number of taps) for the plan's type and taps.
template <template <typename, int> class F, typename T, typename... A>
cudaError_t by_taps(int K, A... a)
{
    switch (K) {
    case 1: return F<T, 1>::go(a...);
    case 2: return F<T, 2>::go(a...);
    case 3: return F<T, 3>::go(a...);
    case 4: return F<T, 4>::go(a...);
    case 5: return F<T, 5>::go(a...);
    case 6: return F<T, 6>::go(a...);
    case 7: return F<T, 7>::go(a...);
    default: return F<T, 8>::go(a...);
    }
}
template <template <typename, int> class F, typename... A>
cudaError_t by_type(int io, int K, A... a)
{
    if (io == 1) return by_taps<F, __half>(K, a...);
    if (io == 2) return by_taps<F, __nv_bfloat16>(K, a...);
    return by_taps<F, float>(K, a...);
}

// Channels of a thread: four (two where the gradient's K taps of four would not fit
// the registers; eight 16-bit ones take twice the registers and no less time), two
// for 16-bit types of even sizes, else one.
template <typename T, int K, bool GRAD>
constexpr int widest()
{
    constexpr int full = 16 / (int)sizeof(T), fits = GRAD && K > 4 ? 2 : 4;
    return full < fits ? full : fits;
}
bool views_fit(std::initializer_list<View> views, std::initializer_list<const void*> states, int64_t D, int elem, int nv)
{
    const int64_t bytes = (int64_t)elem * nv;
    if (D % nv) return false;
    for (const View& v : views)
        if (v.data && ((uintptr_t)v.data % bytes || v.ss * elem % bytes || v.bs * elem % bytes)) return false;
    for (const void* s : states)
        if ((uintptr_t)s % bytes) return false;
    return true;
}

// Steps of a run: the longest that leaves the SMs enough threads (each run
// reads K - 1 inputs again, and writes a partial dW).
int run_of(int64_t S, int64_t threads_a_run, int sms)
{
    int run = 128;
    while (run > 16 && (S + run - 1) / run * threads_a_run < (int64_t)sms * 1024) run /= 2;
    return run;
}
int64_t run_count(int64_t S, int run) { return S > 0 ? (S + run - 1) / run : 1; }
constexpr int64_t kMaxGrid = 0x7fffffff;

template <typename T, int K>
struct RunConv {
    template <int NV>
    static cudaError_t with(const ConvParams& p, cudaStream_t s)
    {
        const int64_t threads = (p.D + NV - 1) / NV, db = (threads + kThreads - 1) / kThreads;
        const int run = run_of(p.S, threads * p.N, p.sms);
        const int64_t runs = run_count(p.S, run);
        if (db * runs > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
        ssm_conv_kernel<T, K, NV><<<(unsigned)(db * runs * p.N), kThreads, 0, s>>>(p, (unsigned)db, (unsigned)runs, run);
        return cudaGetLastError();
    }
    static cudaError_t go(const ConvParams* p, cudaStream_t s)
    {
        constexpr int W = widest<T, K, false>();
        auto fit = [&](int nv) { return views_fit({p->X, p->Y}, {p->h0, p->hT}, p->D, sizeof(T), nv); };
        if (fit(W)) return with<W>(*p, s);
        if constexpr (sizeof(T) == 2 && W > 2)
            if (fit(2)) return with<2>(*p, s);
        return with<1>(*p, s);
    }
};
template <typename T, int K>
struct RunConvGrad {
    template <int NV>
    static cudaError_t with(const ConvGradParams& q, cudaStream_t s)
    {
        const ConvParams& p = q.f;
        const int run = q.run;
        const int64_t threads = (p.D + NV - 1) / NV, db = (threads + kThreads - 1) / kThreads, runs = run_count(p.S, run);
        if (db * runs > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
        ssm_conv_grad_kernel<T, K, NV><<<(unsigned)(db * runs * p.N), kThreads, 0, s>>>(q, (unsigned)db, (unsigned)runs, run);
        return cudaGetLastError();
    }
    static cudaError_t go(const ConvGradParams* q, cudaStream_t s)
    {
        constexpr int W = widest<T, K, true>();
        auto fit = [&](int nv) {
            return views_fit({q->f.X, q->dY, q->dX}, {q->f.h0, q->dhT, q->dh0}, q->f.D, sizeof(T), nv);
        };
        if (fit(W)) return with<W>(*q, s);
        if constexpr (sizeof(T) == 2 && W > 2)
            if (fit(2)) return with<2>(*q, s);
        return with<1>(*q, s);
    }
};
template <typename T, int K>
struct RunConvStep {
    static cudaError_t go(const ConvStepParams* p, unsigned grid, int db, cudaStream_t s)
    {
        ssm_conv_step_kernel<T, K><<<grid, kThreads, 0, s>>>(*p, db);
        return cudaGetLastError();
    }
};

}  // namespace

cudaError_t launch_ssm_conv(const ConvParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    return by_type<RunConv>(p.io, p.K, &p, s);
}

void ssm_conv_grad_plan(ConvGradParams& q)
{
    q.run = run_of(q.f.S, (q.f.D + 1) / 2 * q.f.N, q.f.sms);
    q.parts = q.f.N * run_count(q.f.S, q.run);
}

cudaError_t launch_ssm_conv_grad(const ConvGradParams& q, cudaStream_t s, int* launches)
{
    if (q.f.N > 0) {
        ++*launches;
        cudaError_t e = by_type<RunConvGrad>(q.f.io, q.f.K, &q, s);
        if (e != cudaSuccess) return e;
    }
    if (!q.dW && !q.dbias) return cudaSuccess;
    return launch_sum_parts(q.part, q.parts, q.dW, q.f.D * q.f.K, q.dbias, q.f.D, nullptr, 0, s, launches);
}

cudaError_t launch_ssm_conv_step(const ConvStepParams& p, cudaStream_t s, int* launches)
{
    const int64_t db = (p.D + kThreads - 1) / kThreads;
    if (db > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    ++*launches;
    return by_type<RunConvStep>(p.io, p.K, &p, (unsigned)(db * p.N), (int)db, s);
}

cudaError_t launch_sum_parts(const float* part, int64_t parts, float* out0, int64_t n0, float* out1, int64_t n1,
                             float* out2, int64_t n2, cudaStream_t s, int* launches)
{
    const int64_t blocks = (n0 + n1 + n2 + 31) / 32;
    if (blocks == 0) return cudaSuccess;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    ++*launches;
    sum_parts_kernel<<<(unsigned)blocks, dim3(32, 16), 0, s>>>(part, parts, out0, n0, out1, n1, out2, n2);
    return cudaGetLastError();
}

}  // namespace rnngb
