// Short causal convolution over time for each channel (the formulas stand in
// include/onnx_recurrent.h), its gradients and its single-token form.
//
// A thread takes one channel of one row and walks along a run of steps with
// the last K inputs in registers, so each input is read once (and K - 1 again
// at the start of a run).  The gradient's walk keeps the last K slopes of the
// sums as well: with pre[t] = bias + sum_j W[j] X[t-K+1+j] and
// e[t] = dY[t] f'(pre[t]),
//     dX[u] = sum_j W[j] e[u+K-1-j],   dW[j] = sum_t e[t] X[t-K+1+j],
// so after step t the walk can write dX[t-K+1].
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;          // steps of one thread's walk

template <typename T, int K>
__device__ __forceinline__ float conv_input(const ConvParams& p, int64_t n, int64_t t, int64_t d)
{
    if (t >= 0) return to_f(static_cast<const T*>(p.X.data)[t * p.X.ss + n * p.X.bs + d]);
    if (!p.h0) return 0.0f;
    return to_f(static_cast<const T*>(p.h0)[(n * (K - 1) + (t + K - 1)) * p.D + d]);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) ssm_conv_kernel(const ConvParams p, int dblocks, int runs)
{
    const int64_t d = (int64_t)(blockIdx.x % dblocks) * kThreads + threadIdx.x;
    const int64_t t0 = (int64_t)(blockIdx.x / dblocks % runs) * kRun;
    const int64_t n = blockIdx.x / dblocks / runs;
    if (d >= p.D) return;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t t1 = t0 + kRun < p.S ? t0 + kRun : p.S;
    float w[K], x[K];
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = p.W[d * K + j];
    const float b = p.bias ? p.bias[d] : 0.0f;
#pragma unroll
    for (int j = 1; j < K; ++j) x[j] = t0 < len ? conv_input<T, K>(p, n, t0 - K + j, d) : 0.0f;
    T* y = static_cast<T*>(p.Y.data) + n * p.Y.bs + d;
    for (int64_t t = t0; t < t1; ++t) {
        float v = 0.0f;
        if (t < len) {
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) x[j] = x[j + 1];
            x[K - 1] = conv_input<T, K>(p, n, t, d);
            v = b;
#pragma unroll
            for (int j = 0; j < K; ++j) v = fmaf(w[j], x[j], v);
            if (p.silu) v = silu_f(v);
        }
        y[t * p.Y.ss] = from_f<T>(v);
    }
    if (t0 == 0 && p.hT) {   // the last K-1 inputs, reaching back into the carried ones
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
            static_cast<T*>(p.hT)[(n * (K - 1) + j) * p.D + d] = from_f<T>(conv_input<T, K>(p, n, len - K + 1 + j, d));
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) ssm_conv_grad_kernel(const ConvGradParams q, int dblocks, int runs)
{
    const ConvParams& p = q.f;
    const int64_t d = (int64_t)(blockIdx.x % dblocks) * kThreads + threadIdx.x;
    const int64_t run = blockIdx.x / dblocks % runs;
    const int64_t n = blockIdx.x / dblocks / runs;
    if (d >= p.D) return;
    const int64_t t0 = run * kRun;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t t1 = t0 + kRun < p.S ? t0 + kRun : p.S;
    float w[K], x[K], e[K], dw[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        w[j] = p.W[d * K + j];
        dw[j] = e[j] = 0.0f;
        x[j] = j > 0 && t0 < len ? conv_input<T, K>(p, n, t0 - K + j, d) : 0.0f;
    }
    const float b = p.bias ? p.bias[d] : 0.0f;
    float db = 0.0f;
    const T* dy = static_cast<const T*>(q.dY.data) + n * q.dY.bs + d;
    const T* dhT = static_cast<const T*>(q.dhT);
    // slopes of the run's steps, and of the K-1 after it that its inputs reach
    for (int64_t t = t0; t < t1 + K - 1; ++t) {
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) {
            x[j] = x[j + 1];
            e[j] = e[j + 1];
        }
        x[K - 1] = e[K - 1] = 0.0f;
        if (t < len) {
            x[K - 1] = conv_input<T, K>(p, n, t, d);
            float v = b;
#pragma unroll
            for (int j = 0; j < K; ++j) v = fmaf(w[j], x[j], v);
            const float s = to_f(dy[t * q.dY.ss]);
            e[K - 1] = p.silu ? s * silu_slope(v) : s;
            if (t < t1) {
                db += e[K - 1];
#pragma unroll
                for (int j = 0; j < K; ++j) dw[j] = fmaf(e[K - 1], x[j], dw[j]);
            }
        }
        const int64_t u = t - K + 1;   // the input whose slopes are complete: e[0] belongs to step u
        if (u >= t0 || t0 == 0) {
            float g = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j) g = fmaf(w[K - 1 - j], e[j], g);
            if (dhT && u >= len - (K - 1) && u < len) g += to_f(dhT[(n * (K - 1) + (u - len + K - 1)) * p.D + d]);
            if (u >= 0) {
                if (q.dX.data) static_cast<T*>(q.dX.data)[u * q.dX.ss + n * q.dX.bs + d] = from_f<T>(g);
            } else if (q.dh0) {
                static_cast<T*>(q.dh0)[(n * (K - 1) + (u + K - 1)) * p.D + d] = from_f<T>(g);
            }
        }
    }
    if (q.part) {
        float* part = q.part + (n * runs + run) * p.D * (K + 1);
#pragma unroll
        for (int j = 0; j < K; ++j) part[d * K + j] = dw[j];
        part[p.D * K + d] = db;
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
    *y = from_f<T>(p.silu ? silu_f(v) : v);
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
    if (i < n)
        for (int64_t r = threadIdx.y; r < parts; r += 16) s += part[r * n + i];
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

template <typename T, int K>
struct RunConv {
    static cudaError_t go(const ConvParams* p, unsigned grid, int db, int runs, cudaStream_t s)
    {
        ssm_conv_kernel<T, K><<<grid, kThreads, 0, s>>>(*p, db, runs);
        return cudaGetLastError();
    }
};
template <typename T, int K>
struct RunConvGrad {
    static cudaError_t go(const ConvGradParams* p, unsigned grid, int db, int runs, cudaStream_t s)
    {
        ssm_conv_grad_kernel<T, K><<<grid, kThreads, 0, s>>>(*p, db, runs);
        return cudaGetLastError();
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

int64_t run_count(int64_t S) { return S > 0 ? (S + kRun - 1) / kRun : 1; }
constexpr int64_t kMaxGrid = 0x7fffffff;

}  // namespace

cudaError_t launch_ssm_conv(const ConvParams& p, cudaStream_t s, int* launches)
{
    const int64_t db = (p.D + kThreads - 1) / kThreads, runs = run_count(p.S);
    if (db * runs > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    ++*launches;
    return by_type<RunConv>(p.io, p.K, &p, (unsigned)(db * runs * p.N), (int)db, (int)runs, s);
}

int64_t ssm_conv_grad_parts(const ConvGradParams& p) { return p.f.N * run_count(p.f.S); }

cudaError_t launch_ssm_conv_grad(const ConvGradParams& p, cudaStream_t s, int* launches)
{
    const int64_t db = (p.f.D + kThreads - 1) / kThreads, runs = run_count(p.f.S);
    if (p.f.N > 0) {
        if (db * runs > kMaxGrid / p.f.N) return cudaErrorInvalidConfiguration;
        ++*launches;
        cudaError_t e = by_type<RunConvGrad>(p.f.io, p.f.K, &p, (unsigned)(db * runs * p.f.N), (int)db, (int)runs, s);
        if (e != cudaSuccess) return e;
    }
    if (!p.dW && !p.dbias) return cudaSuccess;
    return launch_sum_parts(p.part, p.parts, p.dW, p.f.D * p.f.K, p.dbias, p.f.D, nullptr, 0, s, launches);
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
