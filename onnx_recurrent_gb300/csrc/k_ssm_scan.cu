// Selective state space scan, its gradients and its single-token form (the
// formulas stand in include/onnx_recurrent.h).
//
// A channel's M states are spread over L lanes (L a power of two), E = 4
// states a lane; states past M have A = B = C = 0 and stay 0.  Every lane
// walks the row's steps in order; y[t] is summed over the channel's lanes.
//
// Gradient, for one channel with g[t,m] the loss's slope in h[t,m],
// a = exp(delta A), p = a h[t-1] and e = dY silu(Z):
//     g[t]   = C e + a[t+1] g[t+1]
//     dX     = delta sum_m g B + Dskip e       dC = e h,  dB = delta X g
//     ddelta = sum_m g (A p + B X)             dA = sum_t delta g p
// The forward run saves h before each tile of kSsmTile steps; the gradient
// takes the tiles from the last to the first, forms a tile's a and p again
// from the saved state and then goes through its steps backwards.
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 128;
constexpr int E = 4;              // states of a lane
constexpr int T = kSsmTile;

// Lanes of a channel of M states: the power of two that holds them.
int lanes_of(int M)
{
    int l = 1;
    while (l * E < M) l *= 2;
    return l;
}

template <typename V>
__device__ __forceinline__ float ld(const View& v, int64_t t, int64_t n, int64_t i)
{
    return to_f(static_cast<const V*>(v.data)[t * v.ss + n * v.bs + i]);
}

template <int L>
__device__ __forceinline__ float sum_lanes(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Blocks take whole channels of one group: kThreads / L of them.
template <typename V, int L>
__global__ void __launch_bounds__(kThreads) ssm_scan_kernel(const ScanParams p, int cblocks)
{
    constexpr int CH = kThreads / L;
    const int lane = threadIdx.x % L;
    const int64_t n = blockIdx.x / (cblocks * p.G);
    const int g = blockIdx.x / cblocks % p.G;
    const int64_t dg = p.D / p.G;
    const int64_t c = (int64_t)(blockIdx.x % cblocks) * CH + threadIdx.x / L;
    const bool on = c < dg;
    const int64_t d = g * dg + (on ? c : 0);
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t tiles = (p.S + T - 1) / T;
    float A[E], h[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int m = lane * E + j;
        A[j] = m < p.M ? p.A[d * p.M + m] : 0.0f;
        h[j] = m < p.M && p.h0 ? p.h0[(n * p.D + d) * p.M + m] : 0.0f;
    }
    const float skip = p.Dskip ? p.Dskip[d] : 0.0f, bias = p.dt_bias ? p.dt_bias[d] : 0.0f;
    V* y = static_cast<V*>(p.Y.data) + n * p.Y.bs + d;
    for (int64_t t = 0; t < len; ++t) {
        if (p.saved && t % T == 0 && on)
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (lane * E + j < p.M) p.saved[((n * tiles + t / T) * p.D + d) * p.M + lane * E + j] = h[j];
        const float x = ld<V>(p.X, t, n, d);
        float delta = ld<V>(p.dt, t, n, d) + bias;
        if (p.softplus) delta = softplus_f(delta);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int m = lane * E + j;
            const float b = m < p.M ? ld<V>(p.B, t, n, g * p.M + m) : 0.0f;
            const float cc = m < p.M ? ld<V>(p.C, t, n, g * p.M + m) : 0.0f;
            h[j] = fmaf(expf(delta * A[j]), h[j], delta * x * b);
            s = fmaf(cc, h[j], s);
        }
        s = sum_lanes<L>(s) + skip * x;
        if (p.Z.data) s *= silu_f(ld<V>(p.Z, t, n, d));
        if (lane == 0 && on) y[t * p.Y.ss] = from_f<V>(s);
    }
    if (!on) return;
    if (lane == 0)
        for (int64_t t = len; t < p.S; ++t) y[t * p.Y.ss] = from_f<V>(0.0f);
    if (p.hT)
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (lane * E + j < p.M) p.hT[(n * p.D + d) * p.M + lane * E + j] = h[j];
}

// Scratch of the gradient: for each row the sums over its steps of dA, dDskip
// and ddt_bias, and for each channel block the sums over its channels of dB
// and dC at every step.
template <typename V, int L>
__global__ void __launch_bounds__(kThreads) ssm_scan_grad_kernel(const ScanGradParams q, int cblocks, float* steps)
{
    constexpr int CH = kThreads / L, W = kThreads / 32;
    const ScanParams& p = q.f;
    __shared__ float bc[W][T][2][L * E];
    const int lane = threadIdx.x % L, warp = threadIdx.x / 32;
    const int cb = blockIdx.x % cblocks;
    const int64_t n = blockIdx.x / (cblocks * p.G);
    const int g = blockIdx.x / cblocks % p.G;
    const int64_t dg = p.D / p.G;
    const int64_t c = (int64_t)cb * CH + threadIdx.x / L;
    const bool on = c < dg;
    const int64_t d = g * dg + (on ? c : 0);
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t tiles = (p.S + T - 1) / T;
    const float some = on ? 1.0f : 0.0f;     // channels past the group add nothing
    float A[E], ahead[E], dA[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int m = lane * E + j;
        A[j] = m < p.M ? p.A[d * p.M + m] : 0.0f;
        ahead[j] = m < p.M && q.dhT && on ? q.dhT[(n * p.D + d) * p.M + m] : 0.0f;
        dA[j] = 0.0f;
    }
    const float skip = p.Dskip ? p.Dskip[d] : 0.0f, bias = p.dt_bias ? p.dt_bias[d] : 0.0f;
    float dskip = 0.0f, dbias = 0.0f;
    for (int64_t k = (len + T - 1) / T - 1; k >= 0; --k) {
        float a[T][E], past[T][E], h[E];
#pragma unroll
        for (int j = 0; j < E; ++j)
            h[j] = lane * E + j < p.M ? p.saved[((n * tiles + k) * p.D + d) * p.M + lane * E + j] : 0.0f;
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int64_t t = k * T + i;
            float x = 0.0f, delta = 0.0f;
            if (t < len) {
                x = ld<V>(p.X, t, n, d);
                delta = ld<V>(p.dt, t, n, d) + bias;
                if (p.softplus) delta = softplus_f(delta);
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int m = lane * E + j;
                const float b = m < p.M && t < len ? ld<V>(p.B, t, n, g * p.M + m) : 0.0f;
                a[i][j] = expf(delta * A[j]);
                past[i][j] = a[i][j] * h[j];
                h[j] = fmaf(delta * x, b, past[i][j]);
            }
        }
#pragma unroll
        for (int i = T - 1; i >= 0; --i) {
            const int64_t t = k * T + i;
            float db[E], dc[E];
            float x = 0.0f, v = 0.0f, delta = 0.0f, e = 0.0f, z = 0.0f, dy = 0.0f;
            if (t < len) {
                x = ld<V>(p.X, t, n, d);
                v = ld<V>(p.dt, t, n, d) + bias;
                delta = p.softplus ? softplus_f(v) : v;
                dy = some * ld<V>(q.dY, t, n, d);
                e = dy;
                if (p.Z.data) {
                    z = ld<V>(p.Z, t, n, d);
                    e = dy * silu_f(z);
                }
            }
            float y = 0.0f, driven = 0.0f, decayed = 0.0f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int m = lane * E + j;
                const float b = m < p.M && t < len ? ld<V>(p.B, t, n, g * p.M + m) : 0.0f;
                const float cc = m < p.M && t < len ? ld<V>(p.C, t, n, g * p.M + m) : 0.0f;
                const float hj = fmaf(delta * x, b, past[i][j]);
                const float slope = fmaf(cc, e, ahead[j]);
                const float sp = slope * past[i][j];
                y = fmaf(cc, hj, y);
                driven = fmaf(slope, b, driven);
                decayed = fmaf(sp, A[j], decayed);
                dA[j] = fmaf(sp, delta, dA[j]);
                db[j] = delta * x * slope;
                dc[j] = e * hj;
                ahead[j] = a[i][j] * slope;
            }
            y = sum_lanes<L>(y) + skip * x;
            driven = sum_lanes<L>(driven);
            decayed = sum_lanes<L>(decayed);
            // over the warp's channels, which share B and C
#pragma unroll
            for (int j = 0; j < E; ++j) {
#pragma unroll
                for (int o = 16; o >= L; o /= 2) {
                    db[j] += __shfl_xor_sync(~0u, db[j], o);
                    dc[j] += __shfl_xor_sync(~0u, dc[j], o);
                }
                if (threadIdx.x % 32 < L) {
                    bc[warp][i][0][lane * E + j] = db[j];
                    bc[warp][i][1][lane * E + j] = dc[j];
                }
            }
            if (t < len && on && lane == 0) {
                float ddt = fmaf(x, driven, decayed);
                if (p.softplus) ddt *= sigmoid_f(v);
                dbias += ddt;
                dskip = fmaf(e, x, dskip);
                if (q.dX.data) static_cast<V*>(q.dX.data)[t * q.dX.ss + n * q.dX.bs + d] = from_f<V>(fmaf(delta, driven, skip * e));
                if (q.ddt.data) static_cast<V*>(q.ddt.data)[t * q.ddt.ss + n * q.ddt.bs + d] = from_f<V>(ddt);
                if (q.dZ.data) static_cast<V*>(q.dZ.data)[t * q.dZ.ss + n * q.dZ.bs + d] = from_f<V>(dy * y * silu_slope(z));
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < T * 2 * p.M; i += kThreads) {
            const int m = i % p.M, w = i / p.M % 2, at = i / p.M / 2;
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < W; ++r) s += bc[r][at][w][m];
            const int64_t t = k * T + at;
            if (t < len) steps[((((int64_t)cb * p.N + n) * p.S + t) * p.G + g) * 2 * p.M + w * p.M + m] = s;
        }
        __syncthreads();
    }
    if (!on) return;
    if (lane == 0) {
        const V zero = from_f<V>(0.0f);
        for (int64_t t = len; t < p.S; ++t) {
            if (q.dX.data) static_cast<V*>(q.dX.data)[t * q.dX.ss + n * q.dX.bs + d] = zero;
            if (q.ddt.data) static_cast<V*>(q.ddt.data)[t * q.ddt.ss + n * q.ddt.bs + d] = zero;
            if (q.dZ.data) static_cast<V*>(q.dZ.data)[t * q.dZ.ss + n * q.dZ.bs + d] = zero;
        }
    }
    float* part = q.part + n * p.D * (p.M + 2);
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int m = lane * E + j;
        if (m < p.M) {
            part[d * p.M + m] = dA[j];
            if (q.dh0) q.dh0[(n * p.D + d) * p.M + m] = ahead[j];
        }
    }
    if (lane == 0) {
        part[p.D * p.M + d] = dskip;
        part[p.D * p.M + p.D + d] = dbias;
    }
}

// dB and dC of every step: the channel blocks' sums in order, zero past a
// row's end.
template <typename V>
__global__ void __launch_bounds__(256) ssm_scan_bc_kernel(const ScanGradParams q, int cblocks, const float* steps)
{
    const ScanParams& p = q.f;
    const int64_t per = (int64_t)p.G * 2 * p.M, count = p.N * p.S * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per % p.S, n = i / per / p.S;
        const int r = (int)(i % per), g = r / (2 * p.M), w = r / p.M % 2, m = r % p.M;
        float s = 0.0f;
        if (t < row_length(p.lens, n, p.S, p.status))
            for (int cb = 0; cb < cblocks; ++cb) s += steps[cb * count + i];
        const View& v = w ? q.dC : q.dB;
        if (v.data) static_cast<V*>(v.data)[t * v.ss + n * v.bs + g * p.M + m] = from_f<V>(s);
    }
}

template <typename V, int L>
__global__ void __launch_bounds__(kThreads) ssm_scan_step_kernel(const ScanStepParams p, int cblocks)
{
    const int lane = threadIdx.x % L;
    const int64_t n = blockIdx.x / cblocks;
    const int64_t c = (int64_t)(blockIdx.x % cblocks) * (kThreads / L) + threadIdx.x / L;
    const bool on = c < p.D;
    const int64_t d = on ? c : 0;
    V* y = static_cast<V*>(p.Y.data) + n * p.Y.bs + d;
    int64_t slot = n;
    if (p.slots) {
        slot = p.slots[n];
        if (slot < 0 || slot >= p.slots_n) {      // the same for the whole block
            if (slot != -1) *p.status = 2;        // RNN_ERR_INVALID_INPUT
            if (on && lane == 0) *y = from_f<V>(0.0f);
            return;
        }
    }
    const int64_t g = d / (p.D / p.G);
    const float x = ld<V>(p.X, 0, n, d);
    float delta = ld<V>(p.dt, 0, n, d) + (p.dt_bias ? p.dt_bias[d] : 0.0f);
    if (p.softplus) delta = softplus_f(delta);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int m = lane * E + j;
        if (m < p.M && on) {
            const int64_t at = (slot * p.D + d) * p.M + m;
            const float h = fmaf(expf(delta * p.A[d * p.M + m]), p.H[at], delta * x * ld<V>(p.B, 0, n, g * p.M + m));
            p.H_out[at] = h;
            s = fmaf(ld<V>(p.C, 0, n, g * p.M + m), h, s);
        }
    }
    s = sum_lanes<L>(s) + (p.Dskip ? p.Dskip[d] : 0.0f) * x;
    if (p.Z.data) s *= silu_f(ld<V>(p.Z, 0, n, d));
    if (lane == 0 && on) *y = from_f<V>(s);
}

constexpr int64_t kMaxGrid = 0x7fffffff;

template <typename V, int L>
cudaError_t scan_l(const ScanParams& p, cudaStream_t s)
{
    const int64_t cb = (p.D / p.G + kThreads / L - 1) / (kThreads / L);
    if (cb * p.G > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    ssm_scan_kernel<V, L><<<(unsigned)(cb * p.G * p.N), kThreads, 0, s>>>(p, (int)cb);
    return cudaGetLastError();
}
template <typename V, int L>
cudaError_t scan_grad_l(const ScanGradParams& q, cudaStream_t s)
{
    const ScanParams& p = q.f;
    const int64_t cb = (p.D / p.G + kThreads / L - 1) / (kThreads / L);
    if (cb * p.G > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    float* steps = q.part + p.N * p.D * (p.M + 2);
    ssm_scan_grad_kernel<V, L><<<(unsigned)(cb * p.G * p.N), kThreads, 0, s>>>(q, (int)cb, steps);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.S == 0) return e;
    const int64_t count = p.N * p.S * p.G * 2 * p.M, blocks = (count + 255) / 256;
    ssm_scan_bc_kernel<V><<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(q, (int)cb, steps);
    return cudaGetLastError();
}
template <typename V, int L>
cudaError_t scan_step_l(const ScanStepParams& p, cudaStream_t s)
{
    const int64_t cb = (p.D + kThreads / L - 1) / (kThreads / L);
    if (cb > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    ssm_scan_step_kernel<V, L><<<(unsigned)(cb * p.N), kThreads, 0, s>>>(p, (int)cb);
    return cudaGetLastError();
}

#define BY_LANES(F, V, M, ...)                       \
    switch (lanes_of(M)) {                           \
    case 1: return F<V, 1>(__VA_ARGS__);             \
    case 2: return F<V, 2>(__VA_ARGS__);             \
    case 4: return F<V, 4>(__VA_ARGS__);             \
    case 8: return F<V, 8>(__VA_ARGS__);             \
    case 16: return F<V, 16>(__VA_ARGS__);           \
    default: return F<V, 32>(__VA_ARGS__);           \
    }
template <typename V>
cudaError_t scan_t(const ScanParams& p, cudaStream_t s) { BY_LANES(scan_l, V, p.M, p, s) }
template <typename V>
cudaError_t scan_grad_t(const ScanGradParams& p, cudaStream_t s) { BY_LANES(scan_grad_l, V, p.f.M, p, s) }
template <typename V>
cudaError_t scan_step_t(const ScanStepParams& p, cudaStream_t s) { BY_LANES(scan_step_l, V, p.M, p, s) }

}  // namespace

int64_t ssm_saved_floats(int64_t S, int64_t N, int64_t D, int64_t M) { return (S + T - 1) / T * N * D * M; }

cudaError_t launch_ssm_scan(const ScanParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    return p.io == 1 ? scan_t<__half>(p, s) : p.io == 2 ? scan_t<__nv_bfloat16>(p, s) : scan_t<float>(p, s);
}

size_t ssm_scan_grad_scratch(const ScanGradParams& q)
{
    const ScanParams& p = q.f;
    const int64_t per = kThreads / lanes_of(p.M), cb = (p.D / p.G + per - 1) / per;
    return sizeof(float) * (size_t)(p.N * p.D * (p.M + 2) + cb * p.N * p.S * p.G * 2 * p.M);
}

cudaError_t launch_ssm_scan_grad(const ScanGradParams& q, cudaStream_t s, int* launches)
{
    if (q.f.N > 0) {
        *launches += q.f.S > 0 ? 2 : 1;
        cudaError_t e = q.f.io == 1 ? scan_grad_t<__half>(q, s) : q.f.io == 2 ? scan_grad_t<__nv_bfloat16>(q, s)
                                                                              : scan_grad_t<float>(q, s);
        if (e != cudaSuccess) return e;
    }
    const int64_t D = q.f.D;
    return launch_sum_parts(q.part, q.f.N, q.dA, D * q.f.M, q.dDskip, D, q.ddt_bias, D, s, launches);
}

cudaError_t launch_ssm_scan_step(const ScanStepParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    return p.io == 1 ? scan_step_t<__half>(p, s) : p.io == 2 ? scan_step_t<__nv_bfloat16>(p, s) : scan_step_t<float>(p, s);
}

}  // namespace rnngb
