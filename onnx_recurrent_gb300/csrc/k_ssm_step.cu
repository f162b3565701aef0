// Single-token form of the selective state space scan (the formulas stand in
// include/onnx_recurrent.h): a channel's M states lie on L lanes, four a lane.
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 128;
constexpr int E = 4;              // states of a lane

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
cudaError_t scan_step_l(const ScanStepParams& p, cudaStream_t s)
{
    const int64_t cb = (p.D + kThreads / L - 1) / (kThreads / L);
    if (cb > kMaxGrid / p.N) return cudaErrorInvalidConfiguration;
    ssm_scan_step_kernel<V, L><<<(unsigned)(cb * p.N), kThreads, 0, s>>>(p, (int)cb);
    return cudaGetLastError();
}

#define BY_LANES(F, V, M, ...)                       \
    switch (ssm_lanes(M)) {                           \
    case 1: return F<V, 1>(__VA_ARGS__);             \
    case 2: return F<V, 2>(__VA_ARGS__);             \
    case 4: return F<V, 4>(__VA_ARGS__);             \
    case 8: return F<V, 8>(__VA_ARGS__);             \
    case 16: return F<V, 16>(__VA_ARGS__);           \
    default: return F<V, 32>(__VA_ARGS__);           \
    }
template <typename V>
cudaError_t scan_step_t(const ScanStepParams& p, cudaStream_t s) { BY_LANES(scan_step_l, V, p.M, p, s) }


}  // namespace

cudaError_t launch_ssm_scan_step(const ScanStepParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    return p.io == 1 ? scan_step_t<__half>(p, s) : p.io == 2 ? scan_step_t<__nv_bfloat16>(p, s) : scan_step_t<float>(p, s);
}

}  // namespace rnngb
