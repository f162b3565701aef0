// The gated delta rule for one token of each row (the formulas stand in
// include/onnx_recurrent.h).
//
// With the state read once: from w = S^T k and z = S^T q,
//     u = beta (v - a w),   S <- a S + k u^T,   Y = scale (a z + (q.k) u)
// so the old state is all that is read, and Y does not wait for the new one.
#include "delta_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 32;                   // columns of a block, 4 a thread
constexpr int kRows = kThreads * 4 / kCols; // threads' rows: a thread has every kRows-th row of its columns
constexpr int kHeld = kDeltaMaxKey / kRows;

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(const DeltaStepParams p)
{
    __shared__ float sq[kDeltaMaxKey], sk[kDeltaMaxKey];
    __shared__ float part[2][kThreads / 32][kCols];
    __shared__ float sqk;
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H;
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK), tid = threadIdx.x;
    const int DK = p.DK, DV = p.DV, v0 = blockIdx.x * kCols;
    int64_t slot = n;
    if (p.slots) {
        slot = p.slots[n];
        if (slot < 0 || slot >= p.slots_n) {
            if (slot != -1 && tid == 0) *p.status = 2;      // RNN_ERR_INVALID_INPUT
            if (tid < kCols && v0 + tid < DV) static_cast<T*>(p.Y.data)[n * p.Y.bs + (int64_t)h * DV + v0 + tid] = from_f<T>(0.f);
            return;
        }
    }
    const int col = tid % (kCols / 4) * 4, row = tid / (kCols / 4);
    const int64_t at = (slot * p.H + h) * DK * DV;
    const bool wide = DV % 4 == 0 && v0 + col < DV && ((uintptr_t)p.state | (uintptr_t)p.state_out) % 16 == 0;
    float S[kHeld][4];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int d = row + i * kRows;
        if (d < DK && wide) {
            const float4 x = *reinterpret_cast<const float4*>(p.state + at + (int64_t)d * DV + v0 + col);
            S[i][0] = x.x, S[i][1] = x.y, S[i][2] = x.z, S[i][3] = x.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) S[i][c] = d < DK && v0 + col + c < DV ? p.state[at + (int64_t)d * DV + v0 + col + c] : 0.f;
        }
    }
    const float g = static_cast<const float*>(p.g.data)[n * p.g.bs + h], a = expf(g);
    const float beta = static_cast<const float*>(p.beta.data)[n * p.beta.bs + h];
    if (tid < kDeltaMaxKey) {
        sq[tid] = tid < DK ? to_f(static_cast<const T*>(p.Q.data)[n * p.Q.bs + (int64_t)hk * DK + tid]) : 0.f;
        sk[tid] = tid < DK ? to_f(static_cast<const T*>(p.K.data)[n * p.K.bs + (int64_t)hk * DK + tid]) : 0.f;
    }
    __syncthreads();
    float w[4] = {}, z[4] = {};
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const float k = sk[row + i * kRows], q = sq[row + i * kRows];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[c] = fmaf(k, S[i][c], w[c]);
            z[c] = fmaf(q, S[i][c], z[c]);
        }
    }
    if (tid < 32) {
        float qk = 0.f;
        for (int d = tid; d < DK; d += 32) qk = fmaf(sq[d], sk[d], qk);
        for (int o = 16; o; o /= 2) qk += __shfl_xor_sync(0xffffffffu, qk, o);
        if (tid == 0) sqk = qk;
    }
#pragma unroll
    for (int o = 16; o >= kCols / 4; o /= 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[c] += __shfl_xor_sync(0xffffffffu, w[c], o);
            z[c] += __shfl_xor_sync(0xffffffffu, z[c], o);
        }
    if (tid % 32 < kCols / 4)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            part[0][tid / 32][col + c] = w[c];
            part[1][tid / 32][col + c] = z[c];
        }
    __syncthreads();
    float u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        w[c] = z[c] = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            w[c] += part[0][i][col + c];
            z[c] += part[1][i][col + c];
        }
        const float v = v0 + col + c < DV ? to_f(static_cast<const T*>(p.V.data)[n * p.V.bs + (int64_t)h * DV + v0 + col + c]) : 0.f;
        u[c] = beta * (v - a * w[c]);
    }
    if (row == 0)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (v0 + col + c < DV)
                static_cast<T*>(p.Y.data)[n * p.Y.bs + (int64_t)h * DV + v0 + col + c] = from_f<T>(p.scale * fmaf(sqk, u[c], a * z[c]));
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int d = row + i * kRows;
        if (d >= DK) continue;
        const float k = sk[d];
#pragma unroll
        for (int c = 0; c < 4; ++c) S[i][c] = fmaf(k, u[c], a * S[i][c]);
        float* out = p.state_out + at + (int64_t)d * DV + v0 + col;
        if (wide) {
            *reinterpret_cast<float4*>(out) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (v0 + col + c < DV) out[c] = S[i][c];
        }
    }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s, int* launches)
{
    const int64_t nh = p.N * p.H, y = nh < 65535 ? nh : 65535;
    const dim3 grid((unsigned)((p.DV + kCols - 1) / kCols), (unsigned)y, (unsigned)((nh + y - 1) / y));
    if (p.io == 0) delta_step_kernel<float><<<grid, kThreads, 0, s>>>(p);
    else if (p.io == 1) delta_step_kernel<__half><<<grid, kThreads, 0, s>>>(p);
    else delta_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace rnngb
