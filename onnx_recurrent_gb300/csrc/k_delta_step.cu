// The gated delta rule for one token of each row (the formulas stand in
// include/onnx_recurrent.h).
//
// With the state read once: from w = S^T k and z = S^T q,
//     u = beta (v - a w),   S <- a S + k u^T,   Y = scale (a z + (q.k) u)
// so the old state is all that is read, and Y does not wait for the new one.
//
// Bytes bound it: the states, read and written once (DK * DV * 8 bytes a row and head).  A warp has 16 columns of a head's
// state to itself, a lane 4 columns of up to 16 neighbouring keys: all its loads are in flight together and the sums over the
// keys are three rounds of shuffles, so no warp waits for another.  (Blocks of 256 threads for 32 columns, whose
// sums met in shared memory, executed five times the instructions: 256 rows, 16 heads of 128 x 128, bf16: 110 us; this 84.5, of which the bytes take 79.5.)
#include "delta_internal.h"
#include "ssm_tile.cuh"

namespace rnngb {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kCols = 16;                   // columns of a warp, 4 a lane
constexpr int kGroups = 128 / kCols;        // lanes of the same columns: 8 parts of the keys
constexpr int kHeld = kDeltaMaxKey / kGroups;
static_assert(kDeltaMaxKey == 128, "a lane brings four keys");

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(const DeltaStepParams p)
{
    // Q and K of each warp's head; a group's keys start four floats further round the banks than the last one's
    __shared__ __align__(16) float sq[kWarps][kDeltaMaxKey + 4 * kGroups], sk[kWarps][kDeltaMaxKey + 4 * kGroups];
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int DK = p.DK, DV = p.DV, v0 = (blockIdx.x * kWarps + warp) * kCols;
    if (nh >= p.N * p.H || v0 >= DV) return;
    const int64_t n = nh / p.H;
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int col = v0 + lane % (kCols / 4) * 4, group = lane / (kCols / 4);
    T* Y = static_cast<T*>(p.Y.data) + n * p.Y.bs + (int64_t)h * DV;
    int64_t slot = n;
    if (p.slots) {
        slot = p.slots[n];
        if (slot < 0 || slot >= p.slots_n) {
            if (slot != -1 && v0 == 0 && lane == 0) *p.status = 2;      // RNN_ERR_INVALID_INPUT
            if (lane < kCols && v0 + lane < DV) Y[v0 + lane] = from_f<T>(0.f);
            return;
        }
    }
    // a group has `per` keys, a multiple of four
    const int per = (DK + 4 * kGroups - 1) / (4 * kGroups) * 4, d0 = group * per;
    const int64_t at = (slot * p.H + h) * DK * (int64_t)DV + (int64_t)d0 * DV + col;
    const bool wide = DV % 4 == 0 && ((uintptr_t)p.state | (uintptr_t)p.state_out) % 16 == 0;
    f2 S[kHeld][2];
    if (wide) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < per && d0 + i < DK && col < DV) x = *reinterpret_cast<const float4*>(p.state + at + (int64_t)i * DV);
            S[i][0] = pack2(x.x, x.y);
            S[i][1] = pack2(x.z, x.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            float x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = i < per && d0 + i < DK && col + c < DV ? p.state[at + (int64_t)i * DV + c] : 0.f;
            S[i][0] = pack2(x[0], x[1]);
            S[i][1] = pack2(x[2], x[3]);
        }
    }
    const float a = expf(static_cast<const float*>(p.g.data)[n * p.g.bs + h]);
    const float beta = static_cast<const float*>(p.beta.data)[n * p.beta.bs + h];
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = col + c < DV ? to_f(static_cast<const T*>(p.V.data)[n * p.V.bs + (int64_t)h * DV + col + c]) : 0.f;
    float qk = 0.f;
    {
        const T* q = static_cast<const T*>(p.Q.data) + n * p.Q.bs + (int64_t)hk * DK;
        const T* k = static_cast<const T*>(p.K.data) + n * p.K.bs + (int64_t)hk * DK;
        float qs[4], ks[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = lane * 4 + e;
            qs[e] = d < DK ? to_f(q[d]) : 0.f;
            ks[e] = d < DK ? to_f(k[d]) : 0.f;
            qk = fmaf(qs[e], ks[e], qk);
        }
        const int to = lane * 4 / per * 4 + lane * 4;       // (past the groups' keys all are 0)
        if (to < kDeltaMaxKey + 4 * kGroups) {
            *reinterpret_cast<float4*>(&sq[warp][to]) = make_float4(qs[0], qs[1], qs[2], qs[3]);
            *reinterpret_cast<float4*>(&sk[warp][to]) = make_float4(ks[0], ks[1], ks[2], ks[3]);
        }
    }
#pragma unroll
    for (int o = 16; o; o /= 2) qk += __shfl_xor_sync(0xffffffffu, qk, o);
    __syncwarp();
    const float *gq = &sq[warp][group * (per + 4)], *gk = &sk[warp][group * (per + 4)];
    f2 w[2] = {}, z[2] = {};
#pragma unroll
    for (int i = 0; i < kHeld; i += 4) {
        if (i >= per) break;
        const float4 q4 = *reinterpret_cast<const float4*>(gq + i), k4 = *reinterpret_cast<const float4*>(gk + i);
        const float qs[4] = {q4.x, q4.y, q4.z, q4.w}, ks[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f2 k = pack2(ks[e], ks[e]), q = pack2(qs[e], qs[e]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                w[c] = fma2(k, S[i + e][c], w[c]);
                z[c] = fma2(q, S[i + e][c], z[c]);
            }
        }
    }
    float ws[4], zs[4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        unpack2(w[c], ws[2 * c], ws[2 * c + 1]);
        unpack2(z[c], zs[2 * c], zs[2 * c + 1]);
    }
#pragma unroll
    for (int o = 16; o >= kCols / 4; o /= 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            ws[c] += __shfl_xor_sync(0xffffffffu, ws[c], o);
            zs[c] += __shfl_xor_sync(0xffffffffu, zs[c], o);
        }
    float u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        u[c] = beta * (v[c] - a * ws[c]);
        if (group == 0 && col + c < DV) Y[col + c] = from_f<T>(p.scale * fmaf(qk, u[c], a * zs[c]));
    }
    const f2 aa = pack2(a, a), uu[2] = {pack2(u[0], u[1]), pack2(u[2], u[3])};
    float* out = p.state_out + at;
#pragma unroll
    for (int i = 0; i < kHeld; i += 4) {
        if (i >= per) break;
        const float4 k4 = *reinterpret_cast<const float4*>(gk + i);
        const float ks[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (d0 + i + e >= DK) break;
            const f2 k = pack2(ks[e], ks[e]);
            float x[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) unpack2(fma2(k, uu[c], mul2(aa, S[i + e][c])), x[2 * c], x[2 * c + 1]);
            if (wide) {
                if (col < DV) *reinterpret_cast<float4*>(out + (int64_t)(i + e) * DV) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col + c < DV) out[(int64_t)(i + e) * DV + c] = x[c];
            }
        }
    }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s, int* launches)
{
    const int64_t nh = p.N * p.H, y = nh < 65535 ? nh : 65535;
    const dim3 grid((unsigned)((p.DV + kWarps * kCols - 1) / (kWarps * kCols)), (unsigned)y, (unsigned)((nh + y - 1) / y));
    if (p.io == 0) delta_step_kernel<float><<<grid, kThreads, 0, s>>>(p);
    else if (p.io == 1) delta_step_kernel<__half><<<grid, kThreads, 0, s>>>(p);
    else delta_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace rnngb
