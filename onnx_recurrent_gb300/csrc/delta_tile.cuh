// Device helpers of the gated delta rule's kernels.
#pragma once

#include "delta_internal.h"
#include "ssm_tile.cuh"

namespace rnngb {
namespace delta {

constexpr int C = kDeltaChunk;
constexpr int kThreads = 256;

// The log decays' sums within a chunk, from its first step, in units of log 2.  Each is two fp32 parts (48 bits), so that the
// difference of two sums is as exact as itself in fp32 however long the sums have grown.  A g below -1000 counts as -1000,
// whose exponential is 0 as well, and whose sums have differences.
//
// The hardware's 2^x is low by 0.1 to 0.5 of 2^-24, always to this side.  What enters a state or an output once may be; what
// a state is multiplied by chunk after chunk adds up over as many as it remembers.  So the whole chunk's decay, where it is
// not far from 1, is 1 and what is left of the exponential without it, whose rounding goes to both sides alike (256 chunks of
// decays of 0.005 were off by 157 of 2^-24, and are by less than 80).
struct Sums {
    float hi[C], lo[C];
    __device__ __forceinline__ float whole() const
    {
        const float x = (hi[C - 1] + lo[C - 1]) * 0.6931471805599453f;
        return x > -0.5f ? 1.f + expm1f(x) : power(C - 1);
    }
    __device__ __forceinline__ float power(int i, int j) const { return ex2((hi[i] - hi[j]) + (lo[i] - lo[j])); }
    __device__ __forceinline__ float power(int i) const { return ex2(hi[i] + lo[i]); }
};
// Thread t < C brings step t's g (read ahead of other work; 0 past the row's end); all threads of the block call.
__device__ __forceinline__ float load_g(const View& g, int64_t n, int h, int64_t t0, int64_t len)
{
    const int t = threadIdx.x;
    return t < C && t0 + t < len ? static_cast<const float*>(g.data)[n * g.bs + (t0 + t) * g.ss + h] : 0.f;
}
// (a, b) + (c, d), each a number and what its rounding left off.
__device__ __forceinline__ void add_pair(float& a, float& b, float c, float d)
{
    const float s = __fadd_rn(a, c), t = __fsub_rn(s, a);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(c, t)), __fadd_rn(b, d));
    a = __fadd_rn(s, e);
    b = __fsub_rn(e, __fsub_rn(a, s));
}
__device__ __forceinline__ void form_sums(Sums& s, float g, float2* carry)
{
    const int t = threadIdx.x;
    float a = 0.f, b = 0.f;
    if (t < C) {
        const float x = g < -1000.f ? -1000.f : g;
        a = __fmul_rn(x, kLog2e);
        b = fmaf(x, 1.925963033500888e-08f, fmaf(x, kLog2e, -a));       // log2 e, and what its rounding to fp32 left off
        for (int o = 1; o < 32; o *= 2) {
            const float c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
            if ((t & 31) >= o) add_pair(a, b, c, d);
        }
        if (t == 31) *carry = make_float2(a, b);
    }
    __syncthreads();
    if (t < C) {
        if (t >= 32) add_pair(a, b, carry->x, carry->y);
        s.hi[t] = a;
        s.lo[t] = b;
    }
    __syncthreads();
}

}  // namespace delta
}  // namespace rnngb
