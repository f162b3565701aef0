// Device helpers of the gated delta rule's kernels.
#pragma once

#include "delta_internal.h"
#include "ssm_tile.cuh"

namespace rnngb {
namespace delta {

constexpr int C = kDeltaChunk;
constexpr int kThreads = 256;

// The log decays' sums within a chunk, from its first step, in units of log 2.  Formed in 64 bits and kept as two fp32 parts, so
// that the difference of two sums is as exact as itself in fp32 however long the sums have grown.  A g below -1000 counts as
// -1000, whose exponential is 0 as well, and whose sums have differences.
struct Sums {
    float hi[C], lo[C];
    __device__ __forceinline__ float power(int i, int j) const { return ex2((hi[i] - hi[j]) + (lo[i] - lo[j])); }
    __device__ __forceinline__ float power(int i) const { return ex2(hi[i] + lo[i]); }
};
// Thread t < C brings step t's g (read ahead of other work; 0 past the row's end); all threads of the block call.
__device__ __forceinline__ float load_g(const View& g, int64_t n, int h, int64_t t0, int64_t len)
{
    const int t = threadIdx.x;
    return t < C && t0 + t < len ? static_cast<const float*>(g.data)[n * g.bs + (t0 + t) * g.ss + h] : 0.f;
}
__device__ __forceinline__ void form_sums(Sums& s, float g, double* carry)
{
    const int t = threadIdx.x;
    double v = 0.0;
    if (t < C) {
        v = 1.4426950408889634074 * (double)(g < -1000.f ? -1000.f : g);
        for (int o = 1; o < 32; o *= 2) {
            const double w = __shfl_up_sync(0xffffffffu, v, o);
            if ((t & 31) >= o) v += w;
        }
        if (t == 31) *carry = v;
    }
    __syncthreads();
    if (t < C) {
        if (t >= 32) v += *carry;
        s.hi[t] = (float)v;
        s.lo[t] = (float)(v - (double)s.hi[t]);
    }
    __syncthreads();
}

}  // namespace delta
}  // namespace rnngb
