// Device helpers of the gated delta rule's kernels.
#pragma once

#include "delta_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace delta {

constexpr int C = kDeltaChunk;
constexpr int kThreads = 256;

// The log decays' sums within a chunk, from its first step: thread t < C has step t's g (0 past
// the row's end).  Formed in 64 bits and kept as two fp32 parts, so that the
// difference of two sums is as exact as itself in fp32 however long the sums have grown.  A g below -1000
// counts as -1000, whose exponential is 0 as well, and whose sums have differences.
struct Sums {
    float hi[C], lo[C];
    __device__ __forceinline__ float between(int i, int j) const { return (hi[i] - hi[j]) + (lo[i] - lo[j]); }
};
__device__ __forceinline__ void form_sums(Sums& s, const View& g, int64_t n, int h, int64_t t0, int64_t len, double* carry)
{
    const int t = threadIdx.x;
    double v = 0.0;
    if (t < C) {
        float x = t0 + t < len ? static_cast<const float*>(g.data)[n * g.bs + (t0 + t) * g.ss + h] : 0.f;
        v = x < -1000.f ? -1000.f : x;
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

// acc[i][j] += sum_k A[k][m0 + i] * B[k][n0 + j], both in shared memory.
template <int RM, int RN>
__device__ __forceinline__ void product(float (&acc)[RM][RN], const float* A, int lda, const float* B, int ldb, int K)
{
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float a[RM], b[RN];
#pragma unroll
        for (int i = 0; i < RM; ++i) a[i] = A[k * lda + i];
#pragma unroll
        for (int j = 0; j < RN; ++j) b[j] = B[k * ldb + j];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}
template <int RM, int RN>
__device__ __forceinline__ void clear(float (&acc)[RM][RN])
{
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) acc[i][j] = 0.f;
}

// A chunk's rows of one head, [C][d], in fp32: natural (row stride ldn) and transposed (ldt), either may
// be NULL; zeros past the row's end.
template <typename T>
__device__ __forceinline__ void load_rows(const View& v, int64_t n, int64_t t0, int64_t len, int64_t at, int d, float* nat, int ldn,
                                          float* tr, int ldt)
{
    for (int i = threadIdx.x; i < C * d; i += blockDim.x) {
        const int t = i / d, c = i - t * d;
        const float x = t0 + t < len ? to_f(static_cast<const T*>(v.data)[n * v.bs + (t0 + t) * v.ss + at + c]) : 0.f;
        if (nat) nat[t * ldn + c] = x;
        if (tr) tr[c * ldt + t] = x;
    }
}

}  // namespace delta
}  // namespace rnngb
