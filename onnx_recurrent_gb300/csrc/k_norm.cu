// Layer normalisation and its gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// A row is read once and held in registers: its mean first, then the mean square of what is left
// of each value (no difference of large sums, so rows far from zero lose nothing).  With z = (x -
// mean) rstd and w = dY W,
//     dX = rstd (w - mean(w) - z mean(w z)),   dW = sum over rows of dY z,   dbias = that of dY.
#include "norm_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace {

// VEC neighbouring values of a row.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
    T v[VEC];
};

// The sums of a row's threads, in all of them.
template <int THREADS, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*shared)[N])
{
#pragma unroll
    for (int o = 16; o; o /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (THREADS == 32) return;
    __syncthreads();
    if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) shared[threadIdx.x / 32][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.f;
        for (int w = 0; w < THREADS / 32; ++w) v[i] += shared[w][i];
    }
}

// A block of THREADS has a row; each thread PER pieces of it.
template <typename T, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormParams p)
{
    __shared__ float sums[THREADS / 32][1];
    const int64_t r = blockIdx.x;
    const Piece<T, VEC>* x = reinterpret_cast<const Piece<T, VEC>*>(static_cast<const T*>(p.X) + r * p.xs);
    const int pieces = p.D / VEC;
    float v[PER][VEC], s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = i * THREADS + threadIdx.x;
        if (at < pieces) {
            const Piece<T, VEC> q = x[at];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[0] += v[i][e] = to_f(q.v[e]);
        }
    }
    row_sums<THREADS>(s, sums);
    const float mean = s[0] / (float)p.D;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i * THREADS + threadIdx.x < pieces)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] -= mean;
                s[0] = fmaf(v[i][e], v[i][e], s[0]);
            }
    row_sums<THREADS>(s, sums);
    const float rstd = 1.f / sqrtf(s[0] / (float)p.D + p.eps);
    if (p.stats && threadIdx.x == 0) {
        p.stats[2 * r] = mean;
        p.stats[2 * r + 1] = rstd;
    }
    Piece<T, VEC>* y = reinterpret_cast<Piece<T, VEC>*>(static_cast<T*>(p.Y) + r * p.ys);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = i * THREADS + threadIdx.x;
        if (at < pieces) {
            Piece<T, VEC> q;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float w = p.W ? p.W[at * VEC + e] : 1.f, b = p.bias ? p.bias[at * VEC + e] : 0.f;
                q.v[e] = from_f<T>(fmaf(v[i][e] * rstd, w, b));
            }
            y[at] = q;
        }
    }
}

template <typename T, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormGradParams p)
{
    __shared__ float sums[THREADS / 32][2];
    const int64_t r = blockIdx.x;
    const Piece<T, VEC>* x = reinterpret_cast<const Piece<T, VEC>*>(static_cast<const T*>(p.f.X) + r * p.f.xs);
    const Piece<T, VEC>* dy = reinterpret_cast<const Piece<T, VEC>*>(static_cast<const T*>(p.dY) + r * p.dys);
    const int pieces = p.f.D / VEC;
    const float mean = p.f.stats[2 * r], rstd = p.f.stats[2 * r + 1];
    float z[PER][VEC], w[PER][VEC], s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = i * THREADS + threadIdx.x;
        if (at < pieces) {
            const Piece<T, VEC> q = x[at], d = dy[at];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                z[i][e] = (to_f(q.v[e]) - mean) * rstd;
                w[i][e] = to_f(d.v[e]) * (p.f.W ? p.f.W[at * VEC + e] : 1.f);
                s[0] += w[i][e];
                s[1] = fmaf(w[i][e], z[i][e], s[1]);
            }
        }
    }
    row_sums<THREADS>(s, sums);
    const float a = s[0] / (float)p.f.D, b = s[1] / (float)p.f.D;
    Piece<T, VEC>* dx = reinterpret_cast<Piece<T, VEC>*>(static_cast<T*>(p.dX) + r * p.dxs);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = i * THREADS + threadIdx.x;
        if (at < pieces) {
            Piece<T, VEC> q;
#pragma unroll
            for (int e = 0; e < VEC; ++e) q.v[e] = from_f<T>(rstd * (w[i][e] - a - z[i][e] * b));
            dx[at] = q;
        }
    }
}

// Column sums of a part of the rows: a block has 32 columns and 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradParams p)
{
    __shared__ float sw[8][33], sb[8][33];
    const int c = threadIdx.x % 32, lane = threadIdx.x / 32, D = p.f.D, at = blockIdx.x * 32 + c;
    const int64_t per = (p.f.rows + p.parts - 1) / p.parts, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < p.f.rows ? r0 + per : p.f.rows;
    float w = 0.f, b = 0.f;
    if (at < D)
        for (int64_t r = r0 + lane; r < r1; r += 8) {
            const float dy = to_f(static_cast<const T*>(p.dY)[r * p.dys + at]), x = to_f(static_cast<const T*>(p.f.X)[r * p.f.xs + at]);
            w = fmaf(dy, (x - p.f.stats[2 * r]) * p.f.stats[2 * r + 1], w);
            b += dy;
        }
    sw[lane][c] = w;
    sb[lane][c] = b;
    __syncthreads();
    if (lane == 0 && at < D) {
        for (int i = 1; i < 8; ++i) {
            w += sw[i][c];
            b += sb[i][c];
        }
        p.part[blockIdx.y * 2 * (int64_t)D + at] = w;
        p.part[(blockIdx.y * 2 + 1) * (int64_t)D + at] = b;
    }
}

template <typename T, int VEC, int PER, int THREADS>
void go(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    if (g) norm_grad_kernel<T, VEC, PER, THREADS><<<(unsigned)p.rows, THREADS, 0, s>>>(*g);
    else norm_kernel<T, VEC, PER, THREADS><<<(unsigned)p.rows, THREADS, 0, s>>>(p);
}

template <typename T, int VEC>
void by_size(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    const int pieces = p.D / VEC;
    constexpr int kMost = 32 / VEC;
    if (pieces <= 128) go<T, VEC, 1, 128>(p, g, s);
    else if (pieces <= 256) go<T, VEC, 1, 256>(p, g, s);
    else if (pieces <= 512) go<T, VEC, 1, 512>(p, g, s);
    else if (pieces <= 1024) go<T, VEC, 2, 512>(p, g, s);
    else if (pieces <= 512 * 4) go<T, VEC, 4, 512>(p, g, s);
    else go<T, VEC, kMost, 1024>(p, g, s);
}

template <typename T>
void by_alignment(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    uintptr_t at = (uintptr_t)p.X;
    int64_t strides = p.D | p.xs;
    if (g) {
        at |= (uintptr_t)g->dY | (uintptr_t)g->dX;
        strides |= g->dys | g->dxs;
    } else {
        at |= (uintptr_t)p.Y;
        strides |= p.ys;
    }
    if (at % 16 == 0 && strides % VEC == 0) by_size<T, VEC>(p, g, s);
    else by_size<T, 1>(p, g, s);
}

void by_type(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    if (p.io == 0) by_alignment<float>(p, g, s);
    else if (p.io == 1) by_alignment<__half>(p, g, s);
    else by_alignment<__nv_bfloat16>(p, g, s);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t s, int* launches)
{
    by_type(p, nullptr, s);
    ++*launches;
    return cudaGetLastError();
}

void norm_grad_plan(NormGradParams& p)
{
    const int64_t blocks = (p.f.D + 31) / 32, want = (int64_t)p.f.sms * 8 / blocks + 1, most = (p.f.rows + 31) / 32;
    p.parts = want < most ? want : most;
    if (p.parts < 1) p.parts = 1;
}

cudaError_t launch_norm_grad(const NormGradParams& p, cudaStream_t s, int* launches)
{
    if (p.dX && p.f.rows) {
        // what dX may overwrite is read by the column sums first
        if (!p.dW && !p.dbias) {
            by_type(p.f, &p, s);
            ++*launches;
            return cudaGetLastError();
        }
    }
    const dim3 grid((unsigned)((p.f.D + 31) / 32), (unsigned)p.parts);
    if (p.f.io == 0) norm_columns_kernel<float><<<grid, 256, 0, s>>>(p);
    else if (p.f.io == 1) norm_columns_kernel<__half><<<grid, 256, 0, s>>>(p);
    else norm_columns_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    ++*launches;
    if (p.dX && p.f.rows) {
        by_type(p.f, &p, s);
        ++*launches;
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // an output that is not wanted goes to its place in the first part, which is read by then
    return launch_sum_parts(p.part, p.parts, p.dW, p.f.D, p.dbias, p.f.D, nullptr, 0, s, launches);
}

}  // namespace rnngb
