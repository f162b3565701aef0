// Layer normalisation and its gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// A row is read once and held in registers: its mean first, then the mean square of what is left
// of each value (no difference of large sums, so rows far from zero lose nothing).  With z = (x -
// mean) rstd and w = dY W,
//     dX = rstd (w - mean(w) - z mean(w z)),   dW = sum over rows of dY z,   dbias = that of dY.
//
// Bytes bound both: each block walks rows, some at a time so that their loads are in flight together and share
// the barriers of their sums; a thread keeps the weights of its columns (and the gradient's sums over the
// rows, until they go to scratch as one of few parts that are added in order).
#include "norm_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace {

// VEC neighbouring values of a row.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
    T v[VEC];
};

// Threads of a row, values a thread holds (NV, in pieces of VEC), rows a thread has at once (R).
template <typename T_, int VEC_, int NV_, int TPR_, int R_>
struct Shape {
    using T = T_;
    static constexpr int VEC = VEC_, NV = NV_, TPR = TPR_, R = R_, PER = NV / VEC;
    static constexpr int threads = TPR < 256 ? 256 : TPR, groups = threads / TPR;
    static constexpr bool weights = NV <= 16;       // in registers
};

// The sums of a row's threads, in all of them.  `shared` must differ from the one of the sums before.
template <typename S, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*shared)[N])
{
#pragma unroll
    for (int o = 16; o; o /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (S::TPR > 32) {
        const int warp = threadIdx.x / 32, first = warp / (S::TPR / 32) * (S::TPR / 32);
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) shared[warp][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < S::TPR / 32; ++w) v[i] += shared[first + w][i];
        }
    }
}

template <typename S>
__device__ __forceinline__ void load_weights(float (&w)[S::NV], const float* from, int D, int t, float otherwise)
{
#pragma unroll
    for (int i = 0; i < S::PER; ++i)
#pragma unroll
        for (int e = 0; e < S::VEC; ++e) {
            const int c = (i * S::TPR + t) * S::VEC + e;
            w[i * S::VEC + e] = from && c < D ? from[c] : otherwise;
        }
}

template <typename S>
__global__ void __launch_bounds__(S::threads) norm_kernel(const NormParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ float sums[2][S::threads / 32][S::R];
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = p.D / S::VEC;
    float w[S::weights ? S::NV : 1], b[S::weights ? S::NV : 1];
    if constexpr (S::weights) {
        load_weights<S>(w, p.W, p.D, t, 1.f);
        load_weights<S>(b, p.bias, p.D, t, 0.f);
    }
    const float per = 1.f / (float)p.D;
    constexpr int rows = S::groups * S::R;
    for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < p.rows; r0 += (int64_t)gridDim.x * rows) {
        P x[S::R][S::PER] = {};
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            const int64_t r = r0 + group * S::R + a;
            const P* from = reinterpret_cast<const P*>(static_cast<const T*>(p.X) + r * p.xs);
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
                if (r < p.rows && i * S::TPR + t < pieces) x[a][i] = from[i * S::TPR + t];
        }
        float s[S::R], mean[S::R], rstd[S::R];
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            s[a] = 0.f;
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) s[a] += to_f(x[a][i].v[e]);
        }
        row_sums<S>(s, sums[0]);
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            mean[a] = s[a] / (float)p.D;
            s[a] = 0.f;
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
                if (i * S::TPR + t < pieces)
#pragma unroll
                    for (int e = 0; e < S::VEC; ++e) {
                        const float d = to_f(x[a][i].v[e]) - mean[a];
                        s[a] = fmaf(d, d, s[a]);
                    }
        }
        row_sums<S>(s, sums[1]);
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            const int64_t r = r0 + group * S::R + a;
            if (r >= p.rows) continue;
            rstd[a] = 1.f / sqrtf(fmaf(s[a], per, p.eps));
            if (p.stats && t == 0) {
                p.stats[2 * r] = mean[a];
                p.stats[2 * r + 1] = rstd[a];
            }
            P* to = reinterpret_cast<P*>(static_cast<T*>(p.Y) + r * p.ys);
#pragma unroll
            for (int i = 0; i < S::PER; ++i) {
                const int at = i * S::TPR + t;
                if (at >= pieces) continue;
                P q;
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) {
                    const float z = (to_f(x[a][i].v[e]) - mean[a]) * rstd[a];
                    float wi, bi;
                    if constexpr (S::weights) wi = w[i * S::VEC + e], bi = b[i * S::VEC + e];
                    else wi = p.W ? p.W[at * S::VEC + e] : 1.f, bi = p.bias ? p.bias[at * S::VEC + e] : 0.f;
                    q.v[e] = from_f<T>(fmaf(z, wi, bi));
                }
                to[at] = q;
            }
        }
    }
}

// SUMS: dW and dbias too.
template <typename S, bool SUMS>
__global__ void __launch_bounds__(S::threads) norm_grad_kernel(const NormGradParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ float sums[2][S::threads / 32][2 * S::R];
    const NormParams& f = p.f;
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = f.D / S::VEC;
    float w[S::weights ? S::NV : 1], dw[SUMS ? S::NV : 1] = {}, db[SUMS ? S::NV : 1] = {};
    if constexpr (S::weights) load_weights<S>(w, f.W, f.D, t, 1.f);
    const float per = 1.f / (float)f.D;
    constexpr int rows = S::groups * S::R;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * rows; r0 < f.rows; r0 += (int64_t)gridDim.x * rows, turn ^= 1) {
        P x[S::R][S::PER] = {}, y[S::R][S::PER] = {};
        float2 stat[S::R];
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            const int64_t r = r0 + group * S::R + a;
            const P* fx = reinterpret_cast<const P*>(static_cast<const T*>(f.X) + r * f.xs);
            const P* fy = reinterpret_cast<const P*>(static_cast<const T*>(p.dY) + r * p.dys);
            stat[a] = make_float2(r < f.rows ? f.stats[2 * r] : 0.f, r < f.rows ? f.stats[2 * r + 1] : 0.f);
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
                if (r < f.rows && i * S::TPR + t < pieces) {
                    x[a][i] = fx[i * S::TPR + t];
                    y[a][i] = fy[i * S::TPR + t];
                }
        }
        float s[2 * S::R];
        auto weight = [&](int i, int e) {
            if constexpr (S::weights) return w[i * S::VEC + e];
            else return f.W && i * S::TPR + t < pieces ? f.W[(i * S::TPR + t) * S::VEC + e] : 1.f;
        };
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            s[2 * a] = s[2 * a + 1] = 0.f;
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) {      // (past the row's end dY is 0, and z is not used but with it)
                    const float z = (to_f(x[a][i].v[e]) - stat[a].x) * stat[a].y, d = to_f(y[a][i].v[e]), g = d * weight(i, e);
                    s[2 * a] += g;
                    s[2 * a + 1] = fmaf(g, z, s[2 * a + 1]);
                    if constexpr (SUMS) {
                        dw[i * S::VEC + e] = fmaf(d, z, dw[i * S::VEC + e]);
                        db[i * S::VEC + e] += d;
                    }
                }
        }
        if (!p.dX) continue;
        row_sums<S>(s, sums[turn]);
#pragma unroll
        for (int a = 0; a < S::R; ++a) {
            const int64_t r = r0 + group * S::R + a;
            if (r >= f.rows) continue;
            const float u = s[2 * a] * per, v = s[2 * a + 1] * per;
            P* to = reinterpret_cast<P*>(static_cast<T*>(p.dX) + r * p.dxs);
#pragma unroll
            for (int i = 0; i < S::PER; ++i) {
                const int at = i * S::TPR + t;
                if (at >= pieces) continue;
                P q;
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) {
                    const float z = (to_f(x[a][i].v[e]) - stat[a].x) * stat[a].y;
                    q.v[e] = from_f<T>(stat[a].y * (to_f(y[a][i].v[e]) * weight(i, e) - u - z * v));
                }
                to[at] = q;
            }
        }
    }
    if constexpr (SUMS) {
        // groups of a block are parts of their own
        float* part = p.part + ((int64_t)blockIdx.x * S::groups + group) * 2 * f.D;
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                const int c = (i * S::TPR + t) * S::VEC + e;
                if (c < f.D) {
                    part[c] = dw[i * S::VEC + e];
                    part[f.D + c] = db[i * S::VEC + e];
                }
            }
    }
}

// Sums over a part of the rows, for rows too long to keep a thread's: a block has 32 columns and 8 rows at a time.
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

// Rows of up to this many values are walked with sums in registers.
constexpr int kWalked = 8192;
int threads_of_row(int D) { return D <= 256 ? 32 : D <= 1024 ? 128 : D <= 4096 ? 256 : D <= kWalked ? 512 : 1024; }
// Rows a block has at once; one a thread where there are too few to fill the multiprocessors otherwise.
struct Split {
    int rows;       // a thread's
    int64_t blocks;
};
Split split_of(const NormParams& p, int a_multiprocessor)
{
    const int tpr = threads_of_row(p.D), groups = tpr < 256 ? 256 / tpr : 1, most = p.D <= 2048 ? 4 : p.D <= 4096 ? 2 : 1;
    const int r = p.rows >= (int64_t)p.sms * 4 * groups * most ? most : 1;
    const int64_t blocks = (p.rows + groups * r - 1) / (groups * r), cap = (int64_t)p.sms * a_multiprocessor;
    return Split{r, blocks < cap ? blocks : cap};
}
constexpr int kRunBlocks = 8, kGradBlocks = 3;      // a multiprocessor's

template <typename S>
void go(const NormParams& p, const NormGradParams* g, int64_t blocks, cudaStream_t s)
{
    if (!g) {
        norm_kernel<S><<<(unsigned)blocks, S::threads, 0, s>>>(p);
        return;
    }
    if constexpr (S::weights) {
        if (g->part) {
            norm_grad_kernel<S, true><<<(unsigned)blocks, S::threads, 0, s>>>(*g);
            return;
        }
    }
    norm_grad_kernel<S, false><<<(unsigned)blocks, S::threads, 0, s>>>(*g);
}

template <typename T, int VEC>
void by_size(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    const Split q = split_of(p, g ? kGradBlocks : kRunBlocks);
    if (p.D <= 256) q.rows == 4 ? go<Shape<T, VEC, 8, 32, 4>>(p, g, q.blocks, s) : go<Shape<T, VEC, 8, 32, 1>>(p, g, q.blocks, s);
    else if (p.D <= 1024) q.rows == 4 ? go<Shape<T, VEC, 8, 128, 4>>(p, g, q.blocks, s) : go<Shape<T, VEC, 8, 128, 1>>(p, g, q.blocks, s);
    else if (p.D <= 2048) q.rows == 4 ? go<Shape<T, VEC, 8, 256, 4>>(p, g, q.blocks, s) : go<Shape<T, VEC, 8, 256, 1>>(p, g, q.blocks, s);
    else if (p.D <= 4096) q.rows == 2 ? go<Shape<T, VEC, 16, 256, 2>>(p, g, q.blocks, s) : go<Shape<T, VEC, 16, 256, 1>>(p, g, q.blocks, s);
    else if (p.D <= kWalked) go<Shape<T, VEC, 16, 512, 1>>(p, g, q.blocks, s);
    else go<Shape<T, VEC, 32, 1024, 1>>(p, g, q.blocks, s);
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
    if (p.f.D <= kWalked) {
        const int tpr = threads_of_row(p.f.D);
        p.parts = split_of(p.f, kGradBlocks).blocks * (tpr < 256 ? 256 / tpr : 1);
        if (p.parts < 1) p.parts = 1;
        return;
    }
    const int64_t blocks = (p.f.D + 31) / 32, want = (int64_t)p.f.sms * 8 / blocks + 1, most = (p.f.rows + 31) / 32;
    p.parts = want < most ? want : most;
    if (p.parts < 1) p.parts = 1;
}

cudaError_t launch_norm_grad(const NormGradParams& p, cudaStream_t s, int* launches)
{
    cudaError_t e = cudaSuccess;
    if (p.part && p.f.rows && p.f.D > kWalked) {
        // (first: dX may be X or dY)
        const dim3 grid((unsigned)((p.f.D + 31) / 32), (unsigned)p.parts);
        if (p.f.io == 0) norm_columns_kernel<float><<<grid, 256, 0, s>>>(p);
        else if (p.f.io == 1) norm_columns_kernel<__half><<<grid, 256, 0, s>>>(p);
        else norm_columns_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
        ++*launches;
    }
    if (p.f.rows && (p.dX || (p.part && p.f.D <= kWalked))) {
        by_type(p.f, &p, s);
        ++*launches;
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.part) return e;
    return launch_sum_parts(p.part, p.f.rows ? p.parts : 0, p.dW, p.f.D, p.dbias, p.f.D, nullptr, 0, s, launches);
}

}  // namespace rnngb
