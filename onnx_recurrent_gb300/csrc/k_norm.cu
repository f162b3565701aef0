// Layer normalisation and its gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// A row is read once and held in registers: its mean first, then the mean square of what is left
// of each value (no difference of large sums, so rows far from zero lose nothing).  With z = (x -
// mean) rstd and w = dY W,
//     dX = rstd (w - mean(w) - z mean(w z)),   dW = sum over rows of dY z,   dbias = that of dY.
//
// Bytes bound both.  Blocks walk rows; in the gradient a thread keeps the sums over rows of its columns, which go to
// scratch as one of few parts that are added in order.  (Several rows at once, or the next row's loads ahead, were no faster:
// the registers cost as many blocks.)
#include "norm_internal.h"
#include "ssm_math.cuh"

namespace rnngb {
namespace {

// VEC neighbouring values of a row.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
    T v[VEC];
};

// Threads of a row, and values a thread holds (NV, in pieces of VEC).
template <typename T_, int VEC_, int NV_, int TPR_>
struct Shape {
    using T = T_;
    static constexpr int VEC = VEC_, NV = NV_, TPR = TPR_, PER = NV / VEC;
    static constexpr int threads = TPR < 256 ? 256 : TPR, groups = threads / TPR;
    static constexpr bool weights = NV <= 16;         // the columns' weights stay in registers
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
        // (rows of a block do not wait for each other)
        if constexpr (S::groups > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / S::TPR), "n"(S::TPR) : "memory");
        else __syncthreads();
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

// The weights of a piece of columns, `wide`: from a 16-byte boundary.
template <int VEC>
__device__ __forceinline__ void piece_weights(float (&w)[VEC], const float* from, int c, bool wide, float otherwise)
{
    if (VEC % 4 == 0 && from && wide) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(from + c + e);
            w[e] = q.x, w[e + 1] = q.y, w[e + 2] = q.z, w[e + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = from ? from[c + e] : otherwise;
    }
}

template <typename S>
__global__ void __launch_bounds__(S::threads, S::NV == 32 && S::VEC > 1 && S::threads == 256 ? 4 : 1) norm_kernel(const NormParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ float sums[2][S::threads / 32][1];
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = p.D / S::VEC;
    float w[S::weights ? S::NV : 1], b[S::weights ? S::NV : 1];
    if constexpr (S::weights) {
        load_weights<S>(w, p.W, p.D, t, 1.f);
        load_weights<S>(b, p.bias, p.D, t, 0.f);
    }
    const bool wide = ((uintptr_t)p.W | (uintptr_t)p.bias) % 16 == 0;
    for (int64_t r0 = (int64_t)blockIdx.x * S::groups; r0 < p.rows; r0 += (int64_t)gridDim.x * S::groups) {
        const int64_t r = r0 + group;
        const bool in = r < p.rows;
        const P* from = reinterpret_cast<const P*>(static_cast<const T*>(p.X) + r * p.xs);
        P x[S::PER] = {};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
            if (in && i * S::TPR + t < pieces) x[i] = from[i * S::TPR + t];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) s[0] += to_f(x[i].v[e]);
        row_sums<S>(s, sums[0]);
        const float mean = s[0] / (float)p.D;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
            if (i * S::TPR + t < pieces)
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) {
                    const float d = to_f(x[i].v[e]) - mean;
                    s[0] = fmaf(d, d, s[0]);
                }
        row_sums<S>(s, sums[1]);
        if (!in) continue;
        const float rstd = 1.f / sqrtf(s[0] / (float)p.D + p.eps);
        if (p.stats && t == 0) {
            p.stats[2 * r] = mean;
            p.stats[2 * r + 1] = rstd;
        }
        P* to = reinterpret_cast<P*>(static_cast<T*>(p.Y) + r * p.ys);
#pragma unroll
        for (int i = 0; i < S::PER; ++i) {
            const int at = i * S::TPR + t;
            if (at >= pieces) continue;
            P q;
            float pw[S::VEC], pb[S::VEC];
            if constexpr (!S::weights) {
                piece_weights(pw, p.W, at * S::VEC, wide, 1.f);
                piece_weights(pb, p.bias, at * S::VEC, wide, 0.f);
            }
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                if constexpr (S::weights) pw[e] = w[i * S::VEC + e], pb[e] = b[i * S::VEC + e];
                q.v[e] = from_f<T>(fmaf((to_f(x[i].v[e]) - mean) * rstd, pw[e], pb[e]));
            }
            to[at] = q;
        }
    }
}

// SUMS: dW and dbias too.
template <typename S, bool SUMS>
__global__ void __launch_bounds__(S::threads) norm_grad_kernel(const NormGradParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ float sums[2][S::threads / 32][2];
    const NormParams& f = p.f;
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = f.D / S::VEC;
    float w[S::weights ? S::NV : 1], dw[SUMS ? S::NV : 1] = {}, db[SUMS ? S::NV : 1] = {};
    if constexpr (S::weights) load_weights<S>(w, f.W, f.D, t, 1.f);
    const float per = 1.f / (float)f.D;
    auto weight = [&](int i, int e) {
        if constexpr (S::weights) return w[i * S::VEC + e];
        else return f.W && i * S::TPR + t < pieces ? f.W[(i * S::TPR + t) * S::VEC + e] : 1.f;
    };
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * S::groups; r0 < f.rows; r0 += (int64_t)gridDim.x * S::groups, turn ^= 1) {
        const int64_t r = r0 + group;
        const bool in = r < f.rows;
        const P* fx = reinterpret_cast<const P*>(static_cast<const T*>(f.X) + r * f.xs);
        const P* fy = reinterpret_cast<const P*>(static_cast<const T*>(p.dY) + r * p.dys);
        P x[S::PER] = {}, y[S::PER] = {};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
            if (in && i * S::TPR + t < pieces) {
                x[i] = fx[i * S::TPR + t];
                y[i] = fy[i * S::TPR + t];
            }
        const float mean = in ? f.stats[2 * r] : 0.f, rstd = in ? f.stats[2 * r + 1] : 0.f;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {      // (past the row's end dY is 0)
                const float z = (to_f(x[i].v[e]) - mean) * rstd, d = to_f(y[i].v[e]), g = d * weight(i, e);
                s[0] += g;
                s[1] = fmaf(g, z, s[1]);
                if constexpr (SUMS) {
                    dw[i * S::VEC + e] = fmaf(d, z, dw[i * S::VEC + e]);
                    db[i * S::VEC + e] += d;
                }
            }
        if (!p.dX) continue;
        row_sums<S>(s, sums[turn]);
        if (!in) continue;
        const float u = s[0] * per, v = s[1] * per;
        P* to = reinterpret_cast<P*>(static_cast<T*>(p.dX) + r * p.dxs);
#pragma unroll
        for (int i = 0; i < S::PER; ++i) {
            const int at = i * S::TPR + t;
            if (at >= pieces) continue;
            P q;
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                const float z = (to_f(x[i].v[e]) - mean) * rstd;
                q.v[e] = from_f<T>(rstd * (to_f(y[i].v[e]) * weight(i, e) - u - z * v));
            }
            to[at] = q;
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

// Rows of up to this many values have the gradient's sums in registers.
constexpr int kWalked = 8192;
int threads_of_row(int D) { return D <= 256 ? 32 : D <= 1024 ? 128 : D <= 4096 ? 256 : D <= kWalked ? 512 : 1024; }
// Blocks that walk `rows` rows, `at_once` each, at most `cap` a multiprocessor.
int64_t blocks_of(const NormParams& p, int at_once, int cap)
{
    const int64_t blocks = (p.rows + at_once - 1) / at_once, most = (int64_t)p.sms * cap;
    return blocks < most ? blocks : most;
}
// (two rows at least a part)
int64_t grad_blocks(const NormParams& p) { return blocks_of(p, 2 * (threads_of_row(p.D) < 256 ? 256 / threads_of_row(p.D) : 1), 4); }

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

// A few rows: many threads a row, for its latency (96 rows of 2048: 3.2 us with 256 threads).  Many: 32 values a thread, their
// weights from the first-level cache, in flight together, four blocks a multiprocessor (16384 x 2048 bf16: 29 us with 64
// threads a row, 33 with three blocks; 8 values a thread with their weights in registers 42 to 50 us, whatever the rows at
// once and blocks; 64 values 39 us).  The gradient has 8 or 16
// values a thread, for its sums (the same case 51 us; 16 values and 128 threads a row, two rows a block, 86).
template <typename T, int VEC>
void by_size(const NormParams& p, const NormGradParams* g, cudaStream_t s)
{
    auto walk = [&](auto shape) {
        using S = decltype(shape);
        go<S>(p, g, g ? grad_blocks(p) : blocks_of(p, S::groups, 8), s);
    };
    if (!g && p.D > 256 && p.rows >= (int64_t)p.sms * 16) {
        if (p.D <= 1024) walk(Shape<T, VEC, 32, 32>{});
        else if (p.D <= 2048) walk(Shape<T, VEC, 32, 64>{});
        else if (p.D <= 4096) walk(Shape<T, VEC, 32, 128>{});
        else if (p.D <= 8192) walk(Shape<T, VEC, 32, 256>{});
        else walk(Shape<T, VEC, 32, 1024>{});
        return;
    }
    if (p.D <= 256) walk(Shape<T, VEC, 8, 32>{});
    else if (p.D <= 1024) walk(Shape<T, VEC, 8, 128>{});
    else if (p.D <= 2048) walk(Shape<T, VEC, 8, 256>{});
    else if (p.D <= 4096) walk(Shape<T, VEC, 16, 256>{});
    else if (p.D <= kWalked) walk(Shape<T, VEC, 16, 512>{});
    else walk(Shape<T, VEC, 32, 1024>{});
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
        p.parts = grad_blocks(p.f) * (threads_of_row(p.f.D) < 256 ? 256 / threads_of_row(p.f.D) : 1);
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
