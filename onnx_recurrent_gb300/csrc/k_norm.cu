// Layer normalisation and its gradient (the formulas stand in
// include/onnx_recurrent.h).
//
// A row is read once and held in registers: its mean first, then the mean square of what is left
// of each value, d = x - mean (no difference of large sums).  That mean is a number of 24 bits, and the sum that it came from
// has rounded: c, the mean of d, is what it is off by, and comes with the squares in one more reduction's second value.  d - c
// is then off by a few units of itself, however far the row is from zero, and so are the variance, mean(d^2) - c^2, and z
// = (d - c) rstd.  (A constant row of 2048 times 1000.1: the mean is off by 6e-5, Y was 0.02 at eps 1e-5.)  The gradient
// has mean + c, rounded, of the statistics, and finds what that is off by where it may matter (off_matters).  With w = dY W,
//     dX = rstd (w - mean(w) - z mean(w z)),   dW = sum over rows of dY z,   dbias = that of dY.
//
// Bytes bound both.  Blocks walk rows; in the gradient a thread keeps the sums over rows of its columns, which go to
// scratch as one of few parts that are added in order.  (Several rows at once, or the next row's loads ahead, were no faster:
// the registers cost as many blocks.)
#include <cfloat>

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
    static_assert(N == 1 || N == 2, "a value, or one a half of a warp");
    const int lane = threadIdx.x % 32;
    if constexpr (S::TPR == 32) {
#pragma unroll
        for (int o = 16; o; o /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {
        // Two values' first round leaves one each half of the warp: 5 exchanges in place of 10.
        float x = v[0];
        if constexpr (N == 1) {
            x += __shfl_xor_sync(0xffffffffu, x, 16);
        } else {
            const float give = lane < 16 ? v[1] : v[0];
            x = (lane < 16 ? v[0] : v[1]) + __shfl_xor_sync(0xffffffffu, give, 16);
        }
#pragma unroll
        for (int o = 8; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        constexpr int warps = S::TPR / 32;
        const int warp = threadIdx.x / 32, first = warp / warps * warps;
        if (lane % 16 == 0 && lane / 16 < N) shared[warp][lane / 16] = x;
        // (rows of a block do not wait for each other)
        if constexpr (S::groups > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / S::TPR), "n"(S::TPR) : "memory");
        else __syncthreads();
        if constexpr (warps == 32) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = shared[lane][i];
#pragma unroll
            for (int o = 16; o; o /= 2)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < warps; ++w) {
                if constexpr (N == 1) {
                    v[0] += shared[first + w][0];
                } else {
                    const float2 both = *reinterpret_cast<const float2*>(shared[first + w]);
                    v[0] += both.x;
                    v[1] += both.y;
                }
            }
        }
    }
}

// Whether what a mean that is held as one fp32 number is off by, at most 2^-24 of itself, may be more than 16 of 2^-24 in z.
__device__ __forceinline__ bool off_matters(float mean, float rstd) { return fabsf(mean) * rstd > 16.f; }

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

// (Blocks a multiprocessor: without a bound the registers of what the mean is off by cost the fourth.)
template <typename S>
__global__ void __launch_bounds__(S::threads, S::NV == 8 || (S::NV == 32 && S::VEC > 1 && S::threads == 256) ? 4 : 1) norm_kernel(const NormParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ __align__(8) float sums[S::threads / 32][1], more[S::threads / 32][2];
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = p.D / S::VEC;
    float w[S::weights ? S::NV : 1], b[S::weights ? S::NV : 1];
    if constexpr (S::weights) {
        load_weights<S>(w, p.W, p.D, t, 1.f);
        load_weights<S>(b, p.bias, p.D, t, 0.f);
    }
    const bool wide = ((uintptr_t)p.W | (uintptr_t)p.bias) % 16 == 0;
    // (32 values a thread leave no register for it: they divide)
    const float per = 1.f / (float)p.D;
    auto over_d = [&](float v) { return S::weights ? v * per : v / (float)p.D; };
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
        row_sums<S>(s, sums);
        const float mean = over_d(s[0]);
        float left[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
            if (i * S::TPR + t < pieces)
#pragma unroll
                for (int e = 0; e < S::VEC; ++e) {
                    const float d = to_f(x[i].v[e]) - mean;
                    left[0] += d;
                    left[1] = fmaf(d, d, left[1]);
                }
        row_sums<S>(left, more);
        if (!in) continue;
        const float c = over_d(left[0]), square = over_d(left[1]);
        // (squares past fp32's range: an infinite variance, as it would be without c, and z = 0; a NaN stays)
        const float var = square <= FLT_MAX ? fmaxf(square - c * c, 0.f) : square;
        const float rstd = 1.f / sqrtf(var + p.eps), off = -c * rstd;
        if (p.stats && t == 0) {
            p.stats[2 * r] = mean + c;
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
                q.v[e] = from_f<T>(fmaf(fmaf(to_f(x[i].v[e]) - mean, rstd, off), pw[e], pb[e]));
            }
            to[at] = q;
        }
    }
}

// SUMS: dW and dbias too.  (Blocks a multiprocessor as above: with three in place of four 16384 rows of 2048 in bf16 took 95 us
// for 67, with one in place of two 8192 rows of 4096 110 for 83.)
template <typename S, bool SUMS>
__global__ void __launch_bounds__(S::threads, S::NV == 8 ? 4 : S::NV == 16 && S::threads == 256 ? 2 : 1) norm_grad_kernel(const NormGradParams p)
{
    using T = typename S::T;
    using P = Piece<T, S::VEC>;
    __shared__ __align__(8) float sums[2][S::threads / 32][2];
    __shared__ float offs[2][S::threads / 32][1];
    const NormParams& f = p.f;
    const int t = threadIdx.x % S::TPR, group = threadIdx.x / S::TPR, pieces = f.D / S::VEC;
    float w[S::weights ? S::NV : 1], dw[SUMS ? S::NV : 1] = {}, db[SUMS ? S::NV : 1] = {};
    if constexpr (S::weights) load_weights<S>(w, f.W, f.D, t, 1.f);
    const float per = 1.f / (float)f.D;
    auto weight = [&](int i, int e) {
        if constexpr (S::weights) return w[i * S::VEC + e];
        else return f.W && i * S::TPR + t < pieces ? f.W[(i * S::TPR + t) * S::VEC + e] : 1.f;
    };
    int turn = 0, found = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * S::groups; r0 < f.rows; r0 += (int64_t)gridDim.x * S::groups, turn ^= 1) {
        const int64_t r = r0 + group;
        const bool in = r < f.rows;
        const float mean = in ? f.stats[2 * r] : 0.f, rstd = in ? f.stats[2 * r + 1] : 0.f;
        const P* fx = reinterpret_cast<const P*>(static_cast<const T*>(f.X) + r * f.xs);
        const P* fy = reinterpret_cast<const P*>(static_cast<const T*>(p.dY) + r * p.dys);
        P x[S::PER] = {}, y[S::PER] = {};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
            if (in && i * S::TPR + t < pieces) {
                x[i] = fx[i * S::TPR + t];
                y[i] = fy[i * S::TPR + t];
            }
        float left = 0.f;       // -c rstd
        if (off_matters(mean, rstd)) {      // (all of a row's threads, which meet here)
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < S::PER; ++i)
                if (i * S::TPR + t < pieces)
#pragma unroll
                    for (int e = 0; e < S::VEC; ++e) s[0] += to_f(x[i].v[e]) - mean;
            row_sums<S>(s, offs[found]);
            found ^= 1;
            left = -(s[0] * per) * rstd;
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < S::PER; ++i)
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {      // (past the row's end dY is 0)
                const float z = fmaf(to_f(x[i].v[e]) - mean, rstd, left), d = to_f(y[i].v[e]), g = d * weight(i, e);
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
                const float z = fmaf(to_f(x[i].v[e]) - mean, rstd, left);
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

// What the statistics' mean of a row is off by (c above), for the sums below: a block a row.
template <typename T>
__global__ void __launch_bounds__(256) norm_off_kernel(const NormGradParams p)
{
    __shared__ float sums[8];
    for (int64_t r = blockIdx.x; r < p.f.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.f.X) + r * p.f.xs;
        const float mean = p.f.stats[2 * r];
        if (!off_matters(mean, p.f.stats[2 * r + 1])) {
            if (threadIdx.x == 0) p.off[r] = 0.f;
            continue;
        }
        float s = 0.f;
        for (int c = threadIdx.x; c < p.f.D; c += 256) s += to_f(x[c]) - mean;
#pragma unroll
        for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 8; ++w) s += sums[w];
            p.off[r] = s / (float)p.f.D;
        }
        __syncthreads();
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
            w = fmaf(dy, ((x - p.f.stats[2 * r]) - p.off[r]) * p.f.stats[2 * r + 1], w);
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

// A few rows: many threads a row, for its latency (96 rows of 2048: 3.6 us with 256 threads).  Many: 32 values a thread, their
// weights from the first-level cache, in flight together, four blocks a multiprocessor (16384 x 2048 bf16: 30.5 us with 64
// threads a row; 8 values a thread with their weights in registers took 1.4 to 1.7 times as long, whatever the rows at
// once and blocks, 64 values 1.3 times, three blocks 1.1 times).  The gradient has 8 or 16
// values a thread, for its sums (the same case 52.5 us; 16 values and 128 threads a row, two rows a block, 1.7 times that).
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

size_t norm_grad_floats(const NormGradParams& p)
{
    return 2 * (size_t)(p.parts * p.f.D) + (p.f.D > kWalked ? (size_t)p.f.rows : 0);
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
        const unsigned rows = (unsigned)blocks_of(p.f, 1, 8);
        const dim3 grid((unsigned)((p.f.D + 31) / 32), (unsigned)p.parts);
        auto sums = [&](auto one) {
            using T = decltype(one);
            norm_off_kernel<T><<<rows, 256, 0, s>>>(p);
            norm_columns_kernel<T><<<grid, 256, 0, s>>>(p);
        };
        if (p.f.io == 0) sums(0.f);
        else if (p.f.io == 1) sums(__half());
        else sums(__nv_bfloat16());
        *launches += 2;
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
