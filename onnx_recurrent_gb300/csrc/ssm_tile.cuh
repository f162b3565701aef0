// Building blocks of the scan kernels: packed pairs of fp32 values, the
// softplus and silu of an elementwise pass, and the staging of tiles of steps
// in shared memory.
#pragma once

#include "ssm_math.cuh"

namespace rnngb {

// Two fp32 values in one 64-bit register: the packed instructions take one
// issue slot for two fused multiply-adds (the pipe's rate is the same), and
// the scan's inner loop is bound by issue slots.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b)
{
    f2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
// 2^x, within 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x)
{
    float v;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
    return v;
}
__device__ __forceinline__ f2 ex2_2(f2 x)
{
    float a, b;
    unpack2(x, a, b);
    return pack2(ex2(a), ex2(b));
}
// exp(d A) of a pair, A carrying log2 e.  The hardware's 2^x is low, measured as
// means over neighbouring d A, by 0.08 to 0.13 of 2^-24 where -d A is below 0.002 and by 0.3
// to 0.5 from 0.003 on, always to the same side, and a state, which remembers
// 1 / (-d A) steps, sums that up.  A nudge of the argument, rounded with the product,
// adds 0.1 of 2^-24 back: what is left then sums up to at most 65 of 2^-24 for all -d A
// above 0.0003 (without a nudge 250 of 2^-24, at 0.0003; with three times this one,
// right for -d A around 0.1, 230 at 0.001 and 700 at 0.0003).  2^nudge rounds to 1, so
// d = 0 leaves a state as it is.
__device__ __forceinline__ f2 decay2(f2 d, f2 A) { return ex2_2(fma2(d, A, pack2(8.6e-9f, 8.6e-9f))); }
__device__ __forceinline__ float rcp(float x)
{
    float v;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + exp(v)) = max(v, 0) + log(1 + t), t = exp(-|v|) in (0, 1], with
// log(1 + t) = t P(t), P the degree-8 polynomial of least relative error on
// [0, 1] (3e-8, and 2.9 * 2^-24 with the roundings of its evaluation): it
// keeps its relative accuracy for the small t that small steps come from,
// which a logarithm of 1 + t would lose.
__device__ __forceinline__ float softplus_fast(float v)
{
    const float t = ex2(-fabsf(v) * kLog2e);
    float p = 0.0052326930941379795f;
    p = fmaf(p, t, -0.02950523979961872f);
    p = fmaf(p, t, 0.07822595536708832f);
    p = fmaf(p, t, -0.13663245737552643f);
    p = fmaf(p, t, 0.19106006622314453f);
    p = fmaf(p, t, -0.2484298199415207f);
    p = fmaf(p, t, 0.3331909775733948f);
    p = fmaf(p, t, -0.4999949336051941f);
    p = fmaf(p, t, 0.9999999403953552f);
    return fmaf(p, t, fmaxf(v, 0.0f));
}
__device__ __forceinline__ f2 dup2(float v) { return pack2(v, v); }
// The same for N pairs at once, so that a coefficient is fetched once for all.
template <int N>
__device__ __forceinline__ void softplus_pairs(f2 (&v)[N])
{
    constexpr float c[9] = {0.9999999403953552f, -0.4999949336051941f, 0.3331909775733948f,
                            -0.2484298199415207f, 0.19106006622314453f, -0.13663245737552643f,
                            0.07822595536708832f, -0.02950523979961872f, 0.0052326930941379795f};
    f2 t[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float a, b;
        unpack2(v[i], a, b);
        t[i] = pack2(ex2(-fabsf(a) * kLog2e), ex2(-fabsf(b) * kLog2e));
        v[i] = pack2(fmaxf(a, 0.0f), fmaxf(b, 0.0f));
        r[i] = dup2(c[8]);
    }
#pragma unroll
    for (int k = 7; k >= 0; --k) {
        const f2 ck = dup2(c[k]);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = fma2(r[i], t[i], ck);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fma2(r[i], t[i], v[i]);
}
// silu(v) = v / (1 + exp(-v)) of a pair.
__device__ __forceinline__ f2 silu_fast2(f2 v)
{
    float a, b;
    unpack2(add2(ex2_2(mul2(v, dup2(-kLog2e))), dup2(1.0f)), a, b);
    return mul2(v, pack2(rcp(a), rcp(b)));
}
__device__ __forceinline__ f2 sigmoid_fast2(f2 v)
{
    float a, b;
    unpack2(add2(ex2_2(mul2(v, dup2(-kLog2e))), dup2(1.0f)), a, b);
    return pack2(rcp(a), rcp(b));
}
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp(1.0f + ex2(-v * kLog2e)); }
__device__ __forceinline__ float silu_fast(float v) { return v * sigmoid_fast(v); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes)
{
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// Copies tiles of T steps x COLS values of a view to shared memory.  A block's THREADS threads each own a 16-byte piece of every
// (THREADS / pieces)-th step.  Values at or past step `live` of the tile or
// column `valid` become zeros without being read.  fast: the rows start on
// 16-byte boundaries, so the copies are asynchronous; else they are plain.
template <typename V, int T, int COLS, int THREADS>
struct Stager {
    static constexpr int EP = 16 / (int)sizeof(V);
    static constexpr int PIECES = (COLS + EP - 1) / EP;
    static constexpr int PITCH = PIECES * EP;                  // of a step in shared memory
    static constexpr int EACH = THREADS / PIECES;              // steps a pass
    static constexpr int PASSES = (T + EACH - 1) / EACH;
    static_assert(THREADS % PIECES == 0, "every thread has one piece of a step");
    __device__ __forceinline__ static int row() { return threadIdx.x / PIECES; }
    __device__ __forceinline__ static int col() { return threadIdx.x % PIECES * EP; }
    __device__ __forceinline__ static void piece(V* to, const V* src, int count, bool fast, const View& v)
    {
        if (fast) {
            cp_async16(to, count > 0 ? src : static_cast<const V*>(v.data), count > 0 ? (count < EP ? count : EP) * (int)sizeof(V) : 0);
        } else {
#pragma unroll
            for (int e = 0; e < EP; ++e) to[e] = e < count ? src[e] : from_f<V>(0.0f);
        }
    }
    // The tile of row n that starts at step t0 and column c0.
    __device__ __forceinline__ static void copy(V* dst, const View& v, int64_t n, int64_t t0, int64_t c0, int live, int valid,
                                                bool fast)
    {
        V* to = dst + row() * PITCH + col();
        const V* src = static_cast<const V*>(v.data) + (t0 + row()) * v.ss + n * v.bs + c0 + col();
        if (fast && live == T && valid >= PITCH) {       // a whole tile
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (EACH <= T || row() < T) cp_async16(to + i * EACH * PITCH, src, 16);
                src += EACH * v.ss;
            }
        } else {
            for (int i = 0; i < PASSES; ++i) {
                if (EACH <= T || row() < T) piece(to + i * EACH * PITCH, src, row() + i * EACH < live ? valid - col() : 0, fast, v);
                src += EACH * v.ss;
            }
        }
    }
};

// The same value, which the compiler takes for a new one: what is formed from
// it inside a loop is not kept in registers across the loop.
__device__ __forceinline__ int64_t anew(int64_t v)
{
    asm volatile("" : "+l"(v));
    return v;
}

// Whether the rows that a Stager takes from a view start on 16-byte
// boundaries: its address and strides, and the column blocks' starts
// (multiples of `block` elements, from multiples of `group`).
inline bool rows_aligned(const View& v, int elem, int64_t block, int64_t group)
{
    return (uintptr_t)v.data % 16 == 0 && v.ss * elem % 16 == 0 && v.bs * elem % 16 == 0 && block * elem % 16 == 0 &&
           group * elem % 16 == 0;
}

// NV neighbouring values (2 or 4) in one access, or `some` of them singly.
template <typename V, int NV>
__device__ __forceinline__ void load_vec(const V* p, float (&v)[NV])
{
    if constexpr (sizeof(V) == 4 && NV == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else if constexpr (sizeof(V) == 4) {
        const float2 q = *reinterpret_cast<const float2*>(p);
        v[0] = q.x, v[1] = q.y;
    } else {
        V raw[NV];
        if constexpr (NV == 4) *reinterpret_cast<uint2*>(raw) = *reinterpret_cast<const uint2*>(p);
        else *reinterpret_cast<unsigned*>(raw) = *reinterpret_cast<const unsigned*>(p);
#pragma unroll
        for (int e = 0; e < NV; ++e) v[e] = to_f(raw[e]);
    }
}
template <typename V, int NV>
__device__ __forceinline__ void store_vec(V* p, const float (&v)[NV], int some, bool vec)
{
    __align__(16) V raw[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) raw[e] = from_f<V>(v[e]);
    if (vec && some == NV) {
        if constexpr (sizeof(V) * NV == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(raw);
        else if constexpr (sizeof(V) * NV == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(raw);
        else *reinterpret_cast<unsigned*>(p) = *reinterpret_cast<unsigned*>(raw);
    } else {
#pragma unroll
        for (int e = 0; e < NV; ++e)
            if (e < some) p[e] = raw[e];
    }
}

template <typename V, int NV>
__device__ __forceinline__ void load_pairs(const V* p, f2 (&v)[NV / 2])
{
    float a[NV];
    load_vec<V, NV>(p, a);
#pragma unroll
    for (int e = 0; e < NV; e += 2) v[e / 2] = pack2(a[e], a[e + 1]);
}

}  // namespace rnngb
