// Single-token form of the selective state space scan (the formulas stand in
// include/onnx_recurrent.h).
//
// The states bound it: 4 bytes read and 4 written for each, against 8 operations.
// A channel's M states lie on L lanes, four (16 bytes) a lane.  A block takes
// a block of channels through ROWS rows: what does not depend on the states (delta,
// delta X, the gate) is formed first, once for a channel and row, in shared memory; then a
// lane keeps its part of A, and its states of the next AHEAD rows are on their way to
// its own places in shared memory: loads in flight are what bandwidth needs,
// and cost no registers there.  256 rows x 4096 channels x 16 states take 29 us (4.6 TB/s
// of states), 256 x 2048 x 64 56 us (4.8 TB/s); with the next rows' states in registers
// 50 to 81 us.  Also measured for the former: 4 blocks an SM 32 us, 6 32 us, 8 38 us;
// 4 rows a block 36 us, 16 34 us; 2 rows ahead 32 us, 8 35 us (6 blocks an SM).  A block's
// first loads and the last, partly filled wave of blocks hold back the rest.
#include "ssm_tile.cuh"

namespace rnngb {
namespace {

constexpr int kThreads = 256;
constexpr int E = 4;              // states of a lane

template <typename V>
__device__ __forceinline__ float ld(const View& v, int64_t n, int64_t i)
{
    return to_f(static_cast<const V*>(v.data)[n * v.bs + i]);
}

// Four states from m on of M; `vec`: in one access.
template <typename V>
__device__ __forceinline__ void load4(const V* from, int m, int M, bool vec, float (&v)[E])
{
    if (vec) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = 0.0f;
        if (m < M) load_vec<V, E>(from, v);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = m + j < M ? to_f(from[j]) : 0.0f;
    }
}

constexpr int kAhead = 4;

template <typename V, int L, int ROWS>
__global__ void __launch_bounds__(kThreads, 5) ssm_scan_step_kernel(const ScanStepParams p, int cblocks, bool vec)
{
    constexpr int CB = kThreads / L, ME = L * E, AHEAD = ROWS < kAhead ? ROWS : kAhead;
    __shared__ int64_t slots[ROWS], first[ROWS];      // -1: no state; its first value
    __shared__ float4 ring[AHEAD][kThreads];
    __shared__ float4 pre[ROWS][CB];                  // delta, delta X, Dskip X, gate
    __shared__ __align__(16) float bc[ROWS][2][ME];
    __shared__ int groups;                            // groups of channels in the block: 1 or more
    const int lane = threadIdx.x % L, m = lane * E;
    const int64_t n0 = (int64_t)(blockIdx.x / cblocks) * ROWS, c0 = (int64_t)(blockIdx.x % cblocks) * CB;
    const int rows = p.N - n0 < ROWS ? (int)(p.N - n0) : ROWS;
    const int ch = threadIdx.x / L;
    const int64_t dg = p.D / p.G, c = c0 + ch;
    const bool on = c < p.D;
    const int64_t d = on ? c : p.D - 1, g = d / dg, g0 = c0 / dg;
    if (threadIdx.x < rows) {
        int64_t slot = n0 + threadIdx.x;
        if (p.slots) {
            slot = p.slots[slot];
            if (slot < 0 || slot >= p.slots_n) {
                if (slot != -1) *p.status = 2;        // RNN_ERR_INVALID_INPUT
                slot = -1;
            }
        }
        slots[threadIdx.x] = slot;
        first[threadIdx.x] = slot * p.D * p.M;
    }
    if (threadIdx.x == 0) groups = (int)(((c0 + CB < p.D ? c0 + CB : p.D) - 1) / dg - g0) + 1;
    __syncthreads();
    // with vec, states come through the ring
    const float* from = p.H + d * p.M + m;
    float* to = p.H_out + d * p.M + m;
    auto start = [&](int r) {
        if (r < rows && first[r] >= 0 && m < p.M) cp_async16(&ring[r % AHEAD][threadIdx.x], from + first[r], 16);
        cp_async_commit();
    };
    if (vec) {
#pragma unroll
        for (int r = 0; r < AHEAD; ++r) start(r);
    }
    float a[E];
    load4(p.A + d * p.M + m, m, p.M, vec, a);
#pragma unroll
    for (int j = 0; j < E; ++j) a[j] *= kLog2e;
    for (int i = threadIdx.x; i < rows * CB; i += kThreads) {
        const int r = i / CB, k = i % CB;
        if (c0 + k >= p.D) continue;
        const int64_t n = n0 + r, at = c0 + k;
        const float x = ld<V>(p.X, n, at);
        float delta = ld<V>(p.dt, n, at) + (p.dt_bias ? p.dt_bias[at] : 0.0f);
        if (p.softplus) delta = softplus_fast(delta);
        pre[r][k] = make_float4(delta, delta * x, p.Dskip ? p.Dskip[at] * x : 0.0f, p.Z.data ? silu_fast(ld<V>(p.Z, n, at)) : 1.0f);
    }
    const bool shared_bc = groups == 1;               // else a lane reads its own group's
    if (shared_bc)
        for (int i = threadIdx.x; i < rows * 2 * ME; i += kThreads) {
            const int r = i / (2 * ME), w = i / ME % 2, k = i % ME;
            bc[r][w][k] = k < p.M ? ld<V>(w ? p.C : p.B, n0 + r, g0 * p.M + k) : 0.0f;
        }
    __syncthreads();
    V* y = static_cast<V*>(p.Y.data) + n0 * p.Y.bs + d;
    if (vec && shared_bc) {       // the ordinary case, in packed pairs and without the others' choices
        const f2 a0 = pack2(a[0], a[1]), a1 = pack2(a[2], a[3]);
        const bool mine = on && m < p.M;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (r >= rows) break;
            const int64_t at = first[r];
            const float4 v = pre[r][on ? ch : 0];
            const ulonglong2 vb = *reinterpret_cast<const ulonglong2*>(&bc[r][0][m]), vc = *reinterpret_cast<const ulonglong2*>(&bc[r][1][m]);
            cp_async_wait<AHEAD - 1>();
            ulonglong2 h = *reinterpret_cast<const ulonglong2*>(&ring[r % AHEAD][threadIdx.x]);
            const f2 delta = dup2(v.x), dx = dup2(v.y);
            h.x = fma2(decay2(delta, a0), h.x, mul2(dx, vb.x));
            h.y = fma2(decay2(delta, a1), h.y, mul2(dx, vb.y));
            if (r + AHEAD < ROWS) start(r + AHEAD);
            else cp_async_commit();
            if (mine && at >= 0) *reinterpret_cast<ulonglong2*>(to + at) = h;
            float s0, s1;
            unpack2(fma2(vc.y, h.y, mul2(vc.x, h.x)), s0, s1);
            float s = m < p.M ? s0 + s1 : 0.0f;
#pragma unroll
            for (int o = L / 2; o > 0; o /= 2) s += __shfl_xor_sync(~0u, s, o);
            if (lane == 0 && on) *y = from_f<V>(at >= 0 ? (s + v.z) * v.w : 0.0f);
            y += p.Y.bs;
        }
        cp_async_wait<0>();
        return;
    }
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        const int64_t n = n0 + r, slot = slots[r];
        float h[E] = {}, vb[E], vc[E];
        if (shared_bc) {
            load_vec<float, E>(&bc[r][0][m], vb);
            load_vec<float, E>(&bc[r][1][m], vc);
        } else {
            load4(static_cast<const V*>(p.B.data) + n * p.B.bs + g * p.M + m, m, p.M, false, vb);
            load4(static_cast<const V*>(p.C.data) + n * p.C.bs + g * p.M + m, m, p.M, false, vc);
        }
        const float4 v = pre[r][on ? ch : 0];
        if (vec) {
            cp_async_wait<AHEAD - 1>();
            if (m < p.M) load_vec<float, E>(reinterpret_cast<const float*>(&ring[r % AHEAD][threadIdx.x]), h);
        } else if (slot >= 0) {
            load4(from + first[r], m, p.M, false, h);
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            unpack2(fma2(decay2(dup2(v.x), pack2(a[j], a[j + 1])), pack2(h[j], h[j + 1]), mul2(dup2(v.y), pack2(vb[j], vb[j + 1]))), h[j],
                    h[j + 1]);
            s = fmaf(vc[j + 1], h[j + 1], fmaf(vc[j], h[j], s));
        }
        if (vec) start(r + AHEAD);
        if (on && m < p.M && slot >= 0) store_vec<float, E>(to + first[r], h, p.M - m < E ? p.M - m : E, vec);
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0 && on) y[r * p.Y.bs] = from_f<V>(slot >= 0 ? (s + v.z) * v.w : 0.0f);
    }
    if (vec) cp_async_wait<0>();
}

constexpr int64_t kMaxGrid = 0x7fffffff;

template <typename V, int L, int ROWS>
cudaError_t scan_step_rows(const ScanStepParams& p, cudaStream_t s)
{
    const int64_t cb = (p.D + kThreads / L - 1) / (kThreads / L), rows = (p.N + ROWS - 1) / ROWS;
    if (cb > kMaxGrid / rows) return cudaErrorInvalidConfiguration;
    const bool vec = p.M % E == 0 && ((uintptr_t)p.H | (uintptr_t)p.H_out | (uintptr_t)p.A) % 16 == 0;
    ssm_scan_step_kernel<V, L, ROWS><<<(unsigned)(cb * rows), kThreads, 0, s>>>(p, (int)cb, vec);
    return cudaGetLastError();
}
// Eight rows a block (fewer with few lanes, whose blocks have many channels)
// where that leaves every SM three blocks, else one.
template <typename V, int L>
cudaError_t scan_step_l(const ScanStepParams& p, cudaStream_t s)
{
    constexpr int ROWS = L >= 4 ? 8 : 4;
    const int64_t cb = (p.D + kThreads / L - 1) / (kThreads / L);
    return cb * (p.N / ROWS) >= p.sms * 3 ? scan_step_rows<V, L, ROWS>(p, s) : scan_step_rows<V, L, 1>(p, s);
}

#define BY_LANES(F, V, M, ...)                       \
    switch (ssm_lanes(M)) {                           \
    case 1: return F<V, 1>(__VA_ARGS__);             \
    case 2: return F<V, 2>(__VA_ARGS__);             \
    case 4: return F<V, 4>(__VA_ARGS__);             \
    case 8: return F<V, 8>(__VA_ARGS__);             \
    case 16: return F<V, 16>(__VA_ARGS__);           \
    default: return F<V, 32>(__VA_ARGS__);           \
    }
template <typename V>
cudaError_t scan_step_t(const ScanStepParams& p, cudaStream_t s) { BY_LANES(scan_step_l, V, p.M, p, s) }


}  // namespace

cudaError_t launch_ssm_scan_step(const ScanStepParams& p, cudaStream_t s, int* launches)
{
    ++*launches;
    return p.io == 1 ? scan_step_t<__half>(p, s) : p.io == 2 ? scan_step_t<__nv_bfloat16>(p, s) : scan_step_t<float>(p, s);
}

}  // namespace rnngb
