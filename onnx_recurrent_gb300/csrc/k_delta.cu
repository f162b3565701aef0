// The gated delta rule over sequences (the formulas stand in
// include/onnx_recurrent.h), in chunks of C = 64 steps as matrix products.
//
// With G_i the sum of the log decays of a chunk's steps up to i, S0 the state
// before it, K, Q [C, DK], V [C, DV] its keys, queries and values, b its
// betas (all sums over a chunk's own steps):
//     A_ij = b_i e^(G_i - G_j) K_i.K_j  (j < i),      T = (1 + A)^-1
//     P_ij = e^(G_i - G_j) Q_i.K_j      (j <= i)
//     U = T b (V - e^G K S0)
//     Y = scale (e^G Q S0 + P U),   S1 = e^(G_last) S0 + (e^(G_last - G) K)^T U
// which are the steps one after another: (1 + A) U = b (V - e^G K S0) is u's formula with
// the state written out.  Only S0 -> S1 is a chain; T and P are formed before it
// for all chunks at once.
#include "delta_tile.cuh"

namespace rnngb {
namespace {

using namespace delta;

// T and P of every chunk: [N][H][chunks][C][C] each, transposed (for the run) or not (for its
// gradient, with a third matrix, e^(G_i - G_j) K_i.K_j below the diagonal).
struct PrepSmem {
    float KT[kDeltaMaxKey][C + 4], QT[kDeltaMaxKey][C + 4];
    float A[C][C + 1];
    float T[C][C + 1];
    Sums sums;
    float beta[C];
    double carry;
};

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(const DeltaParams p, float* mats)
{
    extern __shared__ __align__(16) unsigned char raw[];
    PrepSmem& s = *reinterpret_cast<PrepSmem*>(raw);
    const int64_t chunk = blockIdx.x, chunks = gridDim.x;
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H;
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int64_t len = row_length(p.lens, n, p.S, p.status), t0 = chunk * C;
    if (t0 >= len) return;
    const int tid = threadIdx.x;
    load_rows<T>(p.K, n, t0, len, (int64_t)hk * p.DK, p.DK, nullptr, 0, s.KT[0], C + 4);
    load_rows<T>(p.Q, n, t0, len, (int64_t)hk * p.DK, p.DK, nullptr, 0, s.QT[0], C + 4);
    if (tid < C) s.beta[tid] = t0 + tid < len ? static_cast<const float*>(p.beta.data)[n * p.beta.bs + (t0 + tid) * p.beta.ss + h] : 0.f;
    form_sums(s.sums, p.g, n, h, t0, len, &s.carry);
    const int m0 = tid / 16 * 4, n0 = tid % 16 * 4;
    float kk[4][4], qk[4][4];
    clear(kk);
    clear(qk);
    product<4, 4>(kk, s.KT[0] + m0, C + 4, s.KT[0] + n0, C + 4, p.DK);
    product<4, 4>(qk, s.QT[0] + m0, C + 4, s.KT[0] + n0, C + 4, p.DK);
    float* outT = mats + (nh * chunks + chunk) * (GRAD ? 3 : 2) * C * C;
    float* outP = outT + C * C;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = m0 + a, j = n0 + b;
            const float d = i >= j ? expf(s.sums.between(i, j)) : 0.f;
            const float k = i > j ? d * kk[a][b] : 0.f;
            s.A[i][j] = i > j ? s.beta[i] * k : 0.f;
            const float q = i >= j ? d * qk[a][b] : 0.f;
            if (GRAD) {
                outP[i * C + j] = q;
                outP[C * C + i * C + j] = k;
            } else {
                outP[j * C + i] = q;
            }
        }
    __syncthreads();
    // a thread has a column of T: T_ij = -(sum over j <= m < i of A_im T_mj)
    if (tid < C) {
        const int j = tid;
        for (int i = 0; i < C; ++i) {
            float v = i == j ? 1.f : 0.f;
            for (int m = j; m < i; ++m) v = fmaf(-s.A[i][m], s.T[m][j], v);
            s.T[i][j] = v;
        }
    }
    __syncthreads();
    for (int i = tid; i < C * C; i += kThreads) outT[i] = GRAD ? s.T[i / C][i % C] : s.T[i % C][i / C];
}

constexpr int kBV = 32;         // columns of the state that a block has

struct RunSmem {
    float KT[kDeltaMaxKey][C + 4], QT[kDeltaMaxKey][C + 4];
    float K[C][kDeltaMaxKey + 4];
    float S[kDeltaMaxKey][kBV];
    float TT[C][C], PT[C][C];
    float R[C][kBV], U[C][kBV];
    Sums sums;
    float beta[C], first[C], last[C];
    double carry;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_run_kernel(const DeltaParams p, const float* mats)
{
    extern __shared__ __align__(16) unsigned char raw[];
    RunSmem& s = *reinterpret_cast<RunSmem*>(raw);
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H, chunks = delta_chunks(p.S);
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int v0 = blockIdx.x * kBV, tid = threadIdx.x;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int m0 = tid / 16 * 4, d0 = tid / 16 * 8, n0 = tid % 16 * 2;
    const int DK = p.DK, DV = p.DV;
    float state[8][2];
    float* U = p.saved ? p.saved + p.N * p.H * chunks * DK * DV : nullptr;
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int d = d0 + a, v = v0 + n0 + b;
            state[a][b] = p.h0 && d < DK && v < DV ? p.h0[(nh * DK + d) * DV + v] : 0.f;
            s.S[d][n0 + b] = state[a][b];
        }
    for (int i = tid; i < C * (kDeltaMaxKey + 4); i += kThreads) s.K[0][i] = 0.f;
    for (int64_t chunk = 0; chunk * C < len; ++chunk) {
        const int64_t t0 = chunk * C;
        __syncthreads();
        load_rows<T>(p.K, n, t0, len, (int64_t)hk * DK, DK, s.K[0], kDeltaMaxKey + 4, s.KT[0], C + 4);
        load_rows<T>(p.Q, n, t0, len, (int64_t)hk * DK, DK, nullptr, 0, s.QT[0], C + 4);
        const float* m = mats + (nh * chunks + chunk) * 2 * C * C;
        for (int i = tid; i < C * C; i += kThreads) {
            s.TT[0][i] = m[i];
            s.PT[0][i] = m[C * C + i];
        }
        if (tid < C)
            s.beta[tid] = t0 + tid < len ? static_cast<const float*>(p.beta.data)[n * p.beta.bs + (t0 + tid) * p.beta.ss + h] : 0.f;
        form_sums(s.sums, p.g, n, h, t0, len, &s.carry);
        if (tid < C) {
            s.first[tid] = expf(s.sums.hi[tid]);
            s.last[tid] = expf(s.sums.between(C - 1, tid));
        }
        __syncthreads();
        if (p.saved)
#pragma unroll
            for (int a = 0; a < 8; ++a)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (d0 + a < DK && v0 + n0 + b < DV)
                        p.saved[((nh * chunks + chunk) * DK + d0 + a) * DV + v0 + n0 + b] = state[a][b];
        float ks[4][2], qs[4][2], u[4][2];
        clear(ks);
        clear(qs);
        clear(u);
        product<4, 2>(ks, s.KT[0] + m0, C + 4, s.S[0] + n0, kBV, DK);
        product<4, 2>(qs, s.QT[0] + m0, C + 4, s.S[0] + n0, kBV, DK);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = m0 + a, v = v0 + n0 + b;
                const float x = t0 + t < len && v < DV
                    ? to_f(static_cast<const T*>(p.V.data)[n * p.V.bs + (t0 + t) * p.V.ss + (int64_t)h * DV + v]) : 0.f;
                s.R[t][n0 + b] = s.beta[t] * (x - s.first[t] * ks[a][b]);
            }
        __syncthreads();
        product<4, 2>(u, s.TT[0] + m0, C, s.R[0] + n0, kBV, C);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s.U[m0 + a][n0 + b] = u[a][b];
                if (U && v0 + n0 + b < DV) U[((nh * chunks + chunk) * C + m0 + a) * DV + v0 + n0 + b] = u[a][b];
            }
        __syncthreads();
        clear(ks);
        product<4, 2>(ks, s.PT[0] + m0, C, s.U[0] + n0, kBV, C);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = m0 + a, v = v0 + n0 + b;
                if (t0 + t < len && v < DV)
                    static_cast<T*>(p.Y.data)[n * p.Y.bs + (t0 + t) * p.Y.ss + (int64_t)h * DV + v] =
                        from_f<T>(p.scale * fmaf(s.first[t], qs[a][b], ks[a][b]));
                s.R[t][n0 + b] = s.last[t] * u[a][b];
            }
        __syncthreads();
        const float whole = s.first[C - 1];
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) state[a][b] *= whole;
        product<8, 2>(state, s.K[0] + d0, kDeltaMaxKey + 4, s.R[0] + n0, kBV, C);
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) s.S[d0 + a][n0 + b] = state[a][b];
    }
    if (p.hT)
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (d0 + a < DK && v0 + n0 + b < DV) p.hT[(nh * DK + d0 + a) * DV + v0 + n0 + b] = state[a][b];
    // steps past the row's end
    for (int64_t i = tid; i < (p.S - len) * kBV; i += kThreads) {
        const int64_t t = len + i / kBV;
        const int v = v0 + (int)(i % kBV);
        if (v < DV) static_cast<T*>(p.Y.data)[n * p.Y.bs + t * p.Y.ss + (int64_t)h * DV + v] = from_f<T>(0.f);
    }
}

// Rows and heads over y and z of a grid.
dim3 heads_grid(int64_t x, int64_t nh)
{
    const int64_t y = nh < 65535 ? nh : 65535;
    return dim3((unsigned)x, (unsigned)y, (unsigned)((nh + y - 1) / y));
}

template <typename T>
cudaError_t run(const DeltaParams& p, cudaStream_t st, int* launches)
{
    static std::atomic<uint64_t> prep_done{0}, run_done{0};
    cudaError_t e = allow_shared(delta_prep_kernel<T, false>, sizeof(PrepSmem), prep_done);
    if (e == cudaSuccess) e = allow_shared(delta_run_kernel<T>, sizeof(RunSmem), run_done);
    if (e != cudaSuccess) return e;
    const int64_t nh = p.N * p.H;
    if (p.S > 0) {
        delta_prep_kernel<T, false><<<heads_grid(delta_chunks(p.S), nh), kThreads, sizeof(PrepSmem), st>>>(p, p.scratch);
        ++*launches;
    }
    delta_run_kernel<T><<<heads_grid((p.DV + kBV - 1) / kBV, nh), kThreads, sizeof(RunSmem), st>>>(p, p.scratch);
    ++*launches;
    return cudaGetLastError();
}

template <typename T>
cudaError_t prep_grad(const DeltaParams& p, float* mats, cudaStream_t st, int* launches)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_shared(delta_prep_kernel<T, true>, sizeof(PrepSmem), done);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<T, true><<<heads_grid(delta_chunks(p.S), p.N * p.H), kThreads, sizeof(PrepSmem), st>>>(p, mats);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace

size_t delta_scratch_bytes(const DeltaParams& p)
{
    return sizeof(float) * (size_t)(p.N * p.H * delta_chunks(p.S)) * 2 * C * C;
}

cudaError_t launch_delta(const DeltaParams& p, cudaStream_t s, int* launches)
{
    return p.io == 0 ? run<float>(p, s, launches) : p.io == 1 ? run<__half>(p, s, launches) : run<__nv_bfloat16>(p, s, launches);
}

cudaError_t launch_delta_prep_grad(const DeltaParams& p, float* mats, cudaStream_t s, int* launches)
{
    return p.io == 0 ? prep_grad<float>(p, mats, s, launches)
         : p.io == 1 ? prep_grad<__half>(p, mats, s, launches)
                     : prep_grad<__nv_bfloat16>(p, mats, s, launches);
}

}  // namespace rnngb
