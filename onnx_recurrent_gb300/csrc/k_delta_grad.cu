// Gradient of the gated delta rule, chunk by chunk (the names are those of k_delta.cu; dY' = scale
// dY, and dS1 is the slope in the state after the chunk):
//     dU  = P^T dY' + (e^(G_last - G) K) dS1,        dR = T^T dU
//     dS0 = e^G_last dS1 + (e^G Q)^T dY' - (b e^G K)^T dR
//     dV  = b dR
//     dA  = -dR U^T (below the diagonal),  dP = dY' U^T (up to it)
//     X1 = dY' S0^T,  X2 = dR S0^T,  X3 = U dS1^T
//     EA_ij = b_i e^(G_i - G_j) dA_ij,     EP_ij = e^(G_i - G_j) dP_ij
//     dQ  = e^G X1 + EP K
//     dK  = (EA + EA^T) K + EP^T Q - b e^G X2 + e^(G_last - G) X3
//     db_i = dR_i.V_i - e^G_i K_i.X2_i + sum_j dA_ij e^(G_i - G_j) K_i.K_j
// and with D_ij = EA_ij K_i.K_j + EP_ij Q_i.K_j, the slope in G_i is
//     sum_j D_ij - sum_j D_ji + e^G_i (Q_i.X1_i - b_i K_i.X2_i) - e^(G_last - G_i) K_i.X3_i
// and in G_last also  sum_j e^(G_last - G_j) K_j.X3_j + e^G_last <dS1, S0>; dg_i is their sum from
// i to the chunk's end.  Only dS1 -> dS0 is a chain: a first launch takes it and keeps every
// chunk's dS1 and dR, a second one has the rest for all chunks at once.
#include "delta_tile.cuh"

namespace rnngb {

cudaError_t launch_delta_prep_grad(const DeltaParams& p, float* mats, cudaStream_t s, int* launches);

namespace {

using namespace delta;

constexpr int kBV = 32;

struct ChainSmem {
    float KT[kDeltaMaxKey][C + 4];
    float K[C][kDeltaMaxKey + 4], Q[C][kDeltaMaxKey + 4];
    float G[kDeltaMaxKey][kBV];
    float T[C][C], P[C][C];
    float A[C][kBV], B[C][kBV];
    Sums sums;
    float beta[C], first[C], last[C];
    double carry;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_grad_chain_kernel(const DeltaGradParams q, const float* mats, float* ends, float* dRs)
{
    extern __shared__ __align__(16) unsigned char raw[];
    ChainSmem& s = *reinterpret_cast<ChainSmem*>(raw);
    const DeltaParams& p = q.f;
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H, chunks = delta_chunks(p.S);
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int v0 = blockIdx.x * kBV, tid = threadIdx.x;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int m0 = tid / 16 * 4, d0 = tid / 16 * 8, n0 = tid % 16 * 2;
    const int DK = p.DK, DV = p.DV;
    float G[8][2];
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int d = d0 + a, v = v0 + n0 + b;
            G[a][b] = q.dhT && d < DK && v < DV ? q.dhT[(nh * DK + d) * DV + v] : 0.f;
            s.G[d][n0 + b] = G[a][b];
        }
    for (int i = tid; i < C * (kDeltaMaxKey + 4); i += kThreads) s.K[0][i] = s.Q[0][i] = 0.f;
    for (int64_t chunk = (len + C - 1) / C - 1; chunk >= 0; --chunk) {
        const int64_t t0 = chunk * C;
        __syncthreads();
        load_rows<T>(p.K, n, t0, len, (int64_t)hk * DK, DK, s.K[0], kDeltaMaxKey + 4, s.KT[0], C + 4);
        load_rows<T>(p.Q, n, t0, len, (int64_t)hk * DK, DK, s.Q[0], kDeltaMaxKey + 4, nullptr, 0);
        const float* m = mats + (nh * chunks + chunk) * 3 * C * C;
        for (int i = tid; i < C * C; i += kThreads) {
            s.T[0][i] = m[i];
            s.P[0][i] = m[C * C + i];
        }
        if (tid < C)
            s.beta[tid] = t0 + tid < len ? static_cast<const float*>(p.beta.data)[n * p.beta.bs + (t0 + tid) * p.beta.ss + h] : 0.f;
        form_sums(s.sums, p.g, n, h, t0, len, &s.carry);
        if (tid < C) {
            s.first[tid] = expf(s.sums.hi[tid]);
            s.last[tid] = expf(s.sums.between(C - 1, tid));
        }
        float dy[4][2];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = m0 + a, v = v0 + n0 + b;
                dy[a][b] = t0 + t < len && v < DV
                    ? p.scale * to_f(static_cast<const T*>(q.dY.data)[n * q.dY.bs + (t0 + t) * q.dY.ss + (int64_t)h * DV + v]) : 0.f;
                s.A[t][n0 + b] = dy[a][b];
            }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (d0 + a < DK && v0 + n0 + b < DV)
                    ends[((nh * chunks + chunk) * DK + d0 + a) * DV + v0 + n0 + b] = G[a][b];
        float du[4][2], kg[4][2], dr[4][2];
        clear(du);
        clear(kg);
        clear(dr);
        product<4, 2>(du, s.P[0] + m0, C, s.A[0] + n0, kBV, C);
        product<4, 2>(kg, s.KT[0] + m0, C + 4, s.G[0] + n0, kBV, DK);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) s.B[m0 + a][n0 + b] = fmaf(s.last[m0 + a], kg[a][b], du[a][b]);
        __syncthreads();
        product<4, 2>(dr, s.T[0] + m0, C, s.B[0] + n0, kBV, C);
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = m0 + a, v = v0 + n0 + b;
                const float bt = s.beta[t], f = s.first[t];
                if (v < DV) {
                    dRs[((nh * chunks + chunk) * C + t) * DV + v] = dr[a][b];
                    if (q.dV.data && t0 + t < len)
                        static_cast<T*>(q.dV.data)[n * q.dV.bs + (t0 + t) * q.dV.ss + (int64_t)h * DV + v] = from_f<T>(bt * dr[a][b]);
                }
                s.A[t][n0 + b] = f * dy[a][b];
                s.B[t][n0 + b] = -bt * f * dr[a][b];
            }
        __syncthreads();
        const float whole = s.first[C - 1];
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) G[a][b] *= whole;
        product<8, 2>(G, s.Q[0] + d0, kDeltaMaxKey + 4, s.A[0] + n0, kBV, C);
        product<8, 2>(G, s.K[0] + d0, kDeltaMaxKey + 4, s.B[0] + n0, kBV, C);
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) s.G[d0 + a][n0 + b] = G[a][b];
    }
    if (q.dh0)
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (d0 + a < DK && v0 + n0 + b < DV) q.dh0[(nh * DK + d0 + a) * DV + v0 + n0 + b] = G[a][b];
    if (q.dV.data)
        for (int64_t i = tid; i < (p.S - len) * kBV; i += kThreads) {
            const int64_t t = len + i / kBV;
            const int v = v0 + (int)(i % kBV);
            if (v < DV) static_cast<T*>(q.dV.data)[n * q.dV.bs + t * q.dV.ss + (int64_t)h * DV + v] = from_f<T>(0.f);
        }
}

constexpr int kLd = kDeltaMaxKey + 4;
struct RestSmem {
    float K[C][kLd], Q[C][kLd], dK[C][kLd], dQ[C][kLd];
    union {
        struct {
            float dYT[kBV][C + 4], UT[kBV][C + 4], dRT[kBV][C + 4];
            float ST[kBV][kLd], GT[kBV][kLd];
        } in;
        struct {
            float EP[C][C + 4], EPT[C][C + 4], EA[C][C + 4];      // EA: with its transpose added
        } e;
    };
    Sums sums;
    float beta[C], first[C], last[C];
    float db[C], slope[C], end[C], col[16][C];
    float dot[kThreads / 32];
    double carry;
};

// Sum over the 16 threads that share a row.
__device__ __forceinline__ float row_sum(float v)
{
    for (int o = 8; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_grad_rest_kernel(const DeltaGradParams q, const float* mats, const float* ends, const float* dRs)
{
    extern __shared__ __align__(16) unsigned char raw[];
    RestSmem& s = *reinterpret_cast<RestSmem*>(raw);
    const DeltaParams& p = q.f;
    const int64_t chunk = blockIdx.x, chunks = gridDim.x, nk = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nk >= p.N * p.HK) return;
    const int64_t n = nk / p.HK;
    const int hk = (int)(nk - n * p.HK), per = p.H / p.HK, tid = threadIdx.x;
    const int64_t len = row_length(p.lens, n, p.S, p.status), t0 = chunk * C;
    const int DK = p.DK, DV = p.DV, rows = (int)(p.S - t0 < C ? p.S - t0 : C);
    const int m0 = tid / 16 * 4, n0 = tid % 16 * 4, e0 = tid % 16 * 8;
    for (int i = tid; i < C * kLd; i += kThreads) s.K[0][i] = s.Q[0][i] = s.dK[0][i] = s.dQ[0][i] = 0.f;
    __syncthreads();
    load_rows<T>(p.K, n, t0, len, (int64_t)hk * DK, DK, s.K[0], kLd, nullptr, 0);
    load_rows<T>(p.Q, n, t0, len, (int64_t)hk * DK, DK, s.Q[0], kLd, nullptr, 0);
    const bool live = t0 < len;
    for (int h = hk * per; h < (hk + 1) * per; ++h) {
        const int64_t nh = n * p.H + h, at = nh * chunks + chunk;
        __syncthreads();
        if (live) {
            if (tid < C)
                s.beta[tid] = t0 + tid < len ? static_cast<const float*>(p.beta.data)[n * p.beta.bs + (t0 + tid) * p.beta.ss + h] : 0.f;
            form_sums(s.sums, p.g, n, h, t0, len, &s.carry);
            if (tid < C) {
                s.first[tid] = expf(s.sums.hi[tid]);
                s.last[tid] = expf(s.sums.between(C - 1, tid));
            }
            float dP[4][4], dA[4][4], X1[4][8], X2[4][8], X3[4][8], rv[4] = {0.f, 0.f, 0.f, 0.f}, dot = 0.f;
            clear(dP);
            clear(dA);
            clear(X1);
            clear(X2);
            clear(X3);
            for (int v0 = 0; v0 < DV; v0 += kBV) {
                __syncthreads();
                for (int i = tid; i < C * kBV; i += kThreads) {
                    const int t = i / kBV, v = i % kBV;
                    const bool in = v0 + v < DV, step = in && t0 + t < len;
                    s.in.dYT[v][t] = step ? p.scale * to_f(static_cast<const T*>(q.dY.data)[n * q.dY.bs + (t0 + t) * q.dY.ss + (int64_t)h * DV + v0 + v]) : 0.f;
                    s.in.UT[v][t] = in ? p.saved[p.N * p.H * chunks * DK * DV + (at * C + t) * DV + v0 + v] : 0.f;
                    s.in.dRT[v][t] = in ? dRs[(at * C + t) * DV + v0 + v] : 0.f;
                }
                for (int i = tid; i < kDeltaMaxKey * kBV; i += kThreads) {
                    const int d = i / kBV, v = i % kBV;
                    const bool in = d < DK && v0 + v < DV;
                    const float a = in ? p.saved[(at * DK + d) * DV + v0 + v] : 0.f, b = in ? ends[(at * DK + d) * DV + v0 + v] : 0.f;
                    s.in.ST[v][d] = a;
                    s.in.GT[v][d] = b;
                    dot = fmaf(a, b, dot);
                }
                __syncthreads();
                product<4, 4>(dP, s.in.dYT[0] + m0, C + 4, s.in.UT[0] + n0, C + 4, kBV);
                product<4, 4>(dA, s.in.dRT[0] + m0, C + 4, s.in.UT[0] + n0, C + 4, kBV);
                product<4, 8>(X1, s.in.dYT[0] + m0, C + 4, s.in.ST[0] + e0, kLd, kBV);
                product<4, 8>(X2, s.in.dRT[0] + m0, C + 4, s.in.ST[0] + e0, kLd, kBV);
                product<4, 8>(X3, s.in.UT[0] + m0, C + 4, s.in.GT[0] + e0, kLd, kBV);
                for (int a = 0; a < 4; ++a)
                    for (int b = 0; b < 2; ++b) {
                        const int t = m0 + a, v = tid % 16 * 2 + b;
                        if (t0 + t < len && v0 + v < DV)
                            rv[a] = fmaf(s.in.dRT[v][t], to_f(static_cast<const T*>(p.V.data)[n * p.V.bs + (t0 + t) * p.V.ss + (int64_t)h * DV + v0 + v]), rv[a]);
                    }
            }
            for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (tid % 32 == 0) s.dot[tid / 32] = dot;
            __syncthreads();
            const float* P = mats + at * 3 * C * C + C * C;
            const float* KK = P + C * C;
            float col[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int i = m0 + a;
                const float b = s.beta[i], f = s.first[i], l = s.last[i];
                float db = 0.f, row = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = n0 + c;
                    const float d = i >= j ? expf(s.sums.between(i, j)) : 0.f;
                    const float da = i > j ? -dA[a][c] : 0.f, dp = i >= j ? dP[a][c] : 0.f;
                    const float kk = KK[i * C + j];
                    db = fmaf(da, kk, db);
                    const float D = fmaf(b * da, kk, dp * P[i * C + j]);
                    row += D;
                    col[c] += D;
                    s.e.EP[i][j] = s.e.EPT[j][i] = d * dp;
                    dA[a][c] = d * b * da;
                    s.e.EA[i][j] = dA[a][c];
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float k = s.K[i][e0 + c];
                    x1 = fmaf(s.Q[i][e0 + c], X1[a][c], x1);
                    x2 = fmaf(k, X2[a][c], x2);
                    x3 = fmaf(k, X3[a][c], x3);
                    X1[a][c] *= f;
                    X3[a][c] = l * X3[a][c] - b * f * X2[a][c];
                }
                db = row_sum(db + rv[a] - f * x2);
                row = row_sum(row + f * (x1 - b * x2));
                x3 = row_sum(x3) * l;
                if (tid % 16 == 0) {
                    s.db[i] = db;
                    s.slope[i] = row;
                    s.end[i] = x3;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) s.col[tid / 16][n0 + c] = col[c];
            __syncthreads();
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) dA[a][c] += s.e.EA[n0 + c][m0 + a];
            __syncthreads();
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) s.e.EA[m0 + a][n0 + c] = dA[a][c];
            __syncthreads();
            product<4, 8>(X1, s.e.EPT[0] + m0, C + 4, s.K[0] + e0, kLd, C);
            product<4, 8>(X3, s.e.EA[0] + m0, C + 4, s.K[0] + e0, kLd, C);
            product<4, 8>(X3, s.e.EP[0] + m0, C + 4, s.Q[0] + e0, kLd, C);
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    s.dQ[m0 + a][e0 + c] += X1[a][c];
                    s.dK[m0 + a][e0 + c] += X3[a][c];
                }
            // the decays' slopes, and their sums from each step to the chunk's end
            if (tid < C) {
                float v = s.slope[tid] - s.end[tid];
                for (int w = 0; w < 16; ++w) v -= s.col[w][tid];
                s.slope[tid] = v;
            }
            __syncthreads();
            if (tid < 32) {
                float all = s.end[tid] + s.end[tid + 32], d = tid < kThreads / 32 ? s.dot[tid] : 0.f;
                for (int o = 16; o; o /= 2) {
                    all += __shfl_xor_sync(0xffffffffu, all, o);
                    d += __shfl_xor_sync(0xffffffffu, d, o);
                }
                all += s.first[C - 1] * d;
                float hi = s.slope[tid + 32], lo = s.slope[tid];
                if (tid == 31) hi += all;
                for (int o = 1; o < 32; o *= 2) {
                    const float a = __shfl_down_sync(0xffffffffu, hi, o), b = __shfl_down_sync(0xffffffffu, lo, o);
                    if (tid + o < 32) {
                        hi += a;
                        lo += b;
                    }
                }
                lo += __shfl_sync(0xffffffffu, hi, 0);
                s.slope[tid] = lo;
                s.slope[tid + 32] = hi;
            }
            __syncthreads();
        }
        if (tid < rows) {
            const bool step = t0 + tid < len;
            if (q.dg.data) static_cast<float*>(q.dg.data)[n * q.dg.bs + (t0 + tid) * q.dg.ss + h] = step ? s.slope[tid] : 0.f;
            if (q.dbeta.data) static_cast<float*>(q.dbeta.data)[n * q.dbeta.bs + (t0 + tid) * q.dbeta.ss + h] = step ? s.db[tid] : 0.f;
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * DK; i += kThreads) {
        const int t = i / DK, d = i - t * DK;
        if (q.dQ.data) static_cast<T*>(q.dQ.data)[n * q.dQ.bs + (t0 + t) * q.dQ.ss + (int64_t)hk * DK + d] = from_f<T>(t0 + t < len ? s.dQ[t][d] : 0.f);
        if (q.dK.data) static_cast<T*>(q.dK.data)[n * q.dK.bs + (t0 + t) * q.dK.ss + (int64_t)hk * DK + d] = from_f<T>(t0 + t < len ? s.dK[t][d] : 0.f);
    }
}

dim3 heads_grid(int64_t x, int64_t nh)
{
    const int64_t y = nh < 65535 ? nh : 65535;
    return dim3((unsigned)x, (unsigned)y, (unsigned)((nh + y - 1) / y));
}

template <typename T>
cudaError_t run(const DeltaGradParams& q, cudaStream_t st, int* launches)
{
    static std::atomic<uint64_t> chain_done{0}, rest_done{0};
    cudaError_t e = allow_shared(delta_grad_chain_kernel<T>, sizeof(ChainSmem), chain_done);
    if (e == cudaSuccess) e = allow_shared(delta_grad_rest_kernel<T>, sizeof(RestSmem), rest_done);
    if (e != cudaSuccess) return e;
    const DeltaParams& p = q.f;
    const int64_t chunks = delta_chunks(p.S), all = p.N * p.H * chunks;
    float* mats = p.scratch;
    float* ends = mats + all * 3 * C * C;
    float* dRs = ends + all * p.DK * p.DV;
    if (p.S > 0) {
        e = launch_delta_prep_grad(p, mats, st, launches);
        if (e != cudaSuccess) return e;
    }
    delta_grad_chain_kernel<T><<<heads_grid((p.DV + kBV - 1) / kBV, p.N * p.H), kThreads, sizeof(ChainSmem), st>>>(q, mats, ends, dRs);
    ++*launches;
    if (p.S > 0 && (q.dQ.data || q.dK.data || q.dg.data || q.dbeta.data)) {
        delta_grad_rest_kernel<T><<<heads_grid(chunks, p.N * p.HK), kThreads, sizeof(RestSmem), st>>>(q, mats, ends, dRs);
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace

size_t delta_grad_scratch_bytes(const DeltaGradParams& q)
{
    const DeltaParams& p = q.f;
    return sizeof(float) * (size_t)(p.N * p.H * delta_chunks(p.S)) * (size_t)(3 * C * C + (p.DK + C) * p.DV);
}

cudaError_t launch_delta_grad(const DeltaGradParams& q, cudaStream_t s, int* launches)
{
    return q.f.io == 0 ? run<float>(q, s, launches) : q.f.io == 1 ? run<__half>(q, s, launches) : run<__nv_bfloat16>(q, s, launches);
}

}  // namespace rnngb
