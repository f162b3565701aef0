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
#include "delta_mma.cuh"

namespace rnngb {
namespace {

using namespace delta;

template <int DKB, int KP>
struct PrepSmem {
    union {
        unsigned char KQ[2 * KP * DKB * kBlock];
        unsigned char P[2 * kBlock];        // once K and Q are done with
    };
    alignas(16) float A[C][C + 4], T[C][C + 4];     // (X, a product amid T's, lies above A's diagonal)
    float ek[C], eq[C], beta[C];
    alignas(16) float fac[768];
    Sums sums;
    float2 carry;
};

// T and P, the factors, and K and Q as the second launch wants them.  A block has a chunk of a head.  The two products
// [K; Q] K^T are small (a twentieth of all); they go through the warps' own matrix instructions.  T is
// found by blocks: four of 16 by substitution, a thread a column, then twice T21 = -T22 (A21 T11).
// Instruction issue bounds it, and its eight barriers: 4096 chunks of 64 x 128 in bf16 take 157 us, 0.36 GB at 2.3 TB/s, with
// three blocks a multiprocessor (75 KB of shared memory each).
template <typename T, int DKB, int KP>
__global__ void __launch_bounds__(kThreads, 3) delta_prep_kernel(const DeltaParams p, unsigned char* keys, unsigned char* mats)
{
    extern __shared__ __align__(1024) unsigned char raw[];
    using S = PrepSmem<DKB, KP>;
    S& s = *reinterpret_cast<S*>(raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u));
    const int64_t chunk = blockIdx.x, chunks = gridDim.x;
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H;
    const int per = p.H / p.HK, h = (int)(nh - n * p.H), hk = h / per;
    const int64_t len = row_length(p.lens, n, p.S, p.status), t0 = chunk * C;
    if (t0 >= len) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    {
        const float g = load_g(p.g, n, h, t0, len);
        const bool kw = fours<T>(p.K, p.DK), qw = fours<T>(p.Q, p.DK);
        float k[8][4], q[8][4];
        const int64_t t = t0 + warp * 8;
        auto in = [&](int a) { return t + a < len; };
        const int64_t at = n * p.K.bs + t * p.K.ss + (int64_t)hk * p.DK, qt = n * p.Q.bs + t * p.Q.ss + (int64_t)hk * p.DK;
        load_fours<8>(static_cast<const T*>(p.K.data) + at, p.K.ss, p.DK, kw, in, k);
        load_fours<8>(static_cast<const T*>(p.Q.data) + qt, p.Q.ss, p.DK, qw, in, q);
        if (tid < C) s.beta[tid] = t0 + tid < len ? static_cast<const float*>(p.beta.data)[n * p.beta.bs + (t0 + tid) * p.beta.ss + h] : 0.f;
        form_sums(s.sums, g, &s.carry);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Scale ek = scale_of(row_most(k[i])), eq = scale_of(row_most(q[i]));
            put_row<DKB, KP>(s.KQ, 2 * kBlock, warp * 8 + i, k[i], ek.down);
            put_row<DKB, KP>(s.KQ + kBlock, 2 * kBlock, warp * 8 + i, q[i], eq.down);
            if (lane == 0) s.ek[warp * 8 + i] = ek.up, s.eq[warp * 8 + i] = eq.up;
        }
    }
    __syncthreads();
    if (h % per == 0) {
        uint4* out = reinterpret_cast<uint4*>(keys + ((n * p.HK + hk) * chunks + chunk) * Images<DKB, KP>::keys);
        for (int i = tid; i < (int)Images<DKB, KP>::keys / 16; i += kThreads) out[i] = reinterpret_cast<const uint4*>(s.KQ)[i];
    }
    // warps 0 .. 3: 16 rows of K K^T each; 4 .. 7: of Q K^T
    const int rows = warp % 4 * 16;
    float c[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
    const unsigned a0 = smem_addr(s.KQ) + (warp < 4 ? 0 : kBlock), b0 = smem_addr(s.KQ);
#pragma unroll
    for (int ks = 0; ks < DKB * 4; ++ks) {
        const unsigned blk = ks / 4 * 2 * kBlock;
        const int col = ks % 4 * 16;
        unsigned a[KP][4];
#pragma unroll
        for (int q = 0; q < KP; ++q)
            ld_matrix(a[q], a0 + q * DKB * 2 * kBlock + blk + swizzled(rows + lane % 16, col + lane / 16 * 8));
#pragma unroll
        for (int j = 0; j < 4; ++j) {       // 16 columns
            if (j * 16 > rows) continue;    // above the diagonal
#pragma unroll
            for (int q = 0; q < KP; ++q) {
                unsigned b[4];
                ld_matrix(b, b0 + q * DKB * 2 * kBlock + blk + swizzled(j * 16 + lane % 8 + lane / 16 * 8, col + lane / 8 % 2 * 8));
#pragma unroll
                for (int r = 0; r + q < KP; ++r) {
                    mma_sync(c[2 * j], a[r], b[0], b[1]);
                    mma_sync(c[2 * j + 1], a[r], b[2], b[3]);
                }
            }
        }
    }
    __syncthreads();        // (and written out)
    const float* er = warp < 4 ? s.ek : s.eq;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = rows + lane / 4 + half * 8;
        float m = 0.f;
#pragma unroll
        for (int j8 = 0; j8 < 8; ++j8) {
            if (j8 * 8 > rows + 15) continue;       // above the diagonal, where c is 0
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = j8 * 8 + lane % 4 * 2 + e;
                const bool in = j < i || (j == i && warp >= 4);
                const float v = in ? s.sums.power(i, j) * (c[j8][half * 2 + e] * er[i] * s.ek[j]) : 0.f;
                if (warp < 4 && in) s.A[i][j] = s.beta[i] * v;
                c[j8][half * 2 + e] = v;
                m = fmaxf(m, fabsf(v));
            }
        }
        if (warp >= 4) {
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const Scale sc = scale_of(m);
            if (lane % 4 == 0) s.fac[kP + i] = p.scale * sc.up;
#pragma unroll
            for (int j8 = 0; j8 < 8; ++j8) {
                unsigned hi, lo;
                split_pair(c[j8][half * 2] * sc.down, c[j8][half * 2 + 1] * sc.down, hi, lo);
                unsigned char* at = s.P + swizzled(i, j8 * 8 + lane % 4 * 2);
                *reinterpret_cast<unsigned*>(at) = hi;
                *reinterpret_cast<unsigned*>(at + kBlock) = lo;
            }
        }
    }
    if (tid < C) {
        const float first = s.sums.power(tid);
        s.fac[kBeta + tid] = s.beta[tid];
        s.fac[kDecayed + tid] = s.beta[tid] * first * s.ek[tid];
        s.fac[kLast + tid] = s.sums.power(C - 1, tid) * s.ek[tid];
        s.fac[kQuery + tid] = p.scale * first * s.eq[tid];
        s.fac[kKeyScale + tid] = s.ek[tid];
        s.fac[kQueryScale + tid] = s.eq[tid];
        if (tid == C - 1) s.fac[kWhole] = s.sums.whole();
    }
    __syncthreads();
    if (tid < C) {
        const int b = tid / 16 * 16, j = tid % 16;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            t[i] = i == j ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) t[i] = fmaf(-s.A[b + i][b + m], t[m], t[i]);
            s.T[b + i][b + j] = t[i];
        }
    }
    __syncthreads();
    auto X = [&](int i, int j) { return &s.A[i][32 + j]; };
    {   // two pairs of blocks of 16
        const int at = tid / 128 * 32, i = tid % 128 / 8, j = tid % 8 * 2;
        float x[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 a4 = *reinterpret_cast<const float4*>(&s.A[at + 16 + i][at + m]);
            const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 t = *reinterpret_cast<const float2*>(&s.T[at + m + e][at + j]);
                x[0] = fmaf(a[e], t.x, x[0]);
                x[1] = fmaf(a[e], t.y, x[1]);
            }
        }
        *reinterpret_cast<float2*>(X(at / 2 + i, j)) = make_float2(x[0], x[1]);
        __syncthreads();
        x[0] = x[1] = 0.f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 a4 = *reinterpret_cast<const float4*>(&s.T[at + 16 + i][at + 16 + m]);
            const float a[4] = {-a4.x, -a4.y, -a4.z, -a4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 t = *reinterpret_cast<const float2*>(X(at / 2 + m + e, j));
                x[0] = fmaf(a[e], t.x, x[0]);
                x[1] = fmaf(a[e], t.y, x[1]);
            }
        }
        *reinterpret_cast<float2*>(&s.T[at + 16 + i][at + j]) = make_float2(x[0], x[1]);
        *reinterpret_cast<float2*>(&s.T[at + i][at + 16 + j]) = make_float2(0.f, 0.f);
    }
    __syncthreads();
    {   // the two of 32
        const int i = tid / 8, j = tid % 8 * 4;
        float x[4] = {};
        auto add = [&](const float4& a4, float sign, auto row) {
            const float a[4] = {sign * a4.x, sign * a4.y, sign * a4.z, sign * a4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 t = *reinterpret_cast<const float4*>(row(e));
                x[0] = fmaf(a[e], t.x, x[0]);
                x[1] = fmaf(a[e], t.y, x[1]);
                x[2] = fmaf(a[e], t.z, x[2]);
                x[3] = fmaf(a[e], t.w, x[3]);
            }
        };
#pragma unroll 2
        for (int m = 0; m < 32; m += 4) add(*reinterpret_cast<const float4*>(&s.A[32 + i][m]), 1.f, [&](int e) { return &s.T[m + e][j]; });
        *reinterpret_cast<float4*>(X(i, j)) = make_float4(x[0], x[1], x[2], x[3]);
        x[0] = x[1] = x[2] = x[3] = 0.f;
        __syncthreads();
#pragma unroll 2
        for (int m = 0; m < 32; m += 4) add(*reinterpret_cast<const float4*>(&s.T[32 + i][32 + m]), -1.f, [&](int e) { return X(m + e, j); });
        *reinterpret_cast<float4*>(&s.T[32 + i][j]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&s.T[i][32 + j]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    unsigned char* out = mats + (nh * chunks + chunk) * Images<DKB, KP>::mats;
    {   // T's parts: four threads a row, 16 values each
        const int i = tid / 4, j = tid % 4 * 16;
        float m = 0.f;
        float4 t4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t4[e] = *reinterpret_cast<const float4*>(&s.T[i][j + 4 * e]);
            m = fmaxf(m, fmaxf(fmaxf(fabsf(t4[e].x), fabsf(t4[e].y)), fmaxf(fabsf(t4[e].z), fabsf(t4[e].w))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const Scale sc = scale_of(m);
        if (tid % 4 == 0) s.fac[kT + i] = sc.up;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint4 hi, lo;
            unsigned* hs = &hi.x;
            unsigned* ls = &lo.x;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 t = t4[2 * q + e];
                split_pair(t.x * sc.down, t.y * sc.down, hs[2 * e], ls[2 * e]);
                split_pair(t.z * sc.down, t.w * sc.down, hs[2 * e + 1], ls[2 * e + 1]);
            }
            *reinterpret_cast<uint4*>(out + swizzled(i, j + q * 8)) = hi;
            *reinterpret_cast<uint4*>(out + kBlock + swizzled(i, j + q * 8)) = lo;
        }
    }
    for (int i = tid; i < (int)(2 * kBlock / 16); i += kThreads) reinterpret_cast<uint4*>(out + 2 * kBlock)[i] = reinterpret_cast<const uint4*>(s.P)[i];
    __syncthreads();
    if (tid < 192) reinterpret_cast<float4*>(out + 4 * kBlock)[tid] = reinterpret_cast<const float4*>(s.fac)[tid];
}

// The chain.  A block has 128 columns of a head's state, a lane of tensor memory each: with S^T [value][key], U^T
// and R^T [value][step] in tensor memory as first operands, every product of a chunk has
// them on the left and K, Q, T or P, as they lie in shared memory, on the right.
//   warps 0 .. 7: a thread has half the columns of a lane (32 steps, or half the keys): V, R, U, the state
//     itself (fp32, in registers), the parts of each, and Y;
//   warp 8: issues the products, whose order keeps the tensor cores at work while the others compute:
//     K S0, half of Q S0, T R, the rest of Q S0, U K, P U;
//   warp 9: copies the chunks' images, `stages` of them ahead;
//   warps 10, 11 (16-bit types): a step a thread, lay V out by columns before it is wanted and write Y's rows, 16
//     bytes at a time where they are aligned.
// The latency of a chunk's chain bounds it: products, tensor memory to registers, parts, and back, some 8200 clocks a chunk of
// 128 x 128, of which the tensor cores work 15 %.  128 chains of 32 chunks that keep for their gradient take 220 us (0.77 GB
// at 3.5 TB/s; 209 with first parts on a grid of 2^-11, which are cheaper to form and lose small values), 144 segments of 29 that do not 151 us.
template <int DKB>
struct Columns {     // of tensor memory
    static constexpr uint32_t dS = 0, S = DKB * 64, R = 2 * DKB * 64, U = R + 64, U2 = U + 64, QS = U2 + 64, PU = R;
};

// A chain may be cut into segments, whose states come from one another by what takes a state over a segment, S -> F S + E.  SEARCH:
// finds these, without outputs: E as the state after the segment from zeros (the first one's from initial_state), F as that
// of a head without values from the state 1, in a block of its own.
template <typename T, int DKB, int KP, bool SEARCH>
__global__ void __launch_bounds__(kChainThreads, 1) delta_run_kernel(const DeltaParams p, const unsigned char* keys, const unsigned char* mats)
{
    using Im = Images<DKB, KP>;
    using Co = Columns<DKB>;
    using Sm = ChainSmem<T, DKB, KP>;
    constexpr int ST = Sm::stages, SR = DKB * 32;
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], v_full[2], v_empty[2], y_full, y_empty;
    __shared__ __align__(8) uint64_t s_ready, d_ready, r_ready, u_ready, up_ready, ds_ready, o_ready, done;
    __shared__ float most[4][2][128], warps_most[2][8];
    __shared__ uint32_t slot;
    __shared__ int given_up;
    unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    unsigned char* sheets = base + ST * Sm::stage;       // V, V, Y
    const int64_t nhs = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    const int cuts = SEARCH ? p.cuts - 1 : p.cuts;
    if (nhs >= p.N * p.H * cuts) return;
    const int64_t nh = nhs / cuts;
    const int cut = (int)(nhs - nh * cuts), tiles = (p.DV + 127) / 128;
    const bool of_one = SEARCH && (int)blockIdx.x == tiles;         // F's block
    if (of_one && cut == 0) return;
    const int64_t n = nh / p.H, chunks = delta_chunks(p.S);
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t first = cut * p.cut_chunks, all = (len + C - 1) / C;
    const int live = (int)(all <= first ? 0 : all - first < p.cut_chunks ? all - first : p.cut_chunks);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, v0 = of_one ? 0 : blockIdx.x * 128;
    const int width = of_one ? p.DK : p.DV, cols = width - v0 < 128 ? width - v0 : 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 9);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 2);
            mbar_init(&v_empty[i], 8);
        }
        mbar_init(&y_full, 8);
        mbar_init(&y_empty, 2);
        mbar_init(&s_ready, 8);
        mbar_init(&d_ready, 1);
        mbar_init(&r_ready, 8);
        mbar_init(&u_ready, 1);
        mbar_init(&up_ready, 8);
        mbar_init(&ds_ready, 1);
        mbar_init(&o_ready, 1);
        mbar_init(&done, 1);
        given_up = 0;
        mbar_fence_init();
    }
    if (warp == 8) tmem_alloc(&slot, kTmem);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, slot, 0);
    int never = 0;
    // of 168 registers a thread at launch: 216 for the eight warps that hold the state, 72 for the rest
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 9 && lane == 0) {
            int k = 0;
            for (; k < live; ++k) {
                const int s = k % ST;
                if (k >= ST && !wait(&empty[s], (unsigned)(k / ST - 1) & 1u, &given_up)) break;
                unsigned char* st = base + s * Sm::stage;
                mbar_arrive_expect_tx(&full[s], Sm::stage);
                bulk_g2s(st, keys + ((n * p.HK + hk) * chunks + first + k) * Im::keys, Im::keys, &full[s]);
                bulk_g2s(st + Im::keys, mats + (nh * chunks + first + k) * Im::mats, Im::mats, &full[s]);
            }
            // no copy is in flight when the block ends
            for (int i = k > ST ? k - ST : 0; i < k; ++i) wait(&full[i % ST], (unsigned)(i / ST) & 1u, &never);
        }
        if (warp == 8) {
            const bool leader = elected();
            const unsigned sbase = __shfl_sync(0xffffffffu, smem_addr(base), 0);
            for (int k = 0; k < live; ++k) {
                const int s = k % ST;
                const unsigned ph = (unsigned)k & 1u;
                if (!__all_sync(0xffffffffu, wait(&full[s], (unsigned)(k / ST) & 1u, &given_up) && wait(&s_ready, ph, &given_up))) break;
                fence_after();
                const unsigned kimg = sbase + s * Sm::stage, qimg = kimg + kBlock;
                const unsigned timg = kimg + Im::keys, pimg = timg + 2 * kBlock;
                // parts of S (from the last down, `count` of them) and part b of K or Q, over the keys
                auto keys_product = [&](uint32_t d, unsigned img, int last, int count, int b, bool add) {
#pragma unroll 1
                    for (int a = last; a > last - count; --a)
#pragma unroll
                        for (int ks = 0; ks < DKB * 4; ++ks)
                            if (leader)
                                mma_ts(tm + d, tm + Co::S + a * SR + ks * 8, desc_rows(img + (b * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32), instr(C, false),
                                       add || a < last || ks > 0);
                };
                // R or U and a matrix, over the steps: hi lo, lo hi, hi hi
                auto steps_product = [&](uint32_t d, uint32_t from, unsigned img) {
#pragma unroll 1
                    for (int q = 2; q >= 0; --q)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ts(tm + d, tm + from + ks / 2 * 32 + (q == 1) * 16 + ks % 2 * 8, desc_rows(img + (q == 2) * kBlock + ks * 32), instr(C, false),
                                       q < 2 || ks > 0);
                };
                if (KP == 2) keys_product(Co::R, kimg, 0, 1, 1, false);
                keys_product(Co::R, kimg, 1, 2, 0, KP == 2);
                if (leader) mma_commit(&d_ready);
                if (!SEARCH) keys_product(Co::QS, qimg, 1, 1, 0, false);
                if (!__all_sync(0xffffffffu, wait(&r_ready, ph, &given_up))) break;
                fence_after();
                steps_product(Co::U, Co::R, timg);
                if (leader) mma_commit(&u_ready);
                if (!SEARCH) {
                    if (KP == 2) keys_product(Co::QS, qimg, 0, 1, 1, true);
                    keys_product(Co::QS, qimg, 0, 1, 0, true);
                }
                if (!__all_sync(0xffffffffu, wait(&up_ready, ph, &given_up))) break;
                fence_after();
#pragma unroll 1
                for (int q = KP; q >= 0; --q)        // hi lo, lo hi, hi hi
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (leader)
                            mma_ts(tm + Co::dS, tm + Co::U2 + ks / 2 * 32 + (q == 1) * 16 + ks % 2 * 8,
                                   desc_columns(kimg + (q == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true), q < KP || ks > 0);
                if (leader) mma_commit(&ds_ready);
                if (!SEARCH) steps_product(Co::PU, Co::U, pimg);
                if (leader) {
                    mma_commit(&o_ready);
                    mma_commit(&empty[s]);
                }
            }
            if (leader) mma_commit(&done);
            wait(&done, 0, &never);
        }
        if constexpr (Sm::staged)
        if (warp >= 10) {
            const int t = threadIdx.x - 320;
            const T* from = static_cast<const T*>(p.V.data) + n * p.V.bs + (int64_t)h * p.DV + v0;
            T* to = static_cast<T*>(p.Y.data) + n * p.Y.bs + (int64_t)h * p.DV + v0;
            const bool vw = (uintptr_t)from % 16 == 0 && p.V.ss % 8 == 0, yw = (uintptr_t)to % 16 == 0 && p.Y.ss % 8 == 0;
            auto load_v = [&](int k) {
                const int64_t step = (first + k) * C + t;
                rows_to_sheet(sheets + (k & 1) * kSheet, from + step * p.V.ss, step < len && !of_one, vw, cols, t);
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[k & 1]);
            };
            if (live > 0) load_v(0);
            for (int k = 0; k < live; ++k) {
                if (k + 1 < live) {
                    if (k >= 1 && !__all_sync(0xffffffffu, wait(&v_empty[(k + 1) & 1], (unsigned)((k - 1) / 2) & 1u, &given_up))) break;
                    load_v(k + 1);
                }
                if (SEARCH) continue;
                if (!__all_sync(0xffffffffu, wait(&y_full, (unsigned)k & 1u, &given_up))) break;
                const int64_t step = (first + k) * C + t;
                if (step < len) sheet_to_rows(sheets + 2 * kSheet, to + step * p.Y.ss, yw, cols, t);
                __syncwarp();
                if (lane == 0) mbar_arrive(&y_empty);
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp / 4, row = warp % 4 * 32 + lane;
        const uint32_t my = tm + ((uint32_t)(warp % 4 * 32) << 16);
        const int v = v0 + row;
        const bool col = v < width;
        const int64_t at = nh * p.DK * p.DV + v;         // of this column's state
        const int d0 = half * SR;                        // its keys: SR from here
        f2 S[SR / 2], x[16];
        T vs[Sm::staged ? 1 : 32];
        // where a chunk's parts are kept for the gradient
        unsigned char* kept = !SEARCH && p.kept ? p.kept + ((nh * chunks + first) * gridDim.x + blockIdx.x) * delta_kept_tile(p.DK) : nullptr;
        const float* h0 = SEARCH || p.cuts == 1 ? (cut == 0 && p.h0 ? p.h0 + at : nullptr)
                        : cut == 0 && !p.h0   ? nullptr
                                              : p.starts + (nh * cuts + cut) * (int64_t)p.DK * p.DV + v;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = d0 + 2 * i + e;
                if (of_one) a[e] = d == v ? 1.f : 0.f;
                else a[e] = h0 && col && d < p.DK ? h0[(int64_t)d * p.DV] : 0.f;
            }
            S[i] = pack2(a[0], a[1]);
            m = most_of(m, S[i]);
        }
        auto load_v = [&](int k) {
            if constexpr (!Sm::staged) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int64_t t = (first + k) * C + half * 32 + i;
                    vs[i] = col && !of_one && t < len ? static_cast<const T*>(p.V.data)[n * p.V.bs + t * p.V.ss + (int64_t)h * p.DV + v] : from_f<T>(0.f);
                }
            }
        };
        // a lane's two threads share a scale; false once any wait gave up
        auto both = [&](int i, float& m, bool ok) {
            most[i][half][row] = m;
            if (!meet(1, 256, ok)) return false;
            m = fmaxf(m, most[i][1 - half][row]);
            return true;
        };
        auto tell = [&](uint64_t* bar) {
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto put_state = [&](float down) {
#pragma unroll
            for (int q = 0; q < DKB; ++q)
                put_parts(my + Co::S + d0 / 2 + q * 16, my + Co::S + SR + d0 / 2 + q * 16, S + q * 16, down);
            tmem_st_wait();
        };
        auto write_state = [&](float* to, int apart) {
            to += (int64_t)d0 * apart;
#pragma unroll
            for (int i = 0; i < SR / 2; ++i) {
                float a[2];
                unpack2(S[i], a[0], a[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (d0 + 2 * i + e < p.DK) *to = a[e];
                    to += apart;
                }
            }
        };
        Scale es{1.f, 1.f}, eu{1.f, 1.f}, e2{1.f, 1.f};
        bool ok = true;
        load_v(0);
        // A round ends chunk k - 1 (its state, then its Y) and begins chunk k: the state's parts go out before Y is formed.
        for (int k = 0; k <= live; ++k) {
            const int s = k % ST, sp = (k + ST - 1) % ST;
            const unsigned ph = (unsigned)k & 1u, php = ph ^ 1u;
            const float* stage = reinterpret_cast<const float*>(base + s * Sm::stage + Im::keys + 4 * kBlock) + half * 32;
            const float* before = reinterpret_cast<const float*>(base + sp * Sm::stage + Im::keys + 4 * kBlock) + half * 32;
            auto factors = [](const float* fac, int which, int i) { return *reinterpret_cast<const ulonglong2*>(fac + which + 4 * i); };
            f2 y[16];
            const Scale old = es;
            if (k > 0) {
                ok = __all_sync(0xffffffffu, wait(&ds_ready, php, &given_up));
                m = 0.f;
                if (ok) {
                    fence_after();
                    const f2 w = dup2(before[kWhole - half * 32]), up = dup2(e2.up);
#pragma unroll
                    for (int q = 0; q < DKB; ++q) {
                        tmem_ld(my + Co::dS + d0 + q * 32, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            S[q * 16 + i] = fma2(up, x[i], mul2(w, S[q * 16 + i]));
                            m = most_of(m, S[q * 16 + i]);
                        }
                    }
                }
            }
            if (k < live) {
                if (kept) {
                    const float w = warp_most(m);
                    if (lane == 0) warps_most[0][warp] = w;
                }
                if (!both(3, m, ok)) break;
                es = scale_of(m);
                put_state(es.down);
            }
            if (k > 0) {
                ok = __all_sync(0xffffffffu, ok && wait(&o_ready, php, &given_up));
                if (ok && !SEARCH) {
                    fence_after();
                    tmem_ld(my + Co::QS + half * 32, x);
                    tmem_ld(my + Co::PU + half * 32, y);
                }
            }
            if (k < live) tell(&s_ready);
            if (k > 0) {
                if constexpr (Sm::staged && !SEARCH)
                    if (k > 1) ok = __all_sync(0xffffffffu, ok && wait(&y_empty, ph, &given_up));
                if (ok && !SEARCH) {
                    const f2 qs = dup2(old.up), pu = dup2(eu.up);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const ulonglong2 a = factors(before, kQuery, i), b = factors(before, kP, i);
                        x[2 * i] = fma2(mul2(a.x, qs), x[2 * i], mul2(mul2(b.x, pu), y[2 * i]));
                        x[2 * i + 1] = fma2(mul2(a.y, qs), x[2 * i + 1], mul2(mul2(b.y, pu), y[2 * i + 1]));
                    }
                    if constexpr (Sm::staged) {
                        uint4* sheet = reinterpret_cast<uint4*>(sheets + 2 * kSheet + row * kPitch + half * 64);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sheet[i] = make_uint4(raw_pair<T>(x[4 * i]), raw_pair<T>(x[4 * i + 1]), raw_pair<T>(x[4 * i + 2]), raw_pair<T>(x[4 * i + 3]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int64_t t = (first + k - 1) * C + half * 32 + i;
                            float a[2];
                            unpack2(x[i / 2], a[0], a[1]);
                            if (col && t < len) static_cast<T*>(p.Y.data)[n * p.Y.bs + t * p.Y.ss + (int64_t)h * p.DV + v] = from_f<T>(a[i % 2]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    if constexpr (Sm::staged && !SEARCH) mbar_arrive(&y_full);
                    mbar_arrive(&empty[sp]);
                }
            }
            if (k == live) break;
            if (kept) {
                const Scale one = scale_of(most_of_warps(warps_most[0]));
                keep_parts<SR / 2>(kept, DKB * kSheetImage, row, d0 / 8, S, one.down);
                if (threadIdx.x == 0) *reinterpret_cast<float*>(kept + (2 * DKB + 2) * kSheetImage) = one.up;
            }
            ok = ok && wait(&full[s], (unsigned)(k / ST) & 1u, &given_up);
            if constexpr (Sm::staged) ok = ok && wait(&v_full[k & 1], (unsigned)(k / 2) & 1u, &given_up);
            ok = __all_sync(0xffffffffu, ok && wait(&d_ready, ph, &given_up));
            m = 0.f;
            if (ok) {
                fence_after();
                tmem_ld(my + Co::R + half * 32, x);
                const f2 minus = dup2(-es.up);
                const uint4* sheet = reinterpret_cast<const uint4*>(sheets + (k & 1) * kSheet + row * kPitch + half * 64);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 a = factors(stage, kBeta, i), b = factors(stage, kDecayed, i);
                    f2 w0, w1;
                    if constexpr (Sm::staged) {
                        const uint4 raw4 = sheet[i / 2];
                        w0 = pair_of<T>(i % 2 ? raw4.z : raw4.x);
                        w1 = pair_of<T>(i % 2 ? raw4.w : raw4.y);
                    } else {
                        w0 = pack2(to_f(vs[4 * i]), to_f(vs[4 * i + 1]));
                        w1 = pack2(to_f(vs[4 * i + 2]), to_f(vs[4 * i + 3]));
                    }
                    x[2 * i] = fma2(a.x, w0, mul2(mul2(b.x, minus), x[2 * i]));
                    x[2 * i + 1] = fma2(a.y, w1, mul2(mul2(b.y, minus), x[2 * i + 1]));
                    m = most_of(most_of(m, x[2 * i]), x[2 * i + 1]);
                }
            }
            if (!both(0, m, ok)) break;
            const Scale er = scale_of(m);
            put_parts(my + Co::R + half * 32, my + Co::R + half * 32 + 16, x, er.down);
            tmem_st_wait();
            tell(&r_ready);
            if constexpr (Sm::staged)
                if (lane == 0) mbar_arrive(&v_empty[k & 1]);
            if (k + 1 < live) load_v(k + 1);
            ok = __all_sync(0xffffffffu, wait(&u_ready, ph, &given_up));
            m = 0.f;
            float m2 = 0.f;
            if (ok) {
                fence_after();
                tmem_ld(my + Co::U + half * 32, x);
                const f2 up = dup2(er.up);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 a = factors(stage, kT, i), b = factors(stage, kLast, i);
                    x[2 * i] = mul2(x[2 * i], mul2(a.x, up));
                    x[2 * i + 1] = mul2(x[2 * i + 1], mul2(a.y, up));
                    y[2 * i] = mul2(x[2 * i], b.x);
                    y[2 * i + 1] = mul2(x[2 * i + 1], b.y);
                    m = most_of(most_of(m, x[2 * i]), x[2 * i + 1]);
                    m2 = most_of(most_of(m2, y[2 * i]), y[2 * i + 1]);
                }
            }
            if (kept) {
                const float w = warp_most(m);
                if (lane == 0) warps_most[1][warp] = w;
            }
            most[1][half][row] = m;
            if (!both(2, m2, ok)) break;
            m = fmaxf(m, most[1][1 - half][row]);
            eu = scale_of(m), e2 = scale_of(m2);
            put_parts(my + Co::U2 + half * 32, my + Co::U2 + half * 32 + 16, y, e2.down);
            put_parts(my + Co::U + half * 32, my + Co::U + half * 32 + 16, x, eu.down);
            tmem_st_wait();
            tell(&up_ready);
            if (kept) {
                const Scale one = scale_of(most_of_warps(warps_most[1]));
                keep_parts<16>(kept + 2 * DKB * kSheetImage, kSheetImage, row, half * 4, x, one.down);
                if (threadIdx.x == 0) *reinterpret_cast<float*>(kept + (2 * DKB + 2) * kSheetImage + 4) = one.up;
                kept += gridDim.x * delta_kept_tile(p.DK);
            }
        }
        if (SEARCH) {
            float* over = p.over + (nh * cuts + cut) * p.DK * (int64_t)(p.DV + p.DK);
            if (col) write_state(of_one ? over + (int64_t)p.DK * p.DV + v : over + v, width);
        } else if (cut == cuts - 1) {
            if (p.hT && col) write_state(p.hT + at, p.DV);
            // steps past the row's end
            if (col)
                for (int64_t t = len + half; t < p.S; t += 2)
                    static_cast<T*>(p.Y.data)[n * p.Y.bs + t * p.Y.ss + (int64_t)h * p.DV + v] = from_f<T>(0.f);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        tmem_free(tm, kTmem);
    }
    if (threadIdx.x == 0 && given_up) *p.status = 6;        // RNN_ERR_TIMEOUT
}

// The states before the segments, one after another: S <- F S + E.  A block has 16 columns of a head's state, a thread two
// rows by four columns of it, and the next segment's F and E are on their way while this one's product runs: the launch is as
// long as the segments' products in a row, each DK^2 x 16 multiplications a block, and what it reads lies in L2 (16 heads of
// 128 x 128 in nine segments: 34 us; with 32 columns a block and loads in their turn 102).
constexpr int kJoined = 16;
struct JoinSmem {
    float S[2][kDeltaMaxKey][kJoined];
    float F[kDeltaMaxKey][kDeltaMaxKey + 4];
};
__global__ void __launch_bounds__(kThreads) delta_join_kernel(const DeltaParams p)
{
    extern __shared__ __align__(1024) unsigned char raw[];
    JoinSmem& s = *reinterpret_cast<JoinSmem*>(raw);
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    constexpr int kRows = kDeltaMaxKey / 2, kF = kDeltaMaxKey / (kThreads / 32);
    static_assert(kThreads == kRows * kJoined / 4, "a thread for two rows by four columns");
    const int tid = threadIdx.x, warp = tid / 32, DK = p.DK, DV = p.DV, v0 = blockIdx.x * kJoined, c = tid % 4 * 4, r = tid / 4;
    const bool wide = DK % 4 == 0 && ((uintptr_t)p.over & 15) == 0;
    // (initial_state too: final_state may be the same memory)
    if (p.h0)
        for (int i = tid; i < DK * kJoined; i += kThreads) {
            const int d = i / kJoined, v = v0 + i % kJoined;
            if (v < DV) p.starts[(nh * p.cuts * DK + d) * (int64_t)DV + v] = p.h0[(nh * DK + d) * (int64_t)DV + v];
        }
    float f[kF][4], acc[2][4], next[2][4] = {};
    auto load = [&](int cut) {
        const float* E = p.over + (nh * (p.cuts - 1) + cut) * DK * (int64_t)(DV + DK);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = r + kRows * a, v = v0 + c + e;
                next[a][e] = d < DK && v < DV ? E[(int64_t)d * DV + v] : 0.f;
            }
        // (the first segment has no F: its E begins with the initial state)
        if (cut)
            load_fours<kF>(E + (int64_t)DK * DV + (int64_t)warp * DK, (int64_t)(kThreads / 32) * DK, DK, wide,
                           [&](int a) { return warp + kThreads / 32 * a < DK; }, f);
    };
    load(0);
    for (int cut = 0; cut < p.cuts - 1; ++cut) {
        if (cut)
#pragma unroll
            for (int a = 0; a < kF; ++a)
                *reinterpret_cast<float4*>(&s.F[warp + kThreads / 32 * a][tid % 32 * 4]) = make_float4(f[a][0], f[a][1], f[a][2], f[a][3]);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[a][e] = next[a][e];
        __syncthreads();
        if (cut + 1 < p.cuts - 1) load(cut + 1);
        const float(*old)[kJoined] = s.S[(cut + 1) & 1];
        if (cut)
#pragma unroll 4
            for (int k = 0; k < DK; k += 4) {       // (past DK both are 0)
                const float4 f0 = *reinterpret_cast<const float4*>(&s.F[r][k]), f1 = *reinterpret_cast<const float4*>(&s.F[r + kRows][k]);
                const float fs[2][4] = {{f0.x, f0.y, f0.z, f0.w}, {f1.x, f1.y, f1.z, f1.w}};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(&old[k + w][c]);
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        acc[a][0] = fmaf(fs[a][w], x.x, acc[a][0]);
                        acc[a][1] = fmaf(fs[a][w], x.y, acc[a][1]);
                        acc[a][2] = fmaf(fs[a][w], x.z, acc[a][2]);
                        acc[a][3] = fmaf(fs[a][w], x.w, acc[a][3]);
                    }
                }
            }
        float* out = p.starts + (nh * p.cuts + cut + 1) * DK * (int64_t)DV;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int d = r + kRows * a;
            *reinterpret_cast<float4*>(&s.S[cut & 1][d][c]) = d < DK ? make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3])
                                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d < DK && v0 + c + e < DV) out[(int64_t)d * DV + v0 + c + e] = acc[a][e];
        }
        __syncthreads();
    }
}

template <typename T, int DKB>
cudaError_t run(const DeltaParams& p, cudaStream_t st, int* launches)
{
    constexpr int KP = sizeof(T) == 4 ? 2 : 1;
    constexpr size_t prep_smem = sizeof(PrepSmem<DKB, KP>) + 1024, run_smem = ChainSmem<T, DKB, KP>::bytes;
    static std::atomic<uint64_t> prep_done{0}, run_done{0}, search_done{0}, join_done{0};
    cudaError_t e = allow_shared(delta_prep_kernel<T, DKB, KP>, prep_smem, prep_done);
    if (e == cudaSuccess) e = allow_shared(delta_run_kernel<T, DKB, KP, false>, run_smem, run_done);
    if (e == cudaSuccess && p.cuts > 1) e = allow_shared(delta_run_kernel<T, DKB, KP, true>, run_smem, search_done);
    if (e == cudaSuccess && p.cuts > 1) e = allow_shared(delta_join_kernel, sizeof(JoinSmem), join_done);
    if (e != cudaSuccess) return e;
    const int64_t nh = p.N * p.H;
    unsigned char *keys = p.keys, *mats = p.mats;
    if (p.S > 0) {
        delta_prep_kernel<T, DKB, KP><<<heads_grid(delta_chunks(p.S), nh), kThreads, prep_smem, st>>>(p, keys, mats);
        ++*launches;
    }
    const int64_t tiles = (p.DV + 127) / 128;
    if (p.cuts > 1) {
        delta_run_kernel<T, DKB, KP, true><<<heads_grid(tiles + 1, nh * (p.cuts - 1)), kChainThreads, run_smem, st>>>(p, keys, mats);
        delta_join_kernel<<<heads_grid((p.DV + kJoined - 1) / kJoined, nh), kThreads, sizeof(JoinSmem), st>>>(p);
        *launches += 2;
    }
    delta_run_kernel<T, DKB, KP, false><<<heads_grid(tiles, nh * p.cuts), kChainThreads, run_smem, st>>>(p, keys, mats);
    ++*launches;
    return cudaGetLastError();
}

template <typename T>
cudaError_t run(const DeltaParams& p, cudaStream_t st, int* launches)
{
    return p.DK > 64 ? run<T, 2>(p, st, launches) : run<T, 1>(p, st, launches);
}

}  // namespace

// A chain is cut where there are too few of them for the multiprocessors: the search for what takes a state over a segment costs
// as much again, or twice that (F's blocks), at `cuts` times the blocks.  In waves of blocks times chunks; joining costs a few chunks.
void delta_split(DeltaParams& p)
{
    const int64_t chunks = delta_chunks(p.S), tiles = (p.DV + 127) / 128, chains = p.N * p.H;
    auto waves = [&](int64_t blocks) { return (blocks + p.sms - 1) / p.sms; };
    p.cuts = 1;
    p.cut_chunks = chunks > 0 ? chunks : 1;
    if (p.sms <= 0 || chunks < 16 || chains * tiles * 2 > p.sms) return;
    double best = 0.8 * (double)(waves(chains * tiles) * chunks);
    for (int64_t cuts = 2; cuts <= 64 && cuts * 4 <= chunks; ++cuts) {
        const int64_t per = (chunks + cuts - 1) / cuts, n = (chunks + per - 1) / per;
        const double cost = (double)((waves(chains * (tiles + 1) * (n - 1)) + waves(chains * tiles * n)) * per) + 6.0 + 1.0 * (double)n;
        if (n == cuts && cost < best) {
            best = cost;
            p.cuts = (int)n;
            p.cut_chunks = per;
        }
    }
}

cudaError_t launch_delta(const DeltaParams& p, cudaStream_t s, int* launches)
{
    return p.io == 0 ? run<float>(p, s, launches) : p.io == 1 ? run<__half>(p, s, launches) : run<__nv_bfloat16>(p, s, launches);
}

}  // namespace rnngb
