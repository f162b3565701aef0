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
#include "delta_mma.cuh"

namespace rnngb {
namespace {

using namespace delta;

// The chain, from the last chunk to the first, laid out as the run's (k_delta.cu): G = dS1^T, dU^T, dR^T and dY'^T are the
// products' first operands in tensor memory, the images that the run has kept the second ones.  A
// chunk goes
//     P^T dY'  (its operand put ahead, while the chunk before ends),  K G -> dU -> T^T dU = dR -> K^T dR -> G,
// with (e^G Q)^T dY' while dR is on its way.  Its latency bounds it, as the run's: 128 chains of 32 chunks of 128 x 128 in bf16
// take 206 us, 0.83 GB at 4.0 TB/s.
template <int DKB>
struct Columns {     // of tensor memory
    static constexpr uint32_t dG = 0, G = DKB * 64, U = 2 * DKB * 64, R = U + 64, X = R + 64, PY = X + 64;
};

template <typename T, int DKB, int KP>
__global__ void __launch_bounds__(kChainThreads, 1) delta_grad_chain_kernel(const DeltaGradParams q)
{
    using Im = Images<DKB, KP>;
    using Co = Columns<DKB>;
    using Sm = ChainSmem<T, DKB, KP>;
    constexpr int ST = Sm::stages, SR = DKB * 32;
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], v_full[2], v_empty[2], y_full, y_empty;
    __shared__ __align__(8) uint64_t x_ready, g_ready, d_ready, u_told, r_ready, x2_ready, dq_ready, r_told, dg_ready, done;
    __shared__ float most[5][2][128], warps_most[3][8];
    __shared__ uint32_t slot;
    __shared__ int given_up;
    unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    unsigned char* sheets = base + ST * Sm::stage;       // dY, dY, dV
    const DeltaParams& p = q.f;
    const int64_t nh = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nh >= p.N * p.H) return;
    const int64_t n = nh / p.H, chunks = delta_chunks(p.S);
    const int h = (int)(nh - n * p.H), hk = h / (p.H / p.HK);
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int live = (int)((len + C - 1) / C);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, v0 = blockIdx.x * 128;
    const int cols = p.DV - v0 < 128 ? p.DV - v0 : 128;
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
        mbar_init(&x_ready, 8);
        mbar_init(&g_ready, 8);
        mbar_init(&d_ready, 1);
        mbar_init(&u_told, 8);
        mbar_init(&r_ready, 1);
        mbar_init(&x2_ready, 8);
        mbar_init(&dq_ready, 1);
        mbar_init(&r_told, 8);
        mbar_init(&dg_ready, 1);
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
    // of 168 registers a thread at launch: 216 for the eight warps that hold the slope, 72 for the rest
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 9 && lane == 0) {
            int k = 0;
            for (; k < live; ++k) {
                const int s = k % ST;
                const int64_t chunk = live - 1 - k;
                if (k >= ST && !wait(&empty[s], (unsigned)(k / ST - 1) & 1u, &given_up)) break;
                unsigned char* st = base + s * Sm::stage;
                mbar_arrive_expect_tx(&full[s], Sm::stage);
                bulk_g2s(st, p.keys + ((n * p.HK + hk) * chunks + chunk) * Im::keys, Im::keys, &full[s]);
                bulk_g2s(st + Im::keys, p.mats + (nh * chunks + chunk) * Im::mats, Im::mats, &full[s]);
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
                if (!__all_sync(0xffffffffu, wait(&full[s], (unsigned)(k / ST) & 1u, &given_up) && wait(&x_ready, ph, &given_up))) break;
                fence_after();
                const unsigned kimg = sbase + s * Sm::stage, qimg = kimg + kBlock;
                const unsigned timg = kimg + Im::keys, pimg = timg + 2 * kBlock;
                // the operand at `from` and a matrix transposed, over the steps: hi lo, lo hi, hi hi
                auto steps_product = [&](uint32_t d, uint32_t from, unsigned img) {
#pragma unroll 1
                    for (int r = 2; r >= 0; --r)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ts(tm + d, tm + from + ks / 2 * 32 + (r == 1) * 16 + ks % 2 * 8, desc_columns(img + (r == 2) * kBlock + ks * 2048, kBlock),
                                       instr(C, true), r < 2 || ks > 0);
                };
                // the same with K or Q, into G's increment
                auto state_product = [&](uint32_t from, unsigned img) {
#pragma unroll 1
                    for (int r = KP; r >= 0; --r)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ts(tm + Co::dG, tm + from + ks / 2 * 32 + (r == 1) * 16 + ks % 2 * 8,
                                       desc_columns(img + (r == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true), r < KP || ks > 0);
                };
                steps_product(Co::PY, Co::X, pimg);
                if (!__all_sync(0xffffffffu, wait(&g_ready, ph, &given_up))) break;
                fence_after();
#pragma unroll 1
                for (int r = KP; r >= 0; --r)
#pragma unroll
                    for (int ks = 0; ks < DKB * 4; ++ks)
                        if (leader)
                            mma_ts(tm + Co::U, tm + Co::G + (r == 1) * SR + ks * 8, desc_rows(kimg + ((r == 2) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32),
                                   instr(C, false), r < KP || ks > 0);
                if (leader) mma_commit(&d_ready);
                if (!__all_sync(0xffffffffu, wait(&u_told, ph, &given_up))) break;
                fence_after();
                steps_product(Co::R, Co::U, timg);
                if (leader) mma_commit(&r_ready);
                if (!__all_sync(0xffffffffu, wait(&x2_ready, ph, &given_up))) break;
                fence_after();
                state_product(Co::X, qimg);
                if (leader) mma_commit(&dq_ready);
                if (!__all_sync(0xffffffffu, wait(&r_told, ph, &given_up))) break;
                fence_after();
                state_product(Co::R, kimg);
                if (leader) {
                    mma_commit(&dg_ready);
                    mma_commit(&empty[s]);
                }
            }
            if (leader) mma_commit(&done);
            wait(&done, 0, &never);
        }
        if constexpr (Sm::staged)
        if (warp >= 10) {
            const int t = threadIdx.x - 320;
            const T* from = static_cast<const T*>(q.dY.data) + n * q.dY.bs + (int64_t)h * p.DV + v0;
            T* to = static_cast<T*>(q.dV.data) + n * q.dV.bs + (int64_t)h * p.DV + v0;
            const bool yw = (uintptr_t)from % 16 == 0 && q.dY.ss % 8 == 0, vw = (uintptr_t)to % 16 == 0 && q.dV.ss % 8 == 0;
            auto load = [&](int k) {
                const int64_t step = (int64_t)(live - 1 - k) * C + t;
                rows_to_sheet(sheets + (k & 1) * kSheet, from + step * q.dY.ss, step < len, yw, cols, t);
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[k & 1]);
            };
            if (live > 0) load(0);
            for (int k = 0; k < live; ++k) {
                if (k + 1 < live) {
                    if (k >= 1 && !__all_sync(0xffffffffu, wait(&v_empty[(k + 1) & 1], (unsigned)((k - 1) / 2) & 1u, &given_up))) break;
                    load(k + 1);
                }
                if (!__all_sync(0xffffffffu, wait(&y_full, (unsigned)k & 1u, &given_up))) break;
                const int64_t step = (int64_t)(live - 1 - k) * C + t;
                if (q.dV.data && step < len) sheet_to_rows(sheets + 2 * kSheet, to + step * q.dV.ss, vw, cols, t);
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
        const bool col = v < p.DV;
        const int64_t at = nh * p.DK * p.DV + v;
        const int d0 = half * SR;
        f2 G[SR / 2], x[16], y[16];
        // where a chunk's parts are kept for the second launch: G's, dR's, dY's, the last chunk first
        const int64_t tile = delta_slopes_tile(p.DK, sizeof(T) == 4 ? 0 : 1);
        unsigned char* kept = q.slopes + ((nh * chunks + live - 1) * gridDim.x + blockIdx.x) * tile;
        constexpr unsigned kR = 2 * DKB * kSheetImage, kY = kR + 2 * kSheetImage, kScales = kY + KP * kSheetImage;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) a[e] = q.dhT && col && d0 + 2 * i + e < p.DK ? q.dhT[at + (int64_t)(d0 + 2 * i + e) * p.DV] : 0.f;
            G[i] = pack2(a[0], a[1]);
            m = most_of(m, G[i]);
        }
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
        auto write_state = [&](float* to) {
            to += (int64_t)d0 * p.DV;
#pragma unroll
            for (int i = 0; i < SR / 2; ++i) {
                float a[2];
                unpack2(G[i], a[0], a[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (d0 + 2 * i + e < p.DK) *to = a[e];
                    to += p.DV;
                }
            }
        };
        auto factors = [](const float* fac, int which, int i) { return *reinterpret_cast<const ulonglong2*>(fac + which + 4 * i); };
        auto stage_of = [&](int k) { return reinterpret_cast<const float*>(base + k % ST * Sm::stage + Im::keys + 4 * kBlock) + half * 32; };
        // dY of chunk k times the factors of kind `which`, into y and, in parts, to X; false once any wait gave up
        auto put_dy = [&](int k, int which, int meeting, float& up, bool ok, bool keep) {
            float most_y = 0.f, most_raw = 0.f;
            f2 raw_y[16];
            if (ok) {
                const float* fac = stage_of(k);
                const uint4* sheet = reinterpret_cast<const uint4*>(sheets + (k & 1) * kSheet + row * kPitch + half * 64);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 a = factors(fac, which, i);
                    f2 w0, w1;
                    if constexpr (Sm::staged) {
                        const uint4 raw4 = sheet[i / 2];
                        w0 = pair_of<T>(i % 2 ? raw4.z : raw4.x);
                        w1 = pair_of<T>(i % 2 ? raw4.w : raw4.y);
                    } else {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int64_t t = (int64_t)(live - 1 - k) * C + half * 32 + 4 * i + e;
                            w[e] = col && t < len ? to_f(static_cast<const T*>(q.dY.data)[n * q.dY.bs + t * q.dY.ss + (int64_t)h * p.DV + v]) : 0.f;
                        }
                        w0 = pack2(w[0], w[1]);
                        w1 = pack2(w[2], w[3]);
                    }
                    if (keep) {
                        raw_y[2 * i] = w0;
                        raw_y[2 * i + 1] = w1;
                        most_raw = most_of(most_of(most_raw, w0), w1);
                    }
                    y[2 * i] = mul2(a.x, w0);
                    y[2 * i + 1] = mul2(a.y, w1);
                    most_y = most_of(most_of(most_y, y[2 * i]), y[2 * i + 1]);
                }
            }
            if (keep) {
                const float w = warp_most(most_raw);
                if (lane == 0) warps_most[1][warp] = w;
            }
            if (!both(meeting, most_y, ok)) return false;
            const Scale e = scale_of(most_y);
            put_parts(my + Co::X + half * 32, my + Co::X + half * 32 + 16, y, e.down);
            tmem_st_wait();
            up = e.up;
            if (keep) {
                tell(&x2_ready);
                const Scale one = scale_of(most_of_warps(warps_most[1]));
                if (threadIdx.x == 0) *reinterpret_cast<float*>(kept + kScales + 8) = one.up;
                if constexpr (KP == 2) {
                    keep_parts<16>(kept + kY, kSheetImage, row, half * 4, raw_y, one.down);
                } else {
                    const f2 d = dup2(one.down);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        unsigned v[4];
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) v[e2] = raw_pair<__half>(mul2(raw_y[4 * i + e2], d));
                        *reinterpret_cast<uint4*>(kept + kY + (half * 4 + i) * kPiece + row * 16) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            return true;
        };
        auto arrived = [&](int k) {     // chunk k's factors and dY
            bool ok = wait(&full[k % ST], (unsigned)(k / ST) & 1u, &given_up);
            if constexpr (Sm::staged) ok = ok && wait(&v_full[k & 1], (unsigned)(k / 2) & 1u, &given_up);
            return (bool)__all_sync(0xffffffffu, ok);
        };
        float py_up = 1.f, qy_up = 1.f, r_up = 1.f;
        bool ok = true;
        for (int k = 0; k <= live; ++k) {
            const unsigned ph = (unsigned)k & 1u, php = ph ^ 1u;
            // dY' P's operand, ahead of all else of this chunk
            if (k < live) {
                ok = arrived(k) && ok;
                if (!put_dy(k, kP, 4, py_up, ok, false)) break;
                tell(&x_ready);
            }
            if (k > 0) {        // G of the chunk before is complete
                ok = __all_sync(0xffffffffu, ok && wait(&dg_ready, php, &given_up));
                m = 0.f;
                if (ok) {
                    fence_after();
                    const f2 up = dup2(r_up);
#pragma unroll
                    for (int r = 0; r < DKB; ++r) {
                        tmem_ld(my + Co::dG + d0 + r * 32, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            G[r * 16 + i] = fma2(up, x[i], G[r * 16 + i]);
                            m = most_of(m, G[r * 16 + i]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[(k - 1) % ST]);
            }
            if (k == live) break;
            {
                const float w = warp_most(m);
                if (lane == 0) warps_most[0][warp] = w;
            }
            if (!both(3, m, ok)) break;
            const Scale eg = scale_of(m);
#pragma unroll
            for (int r = 0; r < DKB; ++r)
                put_parts(my + Co::G + d0 / 2 + r * 16, my + Co::G + SR + d0 / 2 + r * 16, G + r * 16, eg.down);
            tmem_st_wait();
            tell(&g_ready);
            const int64_t chunk = live - 1 - k;
            {
                const Scale one = scale_of(most_of_warps(warps_most[0]));
                keep_parts<SR / 2>(kept, DKB * kSheetImage, row, d0 / 8, G, one.down);
                if (threadIdx.x == 0) *reinterpret_cast<float*>(kept + kScales) = one.up;
            }
            const float* fac = stage_of(k);
            ok = __all_sync(0xffffffffu, wait(&d_ready, ph, &given_up));
            m = 0.f;
            if (ok) {
                fence_after();
                tmem_ld(my + Co::U + half * 32, x);
                tmem_ld(my + Co::PY + half * 32, y);
                const f2 g = dup2(eg.up), py = dup2(py_up);
#pragma unroll
                for (int i = 0; i < 8; ++i) {       // dU, times T's rows' scales
                    const ulonglong2 a = factors(fac, kLast, i), b = factors(fac, kT, i);
                    x[2 * i] = mul2(b.x, fma2(mul2(a.x, g), x[2 * i], mul2(py, y[2 * i])));
                    x[2 * i + 1] = mul2(b.y, fma2(mul2(a.y, g), x[2 * i + 1], mul2(py, y[2 * i + 1])));
                    m = most_of(most_of(m, x[2 * i]), x[2 * i + 1]);
                }
            }
            if (!both(0, m, ok)) break;
            const Scale eu = scale_of(m);
            put_parts(my + Co::U + half * 32, my + Co::U + half * 32 + 16, x, eu.down);
            tmem_st_wait();
            tell(&u_told);
            if (!put_dy(k, kQuery, 1, qy_up, ok, true)) break;
            if constexpr (Sm::staged)
                if (lane == 0) mbar_arrive(&v_empty[k & 1]);
            ok = __all_sync(0xffffffffu, wait(&r_ready, ph, &given_up));
            m = 0.f;
            float most_r = 0.f;
            if (ok) {
                fence_after();
                tmem_ld(my + Co::R + half * 32, x);
                const f2 up = dup2(eu.up), minus = dup2(-1.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 a = factors(fac, kDecayed, i);
                    x[2 * i] = mul2(x[2 * i], up);
                    x[2 * i + 1] = mul2(x[2 * i + 1], up);
                    most_r = most_of(most_of(most_r, x[2 * i]), x[2 * i + 1]);
                    y[2 * i] = mul2(mul2(a.x, minus), x[2 * i]);
                    y[2 * i + 1] = mul2(mul2(a.y, minus), x[2 * i + 1]);
                    m = most_of(most_of(m, y[2 * i]), y[2 * i + 1]);
                }
            }
            {
                const float w = warp_most(most_r);
                if (lane == 0) warps_most[2][warp] = w;
            }
            if (!both(2, m, ok)) break;
            const Scale er = scale_of(m);
            r_up = er.up;
            put_parts(my + Co::R + half * 32, my + Co::R + half * 32 + 16, y, er.down);
            tmem_st_wait();
            ok = __all_sync(0xffffffffu, wait(&dq_ready, ph, &given_up));
            if (ok) {
                fence_after();
                const f2 w = dup2(fac[kWhole - half * 32]), up = dup2(qy_up);
#pragma unroll
                for (int r = 0; r < DKB; ++r) {
                    tmem_ld(my + Co::dG + d0 + r * 32, y);
#pragma unroll
                    for (int i = 0; i < 16; ++i) G[r * 16 + i] = fma2(up, y[i], mul2(w, G[r * 16 + i]));
                }
                tell(&r_told);
            }
            {
                const Scale one = scale_of(most_of_warps(warps_most[2]));
                keep_parts<16>(kept + kR, kSheetImage, row, half * 4, x, one.down);
                if (threadIdx.x == 0) *reinterpret_cast<float*>(kept + kScales + 4) = one.up;
                kept -= gridDim.x * tile;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {       // dV
                const ulonglong2 a = factors(fac, kBeta, i);
                x[2 * i] = mul2(a.x, x[2 * i]);
                x[2 * i + 1] = mul2(a.y, x[2 * i + 1]);
            }
            if constexpr (Sm::staged) {
                if (k > 0) ok = __all_sync(0xffffffffu, ok && wait(&y_empty, php, &given_up));
                uint4* sheet = reinterpret_cast<uint4*>(sheets + 2 * kSheet + row * kPitch + half * 64);
                if (ok)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sheet[i] = make_uint4(raw_pair<T>(x[4 * i]), raw_pair<T>(x[4 * i + 1]), raw_pair<T>(x[4 * i + 2]), raw_pair<T>(x[4 * i + 3]));
                __syncwarp();
                if (lane == 0) mbar_arrive(&y_full);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int64_t t = chunk * C + half * 32 + i;
                    float a[2];
                    unpack2(x[i / 2], a[0], a[1]);
                    if (q.dV.data && col && t < len) static_cast<T*>(q.dV.data)[n * q.dV.bs + t * q.dV.ss + (int64_t)h * p.DV + v] = from_f<T>(a[i % 2]);
                }
            }
        }
        if (q.dh0 && col) write_state(q.dh0 + at);
        if (q.dV.data && col)
            for (int64_t t = len + half; t < p.S; t += 2)
                static_cast<T*>(q.dV.data)[n * q.dV.bs + t * q.dV.ss + (int64_t)h * p.DV + v] = from_f<T>(0.f);
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        tmem_free(tm, kTmem);
    }
    if (threadIdx.x == 0 && given_up) *p.status = 6;        // RNN_ERR_TIMEOUT
}

// The rest, a chunk and key head a block.  With what the chains have kept, each [value][step] or [value][key] in two parts,
// the products over the values are
//     [dR; dY'] S0^T = [X2; X1],   [dR; dY'] U^T = [-dA; dP],   [U; not used] dS1^T = [X3; not used],
// 128 rows each: a lane of tensor memory is a step, dR's in the upper half and dY''s in the lower one.  Then [K; Q] K^T
// again, [EA + EA^T; EP] K and [EP^T; not used] Q.  More values than 128 are taken one tile after the other: everything
// below is linear in the five first products.
//
// What decays between two steps i > j, D_ij = EA_ij K_i.K_j + EP_ij Q_i.K_j, has g_t in it for j < t <= i, so that
//     dg_t = sum_{i >= t > j} D_ij + sum_{i >= t} e^G_i (q_i.X1_i - b_i k_i.X2_i) + sum_{j < t} e^(G_last - G_j) k_j.X3_j + e^G_last <dS1, S0>.
// (Sums of the slopes in G_i over i >= t are the same, but hold each D_ij of two later steps twice, with either sign:
// where decays are strong the little that is left had lost three bits.)  The first sum comes from sums along the rows, in
// a thread's 16 columns and those before, added down the rows i >= t.
//
// 240 KB come in a chunk and head of 128 x 128 at 16 bits, copied as they are.  Its phases bound it, five rounds of products
// and what forms their operands, with one block a multiprocessor (231 KB of shared memory, 17 of them static): 4096 chunks take 457 us, 1.25 GB at
// 2.7 TB/s, the tensor cores at 15 %.
constexpr int kRestThreads = 512;
template <int DKB, int KP>
struct RestSmem {
    // u's parts, then [dR; dY] of the first parts and of the second; the states; K and Q (of 32-bit types in the states' place,
    // when these are done with)
    static constexpr unsigned u = 0, r = 2 * kSheetImage, y = 3 * kSheetImage, states = 6 * kSheetImage;
    static constexpr bool early = KP == 1;
    // once [dR; dY] are done with: E; [EA + EA^T; EP].  EP^T has a place of its own, or u's once that is done with
    static constexpr unsigned after = states + 2 * DKB * kSheetImage;
    static constexpr unsigned e = r, a1 = 4 * kSheetImage, a2 = early ? after : u;
    static constexpr unsigned keys = early ? after + 2 * kBlock : states;
    static constexpr unsigned end = early ? keys + Images<DKB, KP>::keys : after;
    // (the products read 128 rows of EP^T's parts, of which 64 are there: what lies behind them must be the block's, too)
    static_assert(a2 + kBlock + 2 * kBlock <= end, "");
    static constexpr size_t bytes = end + 1024;
    static_assert(Images<DKB, KP>::keys <= 2 * DKB * kSheetImage, "");
};

template <typename T, int DKB, int KP>
__global__ void __launch_bounds__(kRestThreads, 1) delta_grad_rest_kernel(const DeltaGradParams q)
{
    using Im = Images<DKB, KP>;
    using Sm = RestSmem<DKB, KP>;
    constexpr uint32_t cX = 0, cX3 = 128, cK = 256, cE = 384, cKQ = 448, cKE = 384;     // columns of tensor memory
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ __align__(8) uint64_t first_full, g_full, k_full, x_done, x3_done, kq_done, k_done, done;
    __shared__ Sums sums;
    __shared__ float k_scale[C], q_scale[C];
    __shared__ __align__(16) float fac[768], scales[8];      // (copied 16 bytes at a time)
    __shared__ float rv[C], part[5][4][128], dots[kRestThreads / 32], scans[5][C], slope[C], db[C];
    __shared__ float2 carry;
    __shared__ uint32_t slot;
    __shared__ int given_up;
    const DeltaParams& p = q.f;
    const int64_t chunk = blockIdx.x, chunks = gridDim.x, nk = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (nk >= p.N * p.HK) return;
    const int64_t n = nk / p.HK, t0 = chunk * C;
    const int hk = (int)(nk - n * p.HK), per = p.H / p.HK, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int DK = p.DK, DV = p.DV, steps = (int)(p.S - t0 < C ? p.S - t0 : C);
    // a thread's step, whether of the upper half (dK) or the lower (dQ), and its quarter of the columns
    const int lane_row = warp % 4 * 32 + lane, i = lane_row % C, quarter = warp / 4;
    const bool upper = lane_row < C;
    float acc[DKB][16];
#pragma unroll
    for (int b = 0; b < DKB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[b][e] = 0.f;
    if (t0 >= len) {
        for (int j = tid; j < steps * per; j += kRestThreads) {
            const int t = j / per, h = hk * per + j % per;
            if (q.dg.data) static_cast<float*>(q.dg.data)[n * q.dg.bs + (t0 + t) * q.dg.ss + h] = 0.f;
            if (q.dbeta.data) static_cast<float*>(q.dbeta.data)[n * q.dbeta.bs + (t0 + t) * q.dbeta.ss + h] = 0.f;
        }
    } else {
        unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
        float* E = reinterpret_cast<float*>(base + Sm::e);
        if (tid == 0) {
            mbar_init(&first_full, 1);
            mbar_init(&g_full, 1);
            mbar_init(&k_full, 1);
            mbar_init(&x_done, 1);
            mbar_init(&x3_done, 1);
            mbar_init(&kq_done, 1);
            mbar_init(&k_done, 1);
            mbar_init(&done, 1);
            given_up = 0;
            mbar_fence_init();
        }
        if (warp == 0) tmem_alloc(&slot, kTmem);
        fence_before();
        __syncthreads();
        fence_after();
        const uint32_t tm = __shfl_sync(0xffffffffu, slot, 0), my = tm + ((uint32_t)(warp % 4 * 32) << 16);
        const unsigned sbase = __shfl_sync(0xffffffffu, smem_addr(base), 0);
        const bool leader = warp == 0 && elected();
        const int tiles = (DV + 127) / 128;
        const int64_t kept_tile = delta_kept_tile(DK), slopes_tile = delta_slopes_tile(DK, KP == 2 ? 0 : 1);
        constexpr unsigned kStates = 2 * DKB * kSheetImage;
        // all threads wait, and know whether all did
        unsigned phase = 0;
        auto await = [&](uint64_t* b) {
            fence_before();
            const bool ok = __syncthreads_and(wait(b, phase, &given_up));
            fence_after();
            return ok;
        };
        bool ok = true;
        for (int round = 0; round < per * tiles; ++round) {
            const int h = hk * per + round / tiles, tile = round % tiles, v0 = tile * 128;
            const int64_t nh = n * p.H + h, at = nh * chunks + chunk;
            const unsigned char *kept = p.kept + (at * tiles + tile) * kept_tile, *slopes = q.slopes + (at * tiles + tile) * slopes_tile;
            const unsigned char* keys = p.keys + (nk * chunks + chunk) * Im::keys;
            const float g = load_g(p.g, n, h, t0, len);
            float4 fac4;
            if (tid < 192) fac4 = reinterpret_cast<const float4*>(p.mats + at * Im::mats + 4 * kBlock)[tid];
            float scale_one = 0.f;
            if (tid < 2) scale_one = reinterpret_cast<const float*>(kept + kStates + 2 * kSheetImage)[tid];
            else if (tid < 5) scale_one = reinterpret_cast<const float*>(slopes + kStates + (2 + KP) * kSheetImage)[tid - 2];
            if (tid == 0) {
                mbar_arrive_expect_tx(&first_full, kStates + (4 + KP) * kSheetImage + (Sm::early ? Im::keys : 0));
                bulk_g2s(base + Sm::r, slopes + kStates, kSheetImage, &first_full);
                bulk_g2s(base + Sm::r + 2 * kSheetImage, slopes + kStates + kSheetImage, kSheetImage, &first_full);
                bulk_g2s(base + Sm::y, slopes + kStates + 2 * kSheetImage, kSheetImage, &first_full);
                if (KP == 2) bulk_g2s(base + Sm::y + 2 * kSheetImage, slopes + kStates + 3 * kSheetImage, kSheetImage, &first_full);
                bulk_g2s(base + Sm::u, kept + kStates, 2 * kSheetImage, &first_full);
                bulk_g2s(base + Sm::states, kept, kStates, &first_full);
                if (Sm::early) bulk_g2s(base + Sm::keys, keys, Im::keys, &first_full);
            }
            if (KP == 1)            // 16-bit values have no second part
                for (int j = tid; j < (int)kSheetImage / 16; j += kRestThreads)
                    reinterpret_cast<uint4*>(base + Sm::y + 2 * kSheetImage)[j] = make_uint4(0, 0, 0, 0);
            fence_shared();
            // V at the warp's four steps, four values 32 apart a lane
            T vs[4][4];
            {
                const T* row = static_cast<const T*>(p.V.data) + n * p.V.bs + (t0 + warp * 4) * p.V.ss + (int64_t)h * DV + v0 + lane;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        vs[t][e] = t0 + warp * 4 + t < len && v0 + lane + 32 * e < DV ? row[t * p.V.ss + 32 * e] : from_f<T>(0.f);
            }
            if (tid < 192) reinterpret_cast<float4*>(fac)[tid] = fac4;
            if (tid < 5) scales[tid] = scale_one;
            form_sums(sums, g, &carry);
            const float s_up = scales[0], u_up = scales[1], g_up = scales[2], r_up = scales[3], y_up = p.scale * scales[4];
            ok = await(&first_full);
            if (!ok) break;
            // What comes next on this multiprocessor, into L2: blocks load and compute at the same times, and their loads alone
            // would wait for one another at the memory.
            if (tid == 32) {
                int64_t next_at = at * tiles + tile + 1, next_keys = -1;
                bool there = true;
                if (round + 1 == per * tiles) {
                    const int64_t b = nk * chunks + chunk + p.sms, bk = b / chunks;
                    there = bk < p.N * p.HK;
                    next_at = ((bk / p.HK * p.H + bk % p.HK * per) * chunks + b % chunks) * tiles;
                    next_keys = b;
                } else if (tile + 1 == tiles) {
                    next_at = (at + chunks) * tiles;
                }
                if (there) {
                    prefetch(p.kept + next_at * kept_tile, (unsigned)kept_tile);
                    prefetch(q.slopes + next_at * slopes_tile, (unsigned)slopes_tile);
                    prefetch(p.mats + next_at / tiles * Im::mats + 4 * kBlock, (unsigned)kDeltaFactors);
                    if (next_keys >= 0) prefetch(p.keys + next_keys * Im::keys, Im::keys);
                }
            }
            const unsigned kimg = sbase + Sm::keys, qimg = kimg + kBlock;
            auto key_products = [&] {
#pragma unroll 1
                for (int r = 2 * KP - 2; r >= 0; --r)         // hi lo, lo hi, hi hi
#pragma unroll
                    for (int ks = 0; ks < DKB * 4; ++ks)
                        if (leader)
                            mma_ss(tm + cKQ, desc_rows(kimg + ((r == 1) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32),
                                   desc_rows(kimg + ((r == 2) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32), instr(C, false), r < 2 * KP - 2 || ks > 0);
                if (leader) mma_commit(&kq_done);
            };
            if (warp == 0) {
#pragma unroll 1
                for (int r = 2; r >= 0; --r)     // [dR; dY'] U^T: hi lo, lo hi, hi hi
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        if (leader)
                            mma_ss(tm + cE, desc_kept(sbase + Sm::r + (r == 1) * 2 * kSheetImage, ks), desc_kept(sbase + Sm::u + (r == 2) * kSheetImage, ks),
                                   instr(C, true) | 1u << 15, r < 2 || ks > 0);
                if (Sm::early) key_products();
#pragma unroll 1
                for (int r = 2; r >= 0; --r)     // [dR; dY'] S0^T
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        if (leader)
                            mma_ss(tm + cX, desc_kept(sbase + Sm::r + (r == 1) * 2 * kSheetImage, ks),
                                   desc_kept(sbase + Sm::states + (r == 2) * DKB * kSheetImage, ks), instr(DKB * 64, true) | 1u << 15, r < 2 || ks > 0);
                if (leader) mma_commit(&x_done);
            }
            {   // dR . V
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                const unsigned char* from = base + Sm::r + warp / 2 * kPiece + warp % 2 * 8 + lane * 16;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint2 a = *reinterpret_cast<const uint2*>(from + e * 512), b = *reinterpret_cast<const uint2*>(from + e * 512 + 2 * kSheetImage);
                    const float2 a0 = pair_value(a.x), a1 = pair_value(a.y), b0 = pair_value(b.x), b1 = pair_value(b.y);
                    sum[0] = fmaf(a0.x + b0.x, to_f(vs[0][e]), sum[0]);
                    sum[1] = fmaf(a0.y + b0.y, to_f(vs[1][e]), sum[1]);
                    sum[2] = fmaf(a1.x + b1.x, to_f(vs[2][e]), sum[2]);
                    sum[3] = fmaf(a1.y + b1.y, to_f(vs[3][e]), sum[3]);
                }
#pragma unroll
                for (int o = 16; o; o /= 2)
#pragma unroll
                    for (int t = 0; t < 4; ++t) sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], o);
                if (lane < 4) rv[warp * 4 + lane] = lane == 0 ? sum[0] : lane == 1 ? sum[1] : lane == 2 ? sum[2] : sum[3];
            }
            const float b_i = fac[kBeta + i];
            float e[16];
            auto form_e = [&] {
                float kq[16], row = 0.f, s = 0.f;
                tmem_ld16(my + cE + quarter * 16, e);
                tmem_ld16(my + cKQ + quarter * 16, kq);
                const float mine = (upper ? -r_up : y_up) * u_up, es = fac[(upper ? kKeyScale : kQueryScale) + i];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int j = quarter * 16 + c;
                    const bool in = upper ? j < i : j <= i;
                    const float decay = in ? sums.power(i, j) : 0.f;
                    const float d = in ? e[c] * mine * decay : 0.f;
                    const float k = in ? kq[c] * es * fac[kKeyScale + j] : 0.f;
                    const float v = upper ? b_i * d : d;
                    s = fmaf(d, k, s);
                    e[c] = v;
                    row = fmaf(v, k, row);
                    kq[c] = j < i ? row : 0.f;      // of D_i., up to column j, where step j + 1 is not past i
                }
                part[0][quarter][lane_row] = row;
                part[1][quarter][lane_row] = s;
                // added over the warp's rows: each round halves the columns that a lane has
#pragma unroll
                for (int o = 16, left = 8; o > 1; o /= 2, left /= 2) {
                    const bool high = lane & o;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < left) {
                            const float keep = high ? kq[c + left] : kq[c], give = high ? kq[c] : kq[c + left];
                            kq[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                }
                kq[0] += __shfl_xor_sync(0xffffffffu, kq[0], 1);
                if (lane % 2 == 0) part[4][warp % 4][quarter * 16 + lane / 2] = kq[0];
            };
            auto put_e = [&] {
#pragma unroll
                for (int c = 0; c < 16; ++c) E[lane_row * C + ((quarter * 16 + c) ^ lane)] = e[c];
            };
            if (Sm::early) {
                ok = await(&kq_done);
                if (!ok) break;
                form_e();
            }
            ok = await(&x_done);
            if (!ok) break;
            // S0 to registers, dS1 in its place
            uint4 s0[DKB][4];
#pragma unroll
            for (int b = 0; b < DKB; ++b)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const unsigned char* from = base + Sm::states + (b * 2 + c) * (kSheetImage / 2) + tid * 16;
                    s0[b][c] = *reinterpret_cast<const uint4*>(from);
                    s0[b][2 + c] = *reinterpret_cast<const uint4*>(from + DKB * kSheetImage);
                }
            fence_shared();
            __syncthreads();
            if (tid == 0) {
                mbar_arrive_expect_tx(&g_full, kStates);
                bulk_g2s(base + Sm::states, slopes, kStates, &g_full);
            }
            // rows of [EA + EA^T; EP] and EP^T, times the scales of K's and Q's rows
            auto pair_to = [&](unsigned img, unsigned second, int r, const float (&v)[2], float down) {
                unsigned hi, lo;
                split_pair(v[0] * down, v[1] * down, hi, lo);
                unsigned char* to = base + img + swizzled(r, 2 * lane);
                *reinterpret_cast<unsigned*>(to) = hi;
                *reinterpret_cast<unsigned*>(to + second) = lo;
            };
            auto at_e = [&](int r, int j) { return E[r * C + (j ^ (r & 31))]; };
            auto convert = [&] {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int r = warp + 16 * a;
                    float ea[2], ep[2], et[2], mk = 0.f, mq = 0.f;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int j = 2 * lane + w;
                        const float ks = fac[kKeyScale + j];
                        ea[w] = (at_e(r, j) + at_e(j, r)) * ks;
                        ep[w] = at_e(C + r, j) * ks;
                        et[w] = at_e(C + j, r) * fac[kQueryScale + j];
                        mk = fmaxf(mk, fmaxf(fabsf(ea[w]), fabsf(et[w])));
                        mq = fmaxf(mq, fabsf(ep[w]));
                    }
                    const Scale sk = scale_of(warp_most(mk)), sq = scale_of(warp_most(mq));
                    pair_to(Sm::a1, kSheetImage, r, ea, sk.down);
                    pair_to(Sm::a1, kSheetImage, C + r, ep, sq.down);
                    pair_to(Sm::a2, kBlock, r, et, sk.down);
                    if (lane == 0) k_scale[r] = sk.up, q_scale[r] = sq.up;
                }
            };
            auto step_products = [&] {
#pragma unroll 1
                for (int r = KP; r >= 0; --r)    // hi lo, lo hi, hi hi
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (leader)
                            mma_ss(tm + cK, desc_rows(sbase + Sm::a1 + (r == 1) * kSheetImage + ks * 32),
                                   desc_columns(kimg + (r == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true), r < KP || ks > 0);
#pragma unroll 1
                for (int r = KP; r >= 0; --r)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (leader)
                            mma_ss(tm + cKE, desc_rows(sbase + Sm::a2 + (r == 1) * kBlock + ks * 32),
                                   desc_columns(qimg + (r == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true), r < KP || ks > 0);
                if (leader) mma_commit(&k_done);
            };
            if (Sm::early) {        // while dS1 is on its way
                put_e();
                __syncthreads();
                convert();
                fence_shared();
            }
            ok = await(&g_full);
            if (!ok) break;
            if (warp == 0) {
#pragma unroll 1
                for (int r = 2; r >= 0; --r)     // U dS1^T
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        if (leader)
                            mma_ss(tm + cX3, desc_kept(sbase + Sm::u + (r == 1) * kSheetImage, ks),
                                   desc_kept(sbase + Sm::states + (r == 2) * DKB * kSheetImage, ks), instr(DKB * 64, true) | 1u << 15,
                                   r < 2 || ks > 0);
                if (leader) mma_commit(&x3_done);
                if (Sm::early) step_products();
            }
            {   // <dS1, S0>
                float dot = 0.f;
#pragma unroll
                for (int b = 0; b < DKB; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const unsigned char* from = base + Sm::states + (b * 2 + c) * (kSheetImage / 2) + tid * 16;
                        const uint4 gh = *reinterpret_cast<const uint4*>(from), gl = *reinterpret_cast<const uint4*>(from + DKB * kSheetImage);
                        const unsigned gs[8] = {gh.x, gh.y, gh.z, gh.w, gl.x, gl.y, gl.z, gl.w};
                        const unsigned ss[8] = {s0[b][c].x, s0[b][c].y, s0[b][c].z, s0[b][c].w, s0[b][2 + c].x, s0[b][2 + c].y, s0[b][2 + c].z, s0[b][2 + c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 a = pair_value(gs[e]), al = pair_value(gs[4 + e]), z = pair_value(ss[e]), zl = pair_value(ss[4 + e]);
                            dot = fmaf(a.x + al.x, z.x + zl.x, fmaf(a.y + al.y, z.y + zl.y, dot));
                        }
                    }
#pragma unroll
                for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (lane == 0) dots[warp] = dot * (g_up * s_up);
            }
            ok = await(&x3_done);
            if (!ok) break;
            if (!Sm::early) {
                fence_shared();
                __syncthreads();
                if (tid == 0) {
                    mbar_arrive_expect_tx(&k_full, Im::keys);
                    bulk_g2s(base + Sm::keys, keys, Im::keys, &k_full);
                }
                ok = await(&k_full);
                if (!ok) break;
                if (warp == 0) key_products();
                ok = await(&kq_done);
                if (!ok) break;
                form_e();
                put_e();
                __syncthreads();
                convert();
                fence_shared();
                __syncthreads();
                if (warp == 0) step_products();
            }
            // in the meantime what the states give, and its sums with K and Q
            const float es = fac[(upper ? kKeyScale : kQueryScale) + i];
            const unsigned char* krow = base + Sm::keys + (upper ? 0 : kBlock);
            auto key_values = [&](int c0, float (&k)[16]) {
#pragma unroll
                for (int c8 = 0; c8 < 2; ++c8) {
                    const unsigned char* row = krow + (c0 / 64) * 2 * kBlock + swizzled(i, c0 % 64 + c8 * 8);
                    const uint4 hi = *reinterpret_cast<const uint4*>(row);
                    uint4 lo = make_uint4(0, 0, 0, 0);
                    if (KP == 2) lo = *reinterpret_cast<const uint4*>(row + DKB * 2 * kBlock);
                    const unsigned his[4] = {hi.x, hi.y, hi.z, hi.w}, los[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 a = pair_value(his[c]), b = pair_value(los[c]);
                        k[c8 * 8 + 2 * c] = KP == 2 ? a.x + b.x : a.x;
                        k[c8 * 8 + 2 * c + 1] = KP == 2 ? a.y + b.y : a.y;
                    }
                }
            };
            {
                const float first = sums.power(i), last = sums.power(C - 1, i);
                const float fx = (upper ? -b_i * r_up : y_up) * s_up * first, f3 = upper ? last * (u_up * g_up) : 0.f;
                float s1 = 0.f, s3 = 0.f;
#pragma unroll
                for (int b = 0; b < DKB; ++b) {
                    const int c0 = quarter * DKB * 16 + b * 16;
                    float x[16], k[16];
                    key_values(c0, k);
                    tmem_ld16(my + cX + c0, x);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        s1 = fmaf(k[c], x[c], s1);
                        acc[b][c] = fmaf(fx, x[c], acc[b][c]);
                    }
                    if (upper) {        // (whole warps are)
                        tmem_ld16(my + cX3 + c0, x);
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            s3 = fmaf(k[c], x[c], s3);
                            acc[b][c] = fmaf(f3, x[c], acc[b][c]);
                        }
                    }
                }
                part[2][quarter][lane_row] = es * ((upper ? r_up : y_up) * s_up * first) * s1;      // e^G k.X2 and e^G q.X1
                part[3][quarter][lane_row] = es * f3 * s3;      // e^(G_last - G) k.X3
            }
            ok = await(&k_done);
            if (!ok) break;
            {
                const float mine = upper ? k_scale[i] : q_scale[i];
#pragma unroll
                for (int b = 0; b < DKB; ++b) {
                    const int c0 = quarter * DKB * 16 + b * 16;
                    float x[16];
                    tmem_ld16(my + cK + c0, x);
#pragma unroll
                    for (int c = 0; c < 16; ++c) acc[b][c] = fmaf(mine, x[c], acc[b][c]);
                    if (upper) {
                        tmem_ld16(my + cKE + c0, x);
#pragma unroll
                        for (int c = 0; c < 16; ++c) acc[b][c] = fmaf(mine, x[c], acc[b][c]);
                    }
                }
            }
            fence_before();
            __syncthreads();
            fence_after();
            // a warp's sum over the steps: of each quarter's D from a step on, of what the states before give from a step
            // on, and of what goes into the state after before a step
            if (warp < 5) {
                float x[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int t = lane + 32 * w;
                    float a = 0.f, b = 0.f;
                    if (warp < 4) {
                        if (warp < 3) a = part[0][warp][t], b = part[0][warp][C + t];
                        else
                            for (int o = 0; o < 4; ++o) a -= part[2][o][t], b += part[2][o][C + t];
                        x[w] = warp < 3 ? a + b : fmaf(fac[kBeta + t], a, b);
                    } else {
                        for (int o = 0; o < 4; ++o) a += part[3][o][t];
                        x[w] = a;
                    }
                }
                const bool back = warp < 4;
#pragma unroll
                for (int o = 1; o < 32; o *= 2)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const float a = back ? __shfl_down_sync(0xffffffffu, x[w], o) : __shfl_up_sync(0xffffffffu, x[w], o);
                        if (back ? lane + o < 32 : lane >= o) x[w] += a;
                    }
                if (back) {
                    x[0] += __shfl_sync(0xffffffffu, x[1], 0);
                    scans[warp][lane] = x[0];
                    scans[warp][lane + 32] = x[1];
                } else {
                    const float all = __shfl_sync(0xffffffffu, x[0], 31);
                    const float a = __shfl_up_sync(0xffffffffu, x[0], 1), b = __shfl_up_sync(0xffffffffu, x[1], 1);
                    scans[4][lane] = lane ? a : 0.f;
                    scans[4][lane + 32] = all + (lane ? b : 0.f);
                }
            } else if (warp < 7) {
                const int t = tid - 5 * 32;
                float s = 0.f, kx2 = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) s += part[1][w][t], kx2 += part[2][w][t];
                db[t] = (tile ? db[t] : 0.f) + s + rv[t] * r_up - kx2;
            } else if (warp == 7) {
                float d = lane < kRestThreads / 32 ? dots[lane] : 0.f;
                for (int o = 16; o; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
                if (lane == 0) carry.x = fac[kWhole] * d;
            }
            __syncthreads();
            if (tid < C) {
                float x = carry.x + scans[4][tid] + scans[3][tid];
                if (tid)
#pragma unroll
                    for (int w = 0; w < 4; ++w) x += part[4][w][tid - 1] + (w < (tid - 1) / 16 ? scans[w][tid] : 0.f);
                if (tile) x += slope[tid];
                slope[tid] = x;
                if (tile == tiles - 1 && tid < steps) {
                    const bool step = t0 + tid < len;
                    const int64_t t = t0 + tid;
                    if (q.dg.data) static_cast<float*>(q.dg.data)[n * q.dg.bs + t * q.dg.ss + h] = step ? x : 0.f;
                    if (q.dbeta.data) static_cast<float*>(q.dbeta.data)[n * q.dbeta.bs + t * q.dbeta.ss + h] = step ? db[tid] : 0.f;
                }
            }
            phase ^= 1u;
            fence_before();
            __syncthreads();        // the next round's images take the place of this one's
            fence_after();
        }
        if (!ok && warp == 0) {     // no product and no copy is in flight when the block ends
            int never = 0;
            if (leader) mma_commit(&done);
            wait(&done, 0, &never);
            for (uint64_t* b : {&first_full, &g_full, &k_full}) {
                never = 0;
                wait(b, phase, &never);
            }
        }
        fence_before();
        __syncthreads();
        if (warp == 0) {
            fence_after();
            tmem_free(tm, kTmem);
        }
        if (tid == 0 && given_up) *p.status = 6;        // RNN_ERR_TIMEOUT
    }
    // Rows of dK and then of dQ through shared memory (nothing reads the first images any more), so that a warp's stores are
    // whole rows: a lane a row, they took 32 lines each.
    constexpr int VEC = 16 / (int)sizeof(T), kUnits = DKB * 64 / VEC, kRowBytes = kUnits * 16 + 16;
    static_assert(128 * kRowBytes <= Sm::states, "");
    unsigned char* rows = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
#pragma unroll
    for (int b = 0; b < DKB; ++b)
#pragma unroll
        for (int c = 0; c < 16; c += VEC) {
            __align__(16) T x[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = from_f<T>(t0 + i < len ? acc[b][c + e] : 0.f);
            *reinterpret_cast<uint4*>(rows + lane_row * kRowBytes + (quarter * DKB * 16 + b * 16 + c) * (int)sizeof(T)) = *reinterpret_cast<const uint4*>(x);
        }
    __syncthreads();
    constexpr int kEach = 128 / (kRestThreads / 32);        // rows of a warp
    const int first = warp * kEach, t1 = first % C;
    const View& to = first < C ? q.dK : q.dQ;
    if (!to.data) return;
    T* at = static_cast<T*>(to.data) + n * to.bs + (t0 + t1) * to.ss + (int64_t)hk * DK;
    if ((uintptr_t)to.data % 16 == 0 && (to.ss | to.bs | DK) % VEC == 0) {
#pragma unroll
        for (int k = 0; k < kEach * kUnits / 32; ++k) {
            const int r = (k * 32 + lane) / kUnits, u = (k * 32 + lane) % kUnits;
            if (t1 + r < steps && u * VEC < DK)
                *reinterpret_cast<uint4*>(at + r * to.ss + u * VEC) = *reinterpret_cast<const uint4*>(rows + (first + r) * kRowBytes + u * 16);
        }
    } else {
        for (int r = 0; r < kEach && t1 + r < steps; ++r)
            for (int d = lane; d < DK; d += 32) at[r * to.ss + d] = reinterpret_cast<const T*>(rows + (first + r) * kRowBytes)[d];
    }
}

template <typename T, int DKB>
cudaError_t run(const DeltaGradParams& q, cudaStream_t st, int* launches)
{
    constexpr int KP = sizeof(T) == 4 ? 2 : 1;
    constexpr size_t chain_smem = ChainSmem<T, DKB, KP>::bytes, rest_smem = RestSmem<DKB, KP>::bytes;
    static std::atomic<uint64_t> chain_done{0}, rest_done{0};
    cudaError_t e = allow_shared(delta_grad_chain_kernel<T, DKB, KP>, chain_smem, chain_done);
    if (e == cudaSuccess) e = allow_shared(delta_grad_rest_kernel<T, DKB, KP>, rest_smem, rest_done);
    if (e != cudaSuccess) return e;
    const DeltaParams& p = q.f;
    delta_grad_chain_kernel<T, DKB, KP><<<heads_grid((p.DV + 127) / 128, p.N * p.H), kChainThreads, chain_smem, st>>>(q);
    ++*launches;
    if (p.S > 0 && (q.dQ.data || q.dK.data || q.dg.data || q.dbeta.data)) {
        delta_grad_rest_kernel<T, DKB, KP><<<heads_grid(delta_chunks(p.S), p.N * p.HK), kRestThreads, rest_smem, st>>>(q);
        ++*launches;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t run(const DeltaGradParams& q, cudaStream_t st, int* launches)
{
    return q.f.DK > 64 ? run<T, 2>(q, st, launches) : run<T, 1>(q, st, launches);
}

}  // namespace

cudaError_t launch_delta_grad(const DeltaGradParams& q, cudaStream_t s, int* launches)
{
    return q.f.io == 0 ? run<float>(q, s, launches) : q.f.io == 1 ? run<__half>(q, s, launches) : run<__nv_bfloat16>(q, s, launches);
}

}  // namespace rnngb
