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
// with (e^G Q)^T dY' while dR is on its way.
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
    __shared__ float most[5][2][128];
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
                // first operand's part a at `from`, a matrix's part b transposed, over the steps
                auto steps_product = [&](uint32_t d, uint32_t from, int a, unsigned img, int b, bool add) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (leader)
                            mma_ts(tm + d, tm + from + ks / 2 * 32 + a * 16 + ks % 2 * 8, desc_columns(img + b * kBlock + ks * 2048, kBlock), instr(C, true), add || ks > 0);
                };
                // the same with K or Q, into G's increment
                auto state_product = [&](uint32_t from, unsigned img) {
#pragma unroll
                    for (int r = 0; r < 1 + KP; ++r)        // hi hi, lo hi, hi lo
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ts(tm + Co::dG, tm + from + ks / 2 * 32 + (r == 1) * 16 + ks % 2 * 8,
                                       desc_columns(img + (r == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true), r > 0 || ks > 0);
                };
                steps_product(Co::PY, Co::X, 0, pimg, 0, false);
                steps_product(Co::PY, Co::X, 0, pimg, 1, true);
                steps_product(Co::PY, Co::X, 1, pimg, 0, true);
                if (!__all_sync(0xffffffffu, wait(&g_ready, ph, &given_up))) break;
                fence_after();
#pragma unroll
                for (int r = 0; r < 1 + KP; ++r)
#pragma unroll
                    for (int ks = 0; ks < DKB * 4; ++ks)
                        if (leader)
                            mma_ts(tm + Co::U, tm + Co::G + (r == 1) * SR + ks * 8, desc_rows(kimg + ((r == 2) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32),
                                   instr(C, false), r > 0 || ks > 0);
                if (leader) mma_commit(&d_ready);
                if (!__all_sync(0xffffffffu, wait(&u_told, ph, &given_up))) break;
                fence_after();
                steps_product(Co::R, Co::U, 0, timg, 0, false);
                steps_product(Co::R, Co::U, 0, timg, 1, true);
                steps_product(Co::R, Co::U, 1, timg, 0, true);
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
        auto put_dy = [&](int k, int which, int meeting, float& up, bool ok) {
            float most_y = 0.f;
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
                    y[2 * i] = mul2(a.x, w0);
                    y[2 * i + 1] = mul2(a.y, w1);
                    most_y = most_of(most_of(most_y, y[2 * i]), y[2 * i + 1]);
                }
            }
            if (!both(meeting, most_y, ok)) return false;
            const Scale e = scale_of(most_y);
            put_parts(my + Co::X + half * 32, my + Co::X + half * 32 + 16, y, e.down);
            tmem_st_wait();
            up = e.up;
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
                if (!put_dy(k, kP, 4, py_up, ok)) break;
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
            if (!both(3, m, ok)) break;
            const Scale eg = scale_of(m);
#pragma unroll
            for (int r = 0; r < DKB; ++r)
                put_parts(my + Co::G + d0 / 2 + r * 16, my + Co::G + SR + d0 / 2 + r * 16, G + r * 16, eg.down);
            tmem_st_wait();
            tell(&g_ready);
            const int64_t chunk = live - 1 - k;
            if (col) write_state(q.ends + (nh * chunks + chunk) * p.DK * p.DV + v);
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
            if (!put_dy(k, kQuery, 1, qy_up, ok)) break;
            tell(&x2_ready);
            if constexpr (Sm::staged)
                if (lane == 0) mbar_arrive(&v_empty[k & 1]);
            ok = __all_sync(0xffffffffu, wait(&r_ready, ph, &given_up));
            m = 0.f;
            if (ok) {
                fence_after();
                tmem_ld(my + Co::R + half * 32, x);
                const f2 up = dup2(eu.up), minus = dup2(-1.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 a = factors(fac, kDecayed, i);
                    x[2 * i] = mul2(x[2 * i], up);
                    x[2 * i + 1] = mul2(x[2 * i + 1], up);
                    y[2 * i] = mul2(mul2(a.x, minus), x[2 * i]);
                    y[2 * i + 1] = mul2(mul2(a.y, minus), x[2 * i + 1]);
                    m = most_of(most_of(m, y[2 * i]), y[2 * i + 1]);
                }
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
            if (col) {
                float* to = q.drs + ((nh * chunks + chunk) * C + half * 32) * p.DV + v;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float a, b;
                    unpack2(x[i], a, b);
                    *to = a;
                    to += p.DV;
                    *to = b;
                    to += p.DV;
                }
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

// The rest, a chunk and key head a block.  With [U; dR; dY'] as rows of one buffer, their products with the two states and with
// U are
//     [dR; dY'] S0^T = [X2; X1],   [dR; dY'] U^T = [-dA; dP],   [U; dR] dS1^T = [X3; not wanted],
// 128 rows each: a lane of tensor memory is a step, in the upper half of dR's results, in the lower of dY''s.  Then [K; Q] K^T
// again, and [EA + EA^T; EP] K and [EP^T; 0] Q.  Everything is read from memory once, as fp32 rows that a warp
// takes to parts (a row's values are the products' sums' direction, so its scale is the result's); the
// reads are what bounds it: 256 KB a chunk and head of 128 x 128, at 16 bits.
constexpr int kRestThreads = 512;
template <int DKB>
struct RestSmem {
    static constexpr unsigned row_block = 192 * 128, state_block = DKB * kBlock;
    static constexpr unsigned rows = 0, states = 4 * row_block, e = states + 4 * state_block, end = e + 128 * C * 4;
    // once the rows are done with: [EA + EA^T; EP], [EP^T; 0] and D; in place of the states, K and Q
    static constexpr unsigned a1 = 0, a2 = 4 * kBlock, d = 8 * kBlock;
    static constexpr size_t bytes = end + 1024;
    static_assert(d + 128 * C * 4 <= states, "");
};

template <typename T, int DKB, int KP>
__global__ void __launch_bounds__(kRestThreads, 1) delta_grad_rest_kernel(const DeltaGradParams q)
{
    using Im = Images<DKB, KP>;
    using Sm = RestSmem<DKB>;
    constexpr uint32_t cX = 0, cE = 128, cX3 = 192, cK = 320, cKQ = 448;     // columns of tensor memory
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ __align__(8) uint64_t bar[4], images, done;
    __shared__ Sums sums;
    __shared__ float scale[192], s_scale[128], g_scale[128], k_scale[C], q_scale[C];
    __shared__ float fac[768];
    __shared__ float rv[C], part[4][4][128], dots[kRestThreads / 32], slope[C], end[C];
    __shared__ double carry;
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
    const View& out = upper ? q.dK : q.dQ;
    float acc[DKB][16];
#pragma unroll
    for (int b = 0; b < DKB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[b][e] = 0.f;
    if (t0 >= len) {
        for (int j = tid; j < steps * p.H; j += kRestThreads) {
            const int t = j / p.H, h = j - t * p.H;
            if (h / per != hk) continue;
            if (q.dg.data) static_cast<float*>(q.dg.data)[n * q.dg.bs + (t0 + t) * q.dg.ss + h] = 0.f;
            if (q.dbeta.data) static_cast<float*>(q.dbeta.data)[n * q.dbeta.bs + (t0 + t) * q.dbeta.ss + h] = 0.f;
        }
    } else {
        unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
        float *E = reinterpret_cast<float*>(base + Sm::e), *D = reinterpret_cast<float*>(base + Sm::d);
        if (tid == 0) {
            for (int b = 0; b < 4; ++b) mbar_init(&bar[b], 1);
            mbar_init(&images, 1);
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
        unsigned phase[3] = {0, 0, 0};      // of bar[0], of bar[1], of the rest (once a head)
        // all threads wait, and know whether all did
        auto await = [&](uint64_t* b, unsigned ph) {
            const bool ok = __syncthreads_and(wait(b, ph, &given_up));
            fence_after();
            return ok;
        };
        bool ok = true;
        for (int h = hk * per; h < (hk + 1) * per && ok; ++h) {
            const int64_t nh = n * p.H + h, at = nh * chunks + chunk;
            const float *us = p.us + at * C * DV, *drs = q.drs + at * C * DV, *states = p.states + at * DK * DV, *ends = q.ends + at * DK * DV;
            const bool wide = DV % 4 == 0 && ((uintptr_t)p.us | (uintptr_t)p.states) % 16 == 0 && ((uintptr_t)q.drs | (uintptr_t)q.ends) % 16 == 0;
            const bool yw = fours<T>(q.dY, DV), vw = fours<T>(p.V, DV);
            for (int j = tid; j < 192; j += kRestThreads)
                reinterpret_cast<float4*>(fac)[j] = reinterpret_cast<const float4*>(p.mats + at * Im::mats + 4 * kBlock)[j];
            form_sums(sums, p.g, n, h, t0, len, &carry);
            // a row's scale; where it has more values than a tile, its others are looked through first
            auto row_scale = [&](const auto* row, bool in, bool vec, const float (&x)[4]) {
                float m = row_most(x);
                if (tiles > 1)
                    for (int v = 0; v < DV; v += 128) {
                        float z[1][4];
                        load_fours<1>(row + v, 0, DV - v, vec, [&](int) { return in; }, z);
                        m = fmaxf(m, row_most(z[0]));
                    }
                return scale_of(m);
            };
            float rv_mine = 0.f, dot = 0.f;     // lane l: the sum for the warp's l-th row of dR
            for (int tile = 0; tile < tiles && ok; ++tile) {
                const int v0 = tile * 128;
                const bool second = DV - v0 > 64;       // two blocks of 64 values
                const int left = DV - v0;
                // a warp's rows: every 16th of U, dR, dY' and V, then of S0
                auto step_in = [&](int a) { return t0 + warp + 16 * a < len; };
                auto key_in = [&](int a) { return warp + 16 * a < DK; };
                auto always = [](int) { return true; };
                const float *u_row = us + warp * (int64_t)DV, *r_row = drs + warp * (int64_t)DV, *s_row = states + warp * (int64_t)DV;
                const T* y_row = static_cast<const T*>(q.dY.data) + n * q.dY.bs + (t0 + warp) * q.dY.ss + (int64_t)h * DV;
                const T* v_row = static_cast<const T*>(p.V.data) + n * p.V.bs + (t0 + warp) * p.V.ss + (int64_t)h * DV;
                {
                    float x[4][4], y[4][4], z[4][4], w[4][4];
                    load_fours<4>(u_row + v0, 16 * (int64_t)DV, left, wide, always, x);
                    load_fours<4>(r_row + v0, 16 * (int64_t)DV, left, wide, always, y);
                    load_fours<4>(y_row + v0, 16 * q.dY.ss, left, yw, step_in, z);
                    load_fours<4>(v_row + v0, 16 * p.V.ss, left, vw, step_in, w);
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const int r = warp + 16 * a;
                        const Scale su = row_scale(u_row + a * 16 * (int64_t)DV, true, wide, x[a]);
                        const Scale sr = row_scale(r_row + a * 16 * (int64_t)DV, true, wide, y[a]);
                        const Scale sy = row_scale(y_row + a * 16 * q.dY.ss, step_in(a), yw, z[a]);
                        put_row<2, 2>(base + Sm::rows, Sm::row_block, r, x[a], su.down);
                        put_row<2, 2>(base + Sm::rows, Sm::row_block, C + r, y[a], sr.down);
                        put_row<2, 2>(base + Sm::rows, Sm::row_block, 2 * C + r, z[a], sy.down);
                        float s = y[a][0] * w[a][0] + y[a][1] * w[a][1] + y[a][2] * w[a][2] + y[a][3] * w[a][3];
#pragma unroll
                        for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
                        if (lane == a) rv_mine += s;
                        if (lane == 0) {
                            scale[r] = su.up;
                            scale[C + r] = sr.up;
                            scale[2 * C + r] = p.scale * sy.up;
                        }
                    }
                }
                {
                    float x[DKB * 4][4];
                    load_fours<DKB * 4>(s_row + v0, 16 * (int64_t)DV, left, wide, key_in, x);
#pragma unroll
                    for (int a = 0; a < DKB * 4; ++a) {
                        const int d = warp + 16 * a;
                        const Scale sc = row_scale(s_row + a * 16 * (int64_t)DV, d < DK, wide, x[a]);
                        put_row<2, 2>(base + Sm::states, Sm::state_block, d, x[a], sc.down);
                        if (lane == 0) s_scale[d] = sc.up;
                    }
                }
                fence_shared();
                __syncthreads();
                const unsigned rows = sbase + Sm::rows, sts = sbase + Sm::states;
                // parts a of the rows from `first` on, b of the other side, over the tile's values
                auto product = [&](uint32_t d, int first, int a, unsigned other, unsigned apart, int b, int nn, bool add) {
                    for (int blk = 0; blk < (second ? 2 : 1); ++blk)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ss(tm + d, desc_rows(rows + (a * 2 + blk) * Sm::row_block + first * 128 + ks * 32),
                                       desc_rows(other + (b * 2 + blk) * apart + ks * 32), instr(nn, false), add || blk > 0 || ks > 0);
                };
                if (warp == 0) {
                    product(cX, C, 0, sts, Sm::state_block, 0, DKB * 64, tile > 0);
                    product(cX, C, 0, sts, Sm::state_block, 1, DKB * 64, true);
                    product(cX, C, 1, sts, Sm::state_block, 0, DKB * 64, true);
                    product(cE, C, 0, rows, Sm::row_block, 0, C, tile > 0);
                    product(cE, C, 0, rows, Sm::row_block, 1, C, true);
                    product(cE, C, 1, rows, Sm::row_block, 0, C, true);
                    if (leader) mma_commit(&bar[0]);
                }
                // dS1 in the meantime, and <dS1, S0> with S0 as its parts have it
                float g[DKB * 4][4];
                const float* e_row = ends + warp * (int64_t)DV;
                load_fours<DKB * 4>(e_row + v0, 16 * (int64_t)DV, left, wide, key_in, g);
#pragma unroll
                for (int a = 0; a < DKB * 4; ++a) {
                    const int d = warp + 16 * a, c = lane * 4;
                    const unsigned char* hi = base + Sm::states + c / 64 * Sm::state_block + swizzled(d, c % 64);
                    const uint2 u = *reinterpret_cast<const uint2*>(hi), w = *reinterpret_cast<const uint2*>(hi + 2 * Sm::state_block);
                    const float2 u0 = pair_value(u.x), u1 = pair_value(u.y), w0 = pair_value(w.x), w1 = pair_value(w.y);
                    dot = fmaf(s_scale[d], g[a][0] * (u0.x + w0.x) + g[a][1] * (u0.y + w0.y) + g[a][2] * (u1.x + w1.x) + g[a][3] * (u1.y + w1.y), dot);
                }
                ok = await(&bar[0], phase[0]);
                phase[0] ^= 1u;
                if (!ok) break;
#pragma unroll
                for (int a = 0; a < DKB * 4; ++a) {
                    const int d = warp + 16 * a;
                    const Scale sc = row_scale(e_row + a * 16 * (int64_t)DV, d < DK, wide, g[a]);
                    put_row<2, 2>(base + Sm::states, Sm::state_block, d, g[a], sc.down);
                    if (lane == 0) g_scale[d] = sc.up;
                }
                fence_shared();
                __syncthreads();
                if (warp == 0) {
                    product(cX3, 0, 0, sts, Sm::state_block, 0, DKB * 64, tile > 0);
                    product(cX3, 0, 0, sts, Sm::state_block, 1, DKB * 64, true);
                    product(cX3, 0, 1, sts, Sm::state_block, 0, DKB * 64, true);
                    if (leader) mma_commit(&bar[1]);
                }
                ok = await(&bar[1], phase[1]);
                phase[1] ^= 1u;
            }
            if (!ok) break;
            if (lane < 4) rv[warp + 16 * lane] = rv_mine;
#pragma unroll
            for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (lane == 0) dots[warp] = dot;
            if (tid == 0) {
                mbar_arrive_expect_tx(&images, Im::keys);
                bulk_g2s(base + Sm::states, p.keys + (nk * chunks + chunk) * Im::keys, Im::keys, &images);
            }
            ok = await(&images, phase[2]);
            if (!ok) break;
            const unsigned kimg = sbase + Sm::states, qimg = kimg + kBlock;
            if (warp == 0) {
#pragma unroll
                for (int r = 0; r < 2 * KP - 1; ++r)         // hi hi, lo hi, hi lo
#pragma unroll
                    for (int ks = 0; ks < DKB * 4; ++ks)
                        if (leader)
                            mma_ss(tm + cKQ, desc_rows(kimg + ((r == 1) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32),
                                   desc_rows(kimg + ((r == 2) * DKB + ks / 4) * 2 * kBlock + ks % 4 * 32), instr(C, false), r > 0 || ks > 0);
                if (leader) mma_commit(&bar[2]);
            }
            ok = await(&bar[2], phase[2]);
            if (!ok) break;
            const float b_i = fac[kBeta + i];
            {
                float e[16], kq[16], row = 0.f, db = 0.f;
                tmem_ld16(my + cE + quarter * 16, e);
                tmem_ld16(my + cKQ + quarter * 16, kq);
                const float mine = scale[upper ? C + i : 128 + i], es = fac[(upper ? kKeyScale : kQueryScale) + i];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int j = quarter * 16 + c;
                    const bool in = upper ? j < i : j <= i;
                    const float decay = in ? expf(sums.between(i, j)) : 0.f;
                    const float d = in ? (upper ? -e[c] : e[c]) * (mine * scale[j]) * decay : 0.f;
                    const float k = in ? kq[c] * (es * fac[kKeyScale + j]) : 0.f;
                    const float v = upper ? b_i * d : d;
                    db = fmaf(d, k, db);
                    E[lane_row * C + (j ^ lane)] = v;
                    D[lane_row * C + (j ^ lane)] = v * k;
                    row = fmaf(v, k, row);
                }
                part[0][quarter][lane_row] = row;
                part[1][quarter][lane_row] = db;
            }
            __syncthreads();
            // rows of [EA + EA^T; EP] and [EP^T; 0], times the scales of K's and Q's rows
            auto pair_to = [&](unsigned img, int r, const float (&v)[2], float down) {
                unsigned hi, lo;
                split_pair(v[0] * down, v[1] * down, hi, lo);
                unsigned char* to = base + img + swizzled(r, 2 * lane);
                *reinterpret_cast<unsigned*>(to) = hi;
                *reinterpret_cast<unsigned*>(to + 2 * kBlock) = lo;
            };
            auto at_e = [&](int r, int j) { return E[r * C + (j ^ (r & 31))]; };
            for (int r = warp; r < C; r += 16) {
                float ea[2], ep[2], et[2], mk = 0.f, mq = 0.f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int j = 2 * lane + w;
                    ea[w] = (at_e(r, j) + at_e(j, r)) * fac[kKeyScale + j];
                    ep[w] = at_e(C + r, j) * fac[kKeyScale + j];
                    et[w] = at_e(C + j, r) * fac[kQueryScale + j];
                    mk = fmaxf(mk, fmaxf(fabsf(ea[w]), fabsf(et[w])));
                    mq = fmaxf(mq, fabsf(ep[w]));
                }
#pragma unroll
                for (int o = 16; o; o /= 2) {
                    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
                    mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
                }
                const Scale sk = scale_of(mk), sq = scale_of(mq);
                pair_to(Sm::a1, r, ea, sk.down);
                pair_to(Sm::a1, C + r, ep, sq.down);
                pair_to(Sm::a2, r, et, sk.down);
                const float zero[2] = {0.f, 0.f};
                pair_to(Sm::a2, C + r, zero, 1.f);
                if (lane == 0) k_scale[r] = sk.up, q_scale[r] = sq.up;
            }
            fence_shared();
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 0; w < 2; ++w)             // with K, with Q
#pragma unroll
                    for (int r = 0; r < 1 + KP; ++r)    // hi hi, lo hi, hi lo
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (leader)
                                mma_ss(tm + cK, desc_rows(sbase + (w ? Sm::a2 : Sm::a1) + (r == 1) * 2 * kBlock + ks * 32),
                                       desc_columns((w ? qimg : kimg) + (r == 2) * DKB * 2 * kBlock + ks * 2048, 2 * kBlock), instr(DKB * 64, true),
                                       w > 0 || r > 0 || ks > 0);
                if (leader) mma_commit(&bar[3]);
            }
            // in the meantime what the states give, and its sums with K and Q
            {
                const float first = expf(sums.hi[i] + sums.lo[i]), last = expf(sums.between(C - 1, i));
                const float mine = scale[upper ? C + i : 128 + i], own = scale[i];
                const float es = fac[(upper ? kKeyScale : kQueryScale) + i];
                const unsigned char* img = base + Sm::states + (upper ? 0 : kBlock);
                float s1 = 0.f, s3 = 0.f;
#pragma unroll
                for (int b = 0; b < DKB; ++b) {
                    const int c0 = quarter * DKB * 16 + b * 16;
                    float x1[16], x3[16];
                    tmem_ld16(my + cX + c0, x1);
                    tmem_ld16(my + cX3 + c0, x3);
#pragma unroll
                    for (int c8 = 0; c8 < 2; ++c8) {
                        const unsigned char* row = img + (c0 / 64) * 2 * kBlock + swizzled(i, c0 % 64 + c8 * 8);
                        const uint4 hi = *reinterpret_cast<const uint4*>(row);
                        uint4 lo = make_uint4(0, 0, 0, 0);
                        if (KP == 2) lo = *reinterpret_cast<const uint4*>(row + DKB * 2 * kBlock);
                        const unsigned his[4] = {hi.x, hi.y, hi.z, hi.w}, los[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int cc = c8 * 8 + c;
                            const float2 u = pair_value(his[c / 2]), w = pair_value(los[c / 2]);
                            const float k = (c % 2 ? u.y : u.x) + (KP == 2 ? (c % 2 ? w.y : w.x) : 0.f);
                            const float a = x1[cc] * (mine * s_scale[c0 + cc]), z = x3[cc] * (own * g_scale[c0 + cc]);
                            s1 = fmaf(k, a, s1);
                            s3 = fmaf(k, z, s3);
                            acc[b][cc] += upper ? last * z - b_i * first * a : first * a;
                        }
                    }
                }
                part[2][quarter][lane_row] = s1 * es;
                part[3][quarter][lane_row] = s3 * es;
            }
            ok = await(&bar[3], phase[2]);
            phase[2] ^= 1u;
            if (!ok) break;
            {
                const float mine = upper ? k_scale[i] : q_scale[i];
#pragma unroll
                for (int b = 0; b < DKB; ++b) {
                    float x[16];
                    tmem_ld16(my + cK + quarter * DKB * 16 + b * 16, x);
#pragma unroll
                    for (int c = 0; c < 16; ++c) acc[b][c] = fmaf(mine, x[c], acc[b][c]);
                }
            }
            // the decays' slopes, and their sums from each step to the chunk's end
            if (tid < C) {
                const float first = expf(sums.hi[tid] + sums.lo[tid]), last = expf(sums.between(C - 1, tid)), b = fac[kBeta + tid];
                float rowsum = 0.f, db = 0.f, qx1 = 0.f, kx2 = 0.f, kx3 = 0.f, column = 0.f;
                for (int w = 0; w < 4; ++w) {
                    rowsum += part[0][w][tid] + part[0][w][C + tid];
                    db += part[1][w][tid];
                    kx2 += part[2][w][tid];
                    qx1 += part[2][w][C + tid];
                    kx3 += part[3][w][tid];
                }
                for (int r = 0; r < 128; ++r) column += D[r * C + (tid ^ (r & 31))];
                kx3 *= last;
                end[tid] = kx3;
                slope[tid] = rowsum - column + first * (qx1 - b * kx2) - kx3;
                const bool step = t0 + tid < len;
                if (q.dbeta.data && tid < steps)
                    static_cast<float*>(q.dbeta.data)[n * q.dbeta.bs + (t0 + tid) * q.dbeta.ss + h] = step ? db + rv[tid] - first * kx2 : 0.f;
            }
            __syncthreads();
            if (tid < 32) {
                float all = end[tid] + end[tid + 32], d = tid < kRestThreads / 32 ? dots[tid] : 0.f;
                for (int o = 16; o; o /= 2) {
                    all += __shfl_xor_sync(0xffffffffu, all, o);
                    d += __shfl_xor_sync(0xffffffffu, d, o);
                }
                all += fac[kWhole] * d;
                float hi = slope[tid + 32], lo = slope[tid];
                if (tid == 31) hi += all;
                for (int o = 1; o < 32; o *= 2) {
                    const float a = __shfl_down_sync(0xffffffffu, hi, o), b = __shfl_down_sync(0xffffffffu, lo, o);
                    if (tid + o < 32) {
                        hi += a;
                        lo += b;
                    }
                }
                lo += __shfl_sync(0xffffffffu, hi, 0);
                if (q.dg.data) {
                    float* dg = static_cast<float*>(q.dg.data) + n * q.dg.bs + h;
                    if (tid < steps) dg[(t0 + tid) * q.dg.ss] = t0 + tid < len ? lo : 0.f;
                    if (tid + 32 < steps) dg[(t0 + tid + 32) * q.dg.ss] = t0 + tid + 32 < len ? hi : 0.f;
                }
            }
            fence_before();
            __syncthreads();        // the next head's rows take the place of this one's
            fence_after();
        }
        if (!ok && warp == 0) {     // no product is in flight when the block ends
            int never = 0;
            if (leader) mma_commit(&done);
            wait(&done, 0, &never);
        }
        fence_before();
        __syncthreads();
        if (warp == 0) {
            fence_after();
            tmem_free(tm, kTmem);
        }
        if (tid == 0 && given_up) *p.status = 6;        // RNN_ERR_TIMEOUT
    }
    if (out.data && i < steps) {
        T* row = static_cast<T*>(out.data) + n * out.bs + (t0 + i) * out.ss + (int64_t)hk * DK;
        const bool in = t0 + i < len;
        constexpr int VEC = 16 / (int)sizeof(T);
        const bool vec = (uintptr_t)out.data % 16 == 0 && (out.ss | out.bs | DK) % VEC == 0;
#pragma unroll
        for (int b = 0; b < DKB; ++b) {
            const int d0 = quarter * DKB * 16 + b * 16;
#pragma unroll
            for (int c = 0; c < 16; c += VEC) {
                __align__(16) T x[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = from_f<T>(in ? acc[b][c + e] : 0.f);
                if (vec) {
                    if (d0 + c < DK) *reinterpret_cast<uint4*>(row + d0 + c) = *reinterpret_cast<const uint4*>(x);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (d0 + c + e < DK) row[d0 + c + e] = x[e];
                }
            }
        }
    }
}

template <typename T, int DKB>
cudaError_t run(const DeltaGradParams& q, cudaStream_t st, int* launches)
{
    constexpr int KP = sizeof(T) == 4 ? 2 : 1;
    constexpr size_t chain_smem = ChainSmem<T, DKB, KP>::bytes, rest_smem = RestSmem<DKB>::bytes;
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
