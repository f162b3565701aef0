// Selective state space scan (the formulas stand in include/onnx_recurrent.h).
//
// Work of one state update h = exp(delta A) h + delta X B, y += C h: one
// exponential (32 lanes a clock and SM, measured) and four fp32 operations
// (128 lanes a clock and SM): both pipes take 4/128 of a clock, so 152 SMs at
// 1.92 GHz need 107 ns for a million updates; the bytes of X, dt, Z and Y
// (8 a channel and step in 16-bit types, 16 updates with M = 16) need 74 ns.
// What the kernel adds to the four operations is kept small:
//   - a lane holds four states of four neighbouring channels: a step's B and C
//     are read once for four channels, delta and delta X once for four states
//     (shared memory returns 128 bytes a clock, whoever asks for the same);
//   - channels are packed in pairs (ssm_tile.cuh): half the issue slots;
//   - delta and delta X are formed once per channel and step, and Y's gate
//     and rounding applied once, by elementwise passes over tiles of T = 16
//     steps; the passes and the loop in between share a warp's own part of
//     shared memory, so a tile costs the block two barriers;
//   - the sum over a channel's lanes goes with the channels, halving the
//     values each time; in the first exchange each lane sends its second pair
//     of channels, which for odd lanes is the first in memory, so nothing is
//     selected.
// The next tile's inputs are copied while a tile is computed.
//
// Measured (38 rows of 1024 steps, 2048 channels, M = 16, bf16: all SMs full):
// 395 us, 3200 updates a ns, a third of the pipes' bound.  Counters: issue slots
// 59 % busy, fp32 pipe 58 %, shared memory 52 %, exponentials 38 %, DRAM 17 %; with
// parts left out, the loop over steps takes 64 % of the time (its loads and
// exchanges half of that), softplus and gate 9 %, copies 7 %, the rest goes to
// the passes' shared memory and barriers.  Four steps a loop body instead of U: 4 %
// slower.  Tried (512 steps, 206 us then) and no faster: 8 channels a lane (252 us, fewer
// warps), 2 (337 us), scalar instead of packed operations, 8 or 32 steps a tile,
// 5 to 8 blocks an SM.
//
// When rows and channels are too few for the SMs, the steps are split in
// chunks: one launch finds each chunk's end state from zero and the sum of
// its delta (the product of its decays is exp(A sum delta)), and the scan runs over
// all chunks at once, each from its first state: with up to kFold chunks the
// block chains the end states before its own, with more a small launch in between
// chains them for all.  That costs another exponential and three operations per update.
#include <cmath>

#include "ssm_tile.cuh"

#pragma nv_diag_suppress 128   // loops that a launch for end states leaves out

namespace rnngb {
namespace {

constexpr int E = 4;              // states of a lane
constexpr int CH = 4;             // channels of a lane
constexpr int T = 16;             // steps of a tile in shared memory
constexpr int U = 8;              // steps of the inner loop's body
constexpr int kFold = 16;         // chunks whose states a block chains itself
struct ScanLaunch {
    int cblocks;          // blocks of channels in a group
    int64_t chunk;        // steps of a chunk (a multiple of T)
    int chunks;
    bool fast_x, fast_dt, fast_z, fast_b, fast_c, vec_y, vec_h, vec_s;
    float* ends;          // [chunks - 1][N][D][M]: end states, then first states of chunks 1 ..
    float* deltas;        // [chunks - 1][N][D]
};

// A block's shape and its shared memory.
template <typename V, int L>
struct Tile {
    static constexpr int W = L >= 4 ? 4 : L;               // warps
    static constexpr int THREADS = 32 * W;
    static constexpr int WC = 32 / L * CH;                 // channels of a warp
    static constexpr int ME = L * E;                       // states, padded
    static constexpr int PW = WC + 4;                      // pitch of delta and delta X
    static constexpr int NV = WC < 4 ? WC : 4;             // channels of an elementwise access
    using Rows = Stager<V, T, W * WC, THREADS>;            // of X, dt, Z
    using Pairs = Stager<V, T, ME, THREADS>;               // of B, C
    static constexpr int RX = T * Rows::PITCH, RB = T * Pairs::PITCH;
    static constexpr size_t bytes(int raws)
    {
        return sizeof(V) * 2 * (size_t)(raws * RX + 2 * RB) + sizeof(float) * 2 * T * ME + sizeof(float) * 2 * W * (T * PW + WC);
    }
};

template <typename V, int L, bool ENDS>
__global__ void __launch_bounds__(Tile<V, L>::THREADS, 16 / Tile<V, L>::W)
    ssm_scan_kernel(const ScanParams p, const ScanLaunch q)
{
    using K = Tile<V, L>;
    constexpr int RAWS = ENDS ? 2 : 3, PAIRS = CH / 2, NP = K::NV / 2;
    extern __shared__ __align__(16) char smem[];
    V* raw = reinterpret_cast<V*>(smem);                          // [2][RAWS][T][..]: dt, X, Z
    V* rawbc = raw + 2 * RAWS * K::RX;                            // [2][2][T][..]: B, C
    float* bc = reinterpret_cast<float*>(rawbc + 2 * 2 * K::RB);  // [T][2][ME]: B, C
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float* sd = bc + 2 * T * K::ME + warp * 2 * (T * K::PW + K::WC);   // the warp's delta
    float* sx = sd + T * K::PW;                                   // delta X, then y
    float* sb = sx + T * K::PW;                                   // dt_bias and Dskip of its channels

    unsigned blk = blockIdx.x;
    const int cb = blk % q.cblocks;
    blk /= q.cblocks;
    const int g = blk % p.G;
    blk /= p.G;
    const int64_t n = blk % (unsigned)p.N;
    const int chunk = blk / (unsigned)p.N;
    const int64_t dg = p.D / p.G;
    const int64_t c0 = (int64_t)cb * K::W * K::WC;                // first channel in the group
    const int valid = dg - c0 < K::W * K::WC ? (int)(dg - c0) : K::W * K::WC;
    const int64_t d0 = g * dg + c0;
    const int64_t len = row_length(p.lens, n, p.S, p.status);
    const int64_t t_first = chunk * q.chunk;
    const int64_t t_end = t_first + q.chunk < p.S ? t_first + q.chunk : p.S;
    const int64_t live = len < t_end ? len : t_end;               // steps of the row end here

    // this lane's channels (of the warp's) and states
    const int sg = lane % L, cg = lane / L;
    // Exchanges over a channel's lanes: one that halves the pairs (SPLIT), then
    // one that halves the last pair (HALVE), if there are lanes for them.
    constexpr int SPLIT = L >= 2 ? 1 : 0, LEFT = PAIRS >> SPLIT;
    constexpr bool HALVE = LEFT == 1 && L > (1 << SPLIT);
    const bool up = HALVE && (sg >> SPLIT & 1);
    static_assert(PAIRS == 2, "the exchanges are those of two pairs");
    int ch[PAIRS];                                                // first channel of each pair
#pragma unroll
    for (int r = 0; r < PAIRS; ++r) {
        const int at = SPLIT && sg & 1 ? r ^ 1 : r;               // what the lane keeps, and what it sends
        ch[r] = cg * CH + 2 * at;
    }
    f2 A[E][PAIRS], h[E][PAIRS];
    // the lane's part of an [.., D, M] table's row n
    auto table = [&](f2 (&v)[E][PAIRS], const float* from, bool vec, float scale) {
#pragma unroll
        for (int r = 0; r < PAIRS; ++r) {
            float s[2][E];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = warp * K::WC + ch[r] + i;
                const float* at = from + (d0 + c) * p.M + sg * E;
                if (vec && from && c < valid && sg * E < p.M) {
                    load_vec<float, E>(at, s[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) s[i][j] = from && c < valid && sg * E + j < p.M ? at[j] : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < E; ++j) v[j][r] = pack2(s[0][j] * scale, s[1][j] * scale);
        }
    };
    table(A, p.A, false, kLog2e);
    {
        const int64_t states = p.N * p.D * p.M, row = n * p.D * p.M;
        const bool fold = q.chunks <= kFold;
        const float* first = ENDS ? nullptr : chunk == 0 || fold ? p.h0 : q.ends + (chunk - 1) * states;
        table(h, first ? first + row : nullptr, false, 1.0f);
        if (!ENDS && fold) {
#pragma unroll 2
            for (int k = 0; k < chunk; ++k) {
                f2 end[E][PAIRS];
                table(end, q.ends + k * states + row, q.vec_h, 1.0f);
                const float* delta = q.deltas + (k * p.N + n) * p.D + d0 + warp * K::WC;
#pragma unroll
                for (int r = 0; r < PAIRS; ++r) {
                    const bool on = warp * K::WC + ch[r] < valid, both = warp * K::WC + ch[r] + 1 < valid;
                    const f2 d = pack2(on ? delta[ch[r]] : 0.0f, both ? delta[ch[r] + 1] : 0.0f);
#pragma unroll
                    for (int j = 0; j < E; ++j) h[j][r] = fma2(ex2_2(mul2(d, A[j][r])), h[j][r], end[j][r]);
                }
            }
        }
    }

    // elementwise accesses: NV channels from ec on, steps er, er + ROWS, ..
    constexpr int PER_ROW = K::WC / K::NV, ROWS = 32 / PER_ROW;
    const int ev = lane % PER_ROW * K::NV, er = lane / PER_ROW;
    const int ec = warp * K::WC + ev;                             // channel in the block
    const int some = valid - ec < K::NV ? (valid - ec > 0 ? valid - ec : 0) : K::NV;
    f2 total[ENDS ? NP : 1];
#pragma unroll
    for (int e = 0; e < (ENDS ? NP : 1); ++e) total[e] = 0;
    for (int i = lane; i < 2 * K::WC; i += 32) {
        const int c = warp * K::WC + i % K::WC;
        const float* from = i < K::WC ? p.dt_bias : p.Dskip;
        sb[i] = from && c < valid ? from[d0 + c] : 0.0f;
    }
    __syncwarp();

    const bool gate = !ENDS && p.Z.data;
    auto stage = [&](int k) {
        const int64_t t0 = t_first + (int64_t)k * T, left = live - t0, row = anew(n);
        const int steps = left < T ? (int)left : T;
        V* r = raw + (k & 1) * RAWS * K::RX;
        V* b = rawbc + (k & 1) * 2 * K::RB;
        K::Rows::copy(r, p.dt, row, t0, d0, steps, valid, q.fast_dt);
        K::Rows::copy(r + K::RX, p.X, row, t0, d0, steps, valid, q.fast_x);
        if (gate) K::Rows::copy(r + 2 * K::RX, p.Z, row, t0, d0, steps, valid, q.fast_z);
        K::Pairs::copy(b, p.B, row, t0, (int64_t)g * p.M, steps, p.M, q.fast_b);
        if (!ENDS) K::Pairs::copy(b + K::RB, p.C, row, t0, (int64_t)g * p.M, steps, p.M, q.fast_c);
        cp_async_commit();
    };
    const int tiles = live > t_first ? (int)((live - t_first + T - 1) / T) : 0;
    if (tiles) stage(0);
    for (int k = 0; k < tiles; ++k) {
        const int64_t left = live - t_first - (int64_t)k * T;
        const int steps = left < T ? (int)left : T;
        const int buf = k & 1;
        cp_async_wait<0>();
        __syncthreads();                       // tile k has landed; tile k-1's buffers are free
        if (k + 1 < tiles) stage(k + 1);
        const V* r = raw + buf * RAWS * K::RX + ec;
        const V* b = rawbc + buf * 2 * K::RB;
        for (int i = threadIdx.x; i < T * K::ME; i += K::THREADS) {
            const int t = i / K::ME, m = i % K::ME;
            bc[t * 2 * K::ME + m] = to_f(b[t * K::Pairs::PITCH + m]);
            if (!ENDS) bc[(t * 2 + 1) * K::ME + m] = to_f(b[K::RB + t * K::Pairs::PITCH + m]);
        }
        constexpr int TURNS = (T + ROWS - 1) / ROWS, BATCH = TURNS < 4 ? TURNS : 4;
#pragma unroll
        for (int i0 = 0; i0 < TURNS; i0 += BATCH) {
            f2 d[BATCH * NP];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                f2 v[NP];
                load_pairs<V, K::NV>(r + (er + (i0 + i) * ROWS) % T * K::Rows::PITCH, v);
#pragma unroll
                for (int e = 0; e < NP; ++e) d[i * NP + e] = add2(v[e], *reinterpret_cast<const f2*>(sb + ev + 2 * e));
            }
            if (p.softplus) softplus_pairs(d);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int t = er + (i0 + i) * ROWS;
                if (ROWS > T && t >= T) break;
                f2 x[NP];
                load_pairs<V, K::NV>(r + K::RX + t * K::Rows::PITCH, x);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    f2& v = d[i * NP + e];
                    if (t >= steps) v = 0;
                    if (ENDS) total[ENDS ? e : 0] = add2(total[ENDS ? e : 0], v);
                    *reinterpret_cast<f2*>(sd + t * K::PW + ev + 2 * e) = v;
                    *reinterpret_cast<f2*>(sx + t * K::PW + ev + 2 * e) = mul2(v, x[e]);
                }
            }
        }
        __syncthreads();                       // B and C are in place (and each warp's own delta)
        if (warp * K::WC >= valid) continue;
        // U steps at a time: their y are stored together, because the loads
        // of a step cannot pass a store before them.
#pragma unroll 1
        for (int t4 = 0; t4 < T; t4 += U) {
            if (!ENDS && p.saved && t4 % kSsmTile == 0 && t4 < steps) {
                const int64_t at = anew(n) * ((p.S + kSsmTile - 1) / kSsmTile) + (t_first + (int64_t)k * T + t4) / kSsmTile;
                float* saved = p.saved + (at * p.D + d0) * p.M + sg * E;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    float s[2][E];
#pragma unroll
                    for (int j = 0; j < E; ++j) unpack2(h[j][i], s[0][j], s[1][j]);
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const int c = warp * K::WC + ch[i] + o;
                        if (c < valid && sg * E < p.M)
                            store_vec<float, E>(saved + (int64_t)c * p.M, s[o], p.M - sg * E < E ? p.M - sg * E : E, q.vec_h);
                    }
                }
            }
            f2 ys[U][LEFT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t4 + u;
                f2 d[PAIRS], dx[PAIRS], y[PAIRS];
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    d[i] = *reinterpret_cast<const f2*>(sd + t * K::PW + ch[i]);
                    dx[i] = *reinterpret_cast<const f2*>(sx + t * K::PW + ch[i]);
                }
                const float4 vb = *reinterpret_cast<const float4*>(bc + t * 2 * K::ME + sg * E);
                float4 vc = vb;
                if (!ENDS) vc = *reinterpret_cast<const float4*>(bc + (t * 2 + 1) * K::ME + sg * E);
                const f2 B[E] = {dup2(vb.x), dup2(vb.y), dup2(vb.z), dup2(vb.w)};
                const f2 C[E] = {dup2(vc.x), dup2(vc.y), dup2(vc.z), dup2(vc.w)};
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        h[j][i] = fma2(decay2(d[i], A[j][i]), h[j][i], mul2(dx[i], B[j]));
                        if (!ENDS) y[i] = j == 0 ? mul2(C[j], h[j][i]) : fma2(C[j], h[j][i], y[i]);
                    }
                if (ENDS) continue;
                // over the channel's lanes
                if (SPLIT) y[0] = add2(y[0], __shfl_xor_sync(~0u, y[1], 1));
                if (HALVE) {
                    float a, b2;
                    unpack2(y[0], a, b2);
                    float one = (up ? b2 : a) + __shfl_xor_sync(~0u, up ? a : b2, 1 << SPLIT);
#pragma unroll
                    for (int o = 2 << SPLIT; o < L; o *= 2) one += __shfl_xor_sync(~0u, one, o);
                    y[0] = pack2(one, one);
                }
#pragma unroll
                for (int i = 0; i < LEFT; ++i) ys[u][i] = y[i];
            }
            if (ENDS) continue;
            // y takes delta X's place
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float* to = sx + (t4 + u) * K::PW;
                if (HALVE) {
                    float a, b2;
                    unpack2(ys[u][0], a, b2);
                    if (sg < (2 << SPLIT)) to[ch[0] + (up ? 1 : 0)] = a;
                } else {
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) *reinterpret_cast<f2*>(to + ch[i]) = ys[u][i];
                }
            }
        }
        if (ENDS) continue;
        __syncwarp();
        V* y_row = static_cast<V*>(p.Y.data) + anew(n) * p.Y.bs + d0 + ec + (t_first + (int64_t)k * T + er) * p.Y.ss;
#pragma unroll
        for (int i = 0; i < (T + ROWS - 1) / ROWS; ++i) {
            const int t = er + i * ROWS;
            if (ROWS > T && t >= T) break;
            f2 x[NP], z[NP];
            float v[K::NV];
            load_pairs<V, K::NV>(r + K::RX + t * K::Rows::PITCH, x);
            if (gate) load_pairs<V, K::NV>(r + 2 * K::RX + t * K::Rows::PITCH, z);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                f2 s = fma2(*reinterpret_cast<const f2*>(sb + K::WC + ev + 2 * e), x[e], *reinterpret_cast<const f2*>(sx + t * K::PW + ev + 2 * e));
                if (gate && p.saved) unpack2(s, v[2 * e], v[2 * e + 1]);
                if (gate) z[e] = s = mul2(s, silu_fast2(z[e]));
                if (!(gate && p.saved)) unpack2(s, v[2 * e], v[2 * e + 1]);
            }
            if (gate && p.saved) {             // y before the gate, for the gate's gradient
                const int64_t at = (anew(n) * p.S + t_first + (int64_t)k * T + t) * p.D + d0 + ec;
                store_vec<float, K::NV>(p.saved + ssm_saved_states(p.S, p.N, p.D, p.M) + at, v, t < steps ? some : 0, q.vec_s);
#pragma unroll
                for (int e = 0; e < NP; ++e) unpack2(z[e], v[2 * e], v[2 * e + 1]);
            }
            store_vec<V, K::NV>(y_row + i * ROWS * p.Y.ss, v, t < steps ? some : 0, q.vec_y);
        }
    }
    if (ENDS) {
        // the chunk's sum of delta, over the steps that the lanes took
#pragma unroll
        for (int e = 0; e < NP; ++e) {
#pragma unroll
            for (int o = PER_ROW; o < 32; o *= 2) total[ENDS ? e : 0] = add2(total[ENDS ? e : 0], __shfl_xor_sync(~0u, total[ENDS ? e : 0], o));
            float v[2];
            unpack2(total[ENDS ? e : 0], v[0], v[1]);
            if (er == 0) store_vec<float, 2>(q.deltas + ((int64_t)chunk * p.N + n) * p.D + d0 + ec + 2 * e, v, some - 2 * e < 2 ? some - 2 * e : 2, false);
        }
    } else {
        const float zero[K::NV] = {};
        V* y = static_cast<V*>(p.Y.data) + n * p.Y.bs + d0 + ec;
        for (int64_t t = (live > t_first ? live : t_first) + er; t < t_end; t += ROWS)
            store_vec<V, K::NV>(y + t * p.Y.ss, zero, some, q.vec_y);
        const bool last = len > 0 ? len > t_first && len <= t_end : chunk == 0;
        if (!p.hT || !last) return;
    }
    float* to = ENDS ? q.ends + (int64_t)chunk * p.N * p.D * p.M : p.hT;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float s[2][E];
#pragma unroll
        for (int j = 0; j < E; ++j) unpack2(h[j][i], s[0][j], s[1][j]);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int c = warp * K::WC + ch[i] + o;
            if (c < valid && sg * E < p.M)
                store_vec<float, E>(to + (n * p.D + d0 + c) * p.M + sg * E, s[o], p.M - sg * E < E ? p.M - sg * E : E, q.vec_h);
        }
    }
}

// First states of chunks 1 .. from the chunks' end states: one state a thread.
__global__ void __launch_bounds__(256) ssm_scan_chain_kernel(const ScanParams p, const ScanLaunch q)
{
    const int64_t per = p.N * p.D * p.M, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int64_t nd = i / p.M;
    const float a = p.A[nd % p.D * p.M + i % p.M] * kLog2e;
    float h = p.h0 ? p.h0[i] : 0.0f;
    constexpr int B = 8;
    for (int c0 = 0; c0 < q.chunks - 1; c0 += B) {
        float e[B], d[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const bool on = c0 + k < q.chunks - 1;
            e[k] = on ? q.ends[(c0 + k) * per + i] : 0.0f;
            d[k] = on ? q.deltas[(int64_t)(c0 + k) * p.N * p.D + nd] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            h = fmaf(ex2(a * d[k]), h, e[k]);
            if (c0 + k < q.chunks - 1) q.ends[(c0 + k) * per + i] = h;
        }
    }
}

constexpr int64_t kMaxGrid = 0x7fffffff;

// Measured times of a step (M = 16, bf16, gate, in ns) with 1 .. 4 warps on
// every scheduler: 239, 342, 375, 402; the chunks' end states cost another 0.72
// of a pass.  With few warps the latency of a step's chain shows, so splitting
// pays: 8 rows of 2048 steps x 2048 channels take 490 us unsplit and 295 us in
// 14 chunks, one row of 16384 steps 288 us in 38; 64 rows of 512 steps fill
// the SMs and take 343 us unsplit, 488 us in two.
constexpr ScanCost kCost{4, {0, 239, 342, 375, 402}, 2500, 0.72};

template <typename V, int L>
cudaError_t run(const ScanParams& p, cudaStream_t s, int* launches)
{
    const ScanChoice& c = p.split;
    static std::atomic<uint64_t> ready_ends{0}, ready{0};
    using K = Tile<V, L>;
    const int elem = (int)sizeof(V);
    const int64_t dg = p.D / p.G, block = K::W * K::WC, group = p.G > 1 ? dg : 0;
    ScanLaunch q{};
    q.cblocks = (int)c.cblocks;
    q.chunk = c.chunk;
    q.chunks = c.chunks;
    q.fast_x = rows_aligned(p.X, elem, block, group);
    q.fast_dt = rows_aligned(p.dt, elem, block, group);
    q.fast_z = rows_aligned(p.Z, elem, block, group);
    q.fast_b = rows_aligned(p.B, elem, 0, p.G > 1 ? p.M : 0);
    q.fast_c = rows_aligned(p.C, elem, 0, p.G > 1 ? p.M : 0);
    const int64_t bytes = elem * K::NV;
    q.vec_y = (uintptr_t)p.Y.data % bytes == 0 && p.Y.ss * elem % bytes == 0 && p.Y.bs * elem % bytes == 0 &&
              group * elem % bytes == 0;
    q.vec_h = p.M % E == 0 && ((uintptr_t)p.hT | (uintptr_t)p.saved) % 16 == 0;
    q.vec_s = p.D % K::NV == 0 && group % K::NV == 0 && ssm_saved_states(p.S, p.N, p.D, p.M) % 4 == 0 && (uintptr_t)p.saved % 16 == 0;
    q.ends = p.scratch;
    q.deltas = p.scratch + (int64_t)(c.chunks - 1) * p.N * p.D * p.M;
    const int64_t blocks = c.cblocks * p.G * p.N;
    if (blocks > kMaxGrid / c.chunks) return cudaErrorInvalidConfiguration;
    if (c.chunks > 1) {
        auto* f = ssm_scan_kernel<V, L, true>;
        const size_t smem = K::bytes(2);
        cudaError_t e = allow_shared(f, smem, ready_ends);
        if (e != cudaSuccess) return e;
        f<<<(unsigned)(blocks * (c.chunks - 1)), K::THREADS, smem, s>>>(p, q);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ++*launches;
        if (c.chunks > kFold) {
            const int64_t states = p.N * p.D * p.M;
            if ((states + 255) / 256 > kMaxGrid) return cudaErrorInvalidConfiguration;
            ssm_scan_chain_kernel<<<(unsigned)((states + 255) / 256), 256, 0, s>>>(p, q);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            ++*launches;
        }
    }
    auto* f = ssm_scan_kernel<V, L, false>;
    const size_t smem = K::bytes(3);
    cudaError_t e = allow_shared(f, smem, ready);
    if (e != cudaSuccess) return e;
    f<<<(unsigned)(blocks * c.chunks), K::THREADS, smem, s>>>(p, q);
    ++*launches;
    return cudaGetLastError();
}

template <typename V>
cudaError_t by_lanes(const ScanParams& p, cudaStream_t s, int* launches)
{
    switch (ssm_lanes(p.M)) {
    case 1: return run<V, 1>(p, s, launches);
    case 2: return run<V, 2>(p, s, launches);
    case 4: return run<V, 4>(p, s, launches);
    case 8: return run<V, 8>(p, s, launches);
    case 16: return run<V, 16>(p, s, launches);
    default: return run<V, 32>(p, s, launches);
    }
}

}  // namespace

int64_t ssm_saved_floats(int64_t S, int64_t N, int64_t D, int64_t M) { return ssm_saved_states(S, N, D, M) + S * N * D; }

ScanChoice ssm_split(const ScanParams& p, int tile, const ScanCost& cost)
{
    const int L = ssm_lanes(p.M), W = L >= 4 ? 4 : L, WC = 32 / L * CH;
    const int64_t dg = p.D / p.G, tiles = (p.S + tile - 1) / tile, blocks = (dg + W * WC - 1) / (W * WC);
    const double all = (double)blocks * W * p.G * p.N / (4.0 * p.sms);       // warps per scheduler
    auto pass = [&](double w, double steps) {
        const double waves = std::floor(w / cost.warps);
        const int r = (int)std::ceil(w - cost.warps * waves);
        return waves * (cost.begin_ns + steps * cost.step_ns[cost.warps]) + (r ? cost.begin_ns + steps * cost.step_ns[r] : 0.0);
    };
    ScanChoice best{1, blocks, (tiles > 0 ? tiles : 1) * tile};
    double least = pass(all, (double)tiles * tile);
    // chunks of fewer and fewer tiles, each number of chunks once
    for (int64_t per = (tiles + 1) / 2; per > 0 && tiles > 1;) {
        const int64_t k = (tiles + per - 1) / per, next = (tiles + k) / (k + 1);      // `per` of k + 1 chunks
        if (k > 512) break;
        const double steps = (double)per * tile;
        // 5 us for two launches more, and a chunk's part of their chain
        const double t = pass(all * (double)k, steps) + cost.ends * pass(all * (double)(k - 1), steps) + 5000.0 + 50.0 * (double)k;
        if (t < least) {
            least = t;
            best.chunks = (int)k;
            best.chunk = per * tile;
        }
        per = next < per ? next : per - 1;
    }
    return best;
}

cudaError_t ssm_sm_count(int* sms)
{
    static std::atomic<int> known[64];          // a call's host time counts
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (*sms = known[dev].load(std::memory_order_relaxed))) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && keep) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

void ssm_scan_plan(ScanParams& p, size_t* bytes)
{
    p.split = ssm_split(p, T, kCost);
    *bytes = sizeof(float) * (size_t)(p.split.chunks - 1) * (size_t)(p.N * p.D * (p.M + 1));
}

cudaError_t launch_ssm_scan(const ScanParams& p, cudaStream_t s, int* launches)
{
    return p.io == 1   ? by_lanes<__half>(p, s, launches)
           : p.io == 2 ? by_lanes<__nv_bfloat16>(p, s, launches)
                       : by_lanes<float>(p, s, launches);
}

}  // namespace rnngb
