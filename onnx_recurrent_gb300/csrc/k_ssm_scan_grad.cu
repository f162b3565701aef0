// Gradients of the selective state space scan (the formulas stand in
// include/onnx_recurrent.h).
//
// For one channel with g[t,m] the loss's slope in h[t,m], a = exp(delta A),
// p = a h[t-1] and e = dY silu(Z):
//     g[t]   = C e + q[t],  q[t] = a[t+1] g[t+1]       (q = dY_h at the row's end)
//     dX     = delta sum_m g B + Dskip e       dC = e h,  dB = delta X g
//     ddelta = sum_m g (A p + B X)             dA = sum_t delta g p
// Going backwards needs every h[t], which the forward run does not keep: it
// saves the state before every kSsmTile-th step.  A tile is kSsmTile = 8
// steps in two halves of 4; for the second half the first is run through once,
// then for each half the 5 states around its steps are formed in registers
// and its steps taken backwards (with a formed again: an exponential is cheaper
// than 16 registers a step).  Saving every 4th state instead would move 8 more
// bytes a channel and step each way (M = 16), keeping a tile's states in
// shared memory 128 bytes a lane and step.
//
// Lanes hold states and channels as in the forward kernel (k_ssm_scan.cu).
// The sums over a channel's states (for dX, ddelta) go over L lanes, those
// over channels (dB, dC) over the other 32 / L, each halving the values at
// every exchange; what a lane sends first is chosen by its place in memory,
// so nothing is selected.  dB and dC are then summed over the block's warps and
// written for each block of channels, dA, dDskip and ddt_bias for each row and
// chunk of steps; a last launch adds both up in order.
//
// Steps are split in chunks as in the forward run, from the end: one launch
// finds the q that each chunk passes on when none enters; with up to kFold
// chunks a block chains those after its own, with more another launch does.
//
// Measured (8 rows of 2048 steps, 2048 channels, M = 16, bf16): 832 us, 650 updates
// a ns with the launch for the chunks' q; 390 instructions for 512 updates, 140 of
// them packed fp32 ones, 43 exponentials.  Counters with the SMs full: issue slots 38 to
// 47 % busy, the fp32 pipe 29 to 46 %, shared memory 30 to 36 %, DRAM 11 to 16 %: three warps
// a scheduler do not hide a step's latencies, and more do not fit the registers
// (three blocks an SM with 168; two with 240: 873 us; four with 128: 919 us).
// Scalar instead of packed operations: 5 to 15 % slower; dA summed in shared memory
// to free registers: no faster.
#include <type_traits>

#include "ssm_tile.cuh"

#pragma nv_diag_suppress 128   // loops that some lane counts leave out

namespace rnngb {
namespace {

constexpr int E = 4;              // states of a lane
constexpr int CH = 4;             // channels of a lane
constexpr int PAIRS = CH / 2;
constexpr int T = kSsmTile;       // steps of a tile
constexpr int U = 4;              // steps of half a tile
constexpr int kFold = 16;         // chunks whose q a block chains itself
constexpr int NV = 4, NP = 2;     // channels of an elementwise access
constexpr float kLn2 = 0.6931471805599453f;

struct GradLaunch {
    int cblocks;          // blocks of channels in a group
    int64_t chunk;        // steps of a chunk (a multiple of T)
    int chunks;
    bool fast_x, fast_dt, fast_z, fast_dy, fast_y, fast_b, fast_c, vec_dx, vec_ddt, vec_dz, vec_h;
    float* ends;          // [chunks - 1][N][D][M]: the q that enters a chunk
    float* deltas;        // [chunks - 1][N][D]: sums of the next chunk's delta
    float* part;          // [chunks][N][D * (M + 2)]: dA, dDskip, ddt_bias
    float* steps;         // [cblocks][N][S][G][2][M]: dB, dC
};

template <typename V, int L>
struct Tile {
    static constexpr int W = L >= 4 ? 4 : L;               // warps
    static constexpr int THREADS = 32 * W;
    static constexpr int WC = 32 / L * CH;                 // channels of a warp
    static constexpr int ME = L * E;                       // states, padded
    static constexpr int PW = WC + 4;                      // pitch of delta, delta X, e
    using Rows = Stager<V, T, W * WC, THREADS>;            // of X, dt, Z, dY
    using Sums = Stager<float, T, W * WC, THREADS>;        // of y
    using Pairs = Stager<V, T, ME, THREADS>;               // of B, C
    static constexpr int RX = T * Rows::PITCH, RB = T * Pairs::PITCH, RY = T * Sums::PITCH;
    static constexpr int WARP = 3 * T * PW + 2 * WC;             // floats of a warp
    static constexpr size_t bytes()
    {
        return sizeof(V) * 2 * (4 * RX + 2 * RB) + sizeof(float) * (2 * RY + 2 * T * ME + W * WARP + W * T * 2 * ME);
    }
    static constexpr size_t bytes_ends()
    {
        return sizeof(V) * 2 * (3 * RX + RB) + sizeof(float) * (T * ME + W * (2 * T * PW + 2 * WC));
    }
};

// Where a lane stands: its channels and states, and how the sums go.
template <int L>
struct Place {
    static constexpr int SPLIT = L >= 2 ? 1 : 0, LEFT = PAIRS >> SPLIT;   // exchanges that halve the pairs; pairs left
    static constexpr bool HALVE = LEFT == 1 && L > 2;                     // one more halves the last pair
    static constexpr int GROUPS = 32 / L;                                 // groups of channels in the warp
    int sg, cg, ch[PAIRS], m0, m1;       // m0, m1: first state of registers 0, 1 and 2, 3
    bool up, up2, up4;

    __device__ __forceinline__ Place()
    {
        const int lane = threadIdx.x % 32;
        sg = lane % L;
        cg = lane / L;
        up = HALVE && (sg & 2);
        const int swap = GROUPS >= 2 ? cg & 1 : 0;
        m0 = sg * E + 2 * swap;
        m1 = sg * E + 2 * (swap ^ 1);
        up2 = GROUPS >= 4 && (cg & 2);
        up4 = GROUPS >= 8 && (cg & 4);
        for (int r = 0; r < PAIRS; ++r) ch[r] = cg * CH + 2 * (SPLIT && sg & 1 ? r ^ 1 : r);
    }
    __device__ __forceinline__ int state(int j) const { return j < 2 ? m0 + j : m1 + j - 2; }

    static constexpr int SV = HALVE ? 1 : 2 * LEFT;                       // sums over states that a lane ends with
    static constexpr int CV = GROUPS >= 8 ? 1 : 8 / GROUPS;               // and sums over channels

    // Sums of v over the channel's lanes; each lane ends with those of some channels.
    __device__ __forceinline__ void sum_states(f2 (&v)[PAIRS], float (&r)[SV]) const
    {
        if constexpr (SPLIT == 1) v[0] = add2(v[0], __shfl_xor_sync(~0u, v[1], 1));
        if constexpr (HALVE) {
            float a, b;
            unpack2(v[0], a, b);
            r[0] = (up ? b : a) + __shfl_xor_sync(~0u, up ? a : b, 2);
#pragma unroll
            for (int o = 4; o < L; o *= 2) r[0] += __shfl_xor_sync(~0u, r[0], o);
        } else {
#pragma unroll
            for (int i = 0; i < LEFT; ++i) unpack2(v[i], r[2 * i], r[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void store_states_sum(const float (&r)[SV], float* to) const
    {
        if constexpr (HALVE) {
            if (L == 4 || sg < 4) to[ch[0] + (up ? 1 : 0)] = r[0];
        } else {
#pragma unroll
            for (int i = 0; i < LEFT; ++i) *reinterpret_cast<float2*>(to + ch[i]) = make_float2(r[2 * i], r[2 * i + 1]);
        }
    }
    // Sums of b and c over the warp's channels; each lane ends with those of some states.
    __device__ __forceinline__ void sum_channels(float (&b)[E], float (&c)[E], float (&r)[CV]) const
    {
        if constexpr (GROUPS == 1) {
#pragma unroll
            for (int j = 0; j < E; ++j) r[j] = b[j], r[E + j] = c[j];
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                b[j] += __shfl_xor_sync(~0u, b[j + 2], L);
                c[j] += __shfl_xor_sync(~0u, c[j + 2], L);
            }
            if constexpr (GROUPS == 2) {
                r[0] = b[0], r[1] = b[1], r[2] = c[0], r[3] = c[1];
            } else {
                float w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j] = (up2 ? c[j] : b[j]) + __shfl_xor_sync(~0u, up2 ? b[j] : c[j], 2 * L);
                if constexpr (GROUPS == 4) {
                    r[0] = w[0], r[1] = w[1];
                } else {
                    r[0] = (up4 ? w[1] : w[0]) + __shfl_xor_sync(~0u, up4 ? w[0] : w[1], 4 * L);
#pragma unroll
                    for (int o = 8 * L; o < 32; o *= 2) r[0] += __shfl_xor_sync(~0u, r[0], o);
                }
            }
        }
    }
    __device__ __forceinline__ void store_channels_sum(const float (&r)[CV], float* to) const      // [2][ME]
    {
        constexpr int ME = L * E;
        if constexpr (GROUPS >= 8) {
            if (GROUPS == 8 || cg < 8) to[(up2 ? ME : 0) + m0 + (up4 ? 1 : 0)] = r[0];
        } else if constexpr (GROUPS == 4) {
            *reinterpret_cast<float2*>(to + (up2 ? ME : 0) + m0) = make_float2(r[0], r[1]);
        } else if constexpr (GROUPS == 2) {
            *reinterpret_cast<float2*>(to + m0) = make_float2(r[0], r[1]);
            *reinterpret_cast<float2*>(to + ME + m0) = make_float2(r[2], r[3]);
        } else {
            *reinterpret_cast<float4*>(to + sg * E) = make_float4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<float4*>(to + ME + sg * E) = make_float4(r[4], r[5], r[6], r[7]);
        }
    }
};

// The lane's part of an [.., M] table of the block's channels (row d0 + c).
template <int L>
__device__ __forceinline__ void load_states(f2 (&v)[E][PAIRS], const float* rows, const Place<L>& at, int c0, int valid,
                                            int M, bool vec, float scale)
{
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float s[2][E];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int c = c0 + at.ch[i] + o;
#pragma unroll
            for (int j = 0; j < E; j += 2) {
                const int m = at.state(j);
                float2 two = make_float2(0.0f, 0.0f);
                if (rows && c < valid) {
                    const float* from = rows + (int64_t)c * M + m;
                    if (vec) {
                        if (m < M) two = *reinterpret_cast<const float2*>(from);
                    } else {
                        if (m < M) two.x = from[0];
                        if (m + 1 < M) two.y = from[1];
                    }
                }
                s[o][j] = two.x * scale;
                s[o][j + 1] = two.y * scale;
            }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) v[j][i] = pack2(s[0][j], s[1][j]);
    }
}
template <int L>
__device__ __forceinline__ void store_states(const f2 (&v)[E][PAIRS], float* rows, const Place<L>& at, int c0, int valid, int M)
{
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float s[2];
            unpack2(v[j][i], s[0], s[1]);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int c = c0 + at.ch[i] + o;
                if (c < valid && at.state(j) < M) rows[(int64_t)c * M + at.state(j)] = s[o];
            }
        }
}

// Which rows, channels and steps a block has.
struct Block {
    int cb, g, chunk, valid;
    int64_t n, d0, len, t_first, t_end, live;

    template <int CB>
    __device__ __forceinline__ void find(const ScanParams& p, const GradLaunch& q, int first_chunk)
    {
        unsigned blk = blockIdx.x;
        cb = blk % q.cblocks;
        blk /= q.cblocks;
        g = blk % p.G;
        blk /= p.G;
        n = blk % (unsigned)p.N;
        chunk = blk / (unsigned)p.N + first_chunk;
        const int64_t dg = p.D / p.G, c0 = (int64_t)cb * CB;
        valid = dg - c0 < CB ? (int)(dg - c0) : CB;
        d0 = g * dg + c0;
        len = row_length(p.lens, n, p.S, p.status);
        t_first = chunk * q.chunk;
        t_end = t_first + q.chunk < p.S ? t_first + q.chunk : p.S;
        live = len < t_end ? len : t_end;
    }
    __device__ __forceinline__ int tiles() const { return live > t_first ? (int)((live - t_first + T - 1) / T) : 0; }
};

// delta and e of a pair of channels, from the raw values.
__device__ __forceinline__ f2 gate_slope(f2 dy, f2 z)
{
    return mul2(dy, silu_fast2(z));
}

template <typename V, int L>
__global__ void __launch_bounds__(Tile<V, L>::THREADS, 12 / Tile<V, L>::W)
    ssm_scan_grad_kernel(const ScanGradParams pp, const GradLaunch q)
{
    using K = Tile<V, L>;
    const ScanParams& p = pp.f;
    extern __shared__ __align__(16) char smem[];
    V* raw = reinterpret_cast<V*>(smem);                          // [2][4][T][..]: dt, X, dY, Z
    V* rawbc = raw + 2 * 4 * K::RX;                               // [2][2][T][..]: B, C
    float* rawy = reinterpret_cast<float*>(rawbc + 2 * 2 * K::RB);      // [2][T][..]: y
    float* bc = rawy + 2 * K::RY;                                 // [T][2][ME]: B, C
    float* sums = bc + 2 * T * K::ME;                             // [W][T][2][ME]: dB, dC of each warp
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float* sd = sums + K::W * T * 2 * K::ME + warp * K::WARP;     // the warp's delta,
    float* sx = sd + T * K::PW;                                   // delta X, then sum g B,
    float* se = sx + T * K::PW;                                   // e, then sum g p A,
    float* sb = se + T * K::PW;                                   // and dt_bias and Dskip

    Block b{};
    b.find<K::W * K::WC>(p, q, 0);
    const Place<L> at;
    const int c0 = warp * K::WC;
    f2 A[E][PAIRS], carry[E][PAIRS], dA[E][PAIRS];
    load_states<L>(A, p.A + b.d0 * p.M, at, c0, b.valid, p.M, false, kLog2e);
    {
        const int64_t states = p.N * p.D * p.M, row = (b.n * p.D + b.d0) * p.M;
        const bool fold = q.chunks <= kFold;
        const float* from = b.chunk + 1 < q.chunks && !fold ? q.ends + b.chunk * states : pp.dhT;
        load_states<L>(carry, from ? from + row : nullptr, at, c0, b.valid, p.M, false, 1.0f);
        if (fold) {
#pragma unroll 2
            for (int k = q.chunks - 2; k >= b.chunk; --k) {
                f2 end[E][PAIRS];
                load_states<L>(end, q.ends + k * states + row, at, c0, b.valid, p.M, p.M % 2 == 0, 1.0f);
                const float* delta = q.deltas + (k * p.N + b.n) * p.D + b.d0 + c0;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const bool on = c0 + at.ch[i] < b.valid, both = c0 + at.ch[i] + 1 < b.valid;
                    const f2 d = pack2(on ? delta[at.ch[i]] : 0.0f, both ? delta[at.ch[i] + 1] : 0.0f);
#pragma unroll
                    for (int j = 0; j < E; ++j) carry[j][i] = fma2(ex2_2(mul2(d, A[j][i])), carry[j][i], end[j][i]);
                }
            }
        }
    }
    float most_a = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            dA[j][i] = 0;
            float x, y;
            unpack2(A[j][i], x, y);
            most_a = fmaxf(most_a, fmaxf(fabsf(x), fabsf(y)));
        }
    }

    most_a = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(most_a)));      // of the warp
    constexpr int PER_ROW = K::WC / NV, ROWS = 32 / PER_ROW, TURNS = (T + ROWS - 1) / ROWS;
    const int ev = lane % PER_ROW * NV, er = lane / PER_ROW, ec = c0 + ev;
    const int some = b.valid - ec < NV ? (b.valid - ec > 0 ? b.valid - ec : 0) : NV;
    f2 dskip[NP] = {0, 0}, dbias[NP] = {0, 0};
    for (int i = lane; i < 2 * K::WC; i += 32) {
        const int c = c0 + i % K::WC;
        const float* from = i < K::WC ? p.dt_bias : p.Dskip;
        sb[i] = from && c < b.valid ? from[b.d0 + c] : 0.0f;
    }
    __syncwarp();

    const bool gate = p.Z.data;
    const float* saved_y = p.saved + ssm_saved_states(p.S, p.N, p.D, p.M);
    const int tiles = b.tiles();
    auto stage = [&](int k) {
        const int64_t t0 = b.t_first + (int64_t)k * T, left = b.live - t0, row = anew(b.n);
        const int steps = left < T ? (int)left : T;
        V* r = raw + (k & 1) * 4 * K::RX;
        V* rb = rawbc + (k & 1) * 2 * K::RB;
        K::Rows::copy(r, p.dt, row, t0, b.d0, steps, b.valid, q.fast_dt);
        K::Rows::copy(r + K::RX, p.X, row, t0, b.d0, steps, b.valid, q.fast_x);
        K::Rows::copy(r + 2 * K::RX, pp.dY, row, t0, b.d0, steps, b.valid, q.fast_dy);
        if (gate) {
            K::Rows::copy(r + 3 * K::RX, p.Z, row, t0, b.d0, steps, b.valid, q.fast_z);
            const View y{const_cast<float*>(saved_y), p.D, p.S * p.D};
            K::Sums::copy(rawy + (k & 1) * K::RY, y, row, t0, b.d0, steps, b.valid, q.fast_y);
        }
        K::Pairs::copy(rb, p.B, row, t0, (int64_t)b.g * p.M, steps, p.M, q.fast_b);
        K::Pairs::copy(rb + K::RB, p.C, row, t0, (int64_t)b.g * p.M, steps, p.M, q.fast_c);
        cp_async_commit();
    };
    if (tiles) stage(tiles - 1);
    for (int k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = b.t_first + (int64_t)k * T;
        const int steps = b.live - t0 < T ? (int)(b.live - t0) : T;
        const V* r = raw + (k & 1) * 4 * K::RX + ec;
        cp_async_wait<0>();
        __syncthreads();                       // tile k has landed; tile k+1's buffers are free
        if (k > 0) stage(k - 1);
        f2 H[U][E][PAIRS];
        auto restart = [&] {
            const int64_t from = anew(b.n) * ((p.S + T - 1) / T) + t0 / T;
            load_states<L>(H[0], p.saved + (from * p.D + b.d0) * p.M, at, c0, b.valid, p.M, q.vec_h, 1.0f);
        };
        restart();
        const V* rb = rawbc + (k & 1) * 2 * K::RB;
        for (int i = threadIdx.x; i < T * K::ME; i += K::THREADS) {
            const int t = i / K::ME, m = i % K::ME;
            bc[t * 2 * K::ME + m] = to_f(rb[t * K::Pairs::PITCH + m]);
            bc[(t * 2 + 1) * K::ME + m] = to_f(rb[K::RB + t * K::Pairs::PITCH + m]);
        }
        // Whether decays below 2^-126 occur, which the exponential flushes but dA may
        // consist of: then they are formed as squares, by a copy of the code (a branch
        // around the squares in one copy cost 10 %).
        bool deep;
        {
            f2 d[TURNS * NP];
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
                f2 v[NP];
                load_pairs<V, NV>(r + (er + i * ROWS) % T * K::Rows::PITCH, v);
#pragma unroll
                for (int e = 0; e < NP; ++e) d[i * NP + e] = add2(v[e], *reinterpret_cast<const f2*>(sb + ev + 2 * e));
            }
            if (p.softplus) softplus_pairs(d);
            float most_d = 0.0f;
#pragma unroll
            for (int i = 0; i < TURNS * NP; ++i) {
                float x, y;
                unpack2(d[i], x, y);
                most_d = fmaxf(most_d, fmaxf(fabsf(x), fabsf(y)));
            }
            deep = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(most_d))) * most_a > 125.0f;
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
                const int t = er + i * ROWS;
                if (ROWS > T && t >= T) break;
                f2 x[NP], dy[NP], z[NP];
                load_pairs<V, NV>(r + K::RX + t * K::Rows::PITCH, x);
                load_pairs<V, NV>(r + 2 * K::RX + t * K::Rows::PITCH, dy);
                if (gate) load_pairs<V, NV>(r + 3 * K::RX + t * K::Rows::PITCH, z);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    f2& v = d[i * NP + e];
                    if (t >= steps) v = 0;
                    *reinterpret_cast<f2*>(sd + t * K::PW + ev + 2 * e) = v;
                    *reinterpret_cast<f2*>(sx + t * K::PW + ev + 2 * e) = mul2(v, x[e]);
                    *reinterpret_cast<f2*>(se + t * K::PW + ev + 2 * e) = gate ? gate_slope(dy[e], z[e]) : dy[e];
                }
            }
        }
        __syncthreads();                       // B and C are in place (and each warp's own delta, delta X, e)
        // One step forward.
        auto ahead = [&](const f2 (&from)[E][PAIRS], f2 (&to)[E][PAIRS], int t) {
            const float2 b0 = *reinterpret_cast<const float2*>(bc + t * 2 * K::ME + at.m0);
            const float2 b1 = *reinterpret_cast<const float2*>(bc + t * 2 * K::ME + at.m1);
            const f2 B[E] = {dup2(b0.x), dup2(b0.y), dup2(b1.x), dup2(b1.y)};
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const f2 d = *reinterpret_cast<const f2*>(sd + t * K::PW + at.ch[i]);
                const f2 dx = *reinterpret_cast<const f2*>(sx + t * K::PW + at.ch[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) to[j][i] = fma2(decay2(d, A[j][i]), from[j][i], mul2(dx, B[j]));
            }
        };
        // The tile's steps backwards.
        auto back = [&](auto is_deep) {
            constexpr bool DEEP = decltype(is_deep)::value;
            if (steps > U) {
#pragma unroll
                for (int u = 0; u < U; ++u) ahead(H[0], H[0], u);
            }
#pragma unroll 1
            for (int t1 = steps > U ? U : 0; t1 >= 0; t1 -= U) {
                if (t1 == 0 && steps > U) restart();
#pragma unroll
                for (int u = 0; u + 1 < U; ++u) ahead(H[u], H[u + 1], t1 + u);
#pragma unroll
                for (int u = U - 1; u >= 0; --u) {
                    const int t = t1 + u;
                    const float2 b0 = *reinterpret_cast<const float2*>(bc + t * 2 * K::ME + at.m0);
                    const float2 b1 = *reinterpret_cast<const float2*>(bc + t * 2 * K::ME + at.m1);
                    const float2 g0 = *reinterpret_cast<const float2*>(bc + (t * 2 + 1) * K::ME + at.m0);
                    const float2 g1 = *reinterpret_cast<const float2*>(bc + (t * 2 + 1) * K::ME + at.m1);
                    const f2 B[E] = {dup2(b0.x), dup2(b0.y), dup2(b1.x), dup2(b1.y)};
                    const f2 C[E] = {dup2(g0.x), dup2(g0.y), dup2(g1.x), dup2(g1.y)};
                    f2 db[E], dc[E], driven[PAIRS], decayed[PAIRS];
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const f2 d = *reinterpret_cast<const f2*>(sd + t * K::PW + at.ch[i]);
                        const f2 dx = *reinterpret_cast<const f2*>(sx + t * K::PW + at.ch[i]);
                        const f2 e = *reinterpret_cast<const f2*>(se + t * K::PW + at.ch[i]);
                        f2 a[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) a[j] = decay2(DEEP ? mul2(d, dup2(0.5f)) : d, A[j][i]);
                        if (DEEP) {
#pragma unroll
                            for (int j = 0; j < E; ++j) a[j] = mul2(a[j], a[j]);
                        }
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const f2 past = mul2(a[j], H[u][j][i]);
                            const f2 now = u + 1 < U ? H[u + 1 < U ? u + 1 : 0][j][i] : fma2(dx, B[j], past);
                            const f2 g = fma2(C[j], e, carry[j][i]), gp = mul2(g, past);
                            driven[i] = j == 0 ? mul2(g, B[0]) : fma2(g, B[j], driven[i]);
                            decayed[i] = j == 0 ? mul2(gp, A[0][i]) : fma2(gp, A[j][i], decayed[i]);
                            dA[j][i] = fma2(gp, d, dA[j][i]);
                            db[j] = i == 0 ? mul2(g, dx) : fma2(g, dx, db[j]);
                            dc[j] = i == 0 ? mul2(e, now) : fma2(e, now, dc[j]);
                            carry[j][i] = mul2(a[j], g);
                        }
                    }
                    float vb[E], vc[E];
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        float x, y;
                        unpack2(db[j], x, y);
                        vb[j] = x + y;
                        unpack2(dc[j], x, y);
                        vc[j] = x + y;
                    }
                    float over_channels[Place<L>::CV], over_states[2][Place<L>::SV];
                    at.sum_channels(vb, vc, over_channels);
                    at.sum_states(driven, over_states[0]);
                    at.sum_states(decayed, over_states[1]);
                    if (Place<L>::GROUPS == 1) __syncwarp();       // every lane has read the step's values
                    at.store_channels_sum(over_channels, sums + (warp * T + t) * 2 * K::ME);
                    at.store_states_sum(over_states[0], sx + t * K::PW);
                    at.store_states_sum(over_states[1], se + t * K::PW);
                }
            }
        };
        if (c0 < b.valid) {
            if (deep) back(std::true_type{});
            else back(std::false_type{});
        } else {
            for (int i = lane; i < T * 2 * K::ME; i += 32) sums[warp * T * 2 * K::ME + i] = 0.0f;
        }
        __syncthreads();                       // every warp's sums are in place
        float* steps_to = q.steps + (((int64_t)b.cb * p.N + anew(b.n)) * p.S + t0) * p.G * 2 * p.M + b.g * 2 * p.M;
        for (int i = threadIdx.x; i < steps * 2 * K::ME; i += K::THREADS) {
            const int t = i / (2 * K::ME), w = i / K::ME % 2, m = i % K::ME;
            float s = 0.0f;
#pragma unroll
            for (int o = 0; o < K::W; ++o) s += sums[o * T * 2 * K::ME + i];
            if (m < p.M) steps_to[(int64_t)t * p.G * 2 * p.M + w * p.M + m] = s;
        }
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int t = er + i * ROWS;
            if (ROWS > T && t >= T) break;
            const int64_t tt = t0 + t, row = anew(b.n);
            const int count = t < steps ? some : 0;
            f2 v[NP], x[NP], dy[NP], z[NP];
            float dx[NV], ddt[NV], dz[NV];
            load_pairs<V, NV>(r + t * K::Rows::PITCH, v);
            load_pairs<V, NV>(r + K::RX + t * K::Rows::PITCH, x);
            load_pairs<V, NV>(r + 2 * K::RX + t * K::Rows::PITCH, dy);
            if (gate) load_pairs<V, NV>(r + 3 * K::RX + t * K::Rows::PITCH, z);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const f2 driven = *reinterpret_cast<const f2*>(sx + t * K::PW + ev + 2 * e);
                const f2 decayed = *reinterpret_cast<const f2*>(se + t * K::PW + ev + 2 * e);
                const f2 d = *reinterpret_cast<const f2*>(sd + t * K::PW + ev + 2 * e);
                const f2 skip = *reinterpret_cast<const f2*>(sb + K::WC + ev + 2 * e);
                f2 slope = dy[e];
                if (gate) {
                    const f2 y = *reinterpret_cast<const f2*>(rawy + (k & 1) * K::RY + t * K::Sums::PITCH + ec + 2 * e);
                    const f2 s = sigmoid_fast2(z[e]), one = dup2(1.0f);
                    // silu's slope s (1 + z (1 - s))
                    const f2 w = mul2(s, fma2(z[e], fma2(s, dup2(-1.0f), one), one));
                    unpack2(mul2(mul2(dy[e], y), w), dz[2 * e], dz[2 * e + 1]);
                    slope = mul2(dy[e], mul2(z[e], s));
                }
                f2 g = fma2(x[e], driven, mul2(decayed, dup2(kLn2)));      // A carries log2 e
                if (p.softplus) g = mul2(g, sigmoid_fast2(add2(v[e], *reinterpret_cast<const f2*>(sb + ev + 2 * e))));
                if (t >= steps) g = 0, slope = 0;
                dskip[e] = fma2(slope, x[e], dskip[e]);
                dbias[e] = add2(dbias[e], g);
                unpack2(fma2(d, driven, mul2(skip, slope)), dx[2 * e], dx[2 * e + 1]);
                unpack2(g, ddt[2 * e], ddt[2 * e + 1]);
            }
            if (pp.dX.data) store_vec<V, NV>(static_cast<V*>(pp.dX.data) + tt * pp.dX.ss + row * pp.dX.bs + b.d0 + ec, dx, count, q.vec_dx);
            if (pp.ddt.data) store_vec<V, NV>(static_cast<V*>(pp.ddt.data) + tt * pp.ddt.ss + row * pp.ddt.bs + b.d0 + ec, ddt, count, q.vec_ddt);
            if (gate && pp.dZ.data) store_vec<V, NV>(static_cast<V*>(pp.dZ.data) + tt * pp.dZ.ss + row * pp.dZ.bs + b.d0 + ec, dz, count, q.vec_dz);
        }
    }

    // steps past the row's end
    const float zero[NV] = {};
    for (int64_t t = (b.live > b.t_first ? b.live : b.t_first) + er; t < b.t_end; t += ROWS) {
        if (pp.dX.data) store_vec<V, NV>(static_cast<V*>(pp.dX.data) + t * pp.dX.ss + b.n * pp.dX.bs + b.d0 + ec, zero, some, q.vec_dx);
        if (pp.ddt.data) store_vec<V, NV>(static_cast<V*>(pp.ddt.data) + t * pp.ddt.ss + b.n * pp.ddt.bs + b.d0 + ec, zero, some, q.vec_ddt);
        if (pp.dZ.data) store_vec<V, NV>(static_cast<V*>(pp.dZ.data) + t * pp.dZ.ss + b.n * pp.dZ.bs + b.d0 + ec, zero, some, q.vec_dz);
    }
    float* part = q.part + ((int64_t)b.chunk * p.N + b.n) * p.D * (p.M + 2);
    store_states<L>(dA, part + b.d0 * p.M, at, c0, b.valid, p.M);
    if (b.chunk == 0 && pp.dh0) store_states<L>(carry, pp.dh0 + (b.n * p.D + b.d0) * p.M, at, c0, b.valid, p.M);
    part += p.D * p.M + b.d0 + ec;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
#pragma unroll
        for (int o = PER_ROW; o < 32; o *= 2) {
            dskip[e] = add2(dskip[e], __shfl_xor_sync(~0u, dskip[e], o));
            dbias[e] = add2(dbias[e], __shfl_xor_sync(~0u, dbias[e], o));
        }
        float s[2], t[2];
        unpack2(dskip[e], s[0], s[1]);
        unpack2(dbias[e], t[0], t[1]);
#pragma unroll
        for (int o = 0; o < 2; ++o)
            if (er == 0 && 2 * e + o < some) {
                part[2 * e + o] = s[o];
                part[p.D + 2 * e + o] = t[o];
            }
    }
}

// The q that chunks 1 .. pass on when none enters them, and the sums of their delta.
template <typename V, int L>
__global__ void __launch_bounds__(Tile<V, L>::THREADS, 16 / Tile<V, L>::W)
    ssm_scan_grad_ends_kernel(const ScanGradParams pp, const GradLaunch q)
{
    using K = Tile<V, L>;
    const ScanParams& p = pp.f;
    extern __shared__ __align__(16) char smem[];
    V* raw = reinterpret_cast<V*>(smem);                          // [2][3][T][..]: dt, dY, Z
    V* rawc = raw + 2 * 3 * K::RX;                                // [2][T][..]: C
    float* sc = reinterpret_cast<float*>(rawc + 2 * K::RB);       // [T][ME]: C
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float* sd = sc + T * K::ME + warp * (2 * T * K::PW + 2 * K::WC);    // the warp's delta, e and dt_bias
    float* se = sd + T * K::PW;
    float* sb = se + T * K::PW;

    Block b{};
    b.find<K::W * K::WC>(p, q, 1);
    const Place<L> at;
    const int c0 = warp * K::WC;
    f2 A[E][PAIRS], carry[E][PAIRS];
    load_states<L>(A, p.A + b.d0 * p.M, at, c0, b.valid, p.M, false, kLog2e);
#pragma unroll
    for (int j = 0; j < E; ++j)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) carry[j][i] = 0;
    constexpr int PER_ROW = K::WC / NV, ROWS = 32 / PER_ROW, TURNS = (T + ROWS - 1) / ROWS;
    const int ev = lane % PER_ROW * NV, er = lane / PER_ROW, ec = c0 + ev;
    const int some = b.valid - ec < NV ? (b.valid - ec > 0 ? b.valid - ec : 0) : NV;
    f2 total[NP] = {0, 0};
    for (int i = lane; i < K::WC; i += 32) sb[i] = p.dt_bias && c0 + i < b.valid ? p.dt_bias[b.d0 + c0 + i] : 0.0f;
    __syncwarp();

    const bool gate = p.Z.data;
    const int tiles = b.tiles();
    auto stage = [&](int k) {
        const int64_t t0 = b.t_first + (int64_t)k * T, left = b.live - t0, row = anew(b.n);
        const int steps = left < T ? (int)left : T;
        V* r = raw + (k & 1) * 3 * K::RX;
        K::Rows::copy(r, p.dt, row, t0, b.d0, steps, b.valid, q.fast_dt);
        K::Rows::copy(r + K::RX, pp.dY, row, t0, b.d0, steps, b.valid, q.fast_dy);
        if (gate) K::Rows::copy(r + 2 * K::RX, p.Z, row, t0, b.d0, steps, b.valid, q.fast_z);
        K::Pairs::copy(rawc + (k & 1) * K::RB, p.C, row, t0, (int64_t)b.g * p.M, steps, p.M, q.fast_c);
        cp_async_commit();
    };
    if (tiles) stage(tiles - 1);
    for (int k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = b.t_first + (int64_t)k * T;
        const int steps = b.live - t0 < T ? (int)(b.live - t0) : T;
        const V* r = raw + (k & 1) * 3 * K::RX + ec;
        cp_async_wait<0>();
        __syncthreads();
        if (k > 0) stage(k - 1);
        for (int i = threadIdx.x; i < T * K::ME; i += K::THREADS)
            sc[i] = to_f(rawc[(k & 1) * K::RB + i / K::ME * K::Pairs::PITCH + i % K::ME]);
        f2 d[TURNS * NP];
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            f2 v[NP];
            load_pairs<V, NV>(r + (er + i * ROWS) % T * K::Rows::PITCH, v);
#pragma unroll
            for (int e = 0; e < NP; ++e) d[i * NP + e] = add2(v[e], *reinterpret_cast<const f2*>(sb + ev + 2 * e));
        }
        if (p.softplus) softplus_pairs(d);
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int t = er + i * ROWS;
            if (ROWS > T && t >= T) break;
            f2 dy[NP], z[NP];
            load_pairs<V, NV>(r + K::RX + t * K::Rows::PITCH, dy);
            if (gate) load_pairs<V, NV>(r + 2 * K::RX + t * K::Rows::PITCH, z);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                f2& v = d[i * NP + e];
                if (t >= steps) v = 0;
                total[e] = add2(total[e], v);
                *reinterpret_cast<f2*>(sd + t * K::PW + ev + 2 * e) = v;
                *reinterpret_cast<f2*>(se + t * K::PW + ev + 2 * e) = gate ? gate_slope(dy[e], z[e]) : dy[e];
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            const float2 g0 = *reinterpret_cast<const float2*>(sc + t * K::ME + at.m0);
            const float2 g1 = *reinterpret_cast<const float2*>(sc + t * K::ME + at.m1);
            const f2 C[E] = {dup2(g0.x), dup2(g0.y), dup2(g1.x), dup2(g1.y)};
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const f2 dd = *reinterpret_cast<const f2*>(sd + t * K::PW + at.ch[i]);
                const f2 e = *reinterpret_cast<const f2*>(se + t * K::PW + at.ch[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) carry[j][i] = mul2(decay2(dd, A[j][i]), fma2(C[j], e, carry[j][i]));
            }
        }
    }
    store_states<L>(carry, q.ends + ((int64_t)(b.chunk - 1) * p.N + b.n) * p.D * p.M + b.d0 * p.M, at, c0, b.valid, p.M);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
#pragma unroll
        for (int o = PER_ROW; o < 32; o *= 2) total[e] = add2(total[e], __shfl_xor_sync(~0u, total[e], o));
        float v[2];
        unpack2(total[e], v[0], v[1]);
#pragma unroll
        for (int o = 0; o < 2; ++o)
            if (er == 0 && 2 * e + o < some) q.deltas[((int64_t)(b.chunk - 1) * p.N + b.n) * p.D + b.d0 + ec + 2 * e + o] = v[o];
    }
}

// The q that enters each chunk but the last, from the last: one state a thread.
__global__ void __launch_bounds__(256) ssm_scan_grad_chain_kernel(const ScanGradParams pp, const GradLaunch q)
{
    const ScanParams& p = pp.f;
    const int64_t per = p.N * p.D * p.M, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int64_t nd = i / p.M;
    const float a = p.A[nd % p.D * p.M + i % p.M] * kLog2e;
    float v = pp.dhT ? pp.dhT[i] : 0.0f;
    constexpr int B = 8;
    for (int c1 = q.chunks - 2; c1 >= 0; c1 -= B) {
        float e[B], d[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            e[k] = c1 >= k ? q.ends[(c1 - k) * per + i] : 0.0f;
            d[k] = c1 >= k ? q.deltas[(int64_t)(c1 - k) * p.N * p.D + nd] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            v = fmaf(ex2(a * d[k]), v, e[k]);
            if (c1 >= k) q.ends[(c1 - k) * per + i] = v;
        }
    }
}

// The sums over blocks, in order.  Blocks below `parts_blocks`: dA, dDskip and
// ddt_bias over rows and chunks (32 values a block, 8 threads' sums each); the others: dB and
// dC of every step over the blocks of channels, zero past a row's end.
template <typename V>
__global__ void __launch_bounds__(256) ssm_scan_grad_sums_kernel(const ScanGradParams pp, const GradLaunch q, int64_t parts_blocks)
{
    const ScanParams& p = pp.f;
    if (blockIdx.x < parts_blocks) {
        __shared__ float sums[8][33];
        const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
        const int64_t n0 = p.D * p.M, n = n0 + 2 * p.D, i = (int64_t)blockIdx.x * 32 + lane, parts = q.chunks * p.N;
        float s = 0.0f;
        if (i < n) {
#pragma unroll 8
            for (int64_t r = w; r < parts; r += 8) s += q.part[r * n + i];
        }
        sums[w][lane] = s;
        __syncthreads();
        if (w != 0 || i >= n) return;
        s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += sums[r][lane];
        if (i < n0) {
            if (pp.dA) pp.dA[i] = s;
        } else if (i < n0 + p.D) {
            if (pp.dDskip) pp.dDskip[i - n0] = s;
        } else if (pp.ddt_bias) {
            pp.ddt_bias[i - n0 - p.D] = s;
        }
        return;
    }
    const int64_t per = (int64_t)p.G * 2 * p.M, count = p.N * p.S * per;
    for (int64_t i = (blockIdx.x - parts_blocks) * 256 + threadIdx.x; i < count; i += (gridDim.x - parts_blocks) * 256) {
        const int64_t step = i / per, t = step % p.S, n = step / p.S;
        const int r = (int)(i - step * per), g = r / (2 * p.M), w = r / p.M % 2, m = r % p.M;
        float s = 0.0f;
        if (t < row_length(p.lens, n, p.S, p.status)) {
#pragma unroll 4
            for (int cb = 0; cb < q.cblocks; ++cb) s += q.steps[cb * count + i];
        }
        const View& v = w ? pp.dC : pp.dB;
        if (v.data) static_cast<V*>(v.data)[t * v.ss + n * v.bs + g * p.M + m] = from_f<V>(s);
    }
}

constexpr int64_t kMaxGrid = 0x7fffffff;

// Measured times of a step (M = 16, bf16, gate, in ns) with 1 .. 3 warps on
// every scheduler: 687, 807, 1120; finding the chunks' q costs another quarter
// of a pass.  8 rows of 2048 steps x 2048 channels take 1408 us unsplit, 832 us in 7
// chunks; one row of 16384 steps 845 us in 57; 64 rows of 512 steps fill the SMs
// and take 1501 us unsplit, 1553 us in two.
constexpr ScanCost kCost{3, {0, 687, 807, 1120}, 3000, 0.25};

template <typename V, int L>
cudaError_t run(const ScanGradParams& pp, cudaStream_t s, int* launches)
{
    using K = Tile<V, L>;
    const ScanParams& p = pp.f;
    const ScanChoice& c = p.split;
    static std::atomic<uint64_t> ready_ends{0}, ready{0};
    const int elem = (int)sizeof(V);
    const int64_t dg = p.D / p.G, block = K::W * K::WC, group = p.G > 1 ? dg : 0;
    GradLaunch q{};
    q.cblocks = (int)c.cblocks;
    q.chunk = c.chunk;
    q.chunks = c.chunks;
    q.fast_x = rows_aligned(p.X, elem, block, group);
    q.fast_dt = rows_aligned(p.dt, elem, block, group);
    q.fast_z = rows_aligned(p.Z, elem, block, group);
    q.fast_dy = rows_aligned(pp.dY, elem, block, group);
    q.fast_y = rows_aligned(View{p.saved + ssm_saved_states(p.S, p.N, p.D, p.M), p.D, p.S * p.D}, 4, block, group);
    q.fast_b = rows_aligned(p.B, elem, 0, p.G > 1 ? p.M : 0);
    q.fast_c = rows_aligned(p.C, elem, 0, p.G > 1 ? p.M : 0);
    const int64_t bytes = elem * NV;
    auto vec = [&](const View& v) {
        return (uintptr_t)v.data % bytes == 0 && v.ss * elem % bytes == 0 && v.bs * elem % bytes == 0 && group * elem % bytes == 0;
    };
    q.vec_dx = vec(pp.dX);
    q.vec_ddt = vec(pp.ddt);
    q.vec_dz = vec(pp.dZ);
    q.vec_h = p.M % 2 == 0 && (uintptr_t)p.saved % 8 == 0;
    const int64_t states = p.N * p.D * p.M;
    q.ends = p.scratch;
    q.deltas = q.ends + (c.chunks - 1) * states;
    q.part = q.deltas + (c.chunks - 1) * p.N * p.D;
    q.steps = q.part + c.chunks * p.N * p.D * (p.M + 2);
    const int64_t blocks = c.cblocks * p.G * p.N;
    if (blocks > kMaxGrid / c.chunks) return cudaErrorInvalidConfiguration;
    if (c.chunks > 1) {
        auto* f = ssm_scan_grad_ends_kernel<V, L>;
        cudaError_t e = allow_shared(f, K::bytes_ends(), ready_ends);
        if (e != cudaSuccess) return e;
        f<<<(unsigned)(blocks * (c.chunks - 1)), K::THREADS, K::bytes_ends(), s>>>(pp, q);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ++*launches;
        if (c.chunks > kFold) {
            if ((states + 255) / 256 > kMaxGrid) return cudaErrorInvalidConfiguration;
            ssm_scan_grad_chain_kernel<<<(unsigned)((states + 255) / 256), 256, 0, s>>>(pp, q);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            ++*launches;
        }
    }
    auto* f = ssm_scan_grad_kernel<V, L>;
    cudaError_t e = allow_shared(f, K::bytes(), ready);
    if (e != cudaSuccess) return e;
    f<<<(unsigned)(blocks * c.chunks), K::THREADS, K::bytes(), s>>>(pp, q);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    const int64_t parts_blocks = (p.D * (p.M + 2) + 31) / 32, steps_blocks = (p.N * p.S * p.G * 2 * p.M + 255) / 256;
    if (parts_blocks > kMaxGrid - 65536) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)(parts_blocks + (steps_blocks < 65536 ? steps_blocks : 65536));
    ssm_scan_grad_sums_kernel<V><<<grid, 256, 0, s>>>(pp, q, parts_blocks);
    ++*launches;
    return cudaGetLastError();
}

template <typename V>
cudaError_t by_lanes(const ScanGradParams& p, cudaStream_t s, int* launches)
{
    switch (ssm_lanes(p.f.M)) {
    case 1: return run<V, 1>(p, s, launches);
    case 2: return run<V, 2>(p, s, launches);
    case 4: return run<V, 4>(p, s, launches);
    case 8: return run<V, 8>(p, s, launches);
    case 16: return run<V, 16>(p, s, launches);
    default: return run<V, 32>(p, s, launches);
    }
}

}  // namespace

void ssm_scan_grad_plan(ScanGradParams& pp, size_t* bytes)
{
    ScanParams& p = pp.f;
    p.split = ssm_split(p, T, kCost);
    const ScanChoice& c = p.split;
    *bytes = sizeof(float) * (size_t)((c.chunks - 1) * p.N * p.D * (p.M + 1) + c.chunks * p.N * p.D * (p.M + 2) +
                                      c.cblocks * p.N * p.S * p.G * 2 * p.M);
}

cudaError_t launch_ssm_scan_grad(const ScanGradParams& p, cudaStream_t s, int* launches)
{
    if (p.f.N == 0) return launch_sum_parts(nullptr, 0, p.dA, p.f.D * p.f.M, p.dDskip, p.f.D, p.ddt_bias, p.f.D, s, launches);
    return p.f.io == 1   ? by_lanes<__half>(p, s, launches)
           : p.f.io == 2 ? by_lanes<__nv_bfloat16>(p, s, launches)
                         : by_lanes<float>(p, s, launches);
}

}  // namespace rnngb
