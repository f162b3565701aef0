// Shared by the gated delta rule's entry points (delta_api.cpp) and kernels.
#pragma once

#include "ssm_internal.h"

namespace rnngb {

// Steps that are taken together as matrix products.
constexpr int kDeltaChunk = 64;
constexpr int kDeltaMaxKey = 128;
constexpr int kDeltaMaxValue = 1024;

struct DeltaParams {
    int64_t S, N;
    int H, HK, DK, DV, io, sms;
    float scale;
    View Q, K, V, g, beta, Y;
    const int32_t* lens;
    const float* h0;        // [N, H, DK, DV]
    float* hT;
    unsigned char *keys, *mats;     // what the chunks' first launch leaves (delta_mma.cuh: Images)
    unsigned char* kept;    // the states before the chunks, and u (delta_kept_bytes); NULL: not kept
    int* status;
    // A run whose chain is cut into `cuts` segments of cut_chunks chunks (delta_split): what takes a state over each of them,
    // and the states before them.
    int cuts;
    int64_t cut_chunks;
    float *over, *starts;   // [N, H, cuts - 1, DK, DV + DK] and [N, H, cuts, DK, DV]
};

struct DeltaGradParams {
    DeltaParams f;          // Y and hT unused
    View dY, dQ, dK, dV, dg, dbeta;
    const float* dhT;
    float* dh0;
    unsigned char* slopes;  // scratch (delta_slopes_bytes): the slopes in the states after the chunks, dR and dY
};

struct DeltaStepParams {
    int64_t N, slots_n;
    int H, HK, DK, DV, io, sms;
    float scale;
    View Q, K, V, g, beta, Y;
    const float* state;
    float* state_out;
    const int32_t* slots;
    int* status;
};

__host__ __device__ inline int64_t delta_chunks(int64_t S) { return (S + kDeltaChunk - 1) / kDeltaChunk; }
// The images of a run's chunks (delta_mma.cuh), and what a run saves for its gradient: them, the states
// before the chunks, and u.
constexpr int64_t kDeltaBlock = 8192, kDeltaFactors = 768 * 4, kDeltaMats = 4 * kDeltaBlock + kDeltaFactors;
inline int64_t delta_keys_bytes(int64_t S, int64_t N, int64_t HK, int64_t DK, int io)
{
    return N * HK * delta_chunks(S) * 2 * (io == 0 ? 2 : 1) * ((DK + 63) / 64) * kDeltaBlock;
}
inline int64_t delta_mats_bytes(int64_t S, int64_t N, int64_t H) { return N * H * delta_chunks(S) * kDeltaMats; }
// Of a chunk, head and 128 values: two parts each of the state (64 keys a block) and of u, and their scales.
__host__ __device__ inline int64_t delta_kept_tile(int DK) { return (2 * ((DK + 63) / 64) + 2) * 2 * kDeltaBlock + 1024; }
// ... of the slope in the state, of dR, and of dY (16-bit ones have one part).
__host__ __device__ inline int64_t delta_slopes_tile(int DK, int io) { return delta_kept_tile(DK) + (io == 0 ? 2 : 1) * 2 * kDeltaBlock; }
inline int64_t delta_tiles(int64_t S, int64_t N, int64_t H, int64_t DV) { return N * H * delta_chunks(S) * ((DV + 127) / 128); }
inline int64_t delta_saved_floats(int64_t S, int64_t N, int64_t H, int64_t HK, int64_t DK, int64_t DV, int io)
{
    return (delta_keys_bytes(S, N, HK, DK, io) + delta_mats_bytes(S, N, H) + delta_tiles(S, N, H, DV) * delta_kept_tile((int)DK)) / 4;
}
inline int64_t delta_slopes_bytes(int64_t S, int64_t N, int64_t H, int64_t DK, int64_t DV, int io)
{
    return delta_tiles(S, N, H, DV) * delta_slopes_tile((int)DK, io);
}

void delta_split(DeltaParams& p);
inline int64_t delta_split_floats(const DeltaParams& p)
{
    return p.cuts > 1 ? p.N * p.H * p.DK * ((p.cuts - 1) * (int64_t)(p.DV + p.DK) + p.cuts * (int64_t)p.DV) : 0;
}
cudaError_t launch_delta(const DeltaParams& p, cudaStream_t s, int* launches);
cudaError_t launch_delta_grad(const DeltaGradParams& p, cudaStream_t s, int* launches);
cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s, int* launches);

}  // namespace rnngb
