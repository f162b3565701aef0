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
    float* saved;           // delta_saved_floats, or NULL
    float* scratch;         // delta_scratch_bytes
    int* status;
};

struct DeltaGradParams {
    DeltaParams f;          // Y and hT unused
    View dY, dQ, dK, dV, dg, dbeta;
    const float* dhT;
    float* dh0;
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
// What a run saves for its gradient: the state before every chunk, [N][H][chunks][DK][DV],
// then the steps' u, [N][H][chunks][kDeltaChunk][DV].
inline int64_t delta_saved_floats(int64_t S, int64_t N, int64_t H, int64_t DK, int64_t DV)
{
    return N * H * delta_chunks(S) * (DK + kDeltaChunk) * DV;
}
size_t delta_scratch_bytes(const DeltaParams& p);
size_t delta_grad_scratch_bytes(const DeltaGradParams& p);

cudaError_t launch_delta(const DeltaParams& p, cudaStream_t s, int* launches);
cudaError_t launch_delta_grad(const DeltaGradParams& p, cudaStream_t s, int* launches);
cudaError_t launch_delta_step(const DeltaStepParams& p, cudaStream_t s, int* launches);

}  // namespace rnngb
