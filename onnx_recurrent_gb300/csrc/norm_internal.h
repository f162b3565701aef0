// Shared by the layer normalisation's and beam search's entry points
// (norm_api.cpp, beam_api.cpp) and kernels.
#pragma once

#include "ssm_internal.h"

namespace rnngb {

constexpr int kNormMaxSize = 32768;
constexpr int kMaxBeams = 32;
constexpr int kReorderTensors = 32;         // of one launch

struct NormParams {
    int64_t rows;
    int D, io, sms;
    float eps;
    const void* X;
    int64_t xs;
    const float *W, *bias;
    void* Y;
    int64_t ys;
    float* stats;           // [rows][2]
};

struct NormGradParams {
    NormParams f;           // Y and bias unused
    const void* dY;
    int64_t dys;
    void* dX;
    int64_t dxs;
    float *dW, *dbias;
    float* part;            // [parts][2][D]
    int64_t parts;          // norm_grad_plan
    float* off;             // [rows], behind the parts (norm_grad_floats): for rows too long to keep a thread's sums
};

struct BeamSelectParams {
    int64_t items, V;
    int B, io, top;         // top: candidates a row has, min(B, V)
    int64_t end;            // -1: none
    int shared;             // an item's beams have one row
    int64_t stride;         // between rows of logits
    const void* logits;
    int sms, parts;         // parts of a row, a block each, and their length (beam_plan)
    int64_t length;
    unsigned char* scratch; // beam_scratch_bytes
    const float* scores;
    const uint8_t* finished;
    int32_t *parents, *ids;
    float* new_scores;
    uint8_t* new_finished;
};
void beam_plan(BeamSelectParams& p);
size_t beam_scratch_bytes(const BeamSelectParams& p);

struct ReorderTensor {
    const void* in;
    void* out;
    int64_t bytes;          // of a row
};
struct ReorderParams {
    int64_t items, n_slots;
    int B, n;
    const int32_t *parents, *slots;
    int* status;
    ReorderTensor t[kReorderTensors];
};

void norm_grad_plan(NormGradParams& p);
size_t norm_grad_floats(const NormGradParams& p);      // of scratch, where dW or dbias is wanted
cudaError_t launch_norm(const NormParams& p, cudaStream_t s, int* launches);
cudaError_t launch_norm_grad(const NormGradParams& p, cudaStream_t s, int* launches);
cudaError_t launch_beam_select(const BeamSelectParams& p, cudaStream_t s, int* launches);
cudaError_t launch_beam_reorder(const ReorderParams& p, cudaStream_t s, int* launches);

}  // namespace rnngb
