// Shared by the state space and token score entry points (ssm_api.cpp) and
// their kernels.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace rnngb {

void set_last_error(const char* message);   // rnn_last_error's text (this thread)

// A [seq, batch, ...] tensor with a dense innermost part; strides in elements.
struct View {
    void* data = nullptr;
    int64_t ss = 0, bs = 0;
};

// What the scan saves for its gradient: the state before every kSsmTile-th
// step, [N][ceil(S / kSsmTile)][D][M] (from which the gradient, in tiles of that many
// steps, forms the others again), then y before its gate, [N][S][D].
constexpr int kSsmTile = 8;
__host__ __device__ inline int64_t ssm_saved_states(int64_t S, int64_t N, int64_t D, int64_t M)
{
    return (S + kSsmTile - 1) / kSsmTile * N * D * M;
}
constexpr int kSsmMaxState = 128;
constexpr int kSsmMaxTaps = 8;
constexpr int kMaxTop = 32;

struct ConvParams {
    int64_t S, N, D;
    int K, io, silu, sms;   // sms: the device's multiprocessors, here and below
    View X, Y;
    const float *W, *bias;
    const int32_t* lens;
    const void* h0;         // [N, K-1, D]
    void* hT;
    int* status;
};

struct ConvGradParams {
    ConvParams f;           // Y and hT unused
    View dY, dX;
    const void* dhT;
    void* dh0;
    float *dW, *dbias;
    int run;                // steps of a run (ssm_conv_grad_plan, as parts)
    float* part;            // [parts, D * K + D]
    int64_t parts;
};

struct ConvStepParams {
    int64_t N, D, slots_n;
    int K, io, silu;
    View X, Y;
    const float *W, *bias;
    const void* state;
    void* state_out;
    const int32_t* slots;
    int* status;
};

// How a scan is split: blocks of channels in a group, and chunks of `chunk`
// steps.
struct ScanChoice {
    int chunks;
    int64_t cblocks, chunk;
};

struct ScanParams {
    int64_t S, N, D;
    int M, G, io, softplus, sms;
    View X, dt, B, C, Z, Y;
    const float *A, *Dskip, *dt_bias;
    const int32_t* lens;
    const float* h0;
    float* hT;
    float* saved;
    ScanChoice split;       // ssm_scan_plan, ssm_scan_grad_plan
    float* scratch;
    int* status;
};

struct ScanGradParams {
    ScanParams f;           // Y and hT unused
    View dY, dX, ddt, dB, dC, dZ;
    const float* dhT;
    float *dA, *dDskip, *ddt_bias, *dh0;
};

struct ScanStepParams {
    int64_t N, D, slots_n;
    int M, G, io, softplus, sms;
    View X, dt, B, C, Z, Y;
    const float *A, *Dskip, *dt_bias, *H;
    float* H_out;
    const int32_t* slots;
    int* status;
};

struct ScoreParams {
    int64_t rows, V, stride;
    int io, top;
    const void* x;
    const int32_t* ids;
    float *logp, *entropy, *lse, *lse_rest;
    int32_t* top_ids;
    float* top_logp;
};

struct ScoreGradParams {
    int64_t rows, V, stride, d_stride;
    int io, top;
    const void* x;
    const int32_t* ids;
    const float *lse, *lse_rest, *entropy, *d_logp, *d_entropy;
    const int32_t* top_ids;
    const float* d_top;
    void* dx;
};

// A split is chosen by a model of the time: `warps` warps fit a scheduler, a
// step takes step_ns[w] with w of them on each, a block begin_ns to begin and end, and
// the launch that finds the chunks' end states the part `ends` of the scan's time.
struct ScanCost {
    int warps;
    double step_ns[5], begin_ns, ends;
};
ScanChoice ssm_split(const ScanParams& p, int tile, const ScanCost& cost);
cudaError_t ssm_sm_count(int* sms);
// Lanes of a channel of M states, four a lane: a power of two.
inline int ssm_lanes(int M)
{
    int l = 1;
    while (l * 4 < M) l *= 2;
    return l;
}

// Lets a kernel have more than 48 KB of dynamic shared memory: once on each device.
template <typename F>
cudaError_t allow_shared(F* kernel, size_t bytes, std::atomic<uint64_t>& done)
{
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Each launcher queues its kernels on `s` and adds their number to *launches.
cudaError_t launch_ssm_conv(const ConvParams& p, cudaStream_t s, int* launches);
void ssm_conv_grad_plan(ConvGradParams& p);
cudaError_t launch_ssm_conv_grad(const ConvGradParams& p, cudaStream_t s, int* launches);
cudaError_t launch_ssm_conv_step(const ConvStepParams& p, cudaStream_t s, int* launches);
int64_t ssm_saved_floats(int64_t S, int64_t N, int64_t D, int64_t M);
void ssm_scan_plan(ScanParams& p, size_t* bytes);            // the split, and the scratch's size
cudaError_t launch_ssm_scan(const ScanParams& p, cudaStream_t s, int* launches);
void ssm_scan_grad_plan(ScanGradParams& p, size_t* bytes);
cudaError_t launch_ssm_scan_grad(const ScanGradParams& p, cudaStream_t s, int* launches);
cudaError_t launch_ssm_scan_step(const ScanStepParams& p, cudaStream_t s, int* launches);
cudaError_t launch_scores(const ScoreParams& p, cudaStream_t s, int* launches);
cudaError_t launch_scores_grad(const ScoreGradParams& p, cudaStream_t s, int* launches);

// Sums of `parts` partial results, in order: out0 takes the first n0 values
// of each, out1 the next n1, out2 the last n2 (a NULL output is skipped).
cudaError_t launch_sum_parts(const float* part, int64_t parts, float* out0, int64_t n0, float* out1, int64_t n1,
                             float* out2, int64_t n2, cudaStream_t s, int* launches);

}  // namespace rnngb
