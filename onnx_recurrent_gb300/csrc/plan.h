// What the plans of the layers' operators have in common: the error text, checks
// of arguments, and a plan's memory on its device (status word, scratch and the
// scratch's order between streams and captured graphs).
#pragma once

#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/onnx_recurrent.h"
#include "ssm_internal.h"

namespace rnngb {

struct Kept {
    char* data;
    Kept* next;
};

struct PlanMemory {
    int device = -1;              // of the first call: what follows lies there
    int sms = 0;
    int* status = nullptr;        // device word the kernels report through
    char* scratch = nullptr;
    size_t scratch_bytes = 0;
    cudaEvent_t used = nullptr;   // after the last call that used the scratch,
    bool pending = false;         // if there is one,
    unsigned long long user = 0;  // on the stream of this id
    bool capturing = false;       // the call at hand is being captured
    char* graph_scratch = nullptr;   // the scratch of captured calls
    size_t graph_bytes = 0;
    Kept* kept = nullptr;         // it and what it grew from: graphs hold their addresses
    int launches = 0;
};

#define NEED(p, name)                                                             \
    do {                                                                          \
        if (!(p)) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is NULL", name);      \
    } while (0)

inline rnn_status fail(rnn_status st, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}

inline rnn_status cuda_fail(cudaError_t e, const char* what)
{
    return fail(e == cudaErrorMemoryAllocation ? RNN_ERR_OOM : RNN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Lets this thread allocate and free while a stream is being captured, which
// would otherwise spoil the capture.
struct AmidCapture {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const cudaError_t status = cudaThreadExchangeStreamCaptureMode(&mode);
    ~AmidCapture()
    {
        if (status == cudaSuccess) cudaThreadExchangeStreamCaptureMode(&mode);
    }
};

inline size_t element(int io) { return io == RNN_IO_F32 ? 4 : 2; }

inline rnn_status check_view(const rnn_view& v, size_t elem, const char* name)
{
    if (v.seq_stride < 0 || v.batch_stride < 0) return fail(RNN_ERR_INVALID_ARGUMENT, "%s has a negative stride", name);
    if ((uintptr_t)v.data % elem) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
    return RNN_OK;
}

// Output views: one whose steps or rows share memory would be written by blocks that run in any order.
struct OutView {
    View v;
    int64_t inner;
    const char* name;
};

template <int K>
rnn_status check_outputs(int64_t S, int64_t N, const OutView (&views)[K])
{
    for (const OutView& o : views)
        if (o.v.data && ((S > 1 && o.v.ss < o.inner) || (N > 1 && o.v.bs < o.inner) || (S > 1 && N > 1 && o.v.ss == o.v.bs)))
            return fail(RNN_ERR_INVALID_ARGUMENT, "%s: its steps or rows share memory", o.name);
    return RNN_OK;
}

struct NamedF32 {
    const void* p;
    const char* name;
};

// fp32 and int32 arrays: whether they are aligned to their elements.
template <int N>
rnn_status check_arrays(const NamedF32 (&arrays)[N])
{
    for (const NamedF32& a : arrays)
        if ((uintptr_t)a.p % 4) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", a.name);
    return RNN_OK;
}

// A state and where it goes: the same memory, or memory apart.
inline rnn_status check_in_place(const void* in, const void* out, size_t bytes, const char* names)
{
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out;
    if (in && out && a != b && (a < b ? b - a : a - b) < bytes)
        return fail(RNN_ERR_INVALID_ARGUMENT, "%s overlap in part", names);
    return RNN_OK;
}

// The plan's status word, on the device of its calls: the current one, which
// must be the same every time.
inline rnn_status ensure_status(PlanMemory* pl)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (pl->status && device != pl->device)
        return fail(RNN_ERR_INVALID_ARGUMENT, "the plan's memory is on device %d, the current device is %d", pl->device, device);
    if (pl->status) return RNN_OK;
    // Cleared on a stream of its own, which alone is waited for: no other work is, and
    // the plan's first call may be a captured one.
    AmidCapture amid;
    int* p = nullptr;
    e = amid.status == cudaSuccess ? cudaMalloc((void**)&p, 256) : amid.status;
    if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc(status)");
    cudaStream_t own = nullptr;
    e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
    if (e == cudaSuccess) {
        e = cudaMemsetAsync(p, 0, 256, own);
        if (e == cudaSuccess) e = cudaStreamSynchronize(own);
        cudaStreamDestroy(own);
    }
    if (e != cudaSuccess) {
        cudaFree(p);
        return cuda_fail(e, "cudaMemset(status)");
    }
    e = ssm_sm_count(&pl->sms);
    if (e != cudaSuccess) {
        cudaFree(p);
        return cuda_fail(e, "reading the device's attributes");
    }
    pl->status = p;
    pl->device = device;
    return RNN_OK;
}

// Scratch of at least `bytes` for a call that is being captured.  A graph keeps
// the address and runs at times that no event of this plan knows, so it is not the
// plain calls' scratch, and not freed before the plan.
inline rnn_status claim_graph_scratch(PlanMemory* pl, size_t bytes)
{
    if (bytes <= pl->graph_bytes) return RNN_OK;
    Kept* k = new (std::nothrow) Kept;
    if (!k) return fail(RNN_ERR_OOM, "host allocation failed");
    cudaError_t e;
    {
        AmidCapture amid;
        e = amid.status == cudaSuccess ? cudaMalloc((void**)&k->data, bytes) : amid.status;
    }
    if (e != cudaSuccess) {
        delete k;
        return cuda_fail(e, "cudaMalloc(scratch of captured calls)");
    }
    k->next = pl->kept;
    pl->kept = k;
    pl->graph_scratch = k->data;
    pl->graph_bytes = bytes;
    return RNN_OK;
}

// The plan's scratch of at least `bytes`, after the previous call's use of it.
inline rnn_status claim_scratch(PlanMemory* pl, size_t bytes, cudaStream_t st, char** scratch)
{
    *scratch = nullptr;
    if (!bytes) return RNN_OK;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cs);
    if (e != cudaSuccess) return cuda_fail(e, "asking whether the stream is being captured");
    pl->capturing = cs != cudaStreamCaptureStatusNone;
    if (pl->capturing) {
        rnn_status rs = claim_graph_scratch(pl, bytes);
        *scratch = pl->graph_scratch;
        return rs;
    }
    if (bytes > pl->scratch_bytes) {
        if (pl->scratch) {
            cudaFree(pl->scratch);   // synchronises with outstanding work
            pl->scratch = nullptr;
            pl->scratch_bytes = 0;
            pl->pending = false;
        }
        e = cudaMalloc((void**)&pl->scratch, bytes);
        if (e != cudaSuccess) {
            pl->scratch = nullptr;
            return cuda_fail(e, "cudaMalloc(scratch)");
        }
        pl->scratch_bytes = bytes;
    }
    if (!pl->used) {
        e = cudaEventCreateWithFlags(&pl->used, cudaEventDisableTiming);
        if (e != cudaSuccess) {
            pl->used = nullptr;
            return cuda_fail(e, "cudaEventCreate");
        }
    }
    unsigned long long id = 0;
    e = cudaStreamGetId(st, &id);
    if (e == cudaSuccess && pl->pending && id != pl->user) e = cudaStreamWaitEvent(st, pl->used, 0);
    pl->user = id;
    *scratch = pl->scratch;
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "ordering the scratch");
}

inline rnn_status release_scratch(PlanMemory* pl, size_t bytes, cudaStream_t st)
{
    if (!bytes || pl->capturing) return RNN_OK;
    cudaError_t e = cudaEventRecord(pl->used, st);
    pl->pending = true;
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "cudaEventRecord");
}

inline rnn_status check_slots(const int32_t* slots, int64_t n_slots)
{
    if (slots && n_slots <= 0)
        return fail(RNN_ERR_INVALID_ARGUMENT, "n_slots is %lld with slots given", (long long)n_slots);
    return RNN_OK;
}

// Frees what the plan holds on its device.
inline void free_plan_memory(PlanMemory* pl)
{
    // a plan may be collected at any time, amid another's capture too
    AmidCapture amid;
    if (pl->scratch) cudaFree(pl->scratch);   // synchronises with outstanding work
    while (Kept* k = pl->kept) {
        pl->kept = k->next;
        cudaFree(k->data);
        delete k;
    }
    if (pl->status) cudaFree(pl->status);
    if (pl->used) cudaEventDestroy(pl->used);
}

// Waits for the device, reads the status word and clears it.
inline rnn_status read_status(PlanMemory* pl, const char* invalid_input)
{
    if (!pl->status) return RNN_OK;   // nothing has run
    int word = 0, current = 0;
    cudaError_t e = cudaGetDevice(&current);
    if (e == cudaSuccess && current != pl->device) e = cudaSetDevice(pl->device);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&word, pl->status, sizeof word, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && word) {
        e = cudaMemset(pl->status, 0, sizeof word);
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
    }
    if (current != pl->device) cudaSetDevice(current);
    if (e != cudaSuccess) return cuda_fail(e, "reading the status");
    if (word == RNN_ERR_TIMEOUT) return fail(RNN_ERR_TIMEOUT, "a kernel gave up waiting for its own copies or products");
    if (word) return fail(RNN_ERR_INVALID_INPUT, "%s", invalid_input);
    return RNN_OK;
}

}  // namespace rnngb
