// C entry points of the layer normalisation: checks of arguments and scratch.
// See include/onnx_recurrent.h for the contract.
#include <cmath>

#include "norm_internal.h"
#include "plan.h"

using namespace rnngb;

struct rnn_norm : PlanMemory {
    int D = 0, io = RNN_IO_F32;
    float eps = 0.f;
};

namespace {

// Rows of D values: *stride in elements.  Output rows must lie apart; an input's may all be one.
rnn_status check_rows(const rnn_norm* pl, const void* data, int64_t rows, int64_t* stride, const char* name, bool out)
{
    const bool one = !out && *stride == RNN_SHARED_ROW;
    if (*stride < 0 && !one) return fail(RNN_ERR_INVALID_ARGUMENT, "%s has a negative stride", name);
    *stride = one ? 0 : *stride == 0 ? pl->D : *stride;
    if (out && data && rows > 1 && *stride < pl->D) return fail(RNN_ERR_INVALID_ARGUMENT, "%s: its rows share memory", name);
    if ((uintptr_t)data % element(pl->io)) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
    return RNN_OK;
}

// An output may be an input itself: every row is read by the block that writes it.
rnn_status check_overlap(const rnn_norm* pl, int64_t rows, const void* in, int64_t is, const void* out, int64_t os, const char* names)
{
    if (!in || !out || rows == 0) return RNN_OK;
    if (in == out && (is == os || rows == 1)) return RNN_OK;
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out, e = element(pl->io);
    const uintptr_t ae = a + e * (uintptr_t)(is * (rows - 1) + pl->D), be = b + e * (uintptr_t)(os * (rows - 1) + pl->D);
    if (a >= be || b >= ae) return RNN_OK;
    // parts of the rows of one wider tensor, side by side
    if (is == os) {
        const uintptr_t gap = (a < b ? b - a : a - b) / e % (uintptr_t)is;
        if ((a < b ? b - a : a - b) % e == 0 && gap >= (uintptr_t)pl->D && (uintptr_t)is - gap >= (uintptr_t)pl->D) return RNN_OK;
    }
    return fail(RNN_ERR_INVALID_ARGUMENT, "%s overlap in part", names);
}

rnn_status check_plan(rnn_norm* pl, const void* args, int64_t rows)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    pl->launches = 0;
    NEED(args, "args");
    if (rows < 0) return fail(RNN_ERR_INVALID_ARGUMENT, "rows %lld", (long long)rows);
    if (rows > 0x7fffff00LL) return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    return RNN_OK;
}

NormParams params(const rnn_norm* pl, int64_t rows)
{
    NormParams p{};
    p.rows = rows;
    p.D = pl->D;
    p.io = pl->io;
    p.sms = pl->sms;
    p.eps = pl->eps;
    return p;
}

}  // namespace

extern "C" {

rnn_status rnn_norm_create(rnn_norm_t* out, int64_t size, float eps)
{
    NEED(out, "out");
    *out = nullptr;
    if (size < 1 || size > kNormMaxSize)
        return fail(RNN_ERR_INVALID_ARGUMENT, "size %lld outside [1, %d]", (long long)size, kNormMaxSize);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(RNN_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
    rnn_norm* pl = new (std::nothrow) rnn_norm;
    if (!pl) return fail(RNN_ERR_OOM, "host allocation failed");
    pl->D = (int)size;
    pl->eps = eps;
    *out = pl;
    return RNN_OK;
}

void rnn_norm_destroy(rnn_norm_t pl)
{
    if (!pl) return;
    free_plan_memory(pl);
    delete pl;
}

rnn_status rnn_norm_set_io_type(rnn_norm_t pl, int io)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (io != RNN_IO_F32 && io != RNN_IO_F16 && io != RNN_IO_BF16)
        return fail(RNN_ERR_INVALID_ARGUMENT, "unknown io type %d", io);
    pl->io = io;
    return RNN_OK;
}

int rnn_norm_last_launch_count(rnn_norm_t pl) { return pl ? pl->launches : 0; }

rnn_status rnn_layer_norm(rnn_norm_t pl, const rnn_norm_args* a)
{
    rnn_status rs = check_plan(pl, a, a ? a->rows : 0);
    if (rs != RNN_OK || a->rows == 0) return rs;
    NEED(a->X, "X");
    NEED(a->Y, "Y");
    int64_t xs = a->x_stride, ys = a->y_stride;
    rs = check_rows(pl, a->X, a->rows, &xs, "X", false);
    if (rs == RNN_OK) rs = check_rows(pl, a->Y, a->rows, &ys, "Y", true);
    if (rs == RNN_OK) rs = check_overlap(pl, a->rows, a->X, xs, a->Y, ys, "X and Y");
    if (rs == RNN_OK) rs = check_arrays({{a->W, "W"}, {a->bias, "bias"}, {a->stats, "stats"}});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    NormParams p = params(pl, a->rows);
    p.X = a->X;
    p.xs = xs;
    p.W = a->W;
    p.bias = a->bias;
    p.Y = a->Y;
    p.ys = ys;
    p.stats = a->stats;
    cudaError_t e = launch_norm(p, (cudaStream_t)a->stream, &pl->launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "normalisation launch");
}

rnn_status rnn_layer_norm_grad(rnn_norm_t pl, const rnn_norm_grad_args* a)
{
    rnn_status rs = check_plan(pl, a, a ? a->rows : 0);
    if (rs != RNN_OK) return rs;
    if (a->rows > 0) {
        NEED(a->dY, "dY");
        NEED(a->X, "X");
        NEED(a->stats, "stats");
    } else if (!a->dW && !a->dbias) {
        return RNN_OK;
    }
    int64_t xs = a->x_stride, dys = a->dy_stride, dxs = a->dx_stride;
    rs = check_rows(pl, a->X, a->rows, &xs, "X", false);
    if (rs == RNN_OK) rs = check_rows(pl, a->dY, a->rows, &dys, "dY", false);
    if (rs == RNN_OK) rs = check_rows(pl, a->dX, a->rows, &dxs, "dX", true);
    if (rs == RNN_OK) rs = check_overlap(pl, a->rows, a->X, xs, a->dX, dxs, "X and dX");
    if (rs == RNN_OK) rs = check_overlap(pl, a->rows, a->dY, dys, a->dX, dxs, "dY and dX");
    if (rs == RNN_OK) rs = check_arrays({{a->W, "W"}, {a->stats, "stats"}, {a->dW, "dW"}, {a->dbias, "dbias"}});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    NormGradParams q{};
    q.f = params(pl, a->rows);
    q.f.X = a->X;
    q.f.xs = xs;
    q.f.W = a->W;
    q.f.stats = const_cast<float*>(a->stats);
    q.dY = a->dY;
    q.dys = dys;
    q.dX = a->dX;
    q.dxs = dxs;
    q.dW = a->dW;
    q.dbias = a->dbias;
    if (!q.dX && !q.dW && !q.dbias) return RNN_OK;
    norm_grad_plan(q);
    const size_t bytes = q.dW || q.dbias ? sizeof(float) * norm_grad_floats(q) : 0;
    cudaStream_t st = (cudaStream_t)a->stream;
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes, st, &scratch);
    if (rs != RNN_OK) return rs;
    q.part = (float*)scratch;
    q.off = q.part + 2 * q.parts * pl->D;
    cudaError_t e = launch_norm_grad(q, st, &pl->launches);
    if (e != cudaSuccess) return cuda_fail(e, "normalisation gradient launch");
    return release_scratch(pl, bytes, st);
}

}  // extern "C"
