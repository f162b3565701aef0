// C entry points of the state space layer's operators and of the token
// scores: checks of arguments, the plan's scratch and its ordering between
// streams.  See include/onnx_recurrent.h for the contract.
#include "plan.h"

using namespace rnngb;

struct rnn_ssm : PlanMemory {
    int64_t D = 0;
    int M = 0, G = 0, K = 0, layout = 0, silu = 0, softplus = 0, io = RNN_IO_F32;
};

namespace {

// A caller's view; both strides 0 stand for a dense tensor in the plan's
// layout whose innermost part holds `inner` values.
View dense(const rnn_view& v, const rnn_ssm* pl, int64_t S, int64_t N, int64_t inner)
{
    View r{v.data, v.seq_stride, v.batch_stride};
    if (r.ss == 0 && r.bs == 0) {
        r.ss = pl->layout == 0 ? N * inner : inner;
        r.bs = pl->layout == 0 ? inner : S * inner;
    }
    return r;
}

View dense_row(const rnn_view& v, int64_t inner) { return View{v.data, 0, v.batch_stride ? v.batch_stride : inner}; }

// Plan, sizes and the views of one call; *none: nothing is to be run.
rnn_status check_sizes(rnn_ssm* pl, const void* args, int64_t S, int64_t N)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    pl->launches = 0;
    NEED(args, "args");
    if (S < 0 || N < 0)
        return fail(RNN_ERR_INVALID_ARGUMENT, "seq_length %lld, batch_size %lld", (long long)S, (long long)N);
    // steps, rows and channel blocks are counted in 32 bits by the launches
    if (S > 0x7fffff00LL || N > 0x7fffff00LL || (N > 0 && pl->D > 0x7fffff00LL))
        return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    return RNN_OK;
}

struct Named {
    const rnn_view* v;
    const char* name;
    bool required;
};

rnn_status check_views(const rnn_ssm* pl, const Named* views, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!views[i].v->data) {
            if (views[i].required) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is NULL", views[i].name);
            continue;
        }
        rnn_status rs = check_view(*views[i].v, element(pl->io), views[i].name);
        if (rs != RNN_OK) return rs;
    }
    return RNN_OK;
}

// The convolution in place: a run of steps begins with the K - 1 inputs before it
// (its gradient ends with the slopes after it), which another block overwrites.
rnn_status check_not_input(const rnn_ssm* pl, int64_t S, const rnn_view& out, const char* name, const rnn_view& in, const char* input)
{
    if (out.data && out.data == in.data && S > 1 && pl->K > 1)
        return fail(RNN_ERR_INVALID_ARGUMENT, "%s must not be %s", name, input);
    return RNN_OK;
}

// Arrays of the plan's io type.
rnn_status check_state(const rnn_ssm* pl, const void* p, const char* name)
{
    if ((uintptr_t)p % element(pl->io)) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
    return RNN_OK;
}

rnn_status check_scores(int64_t rows, int64_t vocab, int64_t stride, int64_t io, int64_t top, const void* x)
{
    if (rows < 0 || vocab <= 0) return fail(RNN_ERR_INVALID_ARGUMENT, "rows %lld, vocab %lld", (long long)rows, (long long)vocab);
    if (rows > 0x7fffff00LL || vocab > 0x7fffff00LL) return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    io &= ~(int64_t)RNN_SCORES_LSE_PAIR;
    if (io != RNN_IO_F32 && io != RNN_IO_F16 && io != RNN_IO_BF16)
        return fail(RNN_ERR_INVALID_ARGUMENT, "unknown io type %lld", (long long)io);
    if (stride != 0 && stride != RNN_SHARED_ROW && stride < vocab)
        return fail(RNN_ERR_INVALID_ARGUMENT, "row_stride %lld is below vocab %lld", (long long)stride, (long long)vocab);
    if (top < 0 || top > kMaxTop || top > vocab)
        return fail(RNN_ERR_INVALID_ARGUMENT, "top %lld outside [0, min(%d, vocab)]", (long long)top, kMaxTop);
    if (rows > 0) {
        NEED(x, "logits");
        if ((uintptr_t)x % element((int)io)) return fail(RNN_ERR_INVALID_ARGUMENT, "logits are not aligned to their elements");
    }
    return RNN_OK;
}

int64_t logits_stride(int64_t stride, int64_t vocab) { return stride == RNN_SHARED_ROW ? 0 : stride ? stride : vocab; }

ConvParams conv_params(const rnn_ssm* pl, int64_t S, int64_t N)
{
    ConvParams p{};
    p.S = S;
    p.N = N;
    p.D = pl->D;
    p.K = pl->K;
    p.io = pl->io;
    p.silu = pl->silu;
    p.sms = pl->sms;
    p.status = pl->status;
    return p;
}

ScanParams scan_params(const rnn_ssm* pl, int64_t S, int64_t N)
{
    ScanParams p{};
    p.S = S;
    p.N = N;
    p.D = pl->D;
    p.M = pl->M;
    p.G = pl->G;
    p.io = pl->io;
    p.softplus = pl->softplus;
    p.sms = pl->sms;
    p.status = pl->status;
    return p;
}

}  // namespace

extern "C" {

rnn_status rnn_ssm_create(rnn_ssm_t* out, int64_t channels, int64_t state_size, int64_t groups, int64_t conv_width,
                          int layout, int conv_silu, int dt_softplus)
{
    NEED(out, "out");
    *out = nullptr;
    if (channels <= 0 || channels > 0x7fffff00LL)
        return fail(RNN_ERR_INVALID_ARGUMENT, "channels must be positive and below 2^31, got %lld", (long long)channels);
    if (state_size < 1 || state_size > kSsmMaxState)
        return fail(RNN_ERR_INVALID_ARGUMENT, "state_size %lld outside [1, %d]", (long long)state_size, kSsmMaxState);
    if (groups <= 0 || channels % groups)
        return fail(RNN_ERR_INVALID_ARGUMENT, "groups %lld does not divide channels %lld", (long long)groups, (long long)channels);
    if (conv_width < 1 || conv_width > kSsmMaxTaps)
        return fail(RNN_ERR_INVALID_ARGUMENT, "conv_width %lld outside [1, %d]", (long long)conv_width, kSsmMaxTaps);
    if ((layout | conv_silu | dt_softplus) & ~1)
        return fail(RNN_ERR_INVALID_ARGUMENT, "layout, conv_silu and dt_softplus are 0 or 1");
    rnn_ssm* pl = new (std::nothrow) rnn_ssm;
    if (!pl) return fail(RNN_ERR_OOM, "host allocation failed");
    pl->D = channels;
    pl->M = (int)state_size;
    pl->G = (int)groups;
    pl->K = (int)conv_width;
    pl->layout = layout;
    pl->silu = conv_silu;
    pl->softplus = dt_softplus;
    *out = pl;
    return RNN_OK;
}

void rnn_ssm_destroy(rnn_ssm_t pl)
{
    if (!pl) return;
    free_plan_memory(pl);
    delete pl;
}

rnn_status rnn_ssm_set_io_type(rnn_ssm_t pl, int io)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (io != RNN_IO_F32 && io != RNN_IO_F16 && io != RNN_IO_BF16)
        return fail(RNN_ERR_INVALID_ARGUMENT, "unknown io type %d", io);
    pl->io = io;
    return RNN_OK;
}

rnn_status rnn_ssm_sync(rnn_ssm_t pl)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    return read_status(pl, "a sequence length outside [0, seq_length] or a slot outside its range");
}

int rnn_ssm_last_launch_count(rnn_ssm_t pl) { return pl ? pl->launches : 0; }

rnn_status rnn_ssm_conv(rnn_ssm_t pl, const rnn_ssm_conv_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0 || (a->seq_length == 0 && (!a->final_state || pl->K == 1))) return RNN_OK;
    const bool steps = a->seq_length > 0;
    const Named views[] = {{&a->X, "X", steps}, {&a->Y, "Y", steps}};
    rs = check_views(pl, views, 2);
    if (rs != RNN_OK) return rs;
    NEED(a->W, "W");
    rs = check_arrays({{a->W, "W"}, {a->bias, "bias"}, {a->sequence_lens, "sequence_lens"}});
    const View Y = dense(a->Y, pl, a->seq_length, a->batch_size, pl->D);
    if (rs == RNN_OK) rs = check_outputs(a->seq_length, a->batch_size, {{Y, pl->D, "Y"}});
    if (rs == RNN_OK) rs = check_state(pl, a->initial_state, "initial_state");
    if (rs == RNN_OK) rs = check_state(pl, a->final_state, "final_state");
    // the same memory needs no copy: a row's first run alone reads it, and its threads have read a value before they write it
    const size_t states = element(pl->io) * (size_t)(a->batch_size * (pl->K - 1) * pl->D);
    if (rs == RNN_OK) rs = check_in_place(a->initial_state, a->final_state, states, "initial_state and final_state");
    if (rs == RNN_OK) rs = check_not_input(pl, a->seq_length, a->Y, "Y", a->X, "X");
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ConvParams p = conv_params(pl, a->seq_length, a->batch_size);
    p.X = dense(a->X, pl, p.S, p.N, p.D);
    p.Y = Y;
    p.W = a->W;
    p.bias = a->bias;
    p.lens = a->sequence_lens;
    p.h0 = a->initial_state;
    p.hT = a->final_state;
    cudaError_t e = launch_ssm_conv(p, (cudaStream_t)a->stream, &pl->launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "convolution launch");
}

rnn_status rnn_ssm_conv_grad(rnn_ssm_t pl, const rnn_ssm_conv_grad_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    const bool steps = a->seq_length > 0 && a->batch_size > 0;
    const Named views[] = {{&a->X, "X", steps}, {&a->dY, "dY", steps}, {&a->dX, "dX", false}};
    rs = check_views(pl, views, 3);
    if (rs != RNN_OK) return rs;
    NEED(a->W, "W");
    rs = check_arrays({{a->W, "W"}, {a->bias, "bias"}, {a->sequence_lens, "sequence_lens"}, {a->dW, "dW"}, {a->dbias, "dbias"}});
    if (rs == RNN_OK) rs = check_state(pl, a->initial_state, "initial_state");
    if (rs == RNN_OK) rs = check_state(pl, a->d_final_state, "d_final_state");
    if (rs == RNN_OK) rs = check_state(pl, a->d_initial_state, "d_initial_state");
    const View dX = dense(a->dX, pl, a->seq_length, a->batch_size, pl->D);
    if (rs == RNN_OK) rs = check_outputs(a->seq_length, a->batch_size, {{dX, pl->D, "dX"}});
    const size_t states = element(pl->io) * (size_t)(a->batch_size * (pl->K - 1) * pl->D);
    if (rs == RNN_OK) rs = check_in_place(a->d_final_state, a->d_initial_state, states, "d_final_state and d_initial_state");
    if (rs == RNN_OK) rs = check_not_input(pl, a->seq_length, a->dX, "dX", a->X, "X");
    if (rs == RNN_OK) rs = check_not_input(pl, a->seq_length, a->dX, "dX", a->dY, "dY");
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ConvGradParams p{};
    p.f = conv_params(pl, a->seq_length, a->batch_size);
    p.f.X = dense(a->X, pl, p.f.S, p.f.N, p.f.D);
    p.f.W = a->W;
    p.f.bias = a->bias;
    p.f.lens = a->sequence_lens;
    p.f.h0 = a->initial_state;
    p.dY = dense(a->dY, pl, p.f.S, p.f.N, p.f.D);
    p.dX = dX;
    p.dhT = a->d_final_state;
    p.dh0 = a->d_initial_state;
    p.dW = a->dW;
    p.dbias = a->dbias;
    cudaStream_t st = (cudaStream_t)a->stream;
    ssm_conv_grad_plan(p);
    const size_t bytes = a->dW || a->dbias ? sizeof(float) * (size_t)p.parts * (size_t)(p.f.D * (p.f.K + 1)) : 0;
    // In place, the blocks of a row's first steps would write what those of its last
    // steps still read: they read a copy, on a 16-byte boundary as the slopes may be.
    const size_t copy = p.dhT && p.dhT == p.dh0 ? states : 0, at = (bytes + 15) / 16 * 16;
    char* scratch = nullptr;
    rs = claim_scratch(pl, copy ? at + copy : bytes, st, &scratch);
    if (rs != RNN_OK) return rs;
    p.part = bytes ? (float*)scratch : nullptr;
    cudaError_t e = cudaSuccess;
    if (copy) {
        e = cudaMemcpyAsync(scratch + at, p.dhT, copy, cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return cuda_fail(e, "copying d_final_state");
        p.dhT = scratch + at;
    }
    e = launch_ssm_conv_grad(p, st, &pl->launches);
    if (e != cudaSuccess) return cuda_fail(e, "convolution gradient launch");
    return release_scratch(pl, bytes + copy, st);
}

rnn_status rnn_ssm_conv_step(rnn_ssm_t pl, const rnn_ssm_conv_step_args* a)
{
    rnn_status rs = check_sizes(pl, a, 1, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0) return RNN_OK;
    const Named views[] = {{&a->X, "X", true}, {&a->Y, "Y", true}};
    rs = check_views(pl, views, 2);
    if (rs != RNN_OK) return rs;
    NEED(a->W, "W");
    if (pl->K > 1) {
        NEED(a->state, "state");
        NEED(a->state_out, "state_out");
    }
    rs = check_slots(a->slots, a->n_slots);
    if (rs == RNN_OK) rs = check_arrays({{a->W, "W"}, {a->bias, "bias"}, {a->slots, "slots"}});
    if (rs == RNN_OK) rs = check_state(pl, a->state, "state");
    if (rs == RNN_OK) rs = check_state(pl, a->state_out, "state_out");
    const size_t states = element(pl->io) * (size_t)((a->slots ? a->n_slots : a->batch_size) * (pl->K - 1) * pl->D);
    if (rs == RNN_OK) rs = check_in_place(a->state, a->state_out, states, "state and state_out");
    const View Y = dense_row(a->Y, pl->D);
    if (rs == RNN_OK) rs = check_outputs(1, a->batch_size, {{Y, pl->D, "Y"}});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ConvStepParams p{};
    p.N = a->batch_size;
    p.D = pl->D;
    p.slots_n = a->n_slots;
    p.K = pl->K;
    p.io = pl->io;
    p.silu = pl->silu;
    p.X = dense_row(a->X, p.D);
    p.Y = Y;
    p.W = a->W;
    p.bias = a->bias;
    p.state = a->state;
    p.state_out = a->state_out;
    p.slots = a->slots;
    p.status = pl->status;
    cudaError_t e = launch_ssm_conv_step(p, (cudaStream_t)a->stream, &pl->launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "convolution step launch");
}

int64_t rnn_ssm_saved_size(rnn_ssm_t pl, int64_t S, int64_t N)
{
    if (!pl || S < 0 || N < 0) return -1;
    return ssm_saved_floats(S, N, pl->D, pl->M);
}

rnn_status rnn_ssm_scan(rnn_ssm_t pl, const rnn_ssm_scan_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0 || (a->seq_length == 0 && !a->Y_h)) return RNN_OK;
    const bool steps = a->seq_length > 0;
    const Named views[] = {{&a->X, "X", steps}, {&a->dt, "dt", steps}, {&a->B, "B", steps},
                           {&a->C, "C", steps}, {&a->Y, "Y", steps},   {&a->Z, "Z", false}};
    rs = check_views(pl, views, 6);
    if (rs != RNN_OK) return rs;
    NEED(a->A, "A");
    rs = check_arrays({{a->A, "A"}, {a->Dskip, "Dskip"}, {a->dt_bias, "dt_bias"}, {a->sequence_lens, "sequence_lens"},
                       {a->initial_h, "initial_h"}, {a->Y_h, "Y_h"}, {a->saved, "saved"}});
    const View Y = dense(a->Y, pl, a->seq_length, a->batch_size, pl->D);
    if (rs == RNN_OK) rs = check_outputs(a->seq_length, a->batch_size, {{Y, pl->D, "Y"}});
    const size_t states = sizeof(float) * (size_t)(a->batch_size * pl->D * pl->M);
    if (rs == RNN_OK) rs = check_in_place(a->initial_h, a->Y_h, states, "initial_h and Y_h");
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ScanParams p = scan_params(pl, a->seq_length, a->batch_size);
    const int64_t gm = (int64_t)p.G * p.M;
    p.X = dense(a->X, pl, p.S, p.N, p.D);
    p.dt = dense(a->dt, pl, p.S, p.N, p.D);
    p.B = dense(a->B, pl, p.S, p.N, gm);
    p.C = dense(a->C, pl, p.S, p.N, gm);
    p.Z = dense(a->Z, pl, p.S, p.N, p.D);
    p.Y = Y;
    p.A = a->A;
    p.Dskip = a->Dskip;
    p.dt_bias = a->dt_bias;
    p.lens = a->sequence_lens;
    p.h0 = a->initial_h;
    p.hT = a->Y_h;
    p.saved = a->saved;
    cudaStream_t st = (cudaStream_t)a->stream;
    size_t bytes = 0;
    cudaError_t e = cudaSuccess;
    ssm_scan_plan(p, &bytes);
    // In place, the last chunk's block would write states that other chunks' blocks
    // still read: they read a copy.  (Unsplit, the thread that writes a state has read it.)
    const size_t copy = p.split.chunks > 1 && p.h0 && p.h0 == p.hT ? states : 0;
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes + copy, st, &scratch);
    if (rs != RNN_OK) return rs;
    p.scratch = (float*)scratch;
    if (copy) {
        e = cudaMemcpyAsync(scratch + bytes, p.h0, copy, cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return cuda_fail(e, "copying initial_h");
        p.h0 = (const float*)(scratch + bytes);
    }
    e = launch_ssm_scan(p, st, &pl->launches);
    if (e != cudaSuccess) return cuda_fail(e, "scan launch");
    return release_scratch(pl, bytes + copy, st);
}

rnn_status rnn_ssm_scan_grad(rnn_ssm_t pl, const rnn_ssm_scan_grad_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    const bool steps = a->seq_length > 0 && a->batch_size > 0;
    const Named views[] = {{&a->X, "X", steps}, {&a->dt, "dt", steps},  {&a->B, "B", steps},    {&a->C, "C", steps},
                           {&a->dY, "dY", steps}, {&a->Z, "Z", false},  {&a->dX, "dX", false},  {&a->ddt, "ddt", false},
                           {&a->dB, "dB", false}, {&a->dC, "dC", false}, {&a->dZ, "dZ", false}};
    rs = check_views(pl, views, 11);
    if (rs != RNN_OK) return rs;
    NEED(a->A, "A");
    if (steps) NEED(a->saved, "saved");
    if (a->dZ.data && !a->Z.data && steps) return fail(RNN_ERR_INVALID_ARGUMENT, "dZ without Z");
    rs = check_arrays({{a->A, "A"}, {a->Dskip, "Dskip"}, {a->dt_bias, "dt_bias"}, {a->sequence_lens, "sequence_lens"},
                       {a->initial_h, "initial_h"}, {a->saved, "saved"}, {a->dY_h, "dY_h"}, {a->dA, "dA"}, {a->dDskip, "dDskip"},
                       {a->ddt_bias, "ddt_bias"}, {a->d_initial_h, "d_initial_h"}});
    if (rs != RNN_OK) return rs;
    const int64_t S = a->seq_length, N = a->batch_size, D = pl->D, gm = (int64_t)pl->G * pl->M;
    ScanGradParams p{};
    p.dX = dense(a->dX, pl, S, N, D);
    p.ddt = dense(a->ddt, pl, S, N, D);
    p.dB = dense(a->dB, pl, S, N, gm);
    p.dC = dense(a->dC, pl, S, N, gm);
    p.dZ = dense(a->dZ, pl, S, N, D);
    rs = check_outputs(S, N, {{p.dX, D, "dX"}, {p.ddt, D, "ddt"}, {p.dB, gm, "dB"}, {p.dC, gm, "dC"}, {p.dZ, D, "dZ"}});
    const size_t states = sizeof(float) * (size_t)(N * D * pl->M);
    if (rs == RNN_OK) rs = check_in_place(a->dY_h, a->d_initial_h, states, "dY_h and d_initial_h");
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    p.f = scan_params(pl, S, N);
    p.f.X = dense(a->X, pl, S, N, D);
    p.f.dt = dense(a->dt, pl, S, N, D);
    p.f.B = dense(a->B, pl, S, N, gm);
    p.f.C = dense(a->C, pl, S, N, gm);
    p.f.Z = dense(a->Z, pl, S, N, D);
    p.f.A = a->A;
    p.f.Dskip = a->Dskip;
    p.f.dt_bias = a->dt_bias;
    p.f.lens = a->sequence_lens;
    p.f.h0 = a->initial_h;
    p.f.saved = const_cast<float*>(a->saved);
    p.dY = dense(a->dY, pl, S, N, D);
    p.dhT = a->dY_h;
    p.dA = a->dA;
    p.dDskip = a->dDskip;
    p.ddt_bias = a->ddt_bias;
    p.dh0 = a->d_initial_h;
    cudaStream_t st = (cudaStream_t)a->stream;
    size_t bytes = 0;
    cudaError_t e = cudaSuccess;
    ssm_scan_grad_plan(p, &bytes);
    // in place, as in the forward run: the first chunk's block would write what the others read
    const size_t copy = p.f.split.chunks > 1 && p.dhT && p.dhT == p.dh0 ? states : 0;
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes + copy, st, &scratch);
    if (rs != RNN_OK) return rs;
    p.f.scratch = (float*)scratch;
    if (copy) {
        e = cudaMemcpyAsync(scratch + bytes, p.dhT, copy, cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return cuda_fail(e, "copying dY_h");
        p.dhT = (const float*)(scratch + bytes);
    }
    e = launch_ssm_scan_grad(p, st, &pl->launches);
    if (e != cudaSuccess) return cuda_fail(e, "scan gradient launch");
    return release_scratch(pl, bytes + copy, st);
}

rnn_status rnn_ssm_scan_step(rnn_ssm_t pl, const rnn_ssm_scan_step_args* a)
{
    rnn_status rs = check_sizes(pl, a, 1, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0) return RNN_OK;
    const Named views[] = {{&a->X, "X", true}, {&a->dt, "dt", true}, {&a->B, "B", true},
                           {&a->C, "C", true}, {&a->Y, "Y", true},   {&a->Z, "Z", false}};
    rs = check_views(pl, views, 6);
    if (rs != RNN_OK) return rs;
    NEED(a->A, "A");
    NEED(a->H, "H");
    NEED(a->H_out, "H_out");
    rs = check_slots(a->slots, a->n_slots);
    if (rs == RNN_OK)
        rs = check_arrays({{a->A, "A"}, {a->Dskip, "Dskip"}, {a->dt_bias, "dt_bias"}, {a->H, "H"}, {a->H_out, "H_out"}, {a->slots, "slots"}});
    const size_t states = sizeof(float) * (size_t)((a->slots ? a->n_slots : a->batch_size) * pl->D * pl->M);
    if (rs == RNN_OK) rs = check_in_place(a->H, a->H_out, states, "H and H_out");
    const View Y = dense_row(a->Y, pl->D);
    if (rs == RNN_OK) rs = check_outputs(1, a->batch_size, {{Y, pl->D, "Y"}});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ScanStepParams p{};
    p.N = a->batch_size;
    p.D = pl->D;
    p.slots_n = a->n_slots;
    p.M = pl->M;
    p.G = pl->G;
    p.io = pl->io;
    p.softplus = pl->softplus;
    p.sms = pl->sms;
    const int64_t gm = (int64_t)p.G * p.M;
    p.X = dense_row(a->X, p.D);
    p.dt = dense_row(a->dt, p.D);
    p.B = dense_row(a->B, gm);
    p.C = dense_row(a->C, gm);
    p.Z = dense_row(a->Z, p.D);
    p.Y = Y;
    p.A = a->A;
    p.Dskip = a->Dskip;
    p.dt_bias = a->dt_bias;
    p.H = a->H;
    p.H_out = a->H_out;
    p.slots = a->slots;
    p.status = pl->status;
    cudaError_t e = launch_ssm_scan_step(p, (cudaStream_t)a->stream, &pl->launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "scan step launch");
}

rnn_status rnn_scores(const rnn_scores_args* a)
{
    NEED(a, "args");
    rnn_status rs = check_scores(a->rows, a->vocab, a->row_stride, a->io, a->top, a->logits);
    if (rs != RNN_OK) return rs;
    if (a->rows == 0) return RNN_OK;
    rs = check_arrays({{a->ids, "ids"}, {a->logp, "logp"}, {a->entropy, "entropy"}, {a->lse, "lse"}, {a->top_ids, "top_ids"},
                       {a->top_logp, "top_logp"}});
    if (rs != RNN_OK) return rs;
    if (a->logp && !a->ids) return fail(RNN_ERR_INVALID_ARGUMENT, "logp without ids");
    if (a->top > 0 && !a->top_ids && !a->top_logp) return fail(RNN_ERR_INVALID_ARGUMENT, "top without top_ids and top_logp");
    ScoreParams p{};
    p.rows = a->rows;
    p.V = a->vocab;
    p.stride = logits_stride(a->row_stride, a->vocab);
    p.io = (int)(a->io & ~RNN_SCORES_LSE_PAIR);
    p.top = (int)a->top;
    p.x = a->logits;
    p.ids = a->ids;
    p.logp = a->logp;
    p.entropy = a->entropy;
    p.lse = a->lse;
    p.lse_rest = a->io & RNN_SCORES_LSE_PAIR && a->lse ? a->lse + a->rows : nullptr;
    p.top_ids = a->top_ids;
    p.top_logp = a->top_logp;
    int launches = 0;
    cudaError_t e = launch_scores(p, (cudaStream_t)a->stream, &launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "scores launch");
}

rnn_status rnn_scores_grad(const rnn_scores_grad_args* a)
{
    NEED(a, "args");
    rnn_status rs = check_scores(a->rows, a->vocab, a->row_stride, a->io, a->top, a->logits);
    if (rs != RNN_OK) return rs;
    if (a->d_row_stride != 0 && a->d_row_stride < a->vocab)
        return fail(RNN_ERR_INVALID_ARGUMENT, "d_row_stride %lld is below vocab", (long long)a->d_row_stride);
    if (a->rows == 0) return RNN_OK;
    NEED(a->lse, "lse");
    NEED(a->dlogits, "dlogits");
    if ((uintptr_t)a->dlogits % element((int)(a->io & ~RNN_SCORES_LSE_PAIR)))
        return fail(RNN_ERR_INVALID_ARGUMENT, "dlogits are not aligned to their elements");
    rs = check_arrays({{a->ids, "ids"}, {a->lse, "lse"}, {a->entropy, "entropy"}, {a->d_logp, "d_logp"}, {a->d_entropy, "d_entropy"},
                       {a->top_ids, "top_ids"}, {a->d_top, "d_top"}});
    if (rs != RNN_OK) return rs;
    if (a->d_logp && !a->ids) return fail(RNN_ERR_INVALID_ARGUMENT, "d_logp without ids");
    if (a->d_entropy && !a->entropy) return fail(RNN_ERR_INVALID_ARGUMENT, "d_entropy without entropy");
    if (a->d_top && (!a->top_ids || a->top == 0)) return fail(RNN_ERR_INVALID_ARGUMENT, "d_top without top_ids");
    ScoreGradParams p{};
    p.rows = a->rows;
    p.V = a->vocab;
    p.stride = logits_stride(a->row_stride, a->vocab);
    p.d_stride = a->d_row_stride ? a->d_row_stride : a->vocab;
    p.io = (int)(a->io & ~RNN_SCORES_LSE_PAIR);
    p.top = a->d_top ? (int)a->top : 0;
    p.x = a->logits;
    p.ids = a->ids;
    p.lse = a->lse;
    p.lse_rest = a->io & RNN_SCORES_LSE_PAIR && a->lse ? a->lse + a->rows : nullptr;
    p.entropy = a->entropy;
    p.d_logp = a->d_logp;
    p.d_entropy = a->d_entropy;
    p.top_ids = a->top_ids;
    p.d_top = a->d_top;
    p.dx = a->dlogits;
    if (p.dx == p.x && p.d_stride != p.stride)
        return fail(RNN_ERR_INVALID_ARGUMENT, "in-place gradients need the logits' row stride");
    int launches = 0;
    cudaError_t e = launch_scores_grad(p, (cudaStream_t)a->stream, &launches);
    return e == cudaSuccess ? RNN_OK : cuda_fail(e, "scores gradient launch");
}

}  // extern "C"
