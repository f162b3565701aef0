// C entry points of the gated delta rule: checks of arguments and scratch.
// See include/onnx_recurrent.h for the contract.
#include <cmath>

#include "delta_internal.h"
#include "plan.h"

using namespace rnngb;

struct rnn_delta : PlanMemory {
    int64_t H = 0, HK = 0;
    int DK = 0, DV = 0, layout = 0, io = RNN_IO_F32;
    float scale = 0.f;
};

namespace {

View dense(const rnn_view& v, const rnn_delta* pl, int64_t S, int64_t N, int64_t inner)
{
    View r{v.data, v.seq_stride, v.batch_stride};
    if (r.ss == 0 && r.bs == 0) {
        r.ss = pl->layout == 0 ? N * inner : inner;
        r.bs = pl->layout == 0 ? inner : S * inner;
    }
    return r;
}

View dense_row(const rnn_view& v, int64_t inner) { return View{v.data, 0, v.batch_stride ? v.batch_stride : inner}; }

// Whether the images and states of all chunks and heads, at most 2^20 bytes each and a tile of 128 values, are counted in 64 bits.
bool countable(const rnn_delta* pl, int64_t S, int64_t N)
{
    return S <= 0x7fffff00LL && N <= 0x7fffff00LL && N * pl->H <= 0x7fffff00LL &&
           (S + 63) / 64 <= ((int64_t)1 << 42) / ((pl->DV + 127) / 128) / (N * pl->H > 0 ? N * pl->H : 1);
}

rnn_status check_sizes(rnn_delta* pl, const void* args, int64_t S, int64_t N)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    pl->launches = 0;
    NEED(args, "args");
    if (S < 0 || N < 0)
        return fail(RNN_ERR_INVALID_ARGUMENT, "seq_length %lld, batch_size %lld", (long long)S, (long long)N);
    // heads of all rows are counted over two dimensions of a grid
    if (!countable(pl, S, N)) return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    return RNN_OK;
}

struct Named {
    const rnn_view* v;
    const char* name;
    bool required;
    size_t elem;
};
template <int K>
rnn_status check_all(const Named (&views)[K])
{
    for (const Named& w : views) {
        if (!w.v->data) {
            if (w.required) return fail(RNN_ERR_INVALID_ARGUMENT, "%s is NULL", w.name);
            continue;
        }
        rnn_status rs = check_view(*w.v, w.elem, w.name);
        if (rs != RNN_OK) return rs;
    }
    return RNN_OK;
}

// Steps and rows of an output apart from one another: whichever stride is the larger steps over
// all that the other one reaches.
template <int K>
rnn_status check_apart(int64_t S, int64_t N, const OutView (&views)[K])
{
    rnn_status rs = check_outputs(S, N, views);
    if (rs != RNN_OK) return rs;
    for (const OutView& o : views) {
        if (!o.v.data || S <= 1 || N <= 1) continue;
        const bool rows_far = o.v.bs > o.v.ss;
        const __int128 far = rows_far ? o.v.bs : o.v.ss, near = rows_far ? o.v.ss : o.v.bs, count = rows_far ? S : N;
        if (far < near * (count - 1) + o.inner)
            return fail(RNN_ERR_INVALID_ARGUMENT, "%s: its steps or rows share memory", o.name);
    }
    return RNN_OK;
}

// A call's array: S steps of N rows of `inner` elements (a state or another dense array: one of each).
struct Laid {
    const void* data;
    int64_t ss, bs, S, N, inner;
    int64_t elem;
    const char* name;
};
Laid laid(const View& v, int64_t S, int64_t N, int64_t inner, size_t elem, const char* name)
{
    return Laid{v.data, v.ss, v.bs, S, N, inner, (int64_t)elem, name};
}
Laid laid(const void* p, int64_t count, const char* name) { return Laid{p, 0, 0, 1, 1, count, 4, name}; }

// Whether two arrays are certain to share memory.  Arrays without gaps are told apart from any other one, and others from those of
// the same strides (parts of wider rows, side by side); of the rest nothing is said.
using wide = __int128;
struct Nested {             // an array's strides and counts, the wider stride first, in bytes
    wide far, near, inner;
    int64_t fars, nears;
};
Nested nested(const Laid& x)
{
    const bool rows_far = x.bs > x.ss;
    return Nested{(wide)(rows_far ? x.bs : x.ss) * x.elem, (wide)(rows_far ? x.ss : x.bs) * x.elem, (wide)x.inner * x.elem,
                  rows_far ? x.N : x.S, rows_far ? x.S : x.N};
}
// Whether any of off + i stride, lo <= i <= hi, that lies between -left and right is what is looked for.
template <typename F>
bool any_between(wide off, wide stride, int64_t lo, int64_t hi, wide left, wide right, F&& found)
{
    if (stride == 0) lo = hi = 0;
    wide i = stride == 0 ? 0 : (-left - off) / stride - 1;
    if (i < lo) i = lo;
    for (int tries = 0; tries < 8 && i <= hi && off + i * stride < right; ++i)
        if (off + i * stride > -left) {
            ++tries;
            if (found(off + i * stride)) return true;
        }
    return false;
}
// Whether a block of `len` bytes meets items of b that begin `off` from it, or (both) that many strides before.
bool block_meets(wide off, wide len, const Nested& b, bool both)
{
    return any_between(off, b.far, both ? 1 - b.fars : 0, b.fars - 1, b.near * (b.nears - 1) + b.inner, len + (both ? b.near * (b.nears - 1) : 0),
                       [&](wide o) { return any_between(o, b.near, both ? 1 - b.nears : 0, b.nears - 1, b.inner, len, [](wide) { return true; }); });
}
bool share(const Laid& a, const Laid& b)
{
    const Nested na = nested(a), nb = nested(b);
    auto span = [](const Nested& x) { return x.far * (x.fars - 1) + x.near * (x.nears - 1) + x.inner; };
    const wide off = (wide)(uintptr_t)b.data - (wide)(uintptr_t)a.data;
    if (off >= span(na) || -off >= span(nb)) return false;
    auto gapless = [](const Nested& x) {
        return (x.nears == 1 || x.near <= x.inner) && (x.fars == 1 || x.far <= x.near * (x.nears - 1) + x.inner);
    };
    if (gapless(na)) return block_meets(off, span(na), nb, false);
    if (gapless(nb)) return block_meets(-off, span(nb), na, false);
    if (a.S != b.S || a.N != b.N || (a.S > 1 && a.ss * a.elem != b.ss * b.elem) || (a.N > 1 && a.bs * a.elem != b.bs * b.elem)) return false;
    return block_meets(off, na.inner, nb, true);
}

// Outputs lie on no input and on no other output.  The first of either is a state and where it goes, which may be the same
// memory (check_in_place).
template <int I, int O>
rnn_status check_shared(const Laid (&in)[I], const Laid (&out)[O])
{
    // what nearly all calls come to: ranges that do not meet (an empty array's is empty)
    struct Range {
        uintptr_t lo, hi;
    };
    auto range = [](const Laid& x) {
        if (!x.data || x.S < 1 || x.N < 1 || x.inner < 1) return Range{0, 0};
        int64_t rows, steps, bytes;
        uintptr_t end;
        const bool past = __builtin_mul_overflow(x.bs, x.N - 1, &rows) || __builtin_mul_overflow(x.ss, x.S - 1, &steps) ||
                          __builtin_add_overflow(rows, steps, &bytes) || __builtin_add_overflow(bytes, x.inner, &bytes) ||
                          __builtin_mul_overflow(bytes, x.elem, &bytes) || __builtin_add_overflow((uintptr_t)x.data, (uintptr_t)bytes, &end);
        return Range{(uintptr_t)x.data, past ? UINTPTR_MAX : end};
    };
    auto meet = [](const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; };
    Range ins[I], outs[O];
    for (int i = 0; i < I; ++i) ins[i] = range(in[i]);
    for (int o = 0; o < O; ++o) {
        outs[o] = range(out[o]);
        for (int i = o == 0; i < I; ++i)
            if (meet(outs[o], ins[i]) && share(out[o], in[i]))
                return fail(RNN_ERR_INVALID_ARGUMENT, "%s overlaps %s", out[o].name, in[i].name);
        for (int i = 0; i < o; ++i)
            if (meet(outs[o], outs[i]) && share(out[o], out[i]))
                return fail(RNN_ERR_INVALID_ARGUMENT, "%s overlaps %s", out[o].name, out[i].name);
    }
    return RNN_OK;
}

DeltaParams params(const rnn_delta* pl, int64_t S, int64_t N)
{
    DeltaParams p{};
    p.S = S;
    p.N = N;
    p.H = (int)pl->H;
    p.HK = (int)pl->HK;
    p.DK = pl->DK;
    p.DV = pl->DV;
    p.io = pl->io;
    p.scale = pl->scale;
    return p;
}

// The parts of what a run saves.
void place(DeltaParams& p, void* saved)
{
    p.keys = static_cast<unsigned char*>(saved);
    p.mats = p.keys + delta_keys_bytes(p.S, p.N, p.HK, p.DK, p.io);
    p.kept = p.mats + delta_mats_bytes(p.S, p.N, p.H);
}

rnn_status check_saved(const void* saved)
{
    if ((uintptr_t)saved % 16) return fail(RNN_ERR_INVALID_ARGUMENT, "saved is not aligned to 16 bytes");
    return RNN_OK;
}

}  // namespace

extern "C" {

rnn_status rnn_delta_create(rnn_delta_t* out, int64_t heads, int64_t key_heads, int64_t key_size, int64_t value_size,
                            int layout, float scale)
{
    NEED(out, "out");
    *out = nullptr;
    if (key_heads <= 0 || heads <= 0 || heads % key_heads)
        return fail(RNN_ERR_INVALID_ARGUMENT, "key_heads %lld does not divide heads %lld", (long long)key_heads, (long long)heads);
    if (key_size < 1 || key_size > kDeltaMaxKey)
        return fail(RNN_ERR_INVALID_ARGUMENT, "key_size %lld outside [1, %d]", (long long)key_size, kDeltaMaxKey);
    if (value_size < 1 || value_size > kDeltaMaxValue)
        return fail(RNN_ERR_INVALID_ARGUMENT, "value_size %lld outside [1, %d]", (long long)value_size, kDeltaMaxValue);
    if (heads > 0x7fffff00LL / value_size || key_heads > 0x7fffff00LL / key_size)
        return fail(RNN_ERR_INVALID_ARGUMENT, "heads times their size is 2^31 or more");
    if (layout & ~1) return fail(RNN_ERR_INVALID_ARGUMENT, "layout is 0 or 1");
    if (!std::isfinite(scale)) return fail(RNN_ERR_INVALID_ARGUMENT, "scale is not finite");
    rnn_delta* pl = new (std::nothrow) rnn_delta;
    if (!pl) return fail(RNN_ERR_OOM, "host allocation failed");
    pl->H = heads;
    pl->HK = key_heads;
    pl->DK = (int)key_size;
    pl->DV = (int)value_size;
    pl->layout = layout;
    pl->scale = scale;
    *out = pl;
    return RNN_OK;
}

void rnn_delta_destroy(rnn_delta_t pl)
{
    if (!pl) return;
    free_plan_memory(pl);
    delete pl;
}

rnn_status rnn_delta_set_io_type(rnn_delta_t pl, int io)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    if (io != RNN_IO_F32 && io != RNN_IO_F16 && io != RNN_IO_BF16)
        return fail(RNN_ERR_INVALID_ARGUMENT, "unknown io type %d", io);
    pl->io = io;
    return RNN_OK;
}

rnn_status rnn_delta_sync(rnn_delta_t pl)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    return read_status(pl, "a sequence length outside [0, seq_length] or a slot outside its range");
}

int rnn_delta_last_launch_count(rnn_delta_t pl) { return pl ? pl->launches : 0; }

int64_t rnn_delta_saved_size(rnn_delta_t pl, int64_t S, int64_t N)
{
    if (!pl || S < 0 || N < 0 || !countable(pl, S, N)) return -1;
    return delta_saved_floats(S, N, pl->H, pl->HK, pl->DK, pl->DV, pl->io);
}

rnn_status rnn_delta_rule(rnn_delta_t pl, const rnn_delta_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0 || (a->seq_length == 0 && !a->final_state)) return RNN_OK;
    const bool steps = a->seq_length > 0;
    const size_t e = element(pl->io);
    rs = check_all({{&a->Q, "Q", steps, e}, {&a->K, "K", steps, e}, {&a->V, "V", steps, e}, {&a->g, "g", steps, 4},
                    {&a->beta, "beta", steps, 4}, {&a->Y, "Y", steps, e}});
    if (rs == RNN_OK)
        rs = check_arrays({{a->sequence_lens, "sequence_lens"}, {a->initial_state, "initial_state"}, {a->final_state, "final_state"}});
    if (rs == RNN_OK) rs = check_saved(a->saved);
    const int64_t S = a->seq_length, N = a->batch_size, dk = pl->HK * pl->DK, dv = pl->H * pl->DV;
    const View Y = dense(a->Y, pl, S, N, dv);
    if (rs == RNN_OK) rs = check_apart(S, N, {{Y, dv, "Y"}});
    const size_t states = sizeof(float) * (size_t)(N * dv * pl->DK);
    // the same memory: the block that writes a part of a state has read it
    if (rs == RNN_OK) rs = check_in_place(a->initial_state, a->final_state, states, "initial_state and final_state");
    if (rs != RNN_OK) return rs;
    DeltaParams p = params(pl, S, N);
    p.Q = dense(a->Q, pl, S, N, dk);
    p.K = dense(a->K, pl, S, N, dk);
    p.V = dense(a->V, pl, S, N, dv);
    p.g = dense(a->g, pl, S, N, pl->H);
    p.beta = dense(a->beta, pl, S, N, pl->H);
    p.Y = Y;
    const int64_t saved = a->saved ? delta_saved_floats(S, N, p.H, p.HK, p.DK, p.DV, p.io) : 0;
    rs = check_shared({laid(a->initial_state, N * dv * pl->DK, "initial_state"), laid(p.Q, S, N, dk, e, "Q"), laid(p.K, S, N, dk, e, "K"),
                       laid(p.V, S, N, dv, e, "V"), laid(p.g, S, N, pl->H, 4, "g"), laid(p.beta, S, N, pl->H, 4, "beta"),
                       laid(a->sequence_lens, N, "sequence_lens")},
                      {laid(a->final_state, N * dv * pl->DK, "final_state"), laid(Y, S, N, dv, e, "Y"), laid(a->saved, saved, "saved")});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    p.sms = pl->sms;
    p.status = pl->status;
    p.lens = a->sequence_lens;
    p.h0 = a->initial_state;
    p.hT = a->final_state;
    cudaStream_t st = (cudaStream_t)a->stream;
    delta_split(p);
    const size_t images = a->saved ? 0 : (size_t)(delta_keys_bytes(S, N, p.HK, p.DK, p.io) + delta_mats_bytes(S, N, p.H));
    const size_t bytes = images + sizeof(float) * (size_t)delta_split_floats(p);
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes, st, &scratch);
    if (rs != RNN_OK) return rs;
    place(p, a->saved ? (void*)a->saved : scratch);
    if (!a->saved) p.kept = nullptr;
    p.over = (float*)(scratch + images);
    p.starts = p.over + N * p.H * (p.cuts - 1) * (int64_t)p.DK * (p.DV + p.DK);
    cudaError_t err = launch_delta(p, st, &pl->launches);
    if (err != cudaSuccess) return cuda_fail(err, "delta rule launch");
    return release_scratch(pl, bytes, st);
}

rnn_status rnn_delta_rule_grad(rnn_delta_t pl, const rnn_delta_grad_args* a)
{
    rnn_status rs = check_sizes(pl, a, a ? a->seq_length : 0, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0) return RNN_OK;
    const bool steps = a->seq_length > 0;
    const size_t e = element(pl->io);
    rs = check_all({{&a->dY, "dY", steps, e}, {&a->Q, "Q", steps, e}, {&a->K, "K", steps, e}, {&a->V, "V", steps, e},
                    {&a->g, "g", steps, 4}, {&a->beta, "beta", steps, 4}, {&a->dQ, "dQ", false, e}, {&a->dK, "dK", false, e},
                    {&a->dV, "dV", false, e}, {&a->dg, "dg", false, 4}, {&a->dbeta, "dbeta", false, 4}});
    if (rs != RNN_OK) return rs;
    if (steps) NEED(a->saved, "saved");
    rs = check_saved(a->saved);
    if (rs == RNN_OK) rs = check_arrays({{a->sequence_lens, "sequence_lens"}, {a->d_final_state, "d_final_state"}, {a->d_initial_state, "d_initial_state"}});
    if (rs != RNN_OK) return rs;
    const int64_t S = a->seq_length, N = a->batch_size, H = pl->H, dk = pl->HK * pl->DK, dv = H * pl->DV;
    DeltaGradParams q{};
    q.dQ = dense(a->dQ, pl, S, N, dk);
    q.dK = dense(a->dK, pl, S, N, dk);
    q.dV = dense(a->dV, pl, S, N, dv);
    q.dg = dense(a->dg, pl, S, N, H);
    q.dbeta = dense(a->dbeta, pl, S, N, H);
    rs = check_apart(S, N, {{q.dQ, dk, "dQ"}, {q.dK, dk, "dK"}, {q.dV, dv, "dV"}, {q.dg, H, "dg"}, {q.dbeta, H, "dbeta"}});
    const size_t states = sizeof(float) * (size_t)(N * dv * pl->DK);
    if (rs == RNN_OK) rs = check_in_place(a->d_final_state, a->d_initial_state, states, "d_final_state and d_initial_state");
    if (rs != RNN_OK) return rs;
    q.f = params(pl, S, N);
    q.f.Q = dense(a->Q, pl, S, N, dk);
    q.f.K = dense(a->K, pl, S, N, dk);
    q.f.V = dense(a->V, pl, S, N, dv);
    q.f.g = dense(a->g, pl, S, N, H);
    q.f.beta = dense(a->beta, pl, S, N, H);
    q.f.lens = a->sequence_lens;
    place(q.f, const_cast<float*>(a->saved));
    q.dY = dense(a->dY, pl, S, N, dv);
    q.dhT = a->d_final_state;
    q.dh0 = a->d_initial_state;
    const int64_t saved = steps ? delta_saved_floats(S, N, H, pl->HK, pl->DK, pl->DV, pl->io) : 0;
    rs = check_shared({laid(a->d_final_state, N * dv * pl->DK, "d_final_state"), laid(q.dY, S, N, dv, e, "dY"), laid(q.f.Q, S, N, dk, e, "Q"),
                       laid(q.f.K, S, N, dk, e, "K"), laid(q.f.V, S, N, dv, e, "V"), laid(q.f.g, S, N, H, 4, "g"),
                       laid(q.f.beta, S, N, H, 4, "beta"), laid(a->sequence_lens, N, "sequence_lens"), laid(a->saved, saved, "saved")},
                      {laid(a->d_initial_state, N * dv * pl->DK, "d_initial_state"), laid(q.dQ, S, N, dk, e, "dQ"), laid(q.dK, S, N, dk, e, "dK"),
                       laid(q.dV, S, N, dv, e, "dV"), laid(q.dg, S, N, H, 4, "dg"), laid(q.dbeta, S, N, H, 4, "dbeta")});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    q.f.sms = pl->sms;
    q.f.status = pl->status;
    cudaStream_t st = (cudaStream_t)a->stream;
    const size_t bytes = (size_t)delta_slopes_bytes(S, N, H, pl->DK, pl->DV, pl->io);
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes, st, &scratch);
    if (rs != RNN_OK) return rs;
    q.slopes = (unsigned char*)scratch;
    cudaError_t err = launch_delta_grad(q, st, &pl->launches);
    if (err != cudaSuccess) return cuda_fail(err, "delta rule gradient launch");
    return release_scratch(pl, bytes, st);
}

rnn_status rnn_delta_step(rnn_delta_t pl, const rnn_delta_step_args* a)
{
    rnn_status rs = check_sizes(pl, a, 1, a ? a->batch_size : 0);
    if (rs != RNN_OK) return rs;
    if (a->batch_size == 0) return RNN_OK;
    const size_t e = element(pl->io);
    rs = check_all({{&a->Q, "Q", true, e}, {&a->K, "K", true, e}, {&a->V, "V", true, e}, {&a->g, "g", true, 4},
                    {&a->beta, "beta", true, 4}, {&a->Y, "Y", true, e}});
    if (rs != RNN_OK) return rs;
    NEED(a->state, "state");
    NEED(a->state_out, "state_out");
    rs = check_slots(a->slots, a->n_slots);
    if (rs == RNN_OK) rs = check_arrays({{a->state, "state"}, {a->state_out, "state_out"}, {a->slots, "slots"}});
    const int64_t dk = pl->HK * pl->DK, dv = pl->H * pl->DV;
    const size_t states = sizeof(float) * (size_t)((a->slots ? a->n_slots : a->batch_size) * dv * pl->DK);
    if (rs == RNN_OK) rs = check_in_place(a->state, a->state_out, states, "state and state_out");
    const View Y = dense_row(a->Y, dv);
    if (rs == RNN_OK) rs = check_outputs(1, a->batch_size, {{Y, dv, "Y"}});
    if (rs != RNN_OK) return rs;
    DeltaStepParams p{};
    p.N = a->batch_size;
    p.slots_n = a->n_slots;
    p.H = (int)pl->H;
    p.HK = (int)pl->HK;
    p.DK = pl->DK;
    p.DV = pl->DV;
    p.io = pl->io;
    p.scale = pl->scale;
    p.Q = dense_row(a->Q, dk);
    p.K = dense_row(a->K, dk);
    p.V = dense_row(a->V, dv);
    p.g = dense_row(a->g, p.H);
    p.beta = dense_row(a->beta, p.H);
    p.Y = Y;
    p.state = a->state;
    p.state_out = a->state_out;
    p.slots = a->slots;
    const int64_t N = a->batch_size, values = (a->slots ? a->n_slots : N) * dv * pl->DK;
    rs = check_shared({laid(a->state, values, "state"), laid(p.Q, 1, N, dk, e, "Q"), laid(p.K, 1, N, dk, e, "K"), laid(p.V, 1, N, dv, e, "V"),
                       laid(p.g, 1, N, p.H, 4, "g"), laid(p.beta, 1, N, p.H, 4, "beta"), laid(a->slots, N, "slots")},
                      {laid(a->state_out, values, "state_out"), laid(Y, 1, N, dv, e, "Y")});
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    p.sms = pl->sms;
    p.status = pl->status;
    cudaError_t err = launch_delta_step(p, (cudaStream_t)a->stream, &pl->launches);
    return err == cudaSuccess ? RNN_OK : cuda_fail(err, "delta rule step launch");
}

}  // extern "C"
