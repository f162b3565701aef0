// C entry points of beam search: checks of arguments and scratch.  See
// include/onnx_recurrent.h for the contract.
#include "norm_internal.h"
#include "plan.h"

using namespace rnngb;

struct rnn_beam : PlanMemory {
    int B = 0;
    int64_t end = -1;
};

namespace {

rnn_status check_plan(rnn_beam* pl, const void* args, int64_t items)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    pl->launches = 0;
    NEED(args, "args");
    if (items < 0) return fail(RNN_ERR_INVALID_ARGUMENT, "items %lld", (long long)items);
    if (items > 0x7fffff00LL / pl->B) return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    return RNN_OK;
}

}  // namespace

extern "C" {

rnn_status rnn_beam_create(rnn_beam_t* out, int64_t beams, int64_t end_id)
{
    NEED(out, "out");
    *out = nullptr;
    if (beams < 1 || beams > kMaxBeams)
        return fail(RNN_ERR_INVALID_ARGUMENT, "beams %lld outside [1, %d]", (long long)beams, kMaxBeams);
    if (end_id < -1 || end_id > 0x7fffffffLL) return fail(RNN_ERR_INVALID_ARGUMENT, "end_id %lld", (long long)end_id);
    rnn_beam* pl = new (std::nothrow) rnn_beam;
    if (!pl) return fail(RNN_ERR_OOM, "host allocation failed");
    pl->B = (int)beams;
    pl->end = end_id;
    *out = pl;
    return RNN_OK;
}

void rnn_beam_destroy(rnn_beam_t pl)
{
    if (!pl) return;
    free_plan_memory(pl);
    delete pl;
}

rnn_status rnn_beam_sync(rnn_beam_t pl)
{
    if (!pl) return fail(RNN_ERR_INVALID_ARGUMENT, "plan is NULL");
    return read_status(pl, "a parent outside [0, beams) or a slot outside its range");
}

int rnn_beam_last_launch_count(rnn_beam_t pl) { return pl ? pl->launches : 0; }

rnn_status rnn_beam_select(rnn_beam_t pl, const rnn_beam_select_args* a)
{
    rnn_status rs = check_plan(pl, a, a ? a->items : 0);
    if (rs != RNN_OK) return rs;
    if (a->vocab <= 0) return fail(RNN_ERR_INVALID_ARGUMENT, "vocab %lld", (long long)a->vocab);
    if (a->vocab > 0x7fffff00LL) return fail(RNN_ERR_UNSUPPORTED, "a size of 2^31 or more");
    if (a->io != RNN_IO_F32 && a->io != RNN_IO_F16 && a->io != RNN_IO_BF16)
        return fail(RNN_ERR_INVALID_ARGUMENT, "unknown io type %lld", (long long)a->io);
    if (a->row_stride != 0 && a->row_stride != RNN_SHARED_ROW && a->row_stride < a->vocab)
        return fail(RNN_ERR_INVALID_ARGUMENT, "row_stride %lld is below vocab %lld", (long long)a->row_stride, (long long)a->vocab);
    if (a->shared & ~(int64_t)1) return fail(RNN_ERR_INVALID_ARGUMENT, "shared is 0 or 1");
    if (pl->end >= a->vocab)
        return fail(RNN_ERR_INVALID_ARGUMENT, "end_id %lld is not below vocab %lld", (long long)pl->end, (long long)a->vocab);
    if (a->finished && pl->end < 0) return fail(RNN_ERR_INVALID_ARGUMENT, "finished beams without an end_id");
    if (a->items == 0) return RNN_OK;
    NEED(a->logits, "logits");
    NEED(a->scores, "scores");
    NEED(a->parents, "parents");
    NEED(a->ids, "ids");
    NEED(a->new_scores, "new_scores");
    if ((uintptr_t)a->logits % element((int)a->io)) return fail(RNN_ERR_INVALID_ARGUMENT, "logits are not aligned to their elements");
    rs = check_arrays({{a->scores, "scores"}, {a->parents, "parents"}, {a->ids, "ids"}, {a->new_scores, "new_scores"}});
    const size_t beams = (size_t)(a->items * pl->B);
    if (rs == RNN_OK) rs = check_in_place(a->scores, a->new_scores, 4 * beams, "scores and new_scores");
    if (rs == RNN_OK) rs = check_in_place(a->finished, a->new_finished, beams, "finished and new_finished");
    if (rs == RNN_OK) rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    BeamSelectParams p{};
    p.items = a->items;
    p.V = a->vocab;
    p.B = pl->B;
    p.io = (int)a->io;
    p.top = a->vocab < pl->B ? (int)a->vocab : pl->B;
    p.end = pl->end;
    p.shared = (int)a->shared;
    p.stride = a->row_stride == RNN_SHARED_ROW ? 0 : a->row_stride ? a->row_stride : a->vocab;
    p.logits = a->logits;
    p.scores = a->scores;
    p.finished = a->finished;
    p.parents = a->parents;
    p.ids = a->ids;
    p.new_scores = a->new_scores;
    p.new_finished = a->new_finished;
    cudaStream_t st = (cudaStream_t)a->stream;
    p.sms = pl->sms;
    beam_plan(p);
    const size_t bytes = beam_scratch_bytes(p);
    char* scratch = nullptr;
    rs = claim_scratch(pl, bytes, st, &scratch);
    if (rs != RNN_OK) return rs;
    p.scratch = (unsigned char*)scratch;
    cudaError_t e = launch_beam_select(p, st, &pl->launches);
    if (e != cudaSuccess) return cuda_fail(e, "beam selection launch");
    return release_scratch(pl, bytes, st);
}

rnn_status rnn_beam_reorder(rnn_beam_t pl, const rnn_beam_reorder_args* a)
{
    rnn_status rs = check_plan(pl, a, a ? a->items : 0);
    if (rs != RNN_OK) return rs;
    if (a->n_tensors < 0) return fail(RNN_ERR_INVALID_ARGUMENT, "n_tensors %lld", (long long)a->n_tensors);
    if (a->items == 0 || a->n_tensors == 0) return RNN_OK;
    NEED(a->parents, "parents");
    NEED(a->tensors, "tensors");
    rs = check_slots(a->slots, a->n_slots);
    if (rs == RNN_OK) rs = check_arrays({{a->parents, "parents"}, {a->slots, "slots"}});
    if (rs != RNN_OK) return rs;
    const int64_t rows = a->slots ? a->n_slots : a->items * pl->B;
    for (int64_t i = 0; i < a->n_tensors; ++i) {
        const rnn_beam_tensor& t = a->tensors[i];
        if (t.row_bytes < 0 || (t.row_bytes > 0 && rows > INT64_MAX / t.row_bytes))
            return fail(RNN_ERR_INVALID_ARGUMENT, "tensor %lld: row_bytes %lld", (long long)i, (long long)t.row_bytes);
        if (t.row_bytes == 0) continue;
        NEED(t.in, "a tensor's in");
        NEED(t.out, "a tensor's out");
        rs = check_in_place(t.in, t.out, (size_t)(rows * t.row_bytes), "a tensor's in and out");
        if (rs != RNN_OK) return rs;
    }
    // Blocks of all tensors run side by side: none may write where another reads or writes.
    auto meet = [](const void* a, uint64_t an, const void* b, uint64_t bn) {
        return (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
    };
    const uint64_t beams = 4 * (uint64_t)(a->items * pl->B);
    for (int64_t i = 0; i < a->n_tensors; ++i) {
        const rnn_beam_tensor& t = a->tensors[i];
        const uint64_t bytes = (uint64_t)(rows * t.row_bytes);
        if (!bytes) continue;
        if (meet(t.out, bytes, a->parents, beams) || (a->slots && meet(t.out, bytes, a->slots, beams)))
            return fail(RNN_ERR_INVALID_ARGUMENT, "tensor %lld's out overlaps parents or slots", (long long)i);
        for (int64_t j = 0; j < i; ++j) {
            const rnn_beam_tensor& o = a->tensors[j];
            const uint64_t others = (uint64_t)(rows * o.row_bytes);
            if (others && (meet(t.out, bytes, o.out, others) || meet(t.out, bytes, o.in, others) || meet(t.in, bytes, o.out, others)))
                return fail(RNN_ERR_INVALID_ARGUMENT, "tensors %lld and %lld overlap", (long long)j, (long long)i);
        }
    }
    rs = ensure_status(pl);
    if (rs != RNN_OK) return rs;
    ReorderParams p{};
    p.items = a->items;
    p.n_slots = a->n_slots;
    p.B = pl->B;
    p.parents = a->parents;
    p.slots = a->slots;
    p.status = pl->status;
    for (int64_t i = 0; i <= a->n_tensors; ++i) {
        if (p.n == kReorderTensors || (i == a->n_tensors && p.n > 0)) {
            cudaError_t e = launch_beam_reorder(p, (cudaStream_t)a->stream, &pl->launches);
            if (e != cudaSuccess) return cuda_fail(e, "reordering launch");
            p.n = 0;
        }
        if (i < a->n_tensors && a->tensors[i].row_bytes > 0)
            p.t[p.n++] = ReorderTensor{a->tensors[i].in, a->tensors[i].out, a->tensors[i].row_bytes};
    }
    return RNN_OK;
}

}  // extern "C"
