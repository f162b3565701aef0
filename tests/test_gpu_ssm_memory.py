"""Which memory the state space operators and token scores use: tensors whose
rows share memory, states updated in place, scratch kept by captured graphs,
streams and devices that are not the current ones."""
import gc

import pytest
import torch

import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).cuda()


# ------------------------------------------------- rows that share memory

@pytest.mark.parametrize("rows,V,top,dtype", [(2, 1, 1, torch.float32), (5, 33, 4, torch.float32), (7, 9001, 20, torch.bfloat16),
                                              (900, 300, 0, torch.float16)])
def test_scores_of_one_row_for_several_tokens(rows, V, top, dtype):
    """An expanded row of logits: the scores and gradients of as many copies of it, bit for bit (the copies start on
    16-byte boundaries as the row does: the order of a row's sums goes by its alignment)."""
    r = _rand(1)
    row = (r(1, V) * 3).to(dtype)
    ids = (torch.arange(rows, device="cuda", dtype=torch.int32) * 7) % V
    d_logp, d_entropy = r(rows), r(rows)
    d_top = r(rows, top) if top else None
    one, copies = row.expand(rows, V), torch.zeros(rows, (V + 7) // 8 * 8, device="cuda", dtype=dtype)[:, :V]
    copies.copy_(one)
    assert one.stride(0) == 0
    got, want = orc.scores(one, ids, top=top), orc.scores(copies, ids, top=top)
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(orc.scores_grad(one, ids, got, d_logp, d_entropy, d_top),
                       orc.scores_grad(copies, ids, want, d_logp, d_entropy, d_top))


def test_gradients_refuse_rows_that_share_memory():
    x = torch.randn(1, 40, device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    s = orc.scores(x.expand(3, 40), ids)
    one = torch.ones(3, device="cuda")
    for logits, out in ((x.expand(3, 40), x.expand(3, 40)), (x.repeat(3, 1), x.expand(3, 40))):
        with pytest.raises(ValueError):
            orc.rnn_scores_grad(logits, ids, s, one, dlogits=out)
    with pytest.raises(orc.RNNError):      # rows that overlap in part
        orc.scores(torch.zeros(100, device="cuda").as_strided((3, 40), (20, 1)), ids)


def test_outputs_refuse_steps_or_rows_that_share_memory():
    N, S, D = 3, 4, 8
    r = _rand(2)
    plan = orc.rnn_ssm_create(D, state_size=4, layout=1)
    X, W, one = r(N, S, D), r(D, 4), torch.zeros(1, S, D, device="cuda")
    with pytest.raises(orc.RNNError) as e:
        orc.rnn_ssm_conv(plan, X, W, Y=one.expand(N, S, D))
    assert e.value.status == 1
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_conv_grad(plan, X, X, W, dX=one.expand(N, S, D))
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_conv(plan, X, W, Y=torch.zeros(N, 1, D, device="cuda").expand(N, S, D))
    B = r(N, S, 1, 4)
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_scan(plan, X, X, -torch.ones(D, 4, device="cuda"), B, B, Y=one.expand(N, S, D))
    # inputs may: a broadcast row gives what its copies give
    x = r(1, S, D).expand(N, S, D)
    assert torch.equal(orc.ssm_conv(plan, x, W)[0], orc.ssm_conv(plan, x.contiguous(), W)[0])


# --------------------------------------------------- states updated in place

def _scan_inputs(N, S, D, M, G, seed, gate=True):
    r = _rand(seed)
    return dict(X=r(N, S, D), dt=r(N, S, D, scale=0.5), A=-torch.exp(r(D, M, scale=0.5)), B=r(N, S, G, M), C=r(N, S, G, M),
                D=r(D), Z=r(N, S, D) if gate else None, dt_bias=r(D, scale=0.5) - 2.0), r(N, D, M)


# unsplit, split with the blocks' own chain, split with the chain's launch: so many launches
IN_PLACE = [((3, 9, 40, 16, 1), 1), ((1, 150, 136, 16, 1), 2), ((2, 300, 64, 16, 2), 3), ((2, 500, 40, 32, 1), 3)]


@pytest.mark.parametrize("size,launches", IN_PLACE, ids=lambda v: str(v))
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_updates_its_state_in_place(size, launches, ragged):
    N, S, D, M, G = size
    v, h0 = _scan_inputs(*size, seed=3)
    lens = torch.tensor([S, 0, S // 2][:N], dtype=torch.int32, device="cuda") if ragged else None
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)
    Y, Y_h, _ = orc.ssm_scan(plan, **v, sequence_lens=lens, initial_h=h0)
    assert orc.rnn_ssm_last_launch_count(plan) == launches
    for _ in range(3):
        h, y = h0.clone(), torch.empty_like(Y)
        orc.rnn_ssm_scan(plan, **v, sequence_lens=lens, initial_h=h, Y=y, Y_h=h)
        assert torch.equal(y, Y) and torch.equal(h, Y_h)
    orc.rnn_ssm_sync(plan)


# launches of the gradient: as above, and one that adds up the sums
GRAD_IN_PLACE = [((3, 9, 40, 16, 1), 2), ((1, 100, 136, 16, 1), 3), ((2, 300, 64, 16, 2), 4), ((2, 500, 40, 32, 1), 4)]


@pytest.mark.parametrize("size,launches", GRAD_IN_PLACE, ids=lambda v: str(v))
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_gradient_updates_its_states_slope_in_place(size, launches, ragged):
    N, S, D, M, G = size
    v, h0 = _scan_inputs(*size, seed=4)
    r = _rand(5)
    dY, dY_h = r(N, S, D), r(N, D, M)
    lens = torch.tensor([S, 0, S // 2][:N], dtype=torch.int32, device="cuda") if ragged else None
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)
    _, _, saved = orc.ssm_scan(plan, **v, sequence_lens=lens, initial_h=h0, save=True)
    want = orc.ssm_scan_grad(plan, dY, saved, **v, sequence_lens=lens, initial_h=h0, dY_h=dY_h)
    assert orc.rnn_ssm_last_launch_count(plan) == launches
    for _ in range(3):
        d = dY_h.clone()
        out = {k: d if k == "d_initial_h" else torch.empty_like(t) for k, t in want.items()}
        orc.rnn_ssm_scan_grad(plan, dY, saved, **v, sequence_lens=lens, initial_h=h0, dY_h=d, **out)
        for k in want:
            assert torch.equal(out[k], want[k]), k
    orc.rnn_ssm_sync(plan)


@pytest.mark.parametrize("N,S,D,K,io", [(3, 1, 40, 4, "f32"), (3, 2, 33, 8, "bf16"), (4, 300, 72, 4, "f16"), (2, 40, 8, 1, "f32")])
def test_convolution_gradient_updates_its_states_slope_in_place(N, S, D, K, io):
    """Runs shorter than the taps, where the first state takes slopes of the last one, and runs of several blocks."""
    r, t = _rand(6), {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[io]
    plan = orc.rnn_ssm_create(D, conv_width=K, layout=1)
    orc.rnn_ssm_set_io_type(plan, io)
    X, dY, W, b = r(N, S, D).to(t), r(N, S, D).to(t), r(D, K), r(D)
    h0, d_state = r(N, K - 1, D).to(t), r(N, K - 1, D).to(t)
    lens = torch.tensor([S, 0, max(S - 1, 0), S // 2][:N], dtype=torch.int32, device="cuda")
    want = orc.ssm_conv_grad(plan, dY, X, W, b, lens, h0, d_state)
    for with_weights in (True, False):
        d = d_state.clone()
        dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty_like(b)
        orc.rnn_ssm_conv_grad(plan, dY, X, W, b, lens, h0, d, dX, dW if with_weights else None, db if with_weights else None, d)
        assert torch.equal(dX, want["dX"]) and torch.equal(d, want["d_initial_state"])
        assert not with_weights or (torch.equal(dW, want["dW"]) and torch.equal(db, want["dbias"]))
    orc.rnn_ssm_sync(plan)


@pytest.mark.parametrize("N,S,D,K,io", [(3, 1, 40, 4, "f32"), (3, 2, 33, 8, "bf16"), (4, 300, 72, 4, "f16"), (3, 0, 8, 5, "f32")])
def test_convolution_updates_its_state_in_place(N, S, D, K, io):
    r, t = _rand(7), {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[io]
    plan = orc.rnn_ssm_create(D, conv_width=K, layout=1)
    orc.rnn_ssm_set_io_type(plan, io)
    X, W, h0 = r(N, S, D).to(t), r(D, K), r(N, K - 1, D).to(t)
    lens = torch.tensor([S, 0, max(S - 1, 0), S // 2][:N], dtype=torch.int32, device="cuda")
    Y, state = orc.ssm_conv(plan, X, W, None, lens, h0)
    y = torch.empty_like(Y)
    orc.rnn_ssm_conv(plan, X, W, None, lens, h0, y, h0)
    assert torch.equal(y, Y) and torch.equal(h0, state)


# ------------------------------------------------------- captured calls

def test_a_plan_that_goes_amid_a_capture():
    """As the garbage collector may have it: the capture goes on, and its graph replays."""
    size = (1, 150, 136, 16, 1)
    v, h0 = _scan_inputs(*size, seed=8)
    N, S, D, M, G = size
    old = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)
    orc.ssm_scan(old, **v, initial_h=h0)             # takes scratch, a status word and an event
    plan, W = orc.rnn_ssm_create(D, layout=1), torch.ones(D, 4, device="cuda")
    want, _ = orc.ssm_conv(plan, v["X"], W)
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orc.rnn_ssm_destroy(old)
        Y, _ = orc.ssm_conv(plan, v["X"], W)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_a_graph_outlives_the_scratch_of_later_calls():
    """A split scan, its gradient and a convolution's captured, then plain calls that need much more scratch, then
    replays: the graph's outputs are those of plain calls on its inputs."""
    size = (1, 150, 136, 16, 1)
    N, S, D, M, G = size
    v, h0 = _scan_inputs(*size, seed=8)
    r = _rand(9)
    dY, dY_h, W, b = r(N, S, D), r(N, D, M), r(D, 4), r(D)
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)

    def calls():
        Y, Y_h, saved = orc.ssm_scan(plan, **v, initial_h=h0, save=True)
        g = orc.ssm_scan_grad(plan, dY, saved, **v, initial_h=h0, dY_h=dY_h)
        c = orc.ssm_conv_grad(plan, dY, v["X"], W, b)
        return [Y, Y_h, *g.values(), *c.values()]
    orc.rnn_ssm_conv(plan, v["X"], W, Y=torch.empty_like(v["X"]))          # the plan's first call: no scratch
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    want = [t.clone() for t in calls()]
    big, H0 = _scan_inputs(4, 1500, D, M, G, seed=10)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        Y, _, saved = orc.ssm_scan(plan, **big, initial_h=H0, save=True)
        orc.ssm_scan_grad(plan, Y, saved, **big, initial_h=H0)
        # whatever took the place of freed memory is not written either
        other = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
        assert all((o == 3.0).all() for o in other)
    orc.rnn_ssm_sync(plan)


def test_plain_calls_beside_a_replay():
    """Plain calls of the plan on another stream while its graph replays: neither uses the other's scratch."""
    size = (2, 300, 64, 16, 2)
    N, S, D, M, G = size
    v, h0 = _scan_inputs(*size, seed=11)
    w, k0 = _scan_inputs(*size, seed=12)
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)
    want_v = [t.clone() for t in orc.ssm_scan(plan, **v, initial_h=h0)[:2]]
    want_w = [t.clone() for t in orc.ssm_scan(plan, **w, initial_h=k0)[:2]]
    gc.collect()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        Y, Y_h, _ = orc.ssm_scan(plan, **v, initial_h=h0)
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            outs.append(orc.ssm_scan(plan, **w, initial_h=k0)[:2])
    torch.cuda.synchronize()
    assert torch.equal(Y, want_v[0]) and torch.equal(Y_h, want_v[1])
    for y, h in outs:
        assert torch.equal(y, want_w[0]) and torch.equal(h, want_w[1])


def test_a_plans_first_call_does_not_wait_for_other_work():
    D = 32
    r = _rand(13)
    X, W = r(2, 5, D), r(D, 4)
    Y = torch.empty_like(X)
    orc.rnn_ssm_conv(orc.rnn_ssm_create(D, layout=1), X, W, Y=Y)           # loads the kernel
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    out, done, side = torch.empty_like(a), torch.cuda.Event(), torch.cuda.Stream()
    torch.mm(a, a, out=out)
    torch.cuda.synchronize()
    for _ in range(200):                                                   # over 100 ms
        torch.mm(a, a, out=out)
    done.record()
    plan = orc.rnn_ssm_create(D, layout=1)
    orc.rnn_ssm_conv(plan, X, W, Y=Y, stream=side)
    assert not done.query()
    torch.cuda.synchronize()
    orc.rnn_ssm_sync(plan)


def test_a_plans_first_call_may_be_captured():
    size = (1, 150, 136, 16, 1)
    N, S, D, M, G = size
    v, h0 = _scan_inputs(*size, seed=14)
    want = orc.ssm_scan(orc.rnn_ssm_create(D, state_size=M, layout=1), **v, initial_h=h0)
    plan = orc.rnn_ssm_create(D, state_size=M, layout=1)
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, Y_h, _ = orc.ssm_scan(plan, **v, sequence_lens=lens, initial_h=h0)
    graph.replay()
    assert torch.equal(Y, want[0]) and torch.equal(Y_h, want[1])
    orc.rnn_ssm_sync(plan)
    lens.fill_(S + 1)                                                      # a length that the kernels report
    graph.replay()
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_sync(plan)
    orc.rnn_ssm_sync(plan)


# ------------------------------------------------------------- streams

@pytest.mark.parametrize("handle", [False, True])
def test_outputs_belong_to_the_stream_of_the_call(handle):
    """Memory that was freed on the current stream, where work queued earlier may still use it, is not what a call on
    another stream writes."""
    N, S, D, M, V = 2, 600, 512, 16, 4096
    v, h0 = _scan_inputs(N, S, D, M, 1, seed=15)
    r = _rand(16)
    W, b, x = r(D, 4), r(D), r(N * S, V)
    plan = orc.rnn_ssm_create(D, state_size=M, layout=1)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    torch.cuda.synchronize()

    def freed(*shapes):
        kept = [torch.empty(s, device="cuda") for s in shapes for _ in range(4)]
        return {t.data_ptr() for t in kept}

    def check(outs, spots):
        assert not {t.data_ptr() for t in outs} & spots
    full, state = (N, S, D), (N, D, M)
    spots = freed(full, (N, 3, D))
    check(orc.ssm_conv(plan, v["X"], W, b, stream=stream), spots)
    spots = freed(full, (D, 4), (D,))
    check(orc.ssm_conv_grad(plan, v["X"], v["X"], W, b, stream=stream).values(), spots)
    side.synchronize()
    spots = freed(full, state, (orc.rnn_ssm_saved_size(plan, S, N),))
    Y, Y_h, saved = orc.ssm_scan(plan, **v, initial_h=h0, save=True, stream=stream)
    check((Y, Y_h, saved), spots)
    side.synchronize()
    spots = freed(full, state, (N, S, 1, M), (D, M), (D,))
    check(orc.ssm_scan_grad(plan, Y, saved, **v, initial_h=h0, stream=stream).values(), spots)
    spots = freed((N * S, V), (N * S,), (N * S, 5))
    s = orc.scores(x, torch.zeros(N * S, dtype=torch.int32, device="cuda"), top=5, stream=stream)
    check(s, spots)
    check([orc.scores_grad(x, None, s, d_top=s.top_logp, stream=stream)], spots)
    torch.cuda.synchronize()
    want = orc.ssm_scan(plan, **v, initial_h=h0)
    assert torch.equal(Y, want[0]) and torch.equal(Y_h, want[1])
