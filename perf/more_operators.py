"""Measured cases of the gated delta rule, layer normalisation and beam search.

Three operators with the forms that a program needs of each: the gated delta
rule (a recurrent layer whose state is a matrix a head) for prompts, for
training and for single tokens; layer normalisation for single tokens and for
training; a step of beam search, which selects over beams and vocabulary and
then reorders the states of the layers.  ``run`` takes one pass of a case: with
``own`` false in plain torch operations, with ``own`` true through this
package's entry points.
"""
import math

import torch

own = False

IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# Most work of a drawn case (each the largest listed case's): steps x heads x
# state of a run of the delta rule and of its training step, states of a token,
# elements of a normalisation, logits of a selection.
MOST_DELTA = 8 * 2048 * 16 * 128 * 128
MOST_STEP, MOST_NORM, MOST_BEAM = 256 * 16 * 128 * 128, 16384 * 2048, 64 * 8 * 50001
CHUNK = 64


def listed():
    def delta(name, **kw):
        return dict(name=name, kind="delta", **kw)

    return [
        # one short prompt through a small layer: latency
        delta("delta_prompt_short_bf16", batch=1, seq=200, heads=8, key_heads=8, key=64, value=64, io="bf16", train=False,
              ragged=False, carried=False, layout=1),
        # one long document: the time axis is the only long one
        delta("delta_prompt_long_bf16", batch=1, seq=16384, heads=16, key_heads=16, key=128, value=128, io="bf16",
              train=False, ragged=False, carried=False, layout=1),
        # prompts of mixed lengths that continue earlier ones, full precision, two value heads a key head
        delta("delta_prompt_ragged_f32", batch=12, seq=777, heads=8, key_heads=4, key=64, value=96, io="f32", train=False,
              ragged=True, carried=True, layout=0),
        # a training step of one wide layer
        delta("delta_train_bf16", batch=8, seq=2048, heads=16, key_heads=16, key=128, value=128, io="bf16", train=True,
              ragged=False, carried=False, layout=1),
        # a small training step where no size is a round one
        delta("delta_train_odd_f16", batch=3, seq=301, heads=6, key_heads=3, key=40, value=72, io="f16", train=True,
              ragged=True, carried=True, layout=1),
        # one token of one sequence: latency
        dict(name="delta_step_one_bf16", kind="delta_step", batch=1, heads=16, key_heads=16, key=128, value=128, io="bf16"),
        # one token for each running sequence of a server: the states' traffic
        dict(name="delta_step_many_bf16", kind="delta_step", batch=256, heads=16, key_heads=8, key=128, value=128,
             io="bf16"),
        # one token for each running sequence of a server, before a layer's projection
        dict(name="norm_step_bf16", kind="norm", rows=96, size=2048, io="bf16", train=False, affine=True),
        # a training step's normalisation of a batch of sequences
        dict(name="norm_train_bf16", kind="norm", rows=16384, size=2048, io="bf16", train=True, affine=True),
        # rows of an odd length in full precision, with their gradients
        dict(name="norm_train_odd_f32", kind="norm", rows=777, size=1001, io="f32", train=True, affine=True),
        # one request's beams: latency
        dict(name="beam_one_f32", kind="beam", items=1, beams=4, vocab=32000, io="f32", finished=False, masked=False,
             state=4096),
        # a batch of requests over an odd vocabulary, some beams at their end, with a layer's states behind them
        dict(name="beam_many_bf16", kind="beam", items=64, beams=8, vocab=50001, io="bf16", finished=True, masked=True,
             state=65536),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["delta", "delta", "delta", "delta_step", "norm", "norm", "beam", "beam"])
    io = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if kind in ("delta", "delta_step"):
        key, value = rng.choice([16, 32, 64, 64, 96, 128, 128]), rng.choice([32, 64, 64, 96, 128, 128, 192])
        if rng.random() < 0.25:
            key, value = rng.randint(5, 128), rng.randint(5, 160)
        key_heads, per = _log_int(rng, 1, 16), rng.choice([1, 1, 2, 3])
        heads = key_heads * per
        c = dict(kind=kind, heads=heads, key_heads=key_heads, key=key, value=value, io=io)
        if kind == "delta_step":
            return dict(c, batch=_log_int(rng, 1, max(1, min(512, MOST_STEP // (heads * key * value)))))
        # narrow heads cost a layer more than their states do, odd types more than bf16
        size = max(key, 64) * max(value, 64)
        most = MOST_DELTA // (heads * size) // (1 if io == "bf16" else 8)
        batch = _log_int(rng, 1, max(1, min(64, most // 64)))
        seq = _log_int(rng, 1 if rng.random() < 0.2 else 48, max(48, min(16384, most // batch)))
        return dict(c, batch=batch, seq=seq, train=rng.random() < 0.5, ragged=rng.random() < 0.4,
                    carried=rng.random() < 0.4, layout=rng.choice([0, 1]))
    if kind == "norm":
        size = _log_int(rng, 32, 16384)
        if rng.random() < 0.6:
            size = max(64, size // 64 * 64)
        return dict(kind=kind, rows=_log_int(rng, 1, max(1, min(65536, MOST_NORM // size // (2 if io == "f32" else 1)))),
                    size=size, io=io, train=rng.random() < 0.6, affine=rng.random() < 0.8)
    beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 10, 16, 32]), _log_int(rng, 100, 130000)
    items = _log_int(rng, 1, max(1, min(128, MOST_BEAM // (beams * vocab) // (2 if io == "f32" else 1))))
    return dict(kind=kind, items=items, beams=beams, vocab=vocab, io=io, finished=rng.random() < 0.5,
                masked=rng.random() < 0.4, state=_log_int(rng, 16, max(16, min(65536, 64 * 8 * 65536 // (items * beams)))))


# ---------------------------------------------------------------- the inputs

def _lengths(c, rnd):
    n, s = c["batch"], c["seq"]
    lens = torch.randint(0, s + 1, (n,), generator=rnd, device="cuda", dtype=torch.int32)
    lens[0] = s
    if n > 1:
        lens[n // 2] = 0        # a row with nothing in it
    return lens


def prepare(case, seed):
    rnd = torch.Generator(device="cuda").manual_seed(int(seed))
    io = IO[case["io"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=rnd, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=rnd, device="cuda") * (hi - lo) + lo

    c, s = case, dict(case=case)
    if c["kind"] in ("delta", "delta_step"):
        n, h, hk, dk, dv = c["batch"], c["heads"], c["key_heads"], c["key"], c["value"]
        if c["kind"] == "delta_step":
            lead = (n,)
        else:
            lead = (n, c["seq"]) if c["layout"] == 1 else (c["seq"], n)

        def unit(*shape):       # queries and keys of length one, as such layers normalise them
            v = normal(*shape)
            return (v / (v * v).sum(-1, keepdim=True).sqrt()).to(io)

        s["Q"], s["K"] = unit(*lead, hk, dk), unit(*lead, hk, dk)
        # V is a part of the convolution's output
        s["V"] = normal(*lead, 2 * hk * dk + h * dv, dtype=io)[..., 2 * hk * dk:].unflatten(-1, (h, dv))
        # rates from 1 to 16, steps from a thousandth to a tenth, as such layers start
        rate, step = uniform(h, lo=1.0, hi=16.0), torch.exp(uniform(h, lo=math.log(1e-3), hi=math.log(0.1)))
        bias = step + torch.log(-torch.expm1(-step))
        s["g"] = -rate * _softplus(normal(*lead, h, scale=0.5) + bias)
        s["beta"] = torch.sigmoid(normal(*lead, h))
        if c["kind"] == "delta_step":
            s["state"] = normal(n, h, dk, dv, scale=0.3)
            s["state_out"], s["Y"] = torch.empty_like(s["state"]), torch.empty(n, h, dv, device="cuda", dtype=io)
        else:
            s["lens"] = _lengths(c, rnd) if c["ragged"] else None
            s["state"] = normal(n, h, dk, dv, scale=0.3) if c["carried"] else None
            if c["train"]:
                s["dY"] = normal(*lead, h, dv, dtype=io)
                s["d_state"] = normal(n, h, dk, dv, scale=0.3) if c["carried"] else None
    elif c["kind"] == "norm":
        r, d = c["rows"], c["size"]
        # rows of a residual stream: a mean and a scale of their own
        s["X"] = (normal(r, d) * uniform(r, 1, lo=0.5, hi=3.0) + normal(r, 1)).to(io)
        s["W"] = 1.0 + normal(d, scale=0.2) if c["affine"] else None
        s["bias"] = normal(d, scale=0.2) if c["affine"] else None
        if c["train"]:
            s["dY"] = normal(r, d, dtype=io)
    else:
        i, b, v = c["items"], c["beams"], c["vocab"]
        s["logits"] = normal(i * b, v, scale=2.5, dtype=io)
        s["scores"] = -20.0 * uniform(i, b)
        s["finished"] = None
        if c["masked"]:         # tokens that a grammar rules out, and a beam that has none left
            s["logits"][torch.rand(i * b, v, generator=rnd, device="cuda") < 0.3] = float("-inf")
            s["logits"][(i * b) // 2] = float("-inf")
        if c["finished"]:       # beams at their end, and a first step, where one beam alone has begun
            s["finished"] = torch.rand(i, b, generator=rnd, device="cuda") < 0.2
            s["scores"][0, 1:], s["finished"][0] = float("-inf"), False
        s["state"] = normal(i * b, c["state"])
        s["ids"] = torch.randint(0, v, (i * b, 64), generator=rnd, device="cuda", dtype=torch.int32)
        s["end"] = v - 1
    if own:
        _handle(s)
    return s


def _handle(s):
    """The plan that a program keeps for a layer or a search."""
    import onnx_recurrent_gb300 as orc
    c = s["case"]
    if c["kind"] in ("delta", "delta_step"):
        s["plan"] = orc.rnn_delta_create(c["heads"], key_size=c["key"], value_size=c["value"], key_heads=c["key_heads"],
                                         layout=c.get("layout", 0))
        orc.rnn_delta_set_io_type(s["plan"], c["io"])
    elif c["kind"] == "norm":
        s["plan"] = orc.rnn_norm_create(c["size"], eps=1e-5)
        orc.rnn_norm_set_io_type(s["plan"], c["io"])
    else:
        s["plan"] = orc.rnn_beam_create(c["beams"], end_id=s["end"])


# ----------------------------------------------------------- the plain forms

def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _delta_plain(s):
    """Chunks of 64 steps as matrix products; the chunks one after another."""
    c = s["case"]
    n, h, hk, dk, dv, seq, io = c["batch"], c["heads"], c["key_heads"], c["key"], c["value"], c["seq"], IO[c["io"]]
    per, scale = h // hk, 1.0 / math.sqrt(dk)
    chunks = (seq + CHUNK - 1) // CHUNK
    pad = chunks * CHUNK - seq
    lens = torch.full((n,), seq, device="cuda") if s["lens"] is None else s["lens"].long()
    valid = torch.arange(chunks * CHUNK, device="cuda")[None, :] < lens[:, None]

    def cut(v, repeat=1):       # [batch, head, chunk, step, ...] in 32 bits, zeros past a row's end
        v = v.float() if c["layout"] == 1 else v.float().transpose(0, 1)
        v = torch.cat([v, v.new_zeros(n, pad, *v.shape[2:])], 1)
        v = torch.where(valid.view(n, -1, *[1] * (v.dim() - 2)), v, 0.0)
        v = v.unflatten(1, (chunks, CHUNK)).movedim(3, 1)
        return v.repeat_interleave(repeat, 1) if repeat > 1 else v

    def back(v, dtype):
        v = v.movedim(1, 3).flatten(1, 2)[:, :seq]
        v = torch.where(valid[:, :seq].view(n, seq, *[1] * (v.dim() - 2)), v, 0.0).to(dtype)
        return v if c["layout"] == 1 else v.transpose(0, 1).contiguous()

    q, k, v, g, beta = cut(s["Q"], per), cut(s["K"], per), cut(s["V"]), cut(s["g"]), cut(s["beta"])
    sums = g.double().cumsum(-1)
    at = torch.arange(CHUNK, device="cuda")
    below, diag = at[:, None] > at[None, :], at[:, None] >= at[None, :]
    decay = torch.where(diag, torch.exp(torch.where(diag, sums[..., :, None] - sums[..., None, :], 0.0)), 0.0).float()
    first, last = torch.exp(sums).float(), torch.exp(sums[..., -1:] - sums).float()     # from the start, to the end
    whole = first[..., -1]
    kk = k @ k.transpose(-1, -2)
    A = torch.where(below, beta[..., None] * decay * kk, 0.0)
    T = torch.eye(CHUNK, device="cuda").expand_as(A).clone()
    for i in range(1, CHUNK):                           # the inverse of 1 + A, a row at a time
        T[..., i, :i] = -(A[..., i, None, :i] @ T[..., :i, :i])[..., 0, :]
    P = torch.where(diag, decay * (q @ k.transpose(-1, -2)), 0.0)
    state = torch.zeros(n, h, dk, dv, device="cuda") if s["state"] is None else s["state"].clone()
    starts, U, Y = [], [], []
    for j in range(chunks):
        starts.append(state)
        r = beta[:, :, j, :, None] * (v[:, :, j] - first[:, :, j, :, None] * (k[:, :, j] @ state))
        u = T[:, :, j] @ r
        Y.append(scale * (first[:, :, j, :, None] * (q[:, :, j] @ state) + P[:, :, j] @ u))
        state = whole[:, :, j, None, None] * state + (last[:, :, j, :, None] * k[:, :, j]).transpose(-1, -2) @ u
        U.append(u)
    out = {"Y": back(torch.stack(Y, 2), io), "state": state}
    if not c["train"]:
        return out
    dy = scale * cut(s["dY"])
    ahead = torch.zeros_like(state) if s["d_state"] is None else s["d_state"].clone()
    dQ, dK, dV, dg, dbeta = [], [], [], [], []
    for j in range(chunks - 1, -1, -1):
        kj, qj, u, s0 = k[:, :, j], q[:, :, j], U[j], starts[j]
        f, l, b, D = first[:, :, j, :, None], last[:, :, j, :, None], beta[:, :, j, :, None], decay[:, :, j]
        du = P[:, :, j].transpose(-1, -2) @ dy[:, :, j] + l * (kj @ ahead)
        dr = T[:, :, j].transpose(-1, -2) @ du
        dA = torch.where(below, -(dr @ u.transpose(-1, -2)), 0.0)
        dP = torch.where(diag, dy[:, :, j] @ u.transpose(-1, -2), 0.0)
        GA, GP = b * D * dA, D * dP
        x1, x2, x3 = dy[:, :, j] @ s0.transpose(-1, -2), dr @ s0.transpose(-1, -2), u @ ahead.transpose(-1, -2)
        dQ.append(f * x1 + GP @ kj)
        dK.append((GA + GA.transpose(-1, -2)) @ kj + GP.transpose(-1, -2) @ qj - b * f * x2 + l * x3)
        dV.append(b * dr)
        kx2 = (kj * x2).sum(-1)
        dbeta.append((dr * v[:, :, j]).sum(-1) - f[..., 0] * kx2 + (dA * D * kk[:, :, j]).sum(-1))
        X = GA * kk[:, :, j] + dP * P[:, :, j]
        end = l[..., 0] * (kj * x3).sum(-1)
        dsum = X.sum(-1) - X.sum(-2) + f[..., 0] * ((qj * x1).sum(-1) - b[..., 0] * kx2) - end
        dsum[..., -1] += end.sum(-1) + whole[:, :, j] * (ahead * s0).sum((-1, -2))
        dg.append(dsum.flip(-1).cumsum(-1).flip(-1))
        ahead = whole[:, :, j, None, None] * ahead + qj.transpose(-1, -2) @ (f * dy[:, :, j]) - kj.transpose(-1, -2) @ (b * f * dr)
    join = lambda parts: torch.stack(parts[::-1], 2)  # noqa: E731
    shared = lambda parts: join(parts).unflatten(1, (hk, per)).sum(2)  # noqa: E731
    out.update(dQ=back(shared(dQ), io), dK=back(shared(dK), io), dV=back(join(dV), io),
               dg=back(join(dg), torch.float32), dbeta=back(join(dbeta), torch.float32))
    if s["state"] is not None:
        out["d_initial_state"] = ahead
    return out


def _delta_step_plain(s):
    c = s["case"]
    per, io = c["heads"] // c["key_heads"], IO[c["io"]]
    q, k = s["Q"].float().repeat_interleave(per, 1), s["K"].float().repeat_interleave(per, 1)
    state = torch.exp(s["g"])[..., None, None] * s["state"]
    u = s["beta"][..., None] * (s["V"].float() - (k[..., None] * state).sum(-2))
    state = state + k[..., None] * u[..., None, :]
    return {"Y": ((q[..., None] * state).sum(-2) / math.sqrt(c["key"])).to(io), "state": state}


def _norm_plain(s):
    c = s["case"]
    io, x = IO[c["io"]], s["X"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5)
    xhat = d * rstd
    out = {"Y": (xhat if s["W"] is None else xhat * s["W"] + s["bias"]).to(io)}
    if c["train"]:
        dy = s["dY"].float()
        w = dy if s["W"] is None else dy * s["W"]
        out["dX"] = (rstd * (w - w.mean(1, keepdim=True) - xhat * (w * xhat).mean(1, keepdim=True))).to(io)
        if s["W"] is not None:
            out.update(dW=(dy * xhat).sum(0), dbias=dy.sum(0))
    return out


def _beam_plain(s):
    c = s["case"]
    i, b, v = c["items"], c["beams"], c["vocab"]
    x = s["logits"].float()
    most = x.max(1, keepdim=True).values
    empty = most == float("-inf")
    total = torch.exp(x - torch.where(empty, 0.0, most)).double().sum(1, keepdim=True)
    # candidates that lie close together are told apart in 64 bits
    lse = torch.where(empty, 0.0, most).double() + torch.log(torch.where(empty, 1.0, total))
    logp = (x.double() - lse).view(i, b, v)
    if s["finished"] is not None:           # a beam at its end goes on as it is, by its last token
        stay = torch.full((v,), float("-inf"), device="cuda", dtype=torch.float64)
        stay[s["end"]] = 0.0
        logp = torch.where(s["finished"][..., None], stay, logp)
    left = (s["scores"].double()[..., None] + logp).view(i, b * v)
    places = torch.arange(b * v, device="cuda")
    scores, parents, ids = [], [], []
    for _ in range(b):                      # the largest, ties to the lowest place, b times
        best = left.max(1, keepdim=True).values
        at = torch.where(left == best, places, b * v).min(1, keepdim=True).values
        scores.append(best[:, 0].float())
        parents.append(torch.div(at[:, 0], v, rounding_mode="floor"))
        ids.append(at[:, 0] % v)
        if len(scores) < b:
            # out of the running for good, below a mask's -inf
            left = left.scatter(1, at, float("nan"))
            left = torch.where(left.isnan(), float("-inf"), left)
            places = torch.where(torch.arange(b * v, device="cuda") == at, b * v, places)
    parents, ids = torch.stack(parents, 1), torch.stack(ids, 1)
    rows = (parents + torch.arange(i, device="cuda")[:, None] * b).view(-1)
    done = ids == s["end"]
    if s["finished"] is not None:
        done = done | s["finished"].gather(1, parents)
    return {"parents": parents.int(), "ids": ids.int(), "scores": torch.stack(scores, 1), "finished": done,
            "state": s["state"][rows], "history": s["ids"][rows]}


# ------------------------------------------------------ the package's operators

def _run_own(s):
    import onnx_recurrent_gb300 as orc
    c = s["case"]
    kind = c["kind"]
    if kind == "delta":
        args = (s["Q"], s["K"], s["V"], s["g"], s["beta"], s["lens"], s["state"])
        Y, state, saved = orc.delta_rule(s["plan"], *args, save=c["train"])
        out = {"Y": Y, "state": state}
        if c["train"]:
            out.update(orc.delta_rule_grad(s["plan"], s["dY"], saved, *args, d_state=s["d_state"]))
        return out
    if kind == "delta_step":
        orc.rnn_delta_step(s["plan"], s["Q"], s["K"], s["V"], s["g"], s["beta"], s["state"], s["Y"],
                           state_out=s["state_out"])
        return {"Y": s["Y"], "state": s["state_out"]}
    if kind == "norm":
        Y, stats = orc.layer_norm(s["plan"], s["X"], s["W"], s["bias"])
        out = {"Y": Y}
        if c["train"]:
            out.update(orc.layer_norm_grad(s["plan"], s["dY"], s["X"], stats, s["W"], s["bias"]))
        return out
    step = orc.beam_select(s["plan"], s["logits"], s["scores"], s["finished"])
    state, history = orc.beam_reorder(s["plan"], step.parents, [s["state"], s["ids"]])
    return {"parents": step.parents, "ids": step.ids, "scores": step.scores, "finished": step.finished, "state": state,
            "history": history}


def run(state):
    if own:
        return _run_own(state)
    return {"delta": _delta_plain, "delta_step": _delta_step_plain, "norm": _norm_plain,
            "beam": _beam_plain}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    e = {"f32": 4, "f16": 2, "bf16": 2}[c["io"]]
    kind = c["kind"]
    if kind == "norm":
        n, w = c["rows"] * c["size"], 4 * c["size"] * (2 if c["affine"] else 0)
        b, f = 2 * n * e + w, 8 * n
        if c["train"]:          # dY read, dX and the weights' gradients written (X is read once in all)
            b, f = b + 2 * n * e + w, f + 14 * n
        return {"bytes": b, "flops": f}
    if kind == "beam":
        rows = c["items"] * c["beams"]
        b = rows * c["vocab"] * e + rows * (4 * 4 + 2) + 2 * rows * (4 * c["state"] + 4 * 64)
        return {"bytes": b, "flops": 5 * rows * c["vocab"]}
    n, h, hk, dk, dv = c["batch"], c["heads"], c["key_heads"], c["key"], c["value"]
    state = 4 * n * h * dk * dv
    if kind == "delta_step":
        return {"bytes": 2 * state + n * ((2 * hk * dk + 2 * h * dv) * e + 8 * h), "flops": n * h * 7 * dk * dv}
    steps = n * c["seq"]
    b = steps * ((2 * hk * dk + 2 * h * dv) * e + 8 * h) + state * (2 if c["carried"] else 1)
    f = steps * h * 7 * dk * dv
    if c["train"]:              # dY read; dQ, dK, dV, dg and dbeta written; the carried state's
        b += steps * ((2 * hk * dk + 2 * h * dv) * e + 8 * h) + (2 * state if c["carried"] else 0)
        f += steps * h * 16 * dk * dv
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------- in 64 bits

def _exact_delta(s, c):
    """The definition, one step after another, and its slopes backwards."""
    n, h, hk, dk, dv, seq = c["batch"], c["heads"], c["key_heads"], c["key"], c["value"], c["seq"]
    time, wide = (1 if c["layout"] == 1 else 0), lambda w: w.repeat_interleave(h // hk, 1)
    step_of = lambda w, t: w.select(time, t).double()  # noqa: E731
    scale = dk ** -0.5
    H = s["state"].double() if s["state"] is not None else torch.zeros(n, h, dk, dv, device="cuda", dtype=torch.float64)
    lens = s["lens"] if s["lens"] is not None else torch.full((n,), seq, device="cuda", dtype=torch.int32)
    Y, kept = [], []
    for t in range(seq):
        live = (lens > t)[:, None, None]
        q, k = wide(step_of(s["Q"], t)), wide(step_of(s["K"], t))
        a, b = torch.exp(step_of(s["g"], t))[..., None, None], step_of(s["beta"], t)[..., None]
        if c["train"]:
            kept.append(H)
        decayed = a * H
        u = b * (step_of(s["V"], t) - torch.einsum("nhk,nhkv->nhv", k, decayed))
        new = decayed + torch.einsum("nhk,nhv->nhkv", k, u)
        H = new if s["lens"] is None else torch.where(live[..., None], new, H)
        Y.append(torch.where(live, scale * torch.einsum("nhk,nhkv->nhv", q, new), 0.0))
    out = {"Y": torch.stack(Y, time), "state": H}
    if not c["train"]:
        return out
    G = s["d_state"].double() if s["d_state"] is not None else torch.zeros_like(H)
    parts = {w: [None] * seq for w in ("dQ", "dK", "dV", "dg", "dbeta")}
    for t in range(seq - 1, -1, -1):
        live = (lens > t)[:, None, None]
        q, k, v, dy = wide(step_of(s["Q"], t)), wide(step_of(s["K"], t)), step_of(s["V"], t), scale * step_of(s["dY"], t)
        a, b = torch.exp(step_of(s["g"], t))[..., None, None], step_of(s["beta"], t)[..., None]
        decayed = a * kept[t]
        miss = v - torch.einsum("nhk,nhkv->nhv", k, decayed)
        new = decayed + torch.einsum("nhk,nhv->nhkv", k, b * miss)
        slope = G + torch.einsum("nhk,nhv->nhkv", q, dy)
        du = torch.einsum("nhk,nhkv->nhv", k, slope)
        dmiss = b * du
        dk_ = torch.einsum("nhkv,nhv->nhk", slope, b * miss) - torch.einsum("nhkv,nhv->nhk", decayed, dmiss)
        dec = slope - torch.einsum("nhk,nhv->nhkv", k, dmiss)       # the slope in the decayed state
        fold = lambda w: torch.where(live, w, 0.0).reshape(n, hk, h // hk, dk).sum(2)  # noqa: E731
        parts["dQ"][t], parts["dK"][t] = fold(torch.einsum("nhkv,nhv->nhk", new, dy)), fold(dk_)
        parts["dV"][t] = torch.where(live, dmiss, 0.0)
        parts["dbeta"][t] = torch.where(live[..., 0], (du * miss).sum(-1), 0.0)
        parts["dg"][t] = torch.where(live[..., 0], (dec * decayed).sum((-1, -2)), 0.0)
        G = a * dec if s["lens"] is None else torch.where(live[..., None], a * dec, G)
        kept[t] = None
    out.update({w: torch.stack(p, time) for w, p in parts.items()})
    if s["state"] is not None:
        out["d_initial_state"] = G
    return out


def _exact_norm(s, c):
    x = s["X"].double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    sd = (var + 1e-5).sqrt()
    z = (x - mean) / sd
    W = torch.ones(c["size"], device="cuda", dtype=torch.float64) if s["W"] is None else s["W"].double()
    out = {"Y": z * W + (0.0 if s["bias"] is None else s["bias"].double())}
    if c["train"]:
        dz = s["dY"].double() * W
        n = c["size"]
        out["dX"] = (dz - (dz.sum(1, keepdim=True) + z * (dz * z).sum(1, keepdim=True)) / n) / sd
        if s["W"] is not None:
            out.update(dW=torch.einsum("rd,rd->d", s["dY"].double(), z), dbias=s["dY"].double().sum(0))
    return out


def _exact_beam(s, c):
    i, b, v = c["items"], c["beams"], c["vocab"]
    out = {q: [] for q in ("parents", "ids", "scores", "finished", "state", "history")}
    for item in range(i):
        x = s["logits"][item * b:(item + 1) * b].double()
        logp = torch.log_softmax(x, 1)
        logp[torch.isneginf(x).all(1)] = float("-inf")
        ended = torch.zeros(b, dtype=torch.bool, device="cuda") if s["finished"] is None else s["finished"][item]
        logp[ended] = float("-inf")
        logp[ended, s["end"]] = 0.0
        total, order = torch.sort((logp + s["scores"][item].double()[:, None]).flatten(), descending=True, stable=True)
        total, order = total[:b], order[:b]
        parent, token = order // v, order % v
        out["parents"].append(parent.int())
        out["ids"].append(token.int())
        out["scores"].append(total)
        out["finished"].append((token == s["end"]) | ended[parent])
        out["state"].append(s["state"][item * b + parent])
        out["history"].append(s["ids"][item * b + parent])
    cat = ("state", "history")
    return {q: torch.cat(w) if q in cat else torch.stack(w) for q, w in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "delta":
        return _exact_delta(s, c)
    if c["kind"] == "norm":
        return _exact_norm(s, c)
    if c["kind"] == "beam":
        return _exact_beam(s, c)
    one = dict(s, lens=None)                         # a sequence of one step with a carried state
    one.update({q: s[q][None] for q in ("Q", "K", "V", "g", "beta")})
    got = _exact_delta(one, dict(c, seq=1, layout=0, train=False))
    return {"Y": got["Y"][0], "state": got["state"]}
