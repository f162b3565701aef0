"""Measured cases of the state space operators and the token scores.

Four operators: the short causal convolution over channels, the selective
state space scan behind it (both for prompts, for training and for single
tokens), and the scores of given tokens under a row of logits.  ``run`` takes
one pass of a case: with ``own`` false in plain torch operations, with
``own`` true through this package's entry points.
"""
import math

import torch

own = False

IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# Most work of a drawn case: elements of X for the convolution, state updates
# for the scan, logits for the scores (each the largest listed case's).
MOST_CONV, MOST_SCAN, MOST_STEP, MOST_SCORES = 8 * 2048 * 2048, 8 * 2048 * 2048 * 16, 256 * 4096 * 16, 8192 * 32000


def listed():
    def conv(name, **kw):
        return dict(name=name, kind="conv", **kw)

    def scan(name, **kw):
        return dict(name=name, kind="scan", **kw)

    return [
        # a batch of full prompts through a wide layer
        conv("conv_prompt_bf16", batch=8, seq=2048, channels=2048, width=4, io="bf16", train=False, ragged=False,
             carried=False, layout=1),
        # a training step over ragged documents, odd channels, carried history
        conv("conv_train_f16_ragged", batch=5, seq=1021, channels=770, width=3, io="f16", train=True, ragged=True,
             carried=True, layout=0),
        # one token for each running sequence of a server
        dict(name="conv_step_bf16", kind="conv_step", batch=96, channels=2048, width=4, io="bf16"),
        # one short prompt: latency
        scan("scan_prompt_short_bf16", batch=1, seq=200, channels=1024, state=16, groups=1, io="bf16", train=False,
             ragged=False, carried=False, gate=True, layout=1),
        # one long document: the time axis is the only long one
        scan("scan_prompt_long_bf16", batch=1, seq=16384, channels=2048, state=16, groups=1, io="bf16", train=False,
             ragged=False, carried=False, gate=True, layout=1),
        # prompts of mixed lengths that continue earlier ones, full precision
        scan("scan_prompt_ragged_f32", batch=24, seq=777, channels=1024, state=16, groups=1, io="f32", train=False,
             ragged=True, carried=True, gate=True, layout=0),
        # a training step of one wide layer
        scan("scan_train_bf16", batch=8, seq=2048, channels=2048, state=16, groups=1, io="bf16", train=True,
             ragged=False, carried=False, gate=True, layout=1),
        # a small training step where no size is a round one
        scan("scan_train_odd_f32", batch=3, seq=301, channels=201, state=12, groups=3, io="f32", train=True,
             ragged=True, carried=True, gate=False, layout=1),
        # one token of one sequence: latency
        dict(name="scan_step_one_bf16", kind="scan_step", batch=1, channels=2048, state=16, groups=1, io="bf16"),
        # one token for each running sequence of a server: the states' traffic
        dict(name="scan_step_many_bf16", kind="scan_step", batch=256, channels=4096, state=16, groups=1, io="bf16"),
        # answers: log probability, entropy and alternatives of a few tokens over an odd vocabulary
        dict(name="scores_serve_f16", kind="scores", rows=48, vocab=50001, top=20, io="f16", train=False, masked=True),
        # a training step's loss with an entropy term, and its gradient
        dict(name="scores_train_bf16", kind="scores", rows=8192, vocab=32000, top=0, io="bf16", train=True,
             masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv", "conv_step", "scan", "scan", "scan", "scan_step", "scores", "scores"])
    io = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("conv", "scan"):
        width, state, groups = rng.choice([2, 3, 4, 4]), rng.choice([4, 8, 12, 16, 16, 24, 32, 64]), rng.choice([1, 1, 1, 2, 4])
        most = MOST_CONV if kind == "conv" else MOST_SCAN // state
        train = rng.random() < 0.5
        channels = _log_int(rng, 16, 512) * groups
        if rng.random() < 0.6:
            channels = max(64, channels // 64 * 64)
        most = min(most, MOST_SCAN // state) if train else most
        batch = _log_int(rng, 1, max(1, min(64, most // channels // 16)))
        seq = _log_int(rng, 16, max(16, min(16384, most // channels // batch)))
        c = dict(kind=kind, batch=batch, seq=seq, channels=channels, io=io, train=train, ragged=rng.random() < 0.4,
                 carried=rng.random() < 0.4, layout=rng.choice([0, 1]))
        return dict(c, width=width) if kind == "conv" else dict(c, state=state, groups=groups, gate=rng.random() < 0.7)
    if kind == "conv_step":
        return dict(kind=kind, batch=_log_int(rng, 1, 512), channels=_log_int(rng, 64, 8192), width=rng.choice([2, 3, 4, 4]), io=io)
    if kind == "scan_step":
        state, groups = rng.choice([4, 8, 12, 16, 16, 24, 32, 64]), rng.choice([1, 1, 1, 2, 4])
        channels = _log_int(rng, 16, 2048) * groups
        batch = _log_int(rng, 1, max(1, min(512, MOST_STEP // (channels * state))))
        return dict(kind=kind, batch=batch, channels=channels, state=state, groups=groups, io=io)
    vocab = _log_int(rng, 200, 130000)
    rows = _log_int(rng, 1, max(1, min(8192, MOST_SCORES // vocab // 2)))
    train = rng.random() < 0.5
    return dict(kind=kind, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 8, 20, 32]), io=io, train=train,
                masked=rng.random() < 0.4)


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
    if c["kind"] in ("conv", "conv_step"):
        n, d, k = c["batch"], c["channels"], c["width"]
        s["W"] = uniform(d, k, lo=-1.0, hi=1.0) / math.sqrt(k)
        s["bias"] = uniform(d, lo=-0.5, hi=0.5)
        if c["kind"] == "conv_step":
            # X is a part of a projection's output
            s["X"] = normal(n, 2 * d, dtype=io)[:, :d]
            s["state"] = normal(n, k - 1, d, dtype=io)
            s["state_out"], s["Y"] = torch.empty_like(s["state"]), torch.empty(n, d, device="cuda", dtype=io)
        else:
            lead = (n, c["seq"]) if c["layout"] == 1 else (c["seq"], n)
            s["X"] = normal(*lead, d, dtype=io)
            s["lens"] = _lengths(c, rnd) if c["ragged"] else None
            s["initial_state"] = normal(n, k - 1, d, dtype=io) if c["carried"] else None
            if c["train"]:
                s["dY"] = normal(*lead, d, dtype=io)
                s["d_state"] = normal(n, k - 1, d, dtype=io) if c["carried"] else None
    elif c["kind"] in ("scan", "scan_step"):
        n, d, m, g = c["batch"], c["channels"], c["state"], c["groups"]
        # rates from 1 to the state size, steps from a thousandth to a tenth,
        # as such layers start
        s["A"] = -torch.arange(1, m + 1, device="cuda", dtype=torch.float32) * uniform(d, m, lo=0.7, hi=1.3)
        step = torch.exp(uniform(d, lo=math.log(1e-3), hi=math.log(0.1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1.0 + normal(d, scale=0.1)
        if c["kind"] == "scan_step":
            lead = (n,)
            s["H"] = normal(n, d, m)
            s["H_out"], s["Y"] = torch.empty_like(s["H"]), torch.empty(n, d, device="cuda", dtype=io)
            gate = True
        else:
            lead = (n, c["seq"]) if c["layout"] == 1 else (c["seq"], n)
            s["lens"] = _lengths(c, rnd) if c["ragged"] else None
            s["H"] = normal(n, d, m) if c["carried"] else None
            gate = c["gate"]
        s["X"], s["dt"] = normal(*lead, d, dtype=io), normal(*lead, d, scale=0.5, dtype=io)
        # B and C lie side by side in one projection's output, Z in another's
        bc = normal(*lead, 2, g, m, dtype=io)
        s["B"], s["C"] = bc[..., 0, :, :], bc[..., 1, :, :]
        s["Z"] = normal(*lead, 2 * d, dtype=io)[..., d:] if gate else None
        if c.get("train"):
            s["dY"] = normal(*lead, d, dtype=io)
            s["dY_h"] = normal(n, d, m) if c["carried"] else None
    else:
        r, v = c["rows"], c["vocab"]
        s["logits"] = normal(r, v, scale=2.5, dtype=io)
        s["ids"] = torch.randint(0, v, (r,), generator=rnd, device="cuda", dtype=torch.int32)
        if c["masked"]:
            # tokens that a grammar rules out, by -inf; positions without a token
            s["logits"][torch.rand(r, v, generator=rnd, device="cuda") < 0.3] = float("-inf")
            s["logits"][torch.arange(r, device="cuda"), s["ids"].long()] = 1.0
            if r > 2:
                s["logits"][r // 2] = float("-inf")
                s["ids"][r - 1] = -1
        if c["train"]:
            # weights of a scaled loss, as half precision gradients need
            s["d_logp"], s["d_entropy"] = normal(r), normal(r, scale=0.1)
    if own:
        _handle(s)
    return s


def _handle(s):
    """The plan that a program keeps for a layer."""
    import onnx_recurrent_gb300 as orc
    c = s["case"]
    if c["kind"] != "scores":
        s["plan"] = orc.rnn_ssm_create(c["channels"], state_size=c.get("state", 16), groups=c.get("groups", 1),
                                       conv_width=c.get("width", 4), layout=c.get("layout", 0))
        orc.rnn_ssm_set_io_type(s["plan"], c["io"])


# ----------------------------------------------------------- the plain forms

def _silu(v):
    return v * torch.sigmoid(v)


def _silu_slope(v):
    q = torch.sigmoid(v)
    return q * (1.0 + v * (1.0 - q))


def _valid(lens, n, seq):
    """[batch, seq] truth values: whether a step belongs to its row."""
    t = torch.arange(seq, device="cuda")
    return t[None, :] < (torch.full((n, 1), seq, device="cuda") if lens is None else lens[:, None])


def _conv_plain(s):
    c = s["case"]
    n, d, k, seq, io = c["batch"], c["channels"], c["width"], c["seq"], IO[c["io"]]
    rows = (lambda v: v.float()) if c["layout"] == 1 else (lambda v: v.float().transpose(0, 1))
    back = (lambda v: v.to(io)) if c["layout"] == 1 else (lambda v: v.to(io).transpose(0, 1).contiguous())
    history = torch.zeros(n, k - 1, d, device="cuda") if s["initial_state"] is None else s["initial_state"].float()
    x = torch.cat([history, rows(s["X"])], 1)
    taps = x.unfold(1, k, 1)                                    # [batch, seq, channels, width]
    pre = (taps * s["W"]).sum(-1) + s["bias"]
    valid = _valid(s["lens"], n, seq)[..., None]
    y = _silu(pre) * valid
    lens = torch.full((n,), seq, device="cuda") if s["lens"] is None else s["lens"].long()
    last = (lens[:, None] + torch.arange(k - 1, device="cuda"))[..., None].expand(n, k - 1, d)
    out = {"Y": back(y), "state": x.gather(1, last).to(io)}
    if c["train"]:
        dpre = rows(s["dY"]) * _silu_slope(pre) * valid
        zeros = torch.zeros(n, k - 1, d, device="cuda")
        dx = (torch.cat([zeros, dpre, zeros], 1).unfold(1, k, 1) * s["W"].flip(1)).sum(-1)
        if s["d_state"] is not None:
            dx = dx.scatter_add(1, last, s["d_state"].float())
        out.update(dX=back(dx[:, k - 1:]), dW=(dpre[..., None] * taps).sum((0, 1)), dbias=dpre.sum((0, 1)))
        if s["initial_state"] is not None:
            out["d_initial_state"] = dx[:, :k - 1].to(io)
    return out


def _conv_step_plain(s):
    io = IO[s["case"]["io"]]
    x = torch.cat([s["state"].float(), s["X"].float()[:, None]], 1)
    return {"Y": _silu((x.transpose(1, 2) * s["W"]).sum(-1) + s["bias"]).to(io), "state": x[:, 1:].to(io)}


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _recurrence(a, b):
    """h[:, t] = a[:, t] * h[:, t - 1] + b[:, t] from h[:, -1] = 0, by doubling the span; overwrites both."""
    span, seq = 1, a.shape[1]
    while span < seq:
        b[:, span:] += a[:, span:] * b[:, :-span]
        if 2 * span < seq:
            a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    return b


def _scan_plain(s):
    c = s["case"]
    n, d, m, g, seq, io = c["batch"], c["channels"], c["state"], c["groups"], c["seq"], IO[c["io"]]
    p = d // g
    rows = (lambda v: v.float()) if c["layout"] == 1 else (lambda v: v.float().transpose(0, 1))
    back = (lambda v: v.to(io)) if c["layout"] == 1 else (lambda v: v.to(io).transpose(0, 1).contiguous())
    x, B, C, A = rows(s["X"]), rows(s["B"]), rows(s["C"]), s["A"]
    valid = _valid(s["lens"], n, seq)[..., None]
    v = rows(s["dt"]) + s["dt_bias"]
    dt = _softplus(v) * valid                                   # steps past a row's end leave its state
    spread = lambda w: w[:, :, :, None, :].expand(n, seq, g, p, m).reshape(n, seq, d, m)  # noqa: E731
    a = torch.exp(dt[..., None] * A)
    b = (dt * x)[..., None] * spread(B)
    if s["H"] is not None:
        b[:, 0] += a[:, 0] * s["H"]
    h = _recurrence(a, b)
    y = (h * spread(C)).sum(-1) + s["D"] * x
    z = None if s["Z"] is None else rows(s["Z"])
    out = {"Y": back((y if z is None else y * _silu(z)) * valid), "Y_h": h[:, -1].clone()}
    if c["train"]:
        dy = rows(s["dY"]) * valid
        if z is not None:
            out["dZ"] = back(dy * y * _silu_slope(z))
            dy = dy * _silu(z)
        a = torch.exp(dt[..., None] * A)
        grad = dy[..., None] * spread(C)
        if s["dY_h"] is not None:
            grad[:, -1] += s["dY_h"]
        ahead = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
        grad = _recurrence(ahead, grad.flip(1)).flip(1)         # the loss's slope in h[:, t]
        first = torch.zeros(n, d, m, device="cuda") if s["H"] is None else s["H"]
        if s["H"] is not None:
            out["d_initial_h"] = a[:, 0] * grad[:, 0]
        out["dC"] = back((dy[..., None] * h).view(n, seq, g, p, m).sum(3))
        decayed = a * torch.cat([first[:, None], h[:, :-1]], 1)
        out["dB"] = back(((dt * x)[..., None] * grad).view(n, seq, g, p, m).sum(3))
        driven = (grad * spread(B)).sum(-1)
        decayed *= grad
        out["dA"] = (decayed * dt[..., None]).sum((0, 1))
        ddt = (x * driven + (decayed * A).sum(-1)) * torch.sigmoid(v) * valid
        out.update(dX=back(dt * driven + s["D"] * dy), ddt=back(ddt), ddt_bias=ddt.sum((0, 1)), dD=(dy * x).sum((0, 1)))
    return out


def _scan_step_plain(s):
    c = s["case"]
    n, d, m, g, io = c["batch"], c["channels"], c["state"], c["groups"], IO[c["io"]]
    spread = lambda w: w.float()[:, :, None, :].expand(n, g, d // g, m).reshape(n, d, m)  # noqa: E731
    x, z = s["X"].float(), s["Z"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["H"] + (dt * x)[..., None] * spread(s["B"])
    y = (h * spread(s["C"])).sum(-1) + s["D"] * x
    return {"Y": (y * _silu(z)).to(io), "H": h}


def _ranked(x, top):
    """The `top` largest of each row and their places, ties to the lowest: one whole number per logit that sorts so."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    place = torch.arange(x.shape[1] - 1, -1, -1, device="cuda")
    key = torch.topk(order * (1 << 32) + place, top).values
    return x.shape[1] - 1 - (key & 0xffffffff)


def _scores_plain(s):
    c = s["case"]
    x, ids = s["logits"].float(), s["ids"].long()
    most = x.max(1, keepdim=True).values
    empty = most == float("-inf")                               # nothing is allowed: no probabilities, no gradient
    shifted = torch.exp(x - torch.where(empty, 0.0, most))
    total = shifted.sum(1, keepdim=True)
    lse = most + torch.log(torch.where(empty, 1.0, total))
    p = shifted / torch.where(empty, 1.0, total)
    logp = torch.where(empty, float("-inf"), x - lse)
    some = torch.where(p > 0, p * logp, 0.0)
    entropy = -some.sum(1)
    given = torch.where(ids < 0, 0.0, logp.gather(1, ids.clamp(min=0)[:, None])[:, 0])
    out = {"logp": given, "entropy": entropy}
    if c["top"]:
        at = _ranked(x, c["top"])
        out["top_ids"], out["top_logp"] = at.int(), logp.gather(1, at)
    if c["train"]:
        weight = torch.where(ids < 0, 0.0, s["d_logp"])[:, None]
        grad = -weight * p - s["d_entropy"][:, None] * (some + p * entropy[:, None])
        grad.scatter_add_(1, ids.clamp(min=0)[:, None], torch.where(empty, 0.0, weight))
        out["dlogits"] = grad.to(s["logits"].dtype)
    return out


# ------------------------------------------------------ the package's operators

def _run_own(s):
    import onnx_recurrent_gb300 as orc
    c = s["case"]
    kind = c["kind"]
    if kind == "conv":
        Y, state = orc.ssm_conv(s["plan"], s["X"], s["W"], s["bias"], s["lens"], s["initial_state"])
        out = {"Y": Y, "state": state}
        if c["train"]:
            out.update(orc.ssm_conv_grad(s["plan"], s["dY"], s["X"], s["W"], s["bias"], s["lens"], s["initial_state"],
                                         s["d_state"]))
        return out
    if kind == "conv_step":
        orc.rnn_ssm_conv_step(s["plan"], s["X"], s["W"], s["bias"], s["state"], s["Y"], state_out=s["state_out"])
        return {"Y": s["Y"], "state": s["state_out"]}
    if kind == "scan":
        args = (s["X"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["Z"], s["dt_bias"], s["lens"], s["H"])
        Y, Y_h, saved = orc.ssm_scan(s["plan"], *args, save=c["train"])
        out = {"Y": Y, "Y_h": Y_h}
        if c["train"]:
            out.update(orc.ssm_scan_grad(s["plan"], s["dY"], saved, *args, dY_h=s["dY_h"]))
        return out
    if kind == "scan_step":
        orc.rnn_ssm_scan_step(s["plan"], s["X"], s["dt"], s["A"], s["B"], s["C"], s["H"], s["Y"], s["D"], s["Z"],
                              s["dt_bias"], H_out=s["H_out"])
        return {"Y": s["Y"], "H": s["H_out"]}
    r = orc.scores(s["logits"], s["ids"], top=c["top"])
    out = {"logp": r.logp, "entropy": r.entropy}
    if c["top"]:
        out.update(top_ids=r.top_ids, top_logp=r.top_logp)
    if c["train"]:
        out["dlogits"] = orc.scores_grad(s["logits"], s["ids"], r, s["d_logp"], s["d_entropy"])
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"conv": _conv_plain, "conv_step": _conv_step_plain, "scan": _scan_plain, "scan_step": _scan_step_plain,
            "scores": _scores_plain}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    e = {"f32": 4, "f16": 2, "bf16": 2}[c["io"]]
    kind = c["kind"]
    if kind == "scores":
        n = c["rows"] * c["vocab"]
        per_row = 4 * (3 + 2 * c["top"] + (2 if c["train"] else 0))
        return {"bytes": n * e * (2 if c["train"] else 1) + c["rows"] * per_row, "flops": n * (10 if c["train"] else 5)}
    n, d = c["batch"], c["channels"]
    if kind in ("conv", "conv_step"):
        k = c["width"]
        weights, state = 4 * d * (k + 1), n * (k - 1) * d * e
        if kind == "conv_step":
            return {"bytes": 2 * n * d * e + 2 * state + weights, "flops": n * d * (2 * k + 4)}
        steps = n * c["seq"] * d
        b = 2 * steps * e + state * (2 if c["carried"] else 1) + weights
        f = steps * (2 * k + 4)
        if c["train"]:      # dY read, dX written; the weights' gradients; the carried state's
            b += 2 * steps * e + weights + (2 * state if c["carried"] else 0)
            f += steps * (4 * k + 8)
        return {"bytes": b, "flops": f}
    m, g = c["state"], c["groups"]
    weights, state = 4 * d * (m + 2), 4 * n * d * m
    if kind == "scan_step":
        return {"bytes": 4 * n * d * e + 2 * n * g * m * e + 2 * state + weights, "flops": n * d * (8 * m + 12)}
    steps, gate = n * c["seq"], int(c["gate"])
    b = steps * (d * (3 + gate) + 2 * g * m) * e + state * (2 if c["carried"] else 1) + weights
    f = steps * d * (8 * m + 12)
    if c["train"]:          # dY read; dX, ddt, dZ, dB, dC written; the weights' gradients; the carried state's
        b += steps * (d * (3 + gate) + 2 * g * m) * e + weights + (2 * state if c["carried"] else 0)
        f += steps * d * (18 * m + 20)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------- in 64 bits

def _exact_conv(s, c):
    n, d, k, seq = c["batch"], c["channels"], c["width"], c["seq"]
    rows = (lambda v: v) if c["layout"] == 1 else (lambda v: v.transpose(0, 1))
    W, X = s["W"].double(), rows(s["X"]).double()
    hist = s["initial_state"].double() if c["carried"] else torch.zeros(n, k - 1, d, device="cuda", dtype=torch.float64)
    lens = s["lens"].tolist() if c["ragged"] else [seq] * n
    Y, state = torch.zeros_like(X), torch.empty_like(hist)
    grads = {q: torch.zeros_like(v) for q, v in (("dX", X), ("dW", W), ("dbias", s["bias"].double()), ("d_initial_state", hist))}
    for i, ln in enumerate(lens):                   # one row of the batch at a time
        line = torch.cat([hist[i], X[i, :ln]])
        state[i] = line[ln:]
        if c["train"]:
            dline = torch.zeros_like(line)
            if s["d_state"] is not None:
                dline[ln:] += s["d_state"][i].double()
        if ln:
            pre = s["bias"].double().expand(ln, d).clone()
            for j in range(k):
                pre += line[j:j + ln] * W[:, j]
            q = 1.0 / (1.0 + torch.exp(-pre))
            Y[i, :ln] = pre * q
            if c["train"]:
                dpre = rows(s["dY"])[i, :ln].double() * (q + pre * q * (1.0 - q))
                for j in range(k):
                    dline[j:j + ln] += dpre * W[:, j]
                    grads["dW"][:, j] += (dpre * line[j:j + ln]).sum(0)
                grads["dbias"] += dpre.sum(0)
        if c["train"]:
            grads["d_initial_state"][i], grads["dX"][i, :ln] = dline[:k - 1], dline[k - 1:]
    out = {"Y": rows(Y), "state": state}
    if c["train"]:
        grads["dX"] = rows(grads["dX"])
        if not c["carried"]:
            del grads["d_initial_state"]
        out.update(grads)
    return out


def _exact_scan(s, c):
    n, d, m, g, seq = c["batch"], c["channels"], c["state"], c["groups"], c["seq"]
    step_of = (lambda v, t: v[:, t].double()) if c["layout"] == 1 else (lambda v, t: v[t].double())
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    h = s["H"].double() if s["H"] is not None else torch.zeros(n, d, m, device="cuda", dtype=torch.float64)
    lens = s["lens"] if s["lens"] is not None else torch.full((n,), seq, device="cuda", dtype=torch.int32)
    wide = lambda w: w.repeat_interleave(d // g, 1)  # noqa: E731
    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    Y, kept = [], []
    for t in range(seq):                             # the definition, one step after another
        live = (lens > t)[:, None]
        x, v = step_of(s["X"], t), step_of(s["dt"], t) + bias
        dt = torch.where(live, torch.logaddexp(v, zero), zero)
        if c["train"]:
            kept.append(h)
        h = torch.exp(dt[..., None] * A) * h + (dt * x)[..., None] * wide(step_of(s["B"], t))
        y = (h * wide(step_of(s["C"], t))).sum(-1) + D * x
        if s["Z"] is not None:
            z = step_of(s["Z"], t)
            y = y * z / (1.0 + torch.exp(-z))
        Y.append(torch.where(live, y, zero))
    time = 1 if c["layout"] == 1 else 0
    out = {"Y": torch.stack(Y, time), "Y_h": h}
    if not c["train"]:
        return out
    ahead = s["dY_h"].double() if s["dY_h"] is not None else torch.zeros_like(h)
    seqs = {q: [None] * seq for q in ("dX", "ddt", "dZ", "dB", "dC")}
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(bias)
    for t in range(seq - 1, -1, -1):
        live = (lens > t)[:, None]
        x, v = step_of(s["X"], t), step_of(s["dt"], t) + bias
        B, C = wide(step_of(s["B"], t)), wide(step_of(s["C"], t))
        dt = torch.where(live, torch.logaddexp(v, zero), zero)
        decay = torch.exp(dt[..., None] * A)
        past = decay * kept[t]
        now = past + (dt * x)[..., None] * B
        dy = torch.where(live, step_of(s["dY"], t), zero)
        if s["Z"] is not None:
            z = step_of(s["Z"], t)
            q = 1.0 / (1.0 + torch.exp(-z))
            seqs["dZ"][t] = dy * ((now * C).sum(-1) + D * x) * (q + z * q * (1.0 - q))
            dy = dy * z * q
        slope = ahead + dy[..., None] * C
        dD += (dy * x).sum(0)
        dA += (slope * past * dt[..., None]).sum(0)
        ddt = torch.where(live, ((slope * B).sum(-1) * x + (slope * past * A).sum(-1)) / (1.0 + torch.exp(-v)), zero)
        dbias += ddt.sum(0)
        seqs["ddt"][t], seqs["dX"][t] = ddt, dt * (slope * B).sum(-1) + D * dy
        seqs["dB"][t] = (slope * (dt * x)[..., None]).reshape(n, g, d // g, m).sum(2)
        seqs["dC"][t] = (dy[..., None] * now).reshape(n, g, d // g, m).sum(2)
        ahead = decay * slope
        kept[t] = None
    out.update({q: torch.stack(w, time) for q, w in seqs.items() if w[0] is not None})
    out.update(dA=dA, dD=dD, ddt_bias=dbias)
    if s["H"] is not None:
        out["d_initial_h"] = ahead
    return out


def _exact_scores(s, c):
    parts = []
    for lo in range(0, c["rows"], 1024):
        x, ids = s["logits"][lo:lo + 1024].double(), s["ids"][lo:lo + 1024].long()
        logp = torch.log_softmax(x, 1)
        logp[torch.isneginf(x).all(1)] = float("-inf")
        p = torch.exp(logp)
        plogp = torch.nan_to_num(p * logp, nan=0.0)
        hit = torch.arange(c["vocab"], device="cuda") == ids[:, None]
        q = {"logp": torch.where(hit, logp, 0.0).sum(1), "entropy": -plogp.sum(1)}
        if c["top"]:
            at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
            q["top_ids"], q["top_logp"] = at.int(), torch.gather(logp, 1, at)
        if c["train"]:
            w = s["d_logp"][lo:lo + 1024].double()[:, None] * (ids >= 0)[:, None]
            e = s["d_entropy"][lo:lo + 1024].double()[:, None]
            some = ~torch.isneginf(x).all(1, keepdim=True)
            q["dlogits"] = torch.where(some, w * hit, 0.0) - w * p - e * (plogp + p * q["entropy"][:, None])
        parts.append(q)
    return {q: torch.cat([v[q] for v in parts]) for q in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "conv":
        return _exact_conv(s, c)
    if c["kind"] == "scan":
        return _exact_scan(s, c)
    if c["kind"] == "scores":
        return _exact_scores(s, c)
    one = dict(s, lens=None)
    lift = lambda v: None if v is None else v[None]  # noqa: E731
    if c["kind"] == "conv_step":                     # a sequence of one step with a carried state
        one.update(X=lift(s["X"]), initial_state=s["state"])
        return _exact_conv(one, dict(c, seq=1, layout=0, train=False, ragged=False, carried=True))
    one.update({q: lift(s[q]) for q in ("X", "dt", "B", "C", "Z")})
    got = _exact_scan(one, dict(c, seq=1, layout=0, train=False))
    return {"Y": got["Y"][0], "H": got["Y_h"]}
