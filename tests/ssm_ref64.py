"""The state space and score operators in 64 bits, straight from their
formulas, one step after another, on the CPU; and bounds on what fp32
arithmetic may differ from them.

Tensors are float64 [N, S, ...] here (layout 1), whatever the GPU run used.

Bounds.  With `magnitude=True` the gradient and forward functions take every
product of a sum in absolute value, which bounds the sum of the absolute
terms of each output.  A term of an output passes through at most S steps of a
recurrence; a step rounds at most 4 times and takes one exponential, whose
argument delta * A carries 3 roundings of its own (the product, and delta's
own relative error of at most 8 roundings counted in the caller's constant),
so each step costs at most (8 + 4 |delta A|) u relative to the term, with
u = 2^-24; a sum of n terms adds n u; gates, softplus and their slopes take at
most 32 roundings together.  `steps_bound` gives that number of u.  An output
rounded to 16 bits adds half a unit in its last place."""
import torch

U = 2.0 ** -24
IO_U = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}     # half a unit in the last place, relative
IO_TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}        # half the smallest subnormal


def steps_bound(S, terms, rate=0.0):
    return ((8 + 4 * rate) * S + terms + 32) * U


def close(got, ref, bound, io, what):
    """|got - ref| <= bound (fp32 arithmetic) + the rounding to io."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = bound + (ref.abs() + bound) * IO_U[io] + IO_TINY[io] + 1e-38
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}{list(i)}: got {got[i]}, expected {ref[i]} +- {tol[i] if tol.dim() else tol}; "
                             f"{int(bad.sum())} of {bad.numel()} outside")


def silu(v):
    return v / (1 + torch.exp(-v))


def silu_slope(v):
    s = 1 / (1 + torch.exp(-v))
    return s + v * s * (1 - s)


def _live(lens, N, S):
    lens = torch.full((N,), S) if lens is None else lens.long()
    return torch.arange(S)[None, :] < lens[:, None], lens


def conv(X, W, bias, lens, h0, act):
    """(Y, final state, pre)."""
    N, S, D = X.shape
    K = W.shape[1]
    live, lens = _live(lens, N, S)
    hist = torch.zeros(N, K - 1, D, dtype=X.dtype) if h0 is None else h0
    line = torch.cat([hist, X], 1)
    pre = torch.zeros_like(X) + (0 if bias is None else bias)
    for k in range(K):
        pre = pre + line[:, k:k + S] * W[:, k]
    Y = torch.where(live[..., None], silu(pre) if act else pre, torch.zeros_like(pre))
    hT = torch.stack([line[n, lens[n]:lens[n] + K - 1] for n in range(N)])
    return Y, hT, pre


def conv_grad(dY, dhT, X, W, bias, lens, h0, act, magnitude=False):
    N, S, D = X.shape
    K = W.shape[1]
    live, lens = _live(lens, N, S)
    pre = conv(X, W, bias, lens, h0, act)[2]
    hist = torch.zeros(N, K - 1, D, dtype=X.dtype) if h0 is None else h0
    ab = torch.abs if magnitude else (lambda v: v)
    slope = ab(silu_slope(pre)) if act else torch.ones_like(pre)
    if magnitude and act:      # the slope's own error follows that of pre, by at most its second slope (< 0.5)
        mag = torch.zeros_like(X) + (0 if bias is None else bias.abs())
        for k in range(K):
            mag = mag + torch.cat([hist, X], 1)[:, k:k + S].abs() * W[:, k].abs()
        slope = slope + mag
    e = torch.where(live[..., None], ab(dY) * slope, torch.zeros_like(dY))
    line, w = ab(torch.cat([hist, X], 1)), ab(W)
    dline = torch.zeros_like(line)
    dW = torch.zeros_like(W)
    for k in range(K):
        dline[:, k:k + S] += e * w[:, k]
        dW[:, k] = (e * line[:, k:k + S]).sum((0, 1))
    if dhT is not None:
        for n in range(N):
            dline[n, lens[n]:lens[n] + K - 1] += ab(dhT[n])
    return dict(dX=dline[:, K - 1:], dW=dW, dbias=e.sum((0, 1)), d_initial_state=dline[:, :K - 1])


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def scan(X, dt, A, B, C, D, Z, dt_bias, lens, h0, soft=True, magnitude=False):
    """(Y, Y_h, y before the gate, h before every step, delta, v)."""
    N, S, Dc = X.shape
    G, M = B.shape[2:]
    live, lens = _live(lens, N, S)
    ab = torch.abs if magnitude else (lambda v: v)
    wide = lambda v: ab(v).repeat_interleave(Dc // G, 1)  # noqa: E731
    v = dt if dt_bias is None else dt + dt_bias
    delta = torch.where(live[..., None], softplus(v) if soft else v, torch.zeros_like(v))
    h = torch.zeros(N, Dc, M, dtype=X.dtype) if h0 is None else ab(h0)
    ys, hs = [], []
    for t in range(S):
        hs.append(h)
        h = torch.exp(delta[:, t, :, None] * A) * h + ab(delta[:, t] * X[:, t])[..., None] * wide(B[:, t])
        y = (h * wide(C[:, t])).sum(-1)
        ys.append(y if D is None else y + ab(D * X[:, t]))
    y = torch.stack(ys, 1)
    Y = y if Z is None else y * ab(silu(Z))
    return torch.where(live[..., None], Y, torch.zeros_like(Y)), h, y, hs, delta, v


def scan_grad(dY, dYh, X, dt, A, B, C, D, Z, dt_bias, lens, h0, soft=True, magnitude=False):
    N, S, Dc = X.shape
    G, M = B.shape[2:]
    live, lens = _live(lens, N, S)
    _, _, y, hs, delta, v = scan(X, dt, A, B, C, D, Z, dt_bias, lens, h0, soft, magnitude)
    ab = torch.abs if magnitude else (lambda w: w)
    wide = lambda w: ab(w).repeat_interleave(Dc // G, 1)  # noqa: E731
    fold = lambda w: w.reshape(N, G, Dc // G, M).sum(2)  # noqa: E731
    skip = torch.zeros(Dc, dtype=X.dtype) if D is None else ab(D)
    X, dY, As = ab(X), torch.where(live[..., None], ab(dY), torch.zeros_like(dY)), ab(A)
    dm = ab(delta)
    out = {}
    e = dY
    if Z is not None:
        out["dZ"] = dY * y * ab(silu_slope(Z))
        e = dY * ab(silu(Z))
    q = torch.sigmoid(v) if soft else torch.ones_like(v)
    ahead = torch.zeros(N, Dc, M, dtype=X.dtype) if dYh is None else ab(dYh)
    rows = {k: [None] * S for k in ("dX", "ddt", "dB", "dC")}
    dA, dD, db = torch.zeros_like(A), torch.zeros_like(skip), torch.zeros_like(skip)
    for t in range(S - 1, -1, -1):
        a = torch.exp(delta[:, t, :, None] * A)
        past = a * hs[t]
        now = past + (dm[:, t] * X[:, t])[..., None] * wide(B[:, t])
        g = wide(C[:, t]) * e[:, t, :, None] + ahead
        driven, decayed = (g * wide(B[:, t])).sum(-1), (g * past * As).sum(-1)
        rows["dX"][t] = dm[:, t] * driven + skip * e[:, t]
        ddt = torch.where(live[:, t, None], (X[:, t] * driven + decayed) * q[:, t], torch.zeros_like(driven))
        rows["ddt"][t] = ddt
        rows["dB"][t] = fold((dm[:, t] * X[:, t])[..., None] * g)
        rows["dC"][t] = fold(e[:, t, :, None] * now)
        dA += (dm[:, t, :, None] * g * past).sum(0)
        dD += (e[:, t] * X[:, t]).sum(0)
        db += ddt.sum(0)
        ahead = a * g
    out.update({k: torch.stack(w, 1) for k, w in rows.items()})
    out.update(dA=dA, dD=dD, ddt_bias=db, d_initial_h=ahead)
    return out


def scores(x, ids, top):
    """dict of logp, entropy, lse, top_ids, top_logp for float64 rows, by the rules of the empty and the bad row."""
    rows, V = x.shape
    out = dict(logp=torch.zeros(rows, dtype=x.dtype), entropy=torch.zeros(rows, dtype=x.dtype),
               lse=torch.zeros(rows, dtype=x.dtype), top_ids=torch.zeros(rows, top, dtype=torch.int32),
               top_logp=torch.zeros(rows, top, dtype=x.dtype))
    inf, nan = float("inf"), float("nan")
    for r in range(rows):
        row = x[r]
        if torch.isnan(row).any() or (row == inf).any():
            lse, ent, logp = nan, nan, torch.full_like(row, nan)
        elif (row == -inf).all():
            lse, ent, logp = -inf, 0.0, torch.full_like(row, -inf)
        else:
            m = row.max()
            lse = m + torch.log(torch.exp(row - m).sum())
            logp = row - lse
            p = torch.exp(logp)
            ent = -(p[p > 0] * logp[p > 0]).sum()
        out["lse"][r], out["entropy"][r] = lse, ent
        if ids is not None:
            i = int(ids[r])
            out["logp"][r] = 0.0 if i < 0 else nan if i >= V else logp[i]
        order = sorted(range(V), key=lambda i: (0, 0, i) if row[i] != row[i] else (1, -float(row[i]), i))[:top]
        out["top_ids"][r] = torch.tensor(order, dtype=torch.int32)
        out["top_logp"][r] = logp[order]
    return out


def scores_grad(x, ids, ref, d_logp, d_entropy, d_top):
    g = torch.zeros_like(x)
    for r in range(x.shape[0]):
        lse = ref["lse"][r]
        if lse == float("-inf"):
            continue
        p = torch.exp(x[r] - lse)
        w = 0.0
        if d_logp is not None and int(ids[r]) >= 0:
            w = w + d_logp[r]
            g[r, int(ids[r])] += d_logp[r]
        if d_top is not None:
            w = w + d_top[r].sum()
            g[r].index_add_(0, ref["top_ids"][r].long(), d_top[r])
        g[r] -= w * p
        if d_entropy is not None:
            g[r] -= d_entropy[r] * torch.where(p > 0, p * (x[r] - lse + ref["entropy"][r]), torch.zeros_like(p))
    return g
