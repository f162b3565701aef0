"""The gated delta rule, layer normalisation and a step of beam search in 64
bits, straight from their formulas, on the CPU; and what 32-bit arithmetic may
differ from them.

Tensors are [N, S, ...] here (layout 1), whatever the GPU run used.

Bounds of the delta rule.  A step's rounding errors reach later states through products of
a (1 - b k k^T), whose norm is at most 1 for keys of length at most 1, betas in [0, 1]
and g <= 0 (all tests have those): they do not grow, they add up.  A step's outputs and state
are sums of at most DK + 2 * 64 products, whose operands' sizes are at most that of the largest
value that the run meets, `size`.  Sums of n products of rounded factors err by at most n u, so
after S steps the error is at most  S (DK + 128) u size  (`worst`).  Errors of either
sign add up as the root of their number does, which the norms are held to:
4 sqrt(S (DK + 128)) u  relative (`norm`; the factor 4 for sums whose terms cancel).  u is 2^-24 in 32-bit
arithmetic.  An output in 16 bits adds half a unit in its last place."""
import torch

U = 2.0 ** -24
IO_U = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
IO_TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def delta(Q, K, V, g, beta, lens, state, scale):
    """(Y, final state); Q, K [N, S, HK, DK], V [N, S, H, DV], g, beta [N, S, H], state [N, H, DK, DV] or None."""
    N, S, HK, DK = Q.shape
    H, DV = V.shape[2:]
    st = torch.zeros(N, H, DK, DV, dtype=Q.dtype) if state is None else state
    Y = []
    for t in range(S):
        q, k = Q[:, t].repeat_interleave(H // HK, 1), K[:, t].repeat_interleave(H // HK, 1)
        decayed = torch.exp(g[:, t])[..., None, None] * st
        u = beta[:, t, :, None] * (V[:, t] - torch.einsum("nhk,nhkv->nhv", k, decayed))
        new = decayed + k[..., None] * u[..., None, :]
        y = scale * torch.einsum("nhk,nhkv->nhv", q, new)
        if lens is not None:
            live = (lens > t)[:, None, None]
            new, y = torch.where(live[..., None], new, st), torch.where(live, y, torch.zeros_like(y))
        st = new
        Y.append(y)
    return torch.stack(Y, 1) if S else V.new_zeros(N, 0, H, DV), st


def delta_grad(dY, d_state, Q, K, V, g, beta, lens, state, scale):
    """Gradients of sum(Y dY) + sum(final state d_state), as a dict."""
    ins = [t.detach().clone().requires_grad_() for t in (Q, K, V, g, beta)]
    st = None if state is None else state.detach().clone().requires_grad_()
    Y, end = delta(*ins, lens, st, scale)
    loss = (Y * dY).sum() + (0 if d_state is None else (end * d_state).sum())
    leaves = ins + ([st] if st is not None else [])
    out = torch.autograd.grad(loss, leaves, allow_unused=True)
    names = ["dQ", "dK", "dV", "dg", "dbeta", "d_initial_state"]
    return {n: (torch.zeros_like(x) if o is None else o) for n, o, x in zip(names, out, leaves)}


def close(got, ref, steps, terms, io, what, u=U, size=None):
    """got against ref: every value within `worst`, and the whole within `norm` (both above) plus the rounding to io."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert bool(got.isfinite().all()), what
    size = max(float(ref.abs().max()), 0.0 if size is None else size)
    worst = max(steps, 1) * terms * u * size
    tol = worst + (ref.abs() + worst) * IO_U[io] + IO_TINY[io] + 1e-38
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, the first at {bad.nonzero()[0].tolist()}"
    norm = 4 * (max(steps, 1) * terms) ** 0.5 * u + IO_U[io]
    err = float((got - ref).norm())
    most = norm * max(float(ref.norm()), size) + IO_TINY[io] * ref.numel() ** 0.5 + 1e-38
    assert err <= most, f"{what}: off by {err} in norm, at most {most}"


def norm(X, W, bias, eps):
    mean = X.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((X - mean) ** 2).mean(-1, keepdim=True) + eps)
    Y = (X - mean) * rstd
    return (Y if W is None else Y * W) + (0 if bias is None else bias), mean[..., 0], rstd[..., 0]


def beam(logits, scores, finished, end):
    """(parents, ids, scores, finished) of a step; logits [items, B, V] in 64 bits."""
    items, B, V = logits.shape
    out = [[], [], [], []]
    for i in range(items):
        cand = []
        for b in range(B):
            s = float(scores[i, b])
            done = finished is not None and bool(finished[i, b])
            lp = torch.full((V,), float("-inf"), dtype=torch.float64)
            lse = torch.logsumexp(logits[i, b], 0)
            if not abs(s) < float("inf"):
                pass
            elif done:
                lp[end] = s
            elif bool(lse.isfinite()):
                lp = s + torch.log_softmax(logits[i, b], 0)         # (logits - lse loses log V where all are -3e38)
            cand.append(lp)
        total, order = torch.sort(torch.cat(cand), descending=True, stable=True)
        parent, token = order[:B] // V, order[:B] % V
        out[0].append(parent)
        out[1].append(token)
        out[2].append(total[:B])
        was = torch.zeros(B, dtype=torch.bool) if finished is None else finished[i]
        out[3].append(was[parent] | (token == end))
    return [torch.stack(o) for o in out]
