"""What the gated delta rule's outputs err by in plain fp32, group by group, and whether other results err no more than some
times that.

A sum's error goes with its terms, not with what they cancel to, so it is that of the same formulas in fp32: of the
steps one after another (dg as its derivative), and of chunks of 64 steps as products (dg summed from pairs of steps), whichever errs
more.  Each is taken with its keys and values in several orders, and the root mean square is a group's: a
group of eight numbers alone is right by chance too often."""
import torch

import delta_ref64 as ref

U = 2.0 ** -24
C = 64


def groups(name, t, size):
    """[N, S, heads, ...] in groups of `size` steps, a row and a head each; a state is a group a row and head."""
    if name in ("state", "d_initial_state"):
        return t.flatten(0, 1).flatten(1)
    N, S, H = t.shape[:3]
    pad = -S % size
    t = torch.cat([t, t.new_zeros(N, pad, *t.shape[2:])], 1).unflatten(1, (-1, size)).movedim(3, 1)
    return t.flatten(0, 2).flatten(1)


def steps(Q, K, V, g, beta, state, dY, d_state, scale):
    """Outputs and gradients in the inputs' type, step by step."""
    Y, end = ref.delta(Q, K, V, g, beta, None, state, scale)
    return dict(Y=Y, state=end, **ref.delta_grad(dY, d_state, Q, K, V, g, beta, None, state, scale))


def chunks(Q, K, V, g, beta, state, dY, d_state, scale):
    """The same by chunks (sums of log decays in 64 bits)."""
    N, S, HK, DK = Q.shape
    H, dt, n = V.shape[2], Q.dtype, -(-S // C)

    def cut(v, rep=1):      # [N, head, chunk, step, ...]
        v = torch.cat([v, v.new_zeros(N, n * C - S, *v.shape[2:])], 1).unflatten(1, (n, C)).movedim(3, 1)
        return v.repeat_interleave(rep, 1) if rep > 1 else v

    t_ = lambda v: v.transpose(-1, -2)  # noqa: E731
    back = lambda v: torch.stack(v, 2).movedim(1, 3).flatten(1, 2)[:, :S]  # noqa: E731
    before = lambda v: torch.cat([v.new_zeros(*v.shape[:-1], 1), v.cumsum(-1)[..., :-1]], -1)  # noqa: E731
    q, k, v, b, dy = cut(Q, H // HK), cut(K, H // HK), cut(V), cut(beta)[..., None], scale * cut(dY)
    G = cut(g).double().cumsum(-1)
    at = torch.arange(C)
    below, diag = at[:, None] > at[None], at[:, None] >= at[None]
    D = torch.where(diag, torch.exp(torch.where(diag, G[..., :, None] - G[..., None, :], 0.0)), 0.0).to(dt)
    first, last = torch.exp(G).to(dt)[..., None], torch.exp(G[..., -1:] - G).to(dt)[..., None]
    whole = first[..., -1, :]
    kk, qk = k @ t_(k), q @ t_(k)
    A = torch.where(below, b * D * kk, 0.0)
    T = torch.linalg.solve_triangular(torch.eye(C, dtype=dt) + A, torch.eye(C, dtype=dt).expand_as(A), upper=False)
    P = D * qk
    starts, us, Y, st = [], [], [], state
    for j in range(n):
        u = T[:, :, j] @ (b[:, :, j] * (v[:, :, j] - first[:, :, j] * (k[:, :, j] @ st)))
        starts.append(st)
        us.append(u)
        Y.append(scale * (first[:, :, j] * (q[:, :, j] @ st) + P[:, :, j] @ u))
        st = whole[:, :, j, None] * st + t_(last[:, :, j] * k[:, :, j]) @ u
    out, parts, ahead = dict(Y=back(Y), state=st), {w: [None] * n for w in ("dQ", "dK", "dV", "dg", "dbeta")}, d_state
    for j in range(n - 1, -1, -1):
        kj, qj, bj, u, s0, f, l, w = (x[:, :, j] if isinstance(x, torch.Tensor) else x[j] for x in (k, q, b, us, starts, first, last, whole))
        dr = t_(T[:, :, j]) @ (t_(P[:, :, j]) @ dy[:, :, j] + l * (kj @ ahead))
        dA, dP = torch.where(below, -(dr @ t_(u)), 0.0), torch.where(diag, dy[:, :, j] @ t_(u), 0.0)
        EA, EP = bj * D[:, :, j] * dA, D[:, :, j] * dP
        x1, x2, x3 = dy[:, :, j] @ t_(s0), dr @ t_(s0), u @ t_(ahead)
        kx2 = f[..., 0] * (kj * x2).sum(-1)
        parts["dQ"][j] = f * x1 + EP @ kj
        parts["dK"][j] = (EA + t_(EA)) @ kj + t_(EP) @ qj - bj * f * x2 + l * x3
        parts["dV"][j] = bj * dr
        parts["dbeta"][j] = (dr * v[:, :, j]).sum(-1) - kx2 + (dA * D[:, :, j] * kk[:, :, j]).sum(-1)
        pairs = torch.where(diag, before(EA * kk[:, :, j] + EP * qk[:, :, j]), 0.0).sum(-2)
        states = f[..., 0] * (qj * x1).sum(-1) - bj[..., 0] * kx2
        parts["dg"][j] = pairs + states.flip(-1).cumsum(-1).flip(-1) + before(l[..., 0] * (kj * x3).sum(-1)) + w * (ahead * s0).sum((-1, -2))[..., None]
        ahead = w[..., None] * ahead + t_(qj) @ (f * dy[:, :, j]) - t_(kj) @ (bj * f * dr)
    for name, p in parts.items():
        p = torch.stack(p, 2)
        p = p.unflatten(1, (HK, H // HK)).sum(2) if name in ("dQ", "dK") else p
        out[name] = p.movedim(1, 3).flatten(1, 2)[:, :S]
    out["d_initial_state"] = ahead
    return out


def plain_errors(ins, want, size, orders=4, forms=(steps, chunks)):
    """Of each output, the error of its groups in norm; `ins` are the eight tensors of `steps`, and the scale."""
    *tensors, scale = ins
    total = {}
    for seed in range(orders):
        g = torch.Generator().manual_seed(seed)
        keys, values = torch.randperm(tensors[0].shape[3], generator=g), torch.randperm(tensors[2].shape[3], generator=g)
        Q, K, V, decay, beta, state, dY, d_state = (t.float() for t in tensors)
        turned = (Q[..., keys], K[..., keys], V[..., values], decay, beta, state[..., keys, :][..., values], dY[..., values],
                  d_state[..., keys, :][..., values], scale)
        for f in forms:
            for name, t in f(*turned).items():
                w = want[name]
                if name in ("dQ", "dK"):
                    w = w[..., keys]
                elif name in ("Y", "dV"):
                    w = w[..., values]
                elif name in ("state", "d_initial_state"):
                    w = w[..., keys, :][..., values]
                e = (groups(name, t.double(), size) - groups(name, w, size)).square().sum(1) / orders
                total[f, name] = total.get((f, name), 0) + e
    return {name: torch.stack([total[f, name] for f in forms]).amax(0).sqrt() for name in want}


def like_plain(name, got, want, plain, io_u=0.0, floor=0.0):
    """Groups (rows) of got err at most 4 times as much as plain's, and 8 u and the outputs' rounding io_u of their norm, and
    `floor` of the largest group's."""
    err, size = (got - want).norm(dim=1), want.norm(dim=1)
    tol = 4 * plain + (8 * U + io_u) * size + floor * size.max() + 1e-37
    bad = ~(err <= tol)
    at = int((err / tol).argmax())
    assert not bad.any(), f"{name}: {int(bad.sum())} of {len(err)} groups, the worst ({at}) off by {float(err[at] / tol[at]):.2f} of what it may be, " \
                          f"{float(err[at] / size[at].clamp_min(1e-37)):.2e} of its norm"
