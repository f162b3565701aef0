"""A small recurrent language model on the state space operators.

    python examples/ssm_language_model.py [--steps 60] [--tokens 48] [--io bf16] [--layers scan,scan] [--beams 0]

Two layers of normalisation -> projection -> causal convolution -> selective
scan -> projection (with --layers delta: the gated delta rule in the scan's and
the convolution's place) learn the sentences of a small grammar (bracketed words
whose brackets close in order).  Training takes whole sentences (the operators
and the scores with their gradients, an entropy bonus in the loss); generation
reads a prompt with the same operators and then continues it a token at a time
from the layers' states, printing each token's log probability and the
alternatives that the model saw; with --beams it also searches for likely
continuations, the layers' states following the beams.  The matrix products are
torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import onnx_recurrent_gb300 as orc  # noqa: E402
from onnx_recurrent_gb300 import autograd  # noqa: E402

WORDS = ["<s>", "(", ")", "[", "]", "a", "b", "c", "."]
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def sentence(rng, length):
    """Token ids of a sentence: brackets nest and close in order, a full stop once all are closed."""
    out, open_ = [0], []
    while len(out) < length:
        r = float(torch.rand((), generator=rng))
        if open_ and (r < 0.3 or len(open_) > 3):
            out.append(open_.pop())
        elif r < 0.55:
            kind = 1 if float(torch.rand((), generator=rng)) < 0.5 else 3
            out.append(kind)
            open_.append(kind + 1)
        elif not open_ and r > 0.9:
            out.append(8)
        else:
            out.append(5 + int(torch.randint(0, 3, (), generator=rng)))
    return out


class Norm(torch.nn.Module):
    """Layer normalisation of rows in the model's own type (fp32)."""

    def __init__(self, width):
        super().__init__()
        self.plan = orc.rnn_norm_create(width)
        self.weight = torch.nn.Parameter(torch.ones(width))
        self.bias = torch.nn.Parameter(torch.zeros(width))

    def forward(self, h):
        return autograd.layer_norm(self.plan, h, self.weight, self.bias)


class Layer(torch.nn.Module):
    def __init__(self, width, inner, state, io):
        super().__init__()
        self.plan = orc.rnn_ssm_create(inner, state_size=state, groups=1, conv_width=4, layout=1)
        orc.rnn_ssm_set_io_type(self.plan, io)
        self.inner, self.state = inner, state
        self.norm = Norm(width)
        self.into = torch.nn.Linear(width, 2 * inner, bias=False)
        self.to_bc = torch.nn.Linear(inner, 2 * state, bias=False)
        self.to_dt = torch.nn.Linear(inner, inner, bias=False)
        self.out = torch.nn.Linear(inner, width, bias=False)
        self.conv_w = torch.nn.Parameter(torch.randn(inner, 4) * 0.3)
        self.conv_b = torch.nn.Parameter(torch.zeros(inner))
        self.a_log = torch.nn.Parameter(torch.log(torch.arange(1, state + 1.0)).repeat(inner, 1))
        self.skip = torch.nn.Parameter(torch.ones(inner))
        self.dt_bias = torch.nn.Parameter(torch.full((inner,), -3.0))

    def project(self, u):
        """dt, B and C of convolved inputs."""
        bc = self.to_bc(u).unflatten(-1, (2, 1, self.state))
        return self.to_dt(u), bc[..., 0, :, :], bc[..., 1, :, :]

    def forward(self, h, states=None):
        """h [batch, seq, width]; states of an earlier part continue it."""
        dtype = self.plan.dtype
        xz = self.into(self.norm(h)).to(dtype)
        x, z = xz.split(self.inner, -1)
        conv0, scan0 = states or (None, None)
        u, conv = autograd.conv(self.plan, x, self.conv_w, self.conv_b, None, conv0)
        dt, B, C = (t.to(dtype) for t in self.project(u.to(h.dtype)))
        y, scan = autograd.scan(self.plan, u, dt, -torch.exp(self.a_log), B, C, self.skip, z, self.dt_bias, None, scan0)
        return h + self.out(y.to(h.dtype)), (conv, scan)

    def step(self, h, states):
        """One token: h [batch, width]; the states are updated in place."""
        dtype = self.plan.dtype
        x, z = self.into(self.norm(h)).to(dtype).split(self.inner, -1)
        u, y = torch.empty_like(x, memory_format=torch.contiguous_format), torch.empty_like(x, memory_format=torch.contiguous_format)
        orc.rnn_ssm_conv_step(self.plan, x, self.conv_w, self.conv_b, states[0], u)
        dt, B, C = (t.to(dtype) for t in self.project(u.to(h.dtype)))
        orc.rnn_ssm_scan_step(self.plan, u, dt, -torch.exp(self.a_log), B, C, states[1], y, self.skip, z, self.dt_bias)
        return h + self.out(y.to(h.dtype))


class DeltaLayer(torch.nn.Module):
    """Heads of 32 values, two to a query and key head of 16."""

    def __init__(self, width, inner, io):
        super().__init__()
        self.heads, self.key_heads, self.key, self.value = inner // 32, max(inner // 64, 1), 16, 32
        self.plan = orc.rnn_delta_create(self.heads, self.key, self.value, self.key_heads, layout=1)
        orc.rnn_delta_set_io_type(self.plan, io)
        self.norm = Norm(width)
        self.sizes = (self.key_heads * self.key, self.key_heads * self.key, self.heads * self.value)
        self.into = torch.nn.Linear(width, sum(self.sizes), bias=False)
        self.to_gates = torch.nn.Linear(width, 2 * self.heads)
        self.out = torch.nn.Linear(self.heads * self.value, width, bias=False)

    def project(self, h):
        """Q, K, V, g and beta of inputs [..., width]."""
        h, dtype = self.norm(h), self.plan.dtype
        q, k, v = self.into(h).split(self.sizes, -1)
        q, k = (torch.nn.functional.normalize(t.unflatten(-1, (self.key_heads, self.key)), dim=-1) for t in (q, k))
        a, b = self.to_gates(h).split(self.heads, -1)
        return (q.to(dtype), k.to(dtype), v.unflatten(-1, (self.heads, self.value)).to(dtype),
                torch.nn.functional.logsigmoid(a + 3), torch.sigmoid(b))

    def forward(self, h, states=None):
        q, k, v, g, beta = self.project(h)
        y, state = autograd.delta_rule(self.plan, q, k, v, g.contiguous(), beta, None, *(states or ()))
        return h + self.out(y.flatten(-2).to(h.dtype)), (state,)

    def step(self, h, states):
        q, k, v, g, beta = self.project(h)
        y = torch.empty_like(v, memory_format=torch.contiguous_format)
        orc.rnn_delta_step(self.plan, q, k, v, g, beta, states[0], y)
        return h + self.out(y.flatten(-2).to(h.dtype))


class Model(torch.nn.Module):
    def __init__(self, width=64, inner=128, state=16, layers=2, io="bf16"):
        """layers: their number, or their kinds ("scan" or "delta")."""
        super().__init__()
        kinds = ["scan"] * layers if isinstance(layers, int) else layers
        self.embed = torch.nn.Embedding(len(WORDS), width)
        self.layers = torch.nn.ModuleList(DeltaLayer(width, inner, io) if kind == "delta" else Layer(width, inner, state, io)
                                          for kind in kinds)
        self.norm = Norm(width)
        self.head = torch.nn.Linear(width, len(WORDS), bias=False)

    def forward(self, ids):
        h, states = self.embed(ids), []
        for layer in self.layers:
            h, s = layer(h)
            states.append(s)
        return self.head(self.norm(h)), states

    def step(self, ids, states):
        h = self.embed(ids)
        for layer, s in zip(self.layers, states):
            h = layer.step(h, s)
        return self.head(self.norm(h))


def train(model, steps, batch=32, length=48, seed=0):
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        ids = torch.tensor([sentence(rng, length + 1) for _ in range(batch)], device="cuda")
        logits, _ = model(ids[:, :-1])
        logp, entropy = autograd.scores(logits.reshape(-1, len(WORDS)), ids[:, 1:].reshape(-1).int())
        loss = -logp.mean() - 0.001 * entropy.mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        torch.nn.utils.clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def generate(model, prompt, tokens):
    """Continue the prompt with the likeliest token each time: (ids, log probabilities, alternatives)."""
    logits, states = model(torch.tensor([prompt], device="cuda"))
    logits = logits[:, -1].contiguous()
    ids, logps, others = list(prompt), [], []
    for _ in range(tokens):
        r = orc.scores(logits, top=3)
        ids.append(int(r.top_ids[0, 0]))
        logps.append(float(r.top_logp[0, 0]))
        others.append([(WORDS[int(i)], round(float(v), 2)) for i, v in zip(r.top_ids[0, 1:], r.top_logp[0, 1:])])
        logits = model.step(r.top_ids[:, 0].long(), states)
    return ids, logps, others


@torch.no_grad()
def search(model, prompt, tokens, beams):
    """Likely continuations of the prompt, best first: (ids [beams, tokens], scores [beams])."""
    plan = orc.rnn_beam_create(beams, end_id=WORDS.index("."))
    logits, states = model(torch.tensor([prompt], device="cuda"))
    # every beam starts from the prompt's states, and the first alone has a score
    states = [tuple(t.expand(beams, *t.shape[1:]).contiguous() for t in s) for s in states]
    scores = torch.full((1, beams), -torch.inf, device="cuda")
    scores[0, 0] = 0
    logits, finished = logits[:, -1].contiguous(), None
    ids = torch.zeros((beams, tokens), dtype=torch.int32, device="cuda")
    for t in range(tokens):
        r = orc.beam_select(plan, logits, scores, finished)
        orc.rnn_beam_reorder(plan, r.parents, [ids, *(x for s in states for x in s)])
        ids[:, t] = r.ids[0]
        scores, finished = r.scores, r.finished
        if t + 1 < tokens:
            logits = model.step(r.ids[0].long(), states)
    orc.rnn_beam_sync(plan)
    return ids, scores[0]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--io", choices=sorted(DTYPES), default="bf16")
    ap.add_argument("--layers", default="scan,scan", help="the layers' kinds: scan or delta, with commas between")
    ap.add_argument("--beams", type=int, default=0)
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(layers=a.layers.split(","), io=a.io).cuda()
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    ids, logps, others = generate(model, [0, 1, 3], a.tokens)
    print(" ".join(WORDS[i] for i in ids))
    for i, lp, alt in list(zip(ids[3:], logps, others))[:8]:
        print(f"  {WORDS[i]:4} log p {lp:6.2f}   else {alt}")
    if a.beams:
        for ids, score in zip(*search(model, [0, 1, 3], 12, a.beams)):
            print(f"  {float(score):7.2f}  " + " ".join(WORDS[i] for i in ids.tolist()))


if __name__ == "__main__":
    main()
