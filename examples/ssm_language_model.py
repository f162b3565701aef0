"""A small recurrent language model on the state space operators.

    python examples/ssm_language_model.py [--steps 60] [--tokens 48] [--io bf16]

Two layers of projection -> causal convolution -> selective scan -> projection
learn the sentences of a small grammar (bracketed words whose brackets close
in order).  Training takes whole sentences (convolution, scan and scores with
their gradients, an entropy bonus in the loss); generation reads a prompt with
the same operators and then continues it a token at a time from the layers'
states, printing each token's log probability and the alternatives that the
model saw.  The matrix products are torch's.
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


class Layer(torch.nn.Module):
    def __init__(self, width, inner, state, io):
        super().__init__()
        self.plan = orc.rnn_ssm_create(inner, state_size=state, groups=1, conv_width=4, layout=1)
        orc.rnn_ssm_set_io_type(self.plan, io)
        self.inner, self.state = inner, state
        self.norm = torch.nn.LayerNorm(width)
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


class Model(torch.nn.Module):
    def __init__(self, width=64, inner=128, state=16, layers=2, io="bf16"):
        super().__init__()
        self.embed = torch.nn.Embedding(len(WORDS), width)
        self.layers = torch.nn.ModuleList(Layer(width, inner, state, io) for _ in range(layers))
        self.norm = torch.nn.LayerNorm(width)
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


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--io", choices=sorted(DTYPES), default="bf16")
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(io=a.io).cuda()
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    ids, logps, others = generate(model, [0, 1, 3], a.tokens)
    print(" ".join(WORDS[i] for i in ids))
    for i, lp, alt in list(zip(ids[3:], logps, others))[:8]:
        print(f"  {WORDS[i]:4} log p {lp:6.2f}   else {alt}")


if __name__ == "__main__":
    main()
