"""The state space operators, the gated delta rule, layer normalisation and token
scores as differentiable functions.

Thin torch.autograd wrappers of ``ssm``, ``delta`` and ``norm``: each forward and each gradient is one
entry point of the CUDA library.  Gradients are those of one backward pass:
differentiating them again raises an error.  Only the gradients that are asked
for are formed, and a scan or a delta rule that needs none saves nothing for
them.  A backward pass that is to be captured needs leaves that no graph built
outside the capture still holds.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import delta, norm, ssm


def _dense(slope):
    return None if slope is None else slope.contiguous()


def _wanted(ctx, inputs):
    """New tensors for the gradients that are needed, under their names: inputs are (name, tensor) in the order of
    forward's arguments after the plan, with no name for what has no gradient."""
    return {name: torch.empty_like(t, memory_format=torch.contiguous_format)
            for (name, t), needed in zip(inputs, ctx.needs_input_grad[1:]) if name and needed}


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, X, W, bias, sequence_lens, initial_state):
        ctx.set_materialize_grads(False)
        Y, state = ssm.ssm_conv(plan, X, W, bias, sequence_lens, initial_state)
        ctx.plan = plan
        ctx.save_for_backward(X, W, bias, sequence_lens, initial_state)
        return Y, state

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, d_state):
        X, W, bias, lens, h0 = ctx.saved_tensors
        dY = torch.zeros_like(X, memory_format=torch.contiguous_format) if dY is None else dY.contiguous()
        g = _wanted(ctx, (("dX", X), ("dW", W), ("dbias", bias), (None, lens), ("d_initial_state", h0)))
        ssm.rnn_ssm_conv_grad(ctx.plan, dY, X, W, bias, lens, h0, _dense(d_state), **g)
        return None, g.get("dX"), g.get("dW"), g.get("dbias"), None, g.get("d_initial_state")


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h):
        ctx.set_materialize_grads(False)
        args = (X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h)
        Y, Y_h, saved = ssm.ssm_scan(plan, *args, save=True)
        ctx.plan = plan
        ctx.save_for_backward(saved, *args)
        return Y, Y_h

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, dY_h):
        saved, *args = ctx.saved_tensors
        X = args[0]
        dY = torch.zeros_like(X, memory_format=torch.contiguous_format) if dY is None else dY.contiguous()
        names = ("dX", "ddt", "dA", "dB", "dC", "dD", "dZ", "ddt_bias", None, "d_initial_h")
        g = _wanted(ctx, zip(names, args))
        ssm.rnn_ssm_scan_grad(ctx.plan, dY, saved, *args, dY_h=_dense(dY_h), **g)
        return (None, *(g.get(name) for name in names))


class _Scores(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, top):
        ctx.set_materialize_grads(False)
        r = ssm.scores(logits, ids, top=top)
        ctx.save_for_backward(logits, ids, *r)
        if r.top_ids is None:
            return r.logp, r.entropy
        ctx.mark_non_differentiable(r.top_ids)
        return r.logp, r.entropy, r.top_ids, r.top_logp

    @staticmethod
    @once_differentiable
    def backward(ctx, d_logp, d_entropy, d_ids=None, d_top=None):
        logits, ids, *r = ctx.saved_tensors
        r = ssm.Scores(*r)
        r.lse._rest = True             # as it was made, whether or not the tensor came back as the same object
        dlogits = ssm.scores_grad(logits, ids, r, _dense(d_logp), _dense(d_entropy),
                                  _dense(d_top))
        return dlogits, None, None


class _Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, Q, K, V, g, beta, sequence_lens, initial_state):
        ctx.set_materialize_grads(False)
        args = (Q, K, V, g, beta, sequence_lens, initial_state)
        Y, state, saved = delta.delta_rule(plan, *args, save=True)
        ctx.plan = plan
        ctx.save_for_backward(saved, *args)
        return Y, state

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, d_state):
        saved, *args = ctx.saved_tensors
        dY = torch.zeros_like(args[2], memory_format=torch.contiguous_format) if dY is None else dY.contiguous()
        names = ("dQ", "dK", "dV", "dg", "dbeta", None, "d_initial_state")
        g = _wanted(ctx, zip(names, args))
        delta.rnn_delta_rule_grad(ctx.plan, dY, saved, *args[:6], _dense(d_state), **g)
        return (None, *(g.get(name) for name in names))


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, X, W, bias):
        Y, stats = norm.layer_norm(plan, X, W, bias)
        ctx.plan = plan
        ctx.save_for_backward(X, stats, W, bias)
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, stats, W, bias = ctx.saved_tensors
        g = _wanted(ctx, (("dX", X), ("dW", W), ("dbias", bias)))
        norm.rnn_layer_norm_grad(ctx.plan, dY.contiguous(), X, stats, W, **g)
        return None, g.get("dX"), g.get("dW"), g.get("dbias")


def conv(plan, X, W, bias=None, sequence_lens=None, initial_state=None):
    """(Y, final_state) of the causal convolution, as ``ssm_conv``."""
    return _Conv.apply(plan, X, W, bias, sequence_lens, initial_state)


def scan(plan, X, dt, A, B, C, D=None, Z=None, dt_bias=None, sequence_lens=None, initial_h=None):
    """(Y, Y_h) of the selective scan, as ``ssm_scan``."""
    args = (X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h)
    if not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in args):
        return ssm.ssm_scan(plan, *args)[:2]
    return _Scan.apply(plan, *args)


def delta_rule(plan, Q, K, V, g, beta, sequence_lens=None, initial_state=None):
    """(Y, final_state) of the gated delta rule, as ``delta.delta_rule``."""
    args = (Q, K, V, g, beta, sequence_lens, initial_state)
    if not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in args):
        return delta.delta_rule(plan, *args)[:2]
    return _Delta.apply(plan, *args)


def layer_norm(plan, X, W=None, bias=None):
    """Y of the layer normalisation, as ``norm.layer_norm``."""
    return _Norm.apply(plan, X, W, bias)


def scores(logits, ids=None, top=0):
    """(logp, entropy), and (top_ids, top_logp) with top > 0, as ``ssm.scores``;
    -logp is the cross entropy of the token (None without ids)."""
    return _Scores.apply(logits, ids, top)
