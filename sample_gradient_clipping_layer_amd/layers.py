"""Layers and the loss of language models under per-sample clipping: torch
modules and autograd functions over the library's calls, for use with
``engine.PrivacyEngine`` (or on their own).

    RMSNorm(width)                      y, or (y, s) with a residual: s = x + residual
    ExpertLinear(experts, d, p)         rows sorted by expert times their expert's weight
    route(expert_ids, experts)          the row order and segments that ExpertLinear takes
    distillation_loss(logits, ids, teacher, temperature, weight)   per-sample losses [B]

The engine keeps what it needs of RMSNorm and ExpertLinear during the backward
pass; without an engine their weights get their ordinary gradients. Everything
is computed by the library's kernels on the current GPU and torch's current
stream; activations are float32 or bfloat16.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (dp_clipped_sum_noise, dp_distill_loss, dp_distill_loss_backward,
               dp_grouped_clipped_sum_noise, dp_grouped_matmul, dp_rms_norm, dp_rms_norm_backward)


def _aligned(t):
    """t contiguous and at a 16-byte boundary, as the grouped and distillation
    calls take it. A contiguous view keeps its offset (a slice of samples, the
    part of a concatenation's gradient): one that starts elsewhere is copied."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, module):
        x = x.contiguous()
        out = torch.empty_like(x)
        s = x
        if residual is not None:
            residual = residual.contiguous()
            s = torch.empty_like(x)
        dp_rms_norm(x, weight, eps, out, residual=residual, sum_out=s if residual is not None else None)
        ctx.save_for_backward(s, weight)
        ctx.eps, ctx.module, ctx.with_residual = eps, module, residual is not None
        ctx.set_materialize_grads(False)
        return (out, s) if residual is not None else out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        s, weight = ctx.saved_tensors
        private = ctx.module is not None and ctx.module.private
        if dy is None:  # only the sum was used: the weight's gradient is zero
            dx = dsum
            rows = torch.zeros(s.shape[0], s.shape[-1], dtype=torch.float32, device=s.device) if private else None
            dw = None
        else:
            dx = torch.empty_like(s) if ctx.needs_input_grad[0] or ctx.needs_input_grad[1] else None
            rows = dw = None
            if private or ctx.needs_input_grad[2]:
                rows = torch.empty(s.shape[0], s.shape[-1], dtype=torch.float32, device=s.device)
            if dx is not None or rows is not None:
                dp_rms_norm_backward(dy.contiguous(), s, weight, ctx.eps, dx=dx,
                                     dsum=None if dsum is None else dsum.contiguous(), gain_rows=rows)
            if not private and ctx.needs_input_grad[2]:
                dw = _sum_rows(rows).to(weight.dtype)
        if private and rows is not None:
            ctx.module.gain_rows = rows
        return dx, (dx if ctx.with_residual else None), dw, None, None


def _sum_rows(rows):
    """The sum over samples of rows [B, d]: the clipped sum under factors 1."""
    B, d = rows.shape
    out = torch.empty(1, d, dtype=torch.float32, device=rows.device)
    ones = torch.ones(B, 1, 1, dtype=torch.float32, device=rows.device)
    dp_clipped_sum_noise(ones, rows.view(B, 1, d), ones.view(B), 1.0, 0.0, 1.0, 0, 0, 0, out)
    return out.view(d)


class RMSNorm(torch.nn.Module):
    """Root-mean-square norm over the last dimension, with the residual's
    addition fused in: forward(x) gives y; forward(x, residual) gives (y, s)
    with s = x + residual, the residual stream after the addition. x is
    [B, ..., width], a sample per index of the first dimension."""

    def __init__(self, width: int, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.eps = float(eps)
        self.private = False   # an engine takes the weight's per-sample gradients
        self.gain_rows = None  # those of the last backward pass, [B, width]

    def forward(self, x, residual=None):
        return _RmsNorm.apply(x, residual, self.weight, self.eps, self)


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, segments, module):
        x = _aligned(x)
        # rows outside the segments belong to no expert: zeros
        out = torch.zeros(x.shape[0], weight.shape[1], dtype=x.dtype, device=x.device)
        dp_grouped_matmul(x, _aligned(weight), segments, out)
        ctx.save_for_backward(x, weight, segments)
        ctx.module = module
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, segments = ctx.saved_tensors
        g = _aligned(g)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.zeros_like(x)
            dp_grouped_matmul(g, _aligned(weight), segments, dx, transpose=True)
        if ctx.needs_input_grad[1] and not ctx.module.private:
            E, p, d = weight.shape
            B = (segments.numel() - 1) // E
            out = torch.empty(E, d, p, dtype=torch.float32, device=x.device)
            dp_grouped_clipped_sum_noise(x, g, segments, torch.ones(B, dtype=torch.float32, device=x.device), 1.0,
                                         0.0, 1.0, 0, 0, 0, out)
            dw = out.transpose(1, 2).to(weight.dtype).contiguous()
        return dx, dw, None, None


class ExpertLinear(torch.nn.Module):
    """A linear layer (no bias) per expert: forward(x [R, in], segments) with
    rows sorted by expert, then sample, as route() gives them, returns
    [R, out]. weight is [experts, out, in]; x and weight share one dtype."""

    def __init__(self, experts: int, in_features: int, out_features: int, device=None, dtype=None):
        super().__init__()
        w = torch.empty(experts, out_features, in_features, device=device, dtype=dtype)
        bound = in_features ** -0.5
        self.weight = torch.nn.Parameter(w.uniform_(-bound, bound))
        self.private = False  # an engine takes the weight's per-sample gradients

    def forward(self, x, segments):
        return _ExpertLinear.apply(x, self.weight, segments, self)


def route(expert_ids, experts: int):
    """Row order and segments of a routing: expert_ids [B, T, top] (int64; a
    negative id drops that place) gives (order [B*T*top], segments
    [experts*B + 1]). Sorted row r is place order[r] of the flattened [B, T, top]
    routing, so its token is order[r] // top of the flattened [B*T]; places
    sort by expert, then sample, dropped ones behind all segments."""
    if expert_ids.dim() != 3 or expert_ids.dtype != torch.int64:
        raise ValueError("expert_ids must be an int64 tensor [B, T, top]")
    B = expert_ids.shape[0]
    sample = torch.arange(B, device=expert_ids.device)[:, None, None]
    inside = (expert_ids >= 0) & (expert_ids < experts)
    key = torch.where(inside, expert_ids * B + sample, experts * B).reshape(-1)
    key, order = torch.sort(key, stable=True)
    segments = torch.searchsorted(key, torch.arange(experts * B + 1, device=key.device))
    return order, segments


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, tau, weight):
        logits = _aligned(logits)
        B, T, _ = logits.shape
        loss = torch.empty(B, dtype=torch.float32, device=logits.device)
        lse = torch.empty(B, T, dtype=torch.float32, device=logits.device)
        dp_distill_loss(logits, ids, teacher, tau, loss, lse, weight=weight)
        ctx.save_for_backward(logits, ids, teacher, lse, weight)
        ctx.tau = tau
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        logits, ids, teacher, lse, weight = ctx.saved_tensors
        grad = torch.empty_like(logits)
        dp_distill_loss_backward(logits, ids, teacher, ctx.tau, lse, grad, weight=weight,
                                 dloss=dloss.float().contiguous())
        return grad, None, None, None, None


def distillation_loss(logits, ids, teacher, temperature: float = 1.0, weight=None):
    """Per-sample distillation losses [B] from a teacher's top logits:

        loss[b] = tau^2 * sum_t weight[b, t] * KL(q || p)

    p = softmax(logits / tau) over the vocabulary, q the softmax of the
    token's used teacher logits / tau (a word named twice is two terms of the
    sum). logits [B, T, V]; ids [B, T, K] int64, -1 where a place is unused;
    teacher [B, T, K]; weight [B, T] float32 or None. Gradients flow to logits only. ``distillation_loss(...).sum()
    .backward()`` is what PrivacyEngine's backward pass asks for."""
    return _Distill.apply(logits, ids.contiguous(), teacher.detach().contiguous(), float(temperature),
                          None if weight is None else weight.detach().float().contiguous())
