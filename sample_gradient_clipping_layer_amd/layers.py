"""Layers and losses of language models under per-sample clipping: torch
modules and autograd functions over the library's calls, for use with
``engine.PrivacyEngine`` (or on their own).

    Embedding(words, width, scale)      rows of a table of words, scaled
    LayerNorm(width), RMSNorm(width)    y, or (y, s) with a residual: s = x + residual
    replace_layer_norms(model)          a model's torch.nn.LayerNorm modules as LayerNorm ones
    ExpertLinear(experts, d, p)         rows sorted by expert times their expert's weight
    route(expert_ids, experts)          the row order and segments that ExpertLinear takes
    balance_loss(logits, expert_ids)    a router's per-sample losses [B], and its rows per expert [B, E]
    token_logprobs(logits, targets)     log probabilities of given tokens, the entropy, top alternatives
    token_loss(logits, targets, weight) per-sample losses [B] from them
    distillation_loss(logits, ids, teacher, temperature, weight)   per-sample losses [B]

The engine keeps what it needs of the modules during the backward pass; without
an engine their weights get their ordinary gradients. Everything is computed by
the library's kernels on the current GPU and torch's current stream;
activations are float32 or bfloat16.

In a captured HIP graph the backward pass is captured with its forward pass, and
no eager graph of the same parameters may be alive then (torch runs a leaf's
accumulation on the stream of the graph that met it first).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (dp_balance_loss, dp_balance_loss_backward, dp_clipped_sum_noise, dp_distill_loss,
               dp_distill_loss_backward, dp_embedding, dp_embedding_clipped_sum_noise, dp_embedding_order,
               dp_grouped_clipped_sum_noise, dp_grouped_matmul, dp_layer_norm, dp_layer_norm_backward, dp_rms_norm,
               dp_rms_norm_backward, dp_token_logprob, dp_token_logprob_backward)


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


def _row_sums(x, most=4096):
    """The sums of rows [B, n], long ones from the sums of their parts: torch
    spreads one row of 131072 or more over workgroups that meet in memory it
    clears by a memset, which has no place in a captured graph."""
    while x.shape[1] > most:
        x = torch.nn.functional.pad(x, (0, -x.shape[1] % most)).view(x.shape[0], -1, most).sum(2)
    return x.sum(1)


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


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, module):
        x = x.contiguous()
        out = torch.empty_like(x)
        s = x
        if residual is not None:
            residual = residual.contiguous()
            s = torch.empty_like(x)
        dp_layer_norm(x, weight, bias, eps, out, residual=residual, sum_out=s if residual is not None else None)
        ctx.save_for_backward(s, weight)
        ctx.eps, ctx.module, ctx.with_residual, ctx.bias_dtype = eps, module, residual is not None, (
            None if bias is None else bias.dtype)
        ctx.set_materialize_grads(False)
        return (out, s) if residual is not None else out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        s, weight = ctx.saved_tensors
        private = ctx.module is not None and ctx.module.private
        has_bias = ctx.bias_dtype is not None
        B, d = s.shape[0] if s.dim() > 1 else 1, s.shape[-1]
        dx, rows, dw, db = dsum, [None, None], None, None
        if dy is None:  # only the sum was used: the gradients of weight and bias are zero
            if private:
                rows = [torch.zeros(B, d, dtype=torch.float32, device=s.device) for _ in range(1 + has_bias)] + [None]
        else:
            dx = torch.empty_like(s) if ctx.needs_input_grad[0] or ctx.needs_input_grad[1] else None
            for k in range(1 + has_bias):
                if private or ctx.needs_input_grad[2 + k]:
                    rows[k] = torch.empty(B, d, dtype=torch.float32, device=s.device)
            if dx is not None or rows[0] is not None or rows[1] is not None:
                dy, v, out, ds = (t if t is None else t.contiguous().view(B, -1, d) for t in (dy, s, dx, dsum))
                dp_layer_norm_backward(dy, v, weight, ctx.eps, dx=out, dsum=ds, gain_rows=rows[0], bias_rows=rows[1])
            if not private:
                dw = _sum_rows(rows[0]).to(weight.dtype) if ctx.needs_input_grad[2] else None
                db = _sum_rows(rows[1]).to(ctx.bias_dtype) if has_bias and ctx.needs_input_grad[3] else None
        if private and rows[0] is not None:
            ctx.module.gain_rows, ctx.module.bias_rows = rows[0], rows[1]
        return dx, (dx if ctx.with_residual else None), dw, db, None, None


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, with the residual's addition fused
    in: forward(x) gives y; forward(x, residual) gives (y, s) with s = x +
    residual, the residual stream after the addition. x is [B, ..., width], a
    sample per index of the first dimension, or one row [width]; weight and bias
    share one dtype."""

    def __init__(self, width: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)
        self.eps = float(eps)
        self.private = False  # an engine takes the per-sample gradients of weight and bias
        self.gain_rows = self.bias_rows = None  # those of the last backward pass, [B, width]

    @classmethod
    def from_torch(cls, norm: torch.nn.LayerNorm):
        """A torch.nn.LayerNorm over the last dimension, sharing its parameters
        and the hooks registered on it (their handles still remove them)."""
        if len(norm.normalized_shape) != 1 or norm.weight is None:
            raise ValueError("LayerNorm must be over the last dimension, with a weight")
        new = cls(1, eps=norm.eps, bias=norm.bias is not None)
        new.weight, new.bias = norm.weight, norm.bias
        new.__dict__.update((n, v) for n, v in norm.__dict__.items() if "_hook" in n)
        return new.train(norm.training)

    def forward(self, x, residual=None):
        return _LayerNorm.apply(x, residual, self.weight, self.bias, self.eps, self)


def replace_layer_norms(model: torch.nn.Module) -> torch.nn.Module:
    """model with every torch.nn.LayerNorm (over the last dimension, with a
    weight) replaced by a LayerNorm that shares its parameters and hooks, so
    that an engine can clip them; names and state_dict stay. Changes model and
    returns it (a model that is a norm itself is returned as a new module). The
    new modules take what LayerNorm takes: float32 or bfloat16 on the GPU, with
    at least one element."""
    new = {}

    def of(m):
        if type(m) is torch.nn.LayerNorm and m.weight is not None and len(m.normalized_shape) == 1:
            if id(m) not in new:  # a module in two places stays one
                new[id(m)] = LayerNorm.from_torch(m)
            return new[id(m)]
        return m

    for m in list(model.modules()):
        for name, child in list(m._modules.items()):
            if child is not None:
                m._modules[name] = of(child)
    return of(model)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, module):
        ids = ids.contiguous()
        out = torch.empty(*ids.shape, weight.shape[1], dtype=weight.dtype, device=weight.device)
        dp_embedding(ids, weight.contiguous(), out, scale=scale)
        ctx.save_for_backward(ids)
        ctx.words, ctx.dtype, ctx.scale, ctx.module = weight.shape[0], weight.dtype, scale, module
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        if ctx.module.private or not ctx.needs_input_grad[1]:
            return None, None, None, None
        ids, = ctx.saved_tensors
        ids = ids.reshape(ids.shape[0], -1) if ids.dim() else ids.reshape(1, 1)
        g = g.contiguous().view(*ids.shape, -1)
        order = torch.empty(ids.numel(), dtype=torch.int64, device=g.device)
        starts = torch.empty(ctx.words + 1, dtype=torch.int64, device=g.device)
        out = torch.empty(ctx.words, g.shape[-1], dtype=torch.float32, device=g.device)
        dp_embedding_order(ids, ctx.words, order, starts)
        dp_embedding_clipped_sum_noise(g, ids, order, starts,
                                       torch.ones(ids.shape[0], dtype=torch.float32, device=g.device), 1.0, 0.0, 1.0, 0,
                                       0, 0, out, scale=ctx.scale)
        return None, out.to(ctx.dtype), None, None


class Embedding(torch.nn.Module):
    """A table of words: forward(ids [B, ...] int64) gives scale * weight[ids],
    and zeros for an id outside the table (padding: -1). weight is [words,
    width]; the rows have its dtype."""

    def __init__(self, words: int, width: int, scale: float = 1.0, device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(words, width, device=device, dtype=dtype).normal_())
        self.scale = float(scale)
        self.private = False  # an engine takes the weight's per-sample gradients

    def forward(self, ids):
        return _Embedding.apply(ids, self.weight, self.scale, self)


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


class _Balance(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids):
        logits = logits.contiguous()
        B, _, E = logits.shape
        loss = torch.empty(B, dtype=torch.float32, device=logits.device)
        counts = torch.empty(B, E, dtype=torch.int64, device=logits.device)
        tokens = torch.empty(B, dtype=torch.int64, device=logits.device)
        dp_balance_loss(logits, ids, loss, counts, tokens)
        ctx.save_for_backward(logits, ids, counts, tokens)
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        logits, ids, counts, tokens = ctx.saved_tensors
        grad = torch.empty_like(logits)
        dp_balance_loss_backward(logits, ids, counts, tokens, grad, dloss=dloss.float().contiguous())
        return grad, None


def balance_loss(logits, expert_ids):
    """(loss [B], counts [B, E]) of a router: its logits [B, T, E] and the
    experts it chose, expert_ids [B, T, top] (int64; as in route(), an id
    outside [0, E) drops that place).

        loss[b] = E * sum_e f_e * P_e

    f_e is the share of the sample's places that name expert e, P_e the mean
    probability of e over the sample's tokens that have a place (0 in a token
    whose logits are all -inf, and so is its gradient); even routing gives 1.
    counts are the places per expert. Each sample's loss is its own, so that it
    can be added to what PrivacyEngine's backward pass sums up. Gradients flow
    to logits only."""
    return _Balance.apply(logits, expert_ids.contiguous())


class _TokenLogprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, tau, top):
        logits = _aligned(logits)
        shape = targets.shape
        logp, entropy = (torch.empty(shape, dtype=torch.float32, device=logits.device) for _ in range(2))
        stats = torch.empty(*shape, 2, dtype=torch.float32, device=logits.device)
        top_ids = top_logp = None
        if top:
            top_ids = torch.empty(*shape, top, dtype=torch.int64, device=logits.device)
            top_logp = torch.empty(*shape, top, dtype=torch.float32, device=logits.device)
        dp_token_logprob(logits, targets, tau, logp, stats, entropy=entropy, top_ids=top_ids, top_logp=top_logp)
        ctx.save_for_backward(logits, targets, stats, entropy)
        ctx.tau = tau
        ctx.set_materialize_grads(False)
        if not top:
            return logp, entropy
        ctx.mark_non_differentiable(top_ids, top_logp)
        return logp, entropy, top_ids, top_logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, *_):
        logits, targets, stats, entropy = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None
        grad = torch.empty_like(logits)
        dp_token_logprob_backward(logits, targets, ctx.tau, stats, grad,
                                  dlogp=None if dlogp is None else dlogp.float().contiguous(), entropy=entropy,
                                  dentropy=None if dentropy is None else dentropy.float().contiguous())
        return grad, None, None, None


def token_logprobs(logits, targets, temperature: float = 1.0, top: int = 0):
    """(logp, entropy), each [...], of softmax(logits [..., V] / temperature):
    the log probability of targets [...] (int64; 0 for a target outside [0, V))
    and the entropy of the distribution. With top = K also (top_ids [..., K],
    top_logp [..., K]), its K most probable words, largest first (of equal ones
    the lower word first): what distillation_loss takes as ids and teacher.
    Gradients flow from logp and entropy to logits."""
    return _TokenLogprob.apply(logits, targets.contiguous(), float(temperature), int(top))


def token_loss(logits, targets, weight=None, temperature: float = 1.0):
    """Per-sample losses [B]: -sum over a sample's tokens of weight * log p of
    its target, for logits [B, ..., V], targets [B, ...] int64 (outside [0, V):
    no loss) and weight [B, ...] float32 or None. A token of weight 0 counts for
    nothing, whatever its logits hold. ``token_loss(...).sum().backward()`` is
    what PrivacyEngine's backward pass asks for."""
    logp = token_logprobs(logits, targets, temperature)[0]
    if weight is not None:
        weight = weight.detach().float()
        logp = torch.where(weight != 0, weight * logp, torch.zeros_like(logp))
    return -_row_sums(logp.reshape(logp.shape[0], -1))


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
