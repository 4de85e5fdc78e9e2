"""Privacy engine front end: per-sample clipping and Gaussian noise for the
Linear, Conv2d, Embedding, LayerNorm, RMSNorm and ExpertLinear layers of a torch
model, through the C ABI.

"Scalable and Efficient Training of Large CNNs with DP", App. E (the privacy
engine with its 'ghost' and 'ghost-mixed' modes) and Sec. 3 (ghost norm, then
the weighted gradient instead of per-sample gradients): hooks keep each
layer's input a and output gradient dL/ds during one ordinary forward and
backward pass of the summed per-sample loss; step() then runs the library's
path over all layers -- the per-sample norm over every layer, the clip
factors, and each layer's clipped noised mean -- and writes the results into
the parameters' .grad. A convolution's input is unfolded into U(a) (same
page, Sec. 2.2: D = C_in * kH * kW features per output position) by the
library (dp_unfold2d), and the conv layers share the multi-layer calls with
the linear ones; with conv_input="folded" the library instead forms U(a)'s
rows inside its kernels (dp_conv_* calls, one per layer; nothing unfolded is
stored), and with conv_input="unfolded" torch unfolds each input (at
ResNet-18 shapes torch's unfold alone takes several times the whole
clipping path).

A root-mean-square norm's gain (layers.RMSNorm, torch.nn.RMSNorm) has the
per-sample gradient sum_t dy u, which dp_rms_norm_backward leaves as [B, d]
rows: the linear layer A = 1 [B, 1, 1], G = rows [B, 1, d] of the multi-layer
calls; layers.LayerNorm's gain and bias are such a layer of 2d columns.
layers.ExpertLinear's rows are grouped by (expert, sample) and take the
dp_grouped_* calls. A table of words (layers.Embedding, torch.nn.Embedding)
takes the dp_embedding_* calls on its tokens sorted by word. All add to the same
per-sample norms and share the clip factors.

Only argument marshalling and layout changes happen here; every step of the
clipping path runs in libdpclip.
"""
from __future__ import annotations

import torch
import torch.nn.functional as F

from . import (DP_BF16, DP_F32, MODE_EXPLICIT, MODE_GHOST, MODE_MIXED, MODE_TIME, conv_geometry, dp_clip_factors,
               dp_clipped_sum_noise_layers, dp_conv_clipped_sum_noise, dp_conv_norm, dp_conv_workspace_bytes,
               dp_embedding_clipped_sum_noise, dp_embedding_norm, dp_embedding_order, dp_embedding_workspace_bytes,
               dp_ghost_norm_clip_layers, dp_ghost_norm_layers, dp_grouped_clipped_sum_noise, dp_grouped_norm,
               dp_grouped_workspace_bytes, dp_layers_workspace_bytes, dp_rms_norm_backward, dp_unfold2d)
from .layers import Embedding, ExpertLinear, LayerNorm, RMSNorm, _aligned

MODES = {"ghost-mixed": MODE_MIXED, "ghost": MODE_GHOST, "explicit": MODE_EXPLICIT, "time": MODE_TIME}


class _Layer:
    def __init__(self, module: torch.nn.Module):
        self.module = module
        self.a = None   # the module's input of the last forward pass
        self.g = None   # dL/d(output) of the last backward pass
        self.passed = True  # that forward pass has had its backward pass
        self.segments = None  # ExpertLinear: its rows' (expert, sample) ranges
        self.version = None  # a table's: that of its ids when they were looked up


def _torch_eps(m, dtype):
    """The eps that a torch.nn.RMSNorm adds to rows of `dtype`. eps=None is the
    machine epsilon of the type torch computes in, which is float32 for the
    16-bit types too."""
    if m.eps is not None:
        return m.eps
    return torch.finfo(torch.float64 if dtype == torch.float64 else torch.float32).eps


_NORMS = (torch.nn.RMSNorm, RMSNorm, LayerNorm)
_TABLES = (torch.nn.Embedding, Embedding)
_OWN = (RMSNorm, LayerNorm, Embedding, ExpertLinear)  # modules that know an engine takes their gradients
_COVERED = (torch.nn.Linear, torch.nn.Conv2d, ExpertLinear) + _NORMS + _TABLES


def _version(t):
    """How often t has been changed in place (a tensor made in inference mode does not say)."""
    return None if t.is_inference() else t._version


def _forget_rows(norm):
    norm.gain_rows = None
    if isinstance(norm, LayerNorm):
        norm.bias_rows = None


class PrivacyEngine:
    """Flat (global) per-sample clipping at bound C with noise multiplier
    sigma for every nn.Linear, nn.Conv2d (groups = 1), nn.Embedding,
    nn.RMSNorm, layers.Embedding, layers.LayerNorm, layers.RMSNorm and
    layers.ExpertLinear with trainable parameters in `model`
    (layers.replace_layer_norms turns torch.nn.LayerNorm into layers.LayerNorm).

    Usage, per step:
        out = model(x)                       # hooks keep the layer inputs
        per_sample_loss(out, y).sum().backward()   # hooks keep dL/ds
        engine.step(step_index)              # .grad = (sum_i c_i g_i + N(0, s^2 C^2 I)) / B

    The backward pass must be of the SUM of the per-sample losses, so that the
    kept output gradients are the per-sample ones. A module may run once per
    forward pass; its input's first dimension is the batch (positions given to
    an Embedding too: one row of them per sample, [B, T]; ids of one dimension
    are refused where another layer has several rows per sample). A torch Embedding's
    padding_idx keeps its row: its gradient is 0, without noise. Any other
    trainable parameter makes the constructor fail: its per-sample gradient
    would go unclipped.

    mode: the per-layer path rule ('ghost-mixed', 'ghost', 'explicit',
    'time') of the linear and convolution layers; expert layers have the ghost
    norm alone. conv_input: 'library-unfold' (the default: the library writes
    each Conv2d input's unfolding, and the layers share the multi-layer
    calls), 'folded' (the library takes each Conv2d input as it is and forms
    the unfolded rows in its kernels, one call per Conv2d layer; no unfolded
    copy in memory) or 'unfolded' (torch unfolds each Conv2d input).
    """

    def __init__(self, model: torch.nn.Module, C: float, sigma: float, seed: int = 0, mode: str = "ghost-mixed",
                 kappa: int = 1, conv_input: str = "library-unfold"):
        if mode not in MODES:
            raise ValueError(f"mode must be one of {sorted(MODES)}")
        if conv_input not in ("library-unfold", "unfolded", "folded"):
            raise ValueError("conv_input must be 'library-unfold', 'unfolded' or 'folded'")
        self.folded = conv_input == "folded"
        self.library_unfold = conv_input == "library-unfold"
        self.C, self.sigma, self.seed = float(C), float(sigma), int(seed)
        self.mode, self.kappa = MODES[mode], int(kappa)
        self.layers: list[_Layer] = []
        covered = {}  # a parameter's id -> the layer's type
        for m in model.modules():
            if isinstance(m, _COVERED) and any(p.requires_grad for p in m.parameters()):
                if isinstance(m, torch.nn.RMSNorm) and len(m.normalized_shape) != 1:
                    raise ValueError("RMSNorm must be over the last dimension")
                if isinstance(m, torch.nn.Conv2d) and m.groups != 1:
                    raise ValueError("Conv2d with groups != 1 is not supported")
                if isinstance(m, torch.nn.Conv2d) and m.padding_mode != "zeros":
                    raise ValueError("Conv2d padding must be zeros")
                if isinstance(m, torch.nn.Conv2d) and isinstance(m.padding, str) and m.padding != "valid":
                    raise ValueError("Conv2d padding must be numeric or 'valid'")
                if isinstance(m, torch.nn.Embedding) and (m.max_norm is not None or m.scale_grad_by_freq or m.sparse):
                    raise ValueError("Embedding with max_norm, scale_grad_by_freq or sparse is not supported")
                if not m.weight.requires_grad:
                    raise ValueError("a layer with a trainable bias needs a trainable weight (one norm covers both)")
                shared = [covered[id(p)] for p in m.parameters() if id(p) in covered]
                if shared and issubclass(type(m), _NORMS + _TABLES + (ExpertLinear,)) or \
                        any(issubclass(c, _NORMS + _TABLES + (ExpertLinear,)) for c in shared):
                    raise ValueError("a norm's, a table's or an expert layer's parameter is shared with another layer: "
                                     "its per-sample gradients would have to be added before their norm")
                self.layers.append(_Layer(m))
                covered.update((id(p), type(m)) for p in m.parameters())
        others = [n for n, p in model.named_parameters() if p.requires_grad and id(p) not in covered]
        if others:
            raise ValueError("trainable parameters outside Linear, Conv2d, Embedding, LayerNorm, RMSNorm and "
                             f"ExpertLinear layers (torch.nn.LayerNorm: see layers.replace_layer_norms): {others}")
        if not self.layers:
            raise ValueError("no Linear, Conv2d, Embedding, LayerNorm, RMSNorm or ExpertLinear layer with trainable "
                             "parameters")
        self._handles = []
        for L in self.layers:
            if isinstance(L.module, _OWN):
                L.module.private = True  # their backward passes leave the weight's gradient to step()
            self._handles.append(L.module.register_forward_hook(self._forward_hook(L), with_kwargs=True))
            self._handles.append(L.module.register_full_backward_hook(self._backward_hook(L)))
        self.last_norms = None  # per-sample norms of the last step

    @staticmethod
    def _forward_hook(L):
        def hook(module, inputs, kwargs, output):  # arguments by position or by name
            if L.a is not None and not L.passed:
                raise RuntimeError("a module ran twice in one forward pass")
            a = inputs[0] if inputs else next(kwargs[n] for n in ("input", "x", "ids") if n in kwargs)
            L.a = a.detach()
            if isinstance(module, _TABLES):
                L.version = _version(a)
            L.g = None
            L.passed = False
            if isinstance(module, ExpertLinear):
                L.segments = inputs[1] if len(inputs) > 1 else kwargs["segments"]
            elif isinstance(module, (RMSNorm, LayerNorm)):
                _forget_rows(module)
        return hook

    @staticmethod
    def _backward_hook(L):
        def hook(module, grad_input, grad_output):
            g = grad_output[0]  # None: a norm of which only the sum was used
            L.g = None if g is None else g.detach()
            L.passed = True
        return hook

    def detach(self):
        """Remove the hooks."""
        for h in self._handles:
            h.remove()
        self._handles = []
        for L in self.layers:
            if isinstance(L.module, _OWN):
                L.module.private = False

    @staticmethod
    def _padding(m):
        return 0 if isinstance(m.padding, str) else m.padding  # 'valid' is no padding

    def _is_folded(self, L):
        return self.folded and isinstance(L.module, torch.nn.Conv2d)

    def _gain_operands(self, L):
        """(A = 1 [B, 1, 1], G = the gain's per-sample gradients [B, 1, d]) of a
        norm layer, in float32; a LayerNorm's with those of a trainable bias
        behind them, [B, 1, 2d]."""
        m, a, g = L.module, L.a, L.g
        if a is None or (g is None and getattr(m, "gain_rows", None) is None):
            raise RuntimeError("step() needs one forward and one backward pass of every layer first")
        if isinstance(m, (RMSNorm, LayerNorm)):
            rows = m.gain_rows
            if rows is None:
                raise RuntimeError("a norm's backward pass did not run")
            if self._norm_bias(m):
                rows = torch.cat([rows, m.bias_rows], dim=1)
        else:
            dt = a.dtype if a.dtype in (torch.float32, torch.bfloat16) else torch.float32
            rows = torch.empty(a.shape[0], a.shape[-1], dtype=torch.float32, device=a.device)
            gain = m.weight.detach()
            if gain.dtype not in (torch.float32, torch.bfloat16):
                gain = gain.float()  # it has no part in the rows, but the call reads it
            dp_rms_norm_backward(g.to(dt).contiguous(), a.to(dt).contiguous(), gain, _torch_eps(m, a.dtype),
                                 gain_rows=rows)
        B = rows.shape[0]
        return torch.ones(B, 1, 1, dtype=torch.float32, device=rows.device), rows.view(B, 1, -1)

    @staticmethod
    def _norm_bias(m):
        return isinstance(m, LayerNorm) and m.bias is not None and m.bias.requires_grad

    def _table_operands(self, L):
        """(ids [B, T], G [B, T, d]) of a table of words, contiguous; tokens that
        have no gradient (an id outside the table, torch's padding_idx) are -1
        or stay outside."""
        m, ids, g = L.module, L.a, L.g
        if ids is None or g is None:
            raise RuntimeError("step() needs one forward and one backward pass of every layer first")
        if _version(ids) != L.version:
            raise RuntimeError("an Embedding's ids were changed in place between its forward pass and step(), which sorts "
                               "the gradients by them")
        if ids.dim() < 1:
            raise RuntimeError("an Embedding's ids must have one row per sample")
        ids = ids.reshape(ids.shape[0], -1).to(torch.int64)
        if getattr(m, "padding_idx", None) is not None:
            ids = torch.where(ids == m.padding_idx, torch.full_like(ids, -1), ids)
        dt = g.dtype if g.dtype in (torch.float32, torch.bfloat16) else torch.float32
        return ids.contiguous(), g.to(dt).reshape(*ids.shape, g.shape[-1]).contiguous()

    def _operands(self, L):
        """(A [B, T, d], G [B, T, p]) of one layer, contiguous, in the activation dtype;
        for a conv layer taken folded, (a [B, C_in, H, W], G [B, T, p], geometry);
        for an expert layer its rows (A [R, d], G [R, p])."""
        m, a, g = L.module, L.a, L.g
        if a is None or g is None:
            raise RuntimeError("step() needs one forward and one backward pass of every layer first")
        B = a.shape[0]
        dt = a.dtype if a.dtype in (torch.float32, torch.bfloat16) else torch.float32
        if isinstance(m, ExpertLinear):
            return _aligned(a.to(dt)), _aligned(g.to(dt))
        elif isinstance(m, torch.nn.Linear):
            A = a.reshape(B, -1, a.shape[-1])
            G = g.reshape(B, -1, g.shape[-1])
        elif self._is_folded(L):
            geo = conv_geometry(a.shape[1], a.shape[2], a.shape[3], m.kernel_size, m.stride, self._padding(m),
                                m.dilation)
            G = g.reshape(B, g.shape[1], -1).transpose(1, 2)
            return a.to(dt).contiguous(), G.to(dt).contiguous(), geo
        elif self.library_unfold:
            geo = conv_geometry(a.shape[1], a.shape[2], a.shape[3], m.kernel_size, m.stride, self._padding(m),
                                m.dilation)
            A = dp_unfold2d(a.to(dt).contiguous(), geo)  # [B, T, D], written by the library
            G = g.reshape(B, g.shape[1], -1).transpose(1, 2)
        else:
            U = F.unfold(a, m.kernel_size, dilation=m.dilation, padding=self._padding(m), stride=m.stride)  # [B, D, L]
            A = U.transpose(1, 2)
            G = g.reshape(B, g.shape[1], -1).transpose(1, 2)
        return A.to(dt).contiguous(), G.to(dt).contiguous()

    def _check_flat_ids(self, ops, B):
        """A table's ids of one dimension are a token of each sample, or positions
        whose rows the whole batch shares: as many of them as samples look the
        same. They are taken where no other layer has several rows per sample."""
        flat = [k for k, L in enumerate(self.layers) if isinstance(L.module, _TABLES) and L.a.dim() == 1]
        if not flat or B == 1:
            return
        for k, (L, op) in enumerate(zip(self.layers, ops)):
            if isinstance(L.module, _NORMS):
                rows = L.a.numel() // L.a.shape[-1]
            elif isinstance(L.module, ExpertLinear):
                rows = op[0].shape[0]
            elif isinstance(L.module, _TABLES):
                rows = op[0].numel()
            else:
                rows = B * op[1].shape[1]
            if rows > B:
                raise RuntimeError("an Embedding's ids have one dimension where another layer has several rows per "
                                   "sample: a row of ids that all samples share has no per-sample gradient. Give each "
                                   "sample its own, [B, T] (one token of each sample: [B, 1])")

    def step(self, step: int, denom: float | None = None):
        """Clipped noised mean gradients into .grad; returns the per-sample norms.

        The noise stream of a layer is its index in the engine's layer list
        (the model's module order), whichever call serves it."""
        gains = [k for k, L in enumerate(self.layers) if isinstance(L.module, _NORMS)]
        tables = [k for k, L in enumerate(self.layers) if isinstance(L.module, _TABLES)]
        experts = [k for k, L in enumerate(self.layers) if isinstance(L.module, ExpertLinear)]
        ops = [self._gain_operands(L) if k in gains else self._table_operands(L) if k in tables else self._operands(L)
               for k, L in enumerate(self.layers)]
        batch = {op[0].shape[0] if k not in experts
                 else (self.layers[k].segments.numel() - 1) // self.layers[k].module.weight.shape[0]
                 for k, op in enumerate(ops)}
        if len(batch) != 1:
            raise RuntimeError(f"all layers must share one batch size, got {sorted(batch)}")
        B = batch.pop()
        self._check_flat_ids(ops, B)
        dev = ops[0][0].device
        dtypes = {op[0].dtype for k, op in enumerate(ops) if k not in gains and k not in tables}
        if len(dtypes) > 1:
            raise RuntimeError("all layers must share one activation dtype")
        dt = DP_BF16 if dtypes == {torch.bfloat16} else DP_F32
        denom = float(B) if denom is None else float(denom)
        has_bias = [k not in gains and getattr(L.module, "bias", None) is not None and L.module.bias.requires_grad
                    for k, L in enumerate(self.layers)]
        others = set(gains) | set(experts) | set(tables)
        # [B, T, d] operands: multi-layer calls; folded conv inputs: dp_conv_* calls
        dense = [k for k, op in enumerate(ops) if len(op) == 2 and k not in others]
        folded = [k for k, op in enumerate(ops) if len(op) == 3]
        sq = torch.empty(B, dtype=torch.float32, device=dev)
        c = torch.empty(B, dtype=torch.float32, device=dev)
        norms = torch.empty(B, dtype=torch.float32, device=dev)
        ws = None
        started = False  # sq holds the layers so far
        if dense:
            dops, dhb = [ops[k] for k in dense], [has_bias[k] for k in dense]
            ws = torch.empty(max(256, dp_layers_workspace_bytes(dops, has_bias=dhb, mode=self.mode,
                                                                kappa=self.kappa)), dtype=torch.uint8, device=dev)
            if folded or others:
                dp_ghost_norm_layers(dops, sq, has_bias=dhb, mode=self.mode, kappa=self.kappa, workspace=ws)
            else:  # every layer in this call: its kernels form the clip factors too (the same bits)
                dp_ghost_norm_clip_layers(dops, sq, self.C, c, norms, has_bias=dhb, mode=self.mode,
                                          kappa=self.kappa, workspace=ws)
            started = True
        wsc = {}
        for k in folded:
            a, G, geo = ops[k]
            wsc[k] = torch.empty(max(256, dp_conv_workspace_bytes(geo, dt, B, G.shape[2], has_bias[k], self.mode,
                                                                  self.kappa)), dtype=torch.uint8, device=dev)
            dp_conv_norm(a, G, geo, sq, has_bias=has_bias[k], mode=self.mode, kappa=self.kappa,
                         accumulate=started, workspace=wsc[k])
            started = True
        if gains:
            gops = [ops[k] for k in gains]
            dp_ghost_norm_layers(gops, sq, accumulate=started)
            started = True
        for k in experts:
            A, G = ops[k]
            E, p, d = self.layers[k].module.weight.shape
            wsc[k] = torch.empty(max(256, dp_grouped_workspace_bytes(dt, A.shape[0], E, B, d, p)), dtype=torch.uint8,
                                 device=dev)
            dp_grouped_norm(A, G, self.layers[k].segments, sq, accumulate=started, workspace=wsc[k])
            started = True
        sorted_tokens = {}
        for k in tables:
            ids, G = ops[k]
            V, d = self.layers[k].module.weight.shape
            order = torch.empty(ids.numel(), dtype=torch.int64, device=dev)
            starts = torch.empty(V + 1, dtype=torch.int64, device=dev)
            dp_embedding_order(ids, V, order, starts)
            sorted_tokens[k] = order, starts
            wsc[k] = torch.empty(dp_embedding_workspace_bytes(DP_BF16 if G.dtype == torch.bfloat16 else DP_F32, B,
                                                              ids.shape[1], V, d), dtype=torch.uint8, device=dev)
            dp_embedding_norm(G, ids, order, starts, sq, scale=getattr(self.layers[k].module, "scale", 1.0),
                              accumulate=started, workspace=wsc[k])
            started = True
        if folded or others:
            dp_clip_factors(sq, self.C, c, norms)
        outs = [torch.empty(self.layers[k].module.weight.transpose(1, 2).shape if k in experts
                            else self.layers[k].module.weight.shape if k in tables
                            else ((op[2].C_in * op[2].kh * op[2].kw if len(op) == 3 else op[0].shape[2]),
                                  op[1].shape[2]), dtype=torch.float32, device=dev) for k, op in enumerate(ops)]
        bouts = [torch.empty(op[1].shape[2], dtype=torch.float32, device=dev) if hb else None
                 for op, hb in zip(ops, has_bias)]
        if dense:
            dp_clipped_sum_noise_layers([ops[k] for k in dense], c, self.C, self.sigma, denom, self.seed, step,
                                        [outs[k] for k in dense],
                                        bias_outs=[bouts[k] for k in dense] if any(dhb) else None, has_bias=dhb,
                                        layer_ids=dense, workspace=ws)
        for k in folded:
            a, G, geo = ops[k]
            dp_conv_clipped_sum_noise(a, G, geo, c, self.C, self.sigma, denom, self.seed, k, step, outs[k],
                                      bias_out=bouts[k], workspace=wsc[k])
        if gains:
            dp_clipped_sum_noise_layers([ops[k] for k in gains], c, self.C, self.sigma, denom, self.seed, step,
                                        [outs[k] for k in gains], layer_ids=gains)
        for k in experts:
            A, G = ops[k]
            dp_grouped_clipped_sum_noise(A, G, self.layers[k].segments, c, self.C, self.sigma, denom, self.seed, k,
                                         step, outs[k], workspace=wsc[k])
        for k in tables:
            ids, G = ops[k]
            dp_embedding_clipped_sum_noise(G, ids, *sorted_tokens[k], c, self.C, self.sigma, denom, self.seed, k, step,
                                           outs[k], scale=getattr(self.layers[k].module, "scale", 1.0),
                                           workspace=wsc[k])
        for L, out, bout in zip(self.layers, outs, bouts):
            w = L.module.weight
            if isinstance(L.module, ExpertLinear):
                w.grad = out.transpose(1, 2).to(w.dtype).contiguous()  # [E, p, d]
            elif isinstance(L.module, _TABLES):
                if getattr(L.module, "padding_idx", None) is not None:
                    out[L.module.padding_idx].zero_()  # no sample has a gradient there: the row needs no noise
                w.grad = out.to(w.dtype)  # [V, d]
            elif isinstance(L.module, LayerNorm):  # [1, d], or [1, 2d] with the bias
                d = w.numel()
                w.grad = out[0, :d].to(w.dtype).contiguous()
                if self._norm_bias(L.module):
                    L.module.bias.grad = out[0, d:].to(L.module.bias.dtype).contiguous()
            elif w.requires_grad:
                w.grad = out.t().reshape(w.shape).to(w.dtype).contiguous()  # [p, d] (conv: [C_out, C_in, kH, kW])
            if bout is not None:
                L.module.bias.grad = bout.to(L.module.bias.dtype)
            L.a = L.g = L.segments = None
            if isinstance(L.module, (RMSNorm, LayerNorm)):
                _forget_rows(L.module)
        self.last_norms = norms
        return norms
