"""What the engine and the modules from tokens to a per-sample loss hand to the
library and make of what it returns, without a GPU: the library's calls are
replaced by plain ones, so that the hooks and the marshalling run on host
tensors."""
from __future__ import annotations

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import sample_gradient_clipping_layer_amd.engine as eng
import sample_gradient_clipping_layer_amd.layers as lay
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine


@pytest.fixture
def calls(monkeypatch):
    """The engine's calls as ones that leave 1 in every norm and factor and 7 in every sum (a noise that is everywhere)."""
    def fill(k, value, *more):
        return lambda *a, **kw: [a[i].fill_(v) for i, v in ((k, value), *more)]

    def sums(ops, c, C, sigma, denom, seed, step, outs, bias_outs=None, **kw):
        for out in outs + [b for b in bias_outs or [] if b is not None]:
            out.fill_(7)

    for name, f in dict(dp_layers_workspace_bytes=lambda *a, **kw: 256, dp_embedding_workspace_bytes=lambda *a: 256,
                        dp_ghost_norm_layers=fill(1, 1.0), dp_ghost_norm_clip_layers=fill(1, 1.0, (3, 1.0), (4, 1.0)),
                        dp_clip_factors=fill(2, 1.0, (3, 1.0)), dp_clipped_sum_noise_layers=sums,
                        dp_embedding_order=fill(2, 0, (3, 0)), dp_embedding_norm=fill(4, 1.0),
                        dp_embedding_clipped_sum_noise=fill(11, 7.0)).items():
        monkeypatch.setattr(eng, name, f)


@pytest.mark.parametrize("padding", [None, 0, 3, -1])
def test_a_padding_words_row_gets_no_noise(calls, padding):
    m = torch.nn.Embedding(5, 3, padding_idx=padding)
    engine = PrivacyEngine(m, C=1.0, sigma=1.0)
    m(torch.tensor([[0, 3, 4], [1, 2, 4]])).sum().backward()
    engine.step(0)
    engine.detach()
    want = torch.full((5, 3), 7.0)
    if padding is not None:
        want[padding] = 0
    assert torch.equal(m.weight.grad, want)


def _parts(*modules):
    model = torch.nn.ModuleList(modules)
    return PrivacyEngine(model, C=1.0, sigma=0.0), modules


@pytest.mark.parametrize("other", ["words", "linear", "conv", "norm"])
def test_one_row_of_positions_for_all_samples_is_refused(calls, monkeypatch, other):
    """As many positions as samples: the batch sizes agree, but a position's gradient is every sample's. (The other layer
    alone, and the positions of every sample, are taken.)"""
    monkeypatch.setattr(eng, "dp_rms_norm_backward", lambda *a, gain_rows=None, **kw: gain_rows.fill_(1))
    B = T = 4
    layer, x = {"words": (torch.nn.Embedding(9, 8), torch.zeros(B, T, dtype=torch.int64)),
                "linear": (torch.nn.Linear(3, 8), torch.ones(B, T, 3)),
                "conv": (torch.nn.Conv2d(2, 8, 1), torch.ones(B, 2, 1, T)),
                "norm": (torch.nn.RMSNorm(8), torch.ones(B, T, 8))}[other]
    engine, (layer, places) = _parts(layer, torch.nn.Embedding(T, 8))
    engine.library_unfold = False  # torch unfolds on the host

    def loss(at):
        h = layer(x)
        return ((h[:, :, 0].transpose(1, 2) if other == "conv" else h) + places(at)).sum()

    loss(torch.arange(T)).backward()
    with pytest.raises(RuntimeError, match=r"\[B, T\]"):
        engine.step(0)
    loss(torch.arange(T).expand(B, T)).backward()
    engine.step(0)
    engine.detach()


def test_one_token_of_each_sample_is_taken(calls):
    """Ids [B] beside layers with one row per sample, and of a batch of one."""
    engine, (labels, head) = _parts(torch.nn.Embedding(5, 8), torch.nn.Linear(8, 2))
    head(labels(torch.tensor([0, 3, 4]))).sum().backward()
    assert engine.step(0).shape == (3,)
    engine.detach()
    engine, (words, places) = _parts(torch.nn.Embedding(5, 8), torch.nn.Embedding(1, 8))
    (words(torch.tensor([[0, 3, 4]])) + places(torch.tensor([0]))).sum().backward()
    assert engine.step(0).shape == (1,)
    engine.detach()


@pytest.mark.parametrize("table,when", [(torch.nn.Embedding, "after the backward pass"),
                                        (lay.Embedding, "after the backward pass"),
                                        (lay.Embedding, "after the forward pass")])  # (where torch's refuses itself)
def test_ids_changed_in_place_are_refused(calls, monkeypatch, table, when):
    """step() sorts the gradients by the ids: others than those looked up would give them to other words."""
    monkeypatch.setattr(lay, "dp_embedding", lambda ids, weight, out, scale: out.copy_(weight[ids]))
    engine, (m,) = _parts(table(5, 3))
    ids = torch.tensor([[0, 3], [1, 4]])
    y = m(ids)
    if when == "after the forward pass":
        ids[ids == 4] = 2
    y.sum().backward()
    if when == "after the backward pass":
        ids.copy_(torch.tensor([[1, 1], [1, 1]]))
    with pytest.raises(RuntimeError, match="in place"):
        engine.step(0)
    m(ids.clone()).sum().backward()  # the next batch
    engine.step(0)
    with torch.inference_mode():  # ids that do not say how often they were changed
        m(torch.tensor([[0, 3], [1, 4]]))
    engine.detach()


class _Sums(TorchDispatchMode):
    """How many values go into one sum, at most."""

    def __init__(self):
        super().__init__()
        self.most = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "sum" in str(func):
            self.most = max(self.most, args[0].numel() // max(1, out.numel()))
        return out


@pytest.mark.parametrize("B,T", [(1, 1), (3, 4096), (2, 4097), (1, 300001), (1, 1 << 20)])
def test_long_losses_are_summed_in_parts(monkeypatch, B, T):
    """Not as one sum of a row of 131072 or more, for which torch records a memset in a captured graph."""
    monkeypatch.setattr(lay, "token_logprobs", lambda logits, targets, temperature: (logits[..., 0], None))
    g = torch.Generator().manual_seed(T)
    z = torch.randn(B, T, 1, generator=g, dtype=torch.float64).requires_grad_()
    w = torch.rand(B, T, generator=g)
    with _Sums() as sums:
        loss = lay.token_loss(z, torch.zeros(B, T, dtype=torch.int64), w)
    assert sums.most <= 1 << 16
    want = -(z[..., 0] * w).sum(1)
    assert loss.shape == (B,) and torch.allclose(loss, want, rtol=1e-12, atol=1e-9)
    loss.sum().backward()
    assert torch.equal(z.grad[..., 0], -w.double())


def test_replaced_layer_norms_keep_their_hooks(monkeypatch):
    """Hooks of every kind run with the module that took the norm's place, in order, until their handles remove them."""
    monkeypatch.setattr(lay, "dp_layer_norm", lambda x, w, b, eps, out, **kw: out.copy_(torch.layer_norm(x, (4,), w, b, eps)))
    monkeypatch.setattr(lay, "dp_layer_norm_backward", lambda dy, s, w, eps, dx=None, **kw: dx.copy_(dy))
    model = torch.nn.Sequential(torch.nn.LayerNorm(4))
    norm, ran = model[0], []
    norm.requires_grad_(False)
    handles = [norm.register_forward_pre_hook(lambda m, a: ran.append((m, "pre"))),
               norm.register_forward_hook(lambda m, a, k, y: ran.append((m, "forward")), with_kwargs=True),
               norm.register_forward_hook(lambda m, a, y: ran.append((m, "always")), always_call=True),
               norm.register_full_backward_pre_hook(lambda m, g: ran.append((m, "backward pre"))),
               norm.register_full_backward_hook(lambda m, gi, go: ran.append((m, "backward"))),
               norm.register_state_dict_pre_hook(lambda m, prefix, keep: ran.append((m, "state")))]
    lay.replace_layer_norms(model)
    x = torch.arange(8.0).view(2, 4).requires_grad_()
    model(x).sum().backward()
    model.state_dict()
    assert [n for _, n in ran] == ["pre", "forward", "always", "backward pre", "backward", "state"]
    assert all(m is model[0] and type(m) is lay.LayerNorm for m, _ in ran)
    for h in handles:
        h.remove()
    model(x).sum().backward()
    model.state_dict()
    assert len(ran) == 6
