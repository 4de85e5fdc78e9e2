"""What the engine and the modules from tokens to a per-sample loss hand to the
library and make of what it returns, without a GPU: the library's calls are
replaced by plain ones, so that the hooks and the marshalling run on host
tensors."""
from __future__ import annotations

import pytest
import torch

import sample_gradient_clipping_layer_amd.engine as eng
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
