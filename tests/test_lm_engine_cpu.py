"""What the engine and the language-model modules hand to the library, without
a GPU: the library's calls are replaced by plain forms, so that the hooks and
the marshalling run on host tensors."""
from __future__ import annotations

import pytest
import torch

import sample_gradient_clipping_layer_amd.engine as eng
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f64": torch.float64}


def _rms_rows(dy, s, gain, eps, dx=None, dsum=None, gain_rows=None, workspace=None, stream=None):
    """dp_rms_norm_backward's gain rows in 64 bits, with its refusals of types."""
    assert dy.dtype == s.dtype and s.dtype in (torch.float32, torch.bfloat16)
    assert gain.dtype in (torch.float32, torch.bfloat16)
    v = s.double()
    u = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    gain_rows.copy_((dy.double() * u).reshape(s.shape[0], -1, s.shape[-1]).sum(1))


@pytest.mark.parametrize("eps", [None, 3e-5])
@pytest.mark.parametrize("dtype", list(DT))
def test_torch_norms_take_torchs_eps(monkeypatch, dtype, eps):
    """A gain's per-sample gradient is sum_t dy y where the gain is 1, y being
    the module's own output: with eps=None and rows far below 1 the engine has
    to add what torch adds."""
    monkeypatch.setattr(eng, "dp_rms_norm_backward", _rms_rows)
    dt = DT[dtype]
    g = torch.Generator().manual_seed(0)
    scale = 1e-8 if dtype == "f64" else 1e-2 if dtype in ("bf16", "f16") else 1e-4
    x = (torch.randn(3, 5, 64, generator=g) * scale).to(dt)
    t = torch.randn(3, 5, 64, generator=g).to(dt)
    m = torch.nn.RMSNorm(64, eps=eps)
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    y = m(x.requires_grad_())
    (y * t).sum().backward()
    ones, rows = engine._gain_operands(engine.layers[0])
    assert (ones == 1).all() and rows.shape == (3, 1, 64) and rows.dtype == torch.float32
    terms = t.double() * y.detach().double()
    # y is off by half a step of its type and a few of the type torch computes in, the rows by one of fp32 (an fp64
    # input enters the library in fp32: one more, for s and for dy)
    steps = torch.finfo(dt).eps / 2 + 200 * torch.finfo(torch.float32).eps / 2
    assert ((rows[:, 0].double() - terms.sum(1)).abs() <= steps * terms.abs().sum(1)).all()
    engine.detach()


@pytest.mark.parametrize("dtype", list(DT))
def test_torch_norms_of_any_floating_type(monkeypatch, dtype):
    """A norm whose gain has the rows' own type, the types the engine takes of
    linear layers among them."""
    monkeypatch.setattr(eng, "dp_rms_norm_backward", _rms_rows)
    dt = DT[dtype]
    g = torch.Generator().manual_seed(1)
    m = torch.nn.RMSNorm(16, eps=1e-6, dtype=dt)
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    x = torch.randn(2, 3, 16, generator=g).to(dt)
    m(x).sum().backward()
    rows = engine._gain_operands(engine.layers[0])[1]
    u = x.double() * torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    assert ((rows[:, 0].double() - u.sum(1)).abs() <= 8 * torch.finfo(torch.float32).eps * u.abs().sum(1)).all()
    engine.detach()
