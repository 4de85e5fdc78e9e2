"""What the engine and the language-model modules hand to the library, without
a GPU: the library's calls are replaced by plain forms, so that the hooks and
the marshalling run on host tensors."""
from __future__ import annotations

import pytest
import torch

import sample_gradient_clipping_layer_amd.engine as eng
import sample_gradient_clipping_layer_amd.layers as lay
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine
from sample_gradient_clipping_layer_amd.layers import ExpertLinear, RMSNorm

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


def _grouped_matmul(X, W, segments, out, transpose=False, workspace=None, stream=None):
    E = W.shape[0]
    B = (segments.numel() - 1) // E
    for e in range(E):
        i, j = int(segments[e * B]), int(segments[(e + 1) * B])
        out[i:j] = X[i:j] @ (W[e] if transpose else W[e].T)


def _rms_norm(x, gain, eps, out, residual=None, sum_out=None, stream=None):
    s = x if residual is None else x + residual
    out.copy_(s * torch.rsqrt((s * s).mean(-1, keepdim=True) + eps) * gain)
    if sum_out is not None:
        sum_out.copy_(s)


def _rms_back(dy, s, gain, eps, dx=None, dsum=None, gain_rows=None, workspace=None, stream=None):
    if gain_rows is not None:
        _rms_rows(dy, s, gain, eps, gain_rows=gain_rows)
    if dx is not None:
        rstd = torch.rsqrt((s * s).mean(-1, keepdim=True) + eps)
        u, h = s * rstd, dy * gain
        dx.copy_(rstd * (h - u * (h * u).mean(-1, keepdim=True)) + (0 if dsum is None else dsum))


@pytest.fixture
def plain_calls(monkeypatch):
    monkeypatch.setattr(eng, "dp_rms_norm_backward", _rms_rows)
    monkeypatch.setattr(lay, "dp_rms_norm", _rms_norm)
    monkeypatch.setattr(lay, "dp_rms_norm_backward", _rms_back)
    monkeypatch.setattr(lay, "dp_grouped_matmul", _grouped_matmul)


SEG = torch.tensor([0, 1, 3, 4, 6])  # 2 experts, 2 samples, 6 rows


@pytest.mark.parametrize("call", [lambda m, x: m(x, SEG), lambda m, x: m(x, segments=SEG), lambda m, x: m(x=x, segments=SEG),
                                  lambda m, x: m(segments=SEG, x=x)])
def test_experts_called_by_keyword(plain_calls, call):
    m = ExpertLinear(2, 3, 4)
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    x = torch.arange(18.0).reshape(6, 3).requires_grad_()
    g = torch.arange(24.0).reshape(6, 4)
    (call(m, x) * g).sum().backward()
    kept = engine.layers[0]
    assert torch.equal(kept.a, x.detach()) and torch.equal(kept.segments, SEG) and torch.equal(kept.g, g)
    engine.detach()


@pytest.mark.parametrize("make,name", [(lambda: RMSNorm(3), "x"), (lambda: torch.nn.RMSNorm(3, eps=1e-6), "x"),
                                       (lambda: torch.nn.Linear(3, 3), "input")])
def test_layers_called_by_keyword(plain_calls, make, name):
    m = make()
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    x = torch.arange(6.0).reshape(2, 3)
    kept = []
    for call in (lambda: m(x), lambda: m(**{name: x})):
        call().sum().backward()
        L = engine.layers[0]
        kept.append((L.a, L.g))
    assert torch.equal(kept[0][0], kept[1][0]) and torch.equal(kept[0][1], kept[1][1])
    engine.detach()


@pytest.mark.parametrize("default", [torch.float32, torch.float64, torch.bfloat16])
def test_expert_gradients_under_another_default_type(plain_calls, monkeypatch, default):
    """Without an engine the weight's gradient is the clipped sum under factors
    1, which the library takes in float32 whatever torch's default type is."""
    def grouped_sum(A, G, segments, c, C, sigma, denom, seed, layer_id, step, out, workspace=None, stream=None):
        assert c.dtype == torch.float32 and out.dtype == torch.float32 and (c == 1).all()
        E, B = out.shape[0], c.numel()
        for e in range(E):
            i, j = int(segments[e * B]), int(segments[(e + 1) * B])
            out[e] = A[i:j].T @ G[i:j] / denom

    monkeypatch.setattr(lay, "dp_grouped_clipped_sum_noise", grouped_sum)
    m = ExpertLinear(2, 3, 4, dtype=torch.float32)
    x, g = torch.arange(18, dtype=torch.float32).reshape(6, 3), torch.arange(24, dtype=torch.float32).reshape(6, 4)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        (m(x, SEG) * g).sum().backward()
    finally:
        torch.set_default_dtype(before)
    want = torch.stack([g[0:3].T @ x[0:3], g[3:6].T @ x[3:6]])
    assert torch.equal(m.weight.grad, want)


def _off(t):
    """t's values in a contiguous view that starts one element off a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def test_views_off_a_16_byte_boundary_reach_the_calls_aligned(plain_calls, monkeypatch):
    """.contiguous() keeps a view's offset; the grouped and distillation calls
    take 16-byte aligned tensors only."""
    seen = []

    def watch(name, f):
        def call(*args, **kw):
            big = args[:4] if name == "dp_grouped_matmul" else args[:2]
            assert all(t.data_ptr() % (8 if t.dtype == torch.int64 else 16) == 0 for t in big), name
            seen.append(name)
            return f(*args, **kw)
        return call

    monkeypatch.setattr(lay, "dp_grouped_matmul", watch("dp_grouped_matmul", _grouped_matmul))
    monkeypatch.setattr(lay, "dp_grouped_clipped_sum_noise", watch("sum", lambda *a, **k: a[10].zero_()))
    monkeypatch.setattr(lay, "dp_distill_loss", lambda z, *a, **k: (seen.append("loss"), a[3].zero_(), a[4].zero_(),
                                                                    [1 / (z.data_ptr() % 16 == 0)]))
    monkeypatch.setattr(lay, "dp_distill_loss_backward", lambda z, ids, t, tau, lse, grad, **k: grad.zero_())
    m = ExpertLinear(2, 3, 5)
    m.weight = torch.nn.Parameter(_off(m.weight.detach()))  # parameters of a flat buffer
    x, g = _off(torch.ones(6, 3)).requires_grad_(), _off(torch.ones(6, 5))
    m(x, SEG).backward(g)
    assert seen == ["dp_grouped_matmul", "dp_grouped_matmul", "sum"]
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    m(x, SEG).backward(g)
    A, G = engine._operands(engine.layers[0])
    assert A.data_ptr() % 16 == 0 and G.data_ptr() % 16 == 0
    assert torch.equal(A, x.detach()) and torch.equal(G, g)
    engine.detach()
    z = _off(torch.ones(2, 3, 5)).requires_grad_()
    lay.distillation_loss(z, torch.zeros(2, 3, 1, dtype=torch.int64), torch.zeros(2, 3, 1)).sum().backward()
    assert "loss" in seen and z.grad.shape == z.shape


@pytest.mark.parametrize("use", ["y", "s", "both"])
def test_a_batch_left_out_does_not_count_as_a_second_run(plain_calls, use):
    """Forward and backward without a step (a batch that is thrown away), then
    the next batch, also where only the norm's sum enters the loss; a forward
    pass without its backward is still told from it."""
    m = RMSNorm(4)
    engine = PrivacyEngine(m, C=1.0, sigma=0.0)
    g = torch.Generator().manual_seed(2)
    for _ in range(3):
        x, r = torch.randn(2, 3, 4, generator=g).requires_grad_(), torch.randn(2, 3, 4, generator=g)
        y, s = m(x, r)
        (y if use == "y" else s if use == "s" else y + s).sum().backward()
    rows = engine._gain_operands(engine.layers[0])[1]
    v = (x + r).detach().double()
    want = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6)).sum(1) * (use != "s")
    assert (rows[:, 0].double() - want).abs().max() < 1e-5
    m(x, r)
    with pytest.raises(RuntimeError, match="twice"):
        m(x, r)
    engine.detach()
