"""The language-model operators without a GPU: refusals of the C ABI (every
call has an invalid argument and returns before any HIP call), of the binding
and of the engine, the workspace sizes, and the routing helper."""
from __future__ import annotations

import os

import pytest
import torch

import sample_gradient_clipping_layer_amd as dpc
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine
from sample_gradient_clipping_layer_amd.layers import ExpertLinear, RMSNorm, distillation_loss, route

FAKE = 0x100000  # aligned, never dereferenced
WS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dpc.LIB_PATH):
        pytest.fail("libdpclip.so is not built (run __graft_entry__.build())")
    return dpc.lib()


NULL, SHAPE, DTYPE, VALUE, WORK, ALIGN = (dpc.DP_ERR_NULL, dpc.DP_ERR_SHAPE, dpc.DP_ERR_DTYPE, dpc.DP_ERR_VALUE,
                                          dpc.DP_ERR_WORKSPACE, dpc.DP_ERR_ALIGN)
INF, NAN = float("inf"), float("nan")


def test_rms_norm_refusals(lib):
    def call(x=FAKE, r=None, gain=FAKE, dt=1, gdt=0, rows=4, d=64, eps=1e-6, out=FAKE, s=None):
        return lib.dp_rms_norm(None, x, r, gain, dt, gdt, rows, d, eps, out, s)

    assert call(x=None) == call(gain=None) == call(out=None) == NULL
    assert call(rows=0) == call(d=0) == call(d=32769) == call(rows=1 << 31) == call(rows=-1) == SHAPE
    assert call(dt=2) == call(gdt=7) == DTYPE
    assert call(eps=-1.0) == call(eps=NAN) == call(eps=INF) == VALUE
    assert call(x=FAKE + 1) == call(out=FAKE + 1) == call(r=FAKE + 1) == call(s=FAKE + 1) == ALIGN
    assert call(dt=0, x=FAKE + 2) == call(gain=FAKE + 2) == ALIGN


def test_rms_norm_backward_refusals(lib):
    def call(dy=FAKE, s=FAKE, dsum=None, gain=FAKE, dt=1, gdt=0, B=2, T=100, d=64, eps=1e-6, ws=FAKE, n=WS, dx=FAKE,
             rows=FAKE):
        return lib.dp_rms_norm_backward(None, dy, s, dsum, gain, dt, gdt, B, T, d, eps, ws, n, dx, rows)

    need = lib.dp_rms_norm_workspace_bytes(1, 2, 100, 64)
    assert need > 0
    assert call(dy=None) == call(s=None) == call(gain=None) == call(dx=None, rows=None) == call(ws=None) == NULL
    assert call(B=0) == call(T=0) == call(d=0) == call(d=40000) == call(B=1 << 31) == SHAPE
    assert call(dt=5) == call(gdt=5) == DTYPE
    assert call(eps=-1e-6) == VALUE
    assert call(n=need - 1) == WORK
    assert call(ws=FAKE + 4) == call(rows=FAKE + 2) == call(dsum=FAKE + 1) == ALIGN
    # too many elements, checked before anything is touched
    assert call(B=(1 << 31) - 1, T=(1 << 31) - 1) == SHAPE


def test_distill_refusals(lib):
    def call(z=FAKE, ids=FAKE, t=FAKE, dt=1, tdt=0, B=2, T=3, V=50, K=4, tau=1.0, w=None, ws=FAKE, n=WS, loss=FAKE,
             lse=FAKE):
        return lib.dp_distill_loss(None, z, ids, t, dt, tdt, B, T, V, K, tau, w, ws, n, loss, lse)

    def back(z=FAKE, ids=FAKE, t=FAKE, dt=1, tdt=0, B=2, T=3, V=50, K=4, tau=1.0, w=None, dl=None, lse=FAKE, g=FAKE):
        return lib.dp_distill_loss_backward(None, z, ids, t, dt, tdt, B, T, V, K, tau, w, dl, lse, g)

    need = lib.dp_distill_workspace_bytes(1, 2, 3, 50, 4)
    assert need > 0
    for f in (call, back):
        assert f(z=None) == f(ids=None) == f(t=None) == f(lse=None) == NULL
        assert f(B=0) == f(T=0) == f(V=0) == f(K=0) == f(K=2049) == f(V=1 << 31) == f(T=1 << 31) == SHAPE
        assert f(dt=3) == f(tdt=3) == DTYPE
        assert f(tau=0.0) == f(tau=-1.0) == f(tau=NAN) == f(tau=INF) == VALUE
        assert f(z=FAKE + 8) == f(ids=FAKE + 4) == f(t=FAKE + 1) == f(w=FAKE + 2) == f(lse=FAKE + 2) == ALIGN
    assert call(loss=None) == call(ws=None) == back(g=None) == NULL
    assert call(n=need - 1) == WORK
    assert back(g=FAKE + 8) == back(dl=FAKE + 1) == ALIGN


def test_grouped_refusals(lib):
    size = dict(R=100, E=3, B=4, d=64, p=128)

    def mm(X=FAKE, W=FAKE, dt=1, seg=FAKE, tr=0, ws=FAKE, n=WS, Y=FAKE, **kw):
        s = {**size, **kw}
        return lib.dp_grouped_matmul(None, X, W, dt, seg, s["R"], s["E"], s["B"], s["d"], s["p"], tr, ws, n, Y)

    def norm(X=FAKE, W=FAKE, dt=1, seg=FAKE, ws=FAKE, n=WS, Y=FAKE, **kw):
        s = {**size, **kw}
        return lib.dp_grouped_norm(None, X, W, dt, seg, s["R"], s["E"], s["B"], s["d"], s["p"], ws, n, Y, 0)

    def csum(X=FAKE, W=FAKE, dt=1, seg=FAKE, c=FAKE, C=1.0, sigma=1.0, denom=1.0, ws=FAKE, n=WS, Y=FAKE, **kw):
        s = {**size, **kw}
        return lib.dp_grouped_clipped_sum_noise(None, X, W, dt, seg, s["R"], s["E"], s["B"], s["d"], s["p"], c, C,
                                                sigma, denom, 0, 0, 0, ws, n, Y)

    for f in (mm, norm, csum):
        assert f(X=None) == f(W=None) == f(seg=None) == f(Y=None) == NULL
        for bad in (dict(R=0), dict(E=0), dict(B=0), dict(d=0), dict(p=0), dict(R=1 << 31), dict(d=(1 << 20) + 1),
                    dict(E=1 << 20, B=1 << 20), dict(E=1 << 16, B=1, d=1 << 18, p=1 << 18), dict(R=-5)):
            assert f(**bad) == SHAPE, bad
        assert f(dt=2) == DTYPE
        assert f(X=FAKE + 8) == f(W=FAKE + 8) == f(seg=FAKE + 4) == f(Y=FAKE + 2) == ALIGN
    assert norm(ws=None) == csum(ws=None) == csum(c=None) == NULL
    assert norm(n=0) == csum(n=16) == WORK
    assert csum(C=0.0) == csum(sigma=-1.0) == csum(denom=0.0) == csum(C=NAN) == csum(denom=INF) == VALUE


def test_workspace_sizes(lib):
    assert lib.dp_rms_norm_workspace_bytes(1, 5000, 3, 64) == 0        # a workgroup or wave per sample
    assert lib.dp_rms_norm_workspace_bytes(2, 2, 100, 64) == 0         # invalid
    assert lib.dp_distill_workspace_bytes(1, 600, 1, 100, 4) == 0      # one workgroup per token, one token each
    assert lib.dp_distill_workspace_bytes(1, 2, 3, 0, 4) == 0
    assert lib.dp_grouped_workspace_bytes(1, 0, 3, 4, 8, 8) == 0
    assert lib.dp_grouped_workspace_bytes(0, 100, 3, 4, 8, 8) > 0


def test_binding_refuses_host_and_misshapen_tensors():
    x, gain = torch.zeros(2, 4), torch.ones(4)
    with pytest.raises(ValueError):
        dpc.dp_rms_norm(x, gain, 1e-6, torch.empty_like(x))
    with pytest.raises(TypeError):
        dpc.dp_rms_norm(x.half(), gain, 1e-6, x.half())
    with pytest.raises(ValueError):
        dpc.dp_rms_norm(torch.zeros(0, 4), gain, 1e-6, torch.zeros(0, 4))
    with pytest.raises(ValueError):
        dpc.dp_rms_norm_backward(x[0], x[0], gain, 1e-6, dx=x[0])
    with pytest.raises(ValueError):
        dpc.dp_distill_loss(x, x, x, 1.0, x, x)
    with pytest.raises(ValueError):
        dpc.dp_grouped_matmul(x, torch.zeros(3, 5, 4), torch.zeros(6, dtype=torch.int64), torch.zeros(2, 5))
    with pytest.raises(ValueError):
        dpc.dp_grouped_norm(x, x, torch.zeros(7, dtype=torch.int64), torch.zeros(3))
    with pytest.raises(ValueError):
        route(torch.zeros(3, 4, dtype=torch.int64), 2)


def test_engine_covers_norms_and_experts():
    model = torch.nn.Sequential(RMSNorm(8), ExpertLinear(2, 8, 8), torch.nn.RMSNorm(8), torch.nn.Linear(8, 2))
    e = PrivacyEngine(model, C=1.0, sigma=1.0)
    assert len(e.layers) == 4 and model[0].private and model[1].private
    e.detach()
    assert not model[0].private and not model[1].private
    with pytest.raises(ValueError):
        PrivacyEngine(torch.nn.RMSNorm((4, 8)), C=1.0, sigma=1.0)
    frozen = RMSNorm(8)
    frozen.weight.requires_grad_(False)
    e = PrivacyEngine(torch.nn.Sequential(frozen, torch.nn.Linear(8, 2)), C=1.0, sigma=1.0)
    assert len(e.layers) == 1 and not frozen.private
    e.detach()
    with pytest.raises(RuntimeError):
        PrivacyEngine(RMSNorm(8), C=1.0, sigma=1.0).step(0)


def test_engine_refuses_shared_norm_and_expert_weights():
    for make in (lambda: RMSNorm(8), lambda: torch.nn.RMSNorm(8), lambda: ExpertLinear(2, 8, 8)):
        a, b = make(), make()
        b.weight = a.weight
        with pytest.raises(ValueError):
            PrivacyEngine(torch.nn.Sequential(a, b), C=1.0, sigma=1.0)
        assert not getattr(a, "private", False)


def test_route_orders_by_expert_then_sample():
    g = torch.Generator().manual_seed(0)
    ids = torch.randint(-1, 5, (3, 7, 2), generator=g)
    order, seg = route(ids, 5)
    flat = ids.reshape(-1)
    assert sorted(order.tolist()) == list(range(42))
    for e in range(5):
        for b in range(3):
            rows = order[seg[e * 3 + b]:seg[e * 3 + b + 1]]
            assert (flat[rows] == e).all() and (rows // 14 == b).all()
            assert rows.tolist() == sorted(rows.tolist())
            assert rows.numel() == int((ids[b] == e).sum())
    assert (flat[order[seg[-1]:]] < 0).all()


def test_layers_refuse_host_tensors():
    with pytest.raises(ValueError):
        RMSNorm(4)(torch.zeros(2, 4))
    with pytest.raises(ValueError):
        ExpertLinear(2, 4, 4)(torch.zeros(3, 4), torch.tensor([0, 1, 3]))
    with pytest.raises(ValueError):
        distillation_loss(torch.zeros(1, 2, 4), torch.zeros(1, 2, 1, dtype=torch.int64), torch.zeros(1, 2, 1))
