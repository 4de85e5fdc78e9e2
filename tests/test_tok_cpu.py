"""The operators from tokens to a per-sample loss without a GPU: refusals of
the C ABI (every call has an invalid argument and returns before any HIP call)
and of the binding, and the workspace sizes."""
from __future__ import annotations

import os

import pytest
import torch

import sample_gradient_clipping_layer_amd as dpc
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine
from sample_gradient_clipping_layer_amd.layers import Embedding, LayerNorm, RMSNorm, replace_layer_norms, token_loss

FAKE = 0x100000  # aligned, never dereferenced
WS = 1 << 40
NULL, SHAPE, DTYPE, VALUE, WORK, ALIGN = (dpc.DP_ERR_NULL, dpc.DP_ERR_SHAPE, dpc.DP_ERR_DTYPE, dpc.DP_ERR_VALUE,
                                          dpc.DP_ERR_WORKSPACE, dpc.DP_ERR_ALIGN)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dpc.LIB_PATH):
        pytest.fail("libdpclip.so is not built (run __graft_entry__.build())")
    return dpc.lib()


def test_layer_norm_refusals(lib):
    def call(x=FAKE, r=None, gain=FAKE, bias=None, dt=1, gdt=0, rows=4, d=64, eps=1e-6, out=FAKE, s=None):
        return lib.dp_layer_norm(None, x, r, gain, bias, dt, gdt, rows, d, eps, out, s)

    assert call(x=None) == call(gain=None) == call(out=None) == NULL
    assert call(rows=0) == call(d=0) == call(d=32769) == call(rows=1 << 31) == call(rows=-1) == SHAPE
    assert call(dt=2) == call(gdt=7) == DTYPE
    assert call(eps=-1.0) == call(eps=NAN) == call(eps=INF) == VALUE
    assert call(x=FAKE + 1) == call(out=FAKE + 1) == call(r=FAKE + 1) == call(s=FAKE + 1) == ALIGN
    assert call(dt=0, x=FAKE + 2) == call(gain=FAKE + 2) == call(bias=FAKE + 2) == ALIGN


def test_layer_norm_backward_refusals(lib):
    def call(dy=FAKE, s=FAKE, dsum=None, gain=FAKE, dt=1, gdt=0, B=2, T=100, d=64, eps=1e-6, ws=FAKE, n=WS, dx=FAKE,
             rows=FAKE, brows=FAKE):
        return lib.dp_layer_norm_backward(None, dy, s, dsum, gain, dt, gdt, B, T, d, eps, ws, n, dx, rows, brows)

    need = lib.dp_layer_norm_workspace_bytes(1, 2, 100, 64)
    assert need > 0
    assert call(dy=None) == call(s=None) == call(gain=None) == call(dx=None, rows=None, brows=None) == NULL
    assert call(ws=None) == call(ws=None, rows=None) == call(ws=None, brows=None) == NULL
    assert call(B=0) == call(T=0) == call(d=0) == call(d=40000) == call(B=1 << 31) == SHAPE
    assert call(dt=5) == call(gdt=5) == DTYPE
    assert call(eps=-1e-6) == VALUE
    assert call(n=need - 1) == WORK
    assert call(ws=FAKE + 4) == call(rows=FAKE + 2) == call(brows=FAKE + 2) == call(dsum=FAKE + 1) == ALIGN
    assert call(B=(1 << 31) - 1, T=(1 << 31) - 1) == SHAPE


def test_embedding_refusals(lib):
    def look(ids=FAKE, w=FAKE, dt=1, wdt=0, N=5, V=10, d=8, scale=1.0, out=FAKE):
        return lib.dp_embedding(None, ids, w, dt, wdt, N, V, d, scale, out)

    assert look(ids=None) == look(w=None) == look(out=None) == NULL
    for bad in (dict(N=0), dict(V=0), dict(d=0), dict(d=(1 << 20) + 1), dict(N=1 << 31), dict(V=1 << 31), dict(N=-1),
                dict(N=(1 << 31) - 1, d=1 << 20)):
        assert look(**bad) == SHAPE, bad
    assert look(dt=2) == look(wdt=2) == DTYPE
    assert look(scale=NAN) == look(scale=INF) == VALUE
    assert look(ids=FAKE + 4) == look(w=FAKE + 2) == look(out=FAKE + 1) == ALIGN

    def sort(ids=FAKE, N=5, V=10, ws=FAKE, n=WS, o=FAKE, s=FAKE):
        return lib.dp_embedding_order(None, ids, N, V, ws, n, o, s)

    need = lib.dp_embedding_order_workspace_bytes(5, 10)
    assert need > 0 and lib.dp_embedding_order_workspace_bytes(0, 10) == 0
    assert sort(ids=None) == sort(o=None) == sort(s=None) == sort(ws=None) == NULL
    assert sort(N=0) == sort(V=0) == sort(N=1 << 31) == sort(V=1 << 31) == SHAPE
    assert sort(n=need - 1) == WORK
    assert sort(ids=FAKE + 4) == sort(o=FAKE + 4) == sort(s=FAKE + 4) == sort(ws=FAKE + 8) == ALIGN


def test_embedding_gradient_refusals(lib):
    def norm(G=FAKE, dt=1, o=FAKE, B=2, T=30, V=10, d=8, scale=1.0, ws=FAKE, n=WS, sq=FAKE):
        return lib.dp_embedding_norm(None, G, dt, o, B, T, V, d, scale, ws, n, sq, 0)

    def csum(G=FAKE, dt=1, o=FAKE, st=FAKE, B=2, T=30, V=10, d=8, scale=1.0, c=FAKE, C=1.0, sigma=1.0,
             denom=1.0, ws=FAKE, n=WS, out=FAKE):
        return lib.dp_embedding_clipped_sum_noise(None, G, dt, o, st, B, T, V, d, scale, c, C, sigma, denom, 0, 0, 0, ws,
                                                  n, out)

    need = lib.dp_embedding_workspace_bytes(1, 2, 30, 10, 8)
    assert need > 0 and lib.dp_embedding_workspace_bytes(3, 2, 30, 10, 8) == 0
    for f in (norm, csum):
        assert f(G=None) == f(o=None) == f(ws=None) == NULL
        for bad in (dict(B=0), dict(T=0), dict(V=0), dict(d=0), dict(d=(1 << 20) + 1), dict(B=1 << 31), dict(T=1 << 31),
                    dict(B=1 << 16, T=1 << 15), dict(V=1 << 31)):
            assert f(**bad) == SHAPE, bad
        assert f(dt=2) == DTYPE
        assert f(scale=NAN) == VALUE
        assert f(n=need - 1) == WORK
        assert f(G=FAKE + 1) == f(o=FAKE + 4) == f(ws=FAKE + 8) == ALIGN
    assert norm(sq=None) == csum(st=None) == csum(c=None) == csum(out=None) == NULL
    assert norm(sq=FAKE + 2) == csum(st=FAKE + 4) == csum(c=FAKE + 2) == csum(out=FAKE + 2) == ALIGN
    assert csum(C=0.0) == csum(sigma=-1.0) == csum(denom=0.0) == csum(C=NAN) == csum(denom=INF) == VALUE
    assert csum(V=1 << 30, d=1 << 10) == SHAPE  # the noise's group index


def test_token_logprob_refusals(lib):
    def call(z=FAKE, y=FAKE, dt=1, rows=3, V=50, tau=1.0, K=4, lp=FAKE, st=FAKE, h=None, ti=FAKE, tl=FAKE):
        return lib.dp_token_logprob(None, z, y, dt, rows, V, tau, K, lp, st, h, ti, tl)

    def back(z=FAKE, y=FAKE, dt=1, rows=3, V=50, tau=1.0, st=FAKE, dl=FAKE, h=None, dh=None, g=FAKE):
        return lib.dp_token_logprob_backward(None, z, y, dt, rows, V, tau, st, dl, h, dh, g)

    for f in (call, back):
        assert f(z=None) == f(y=None) == f(st=None) == NULL
        assert f(rows=0) == f(V=0) == f(rows=1 << 31) == f(V=1 << 31) == f(rows=1 << 30, V=1 << 30) == SHAPE
        assert f(dt=3) == DTYPE
        assert f(tau=0.0) == f(tau=-1.0) == f(tau=NAN) == f(tau=INF) == f(tau=1e-30) == VALUE
        assert f(z=FAKE + 8) == f(y=FAKE + 4) == f(st=FAKE + 2) == f(h=FAKE + 2) == ALIGN
    assert call(lp=None) == call(ti=None) == call(tl=None) == NULL
    assert call(K=-1) == call(K=51) == call(K=257, V=1000) == SHAPE
    assert call(lp=FAKE + 1) == call(ti=FAKE + 4) == call(tl=FAKE + 2) == ALIGN
    assert back(g=None) == back(dl=None) == back(dh=FAKE) == NULL
    assert back(g=FAKE + 8) == back(dl=FAKE + 1) == back(h=FAKE, dh=FAKE + 2) == ALIGN


def test_balance_refusals(lib):
    def call(z=FAKE, ids=FAKE, dt=1, B=2, T=5000, E=8, top=2, ws=FAKE, n=WS, loss=FAKE, c=FAKE, t=FAKE):
        return lib.dp_balance_loss(None, z, ids, dt, B, T, E, top, ws, n, loss, c, t)

    def back(z=FAKE, ids=FAKE, dt=1, B=2, T=100, E=8, top=2, c=FAKE, t=FAKE, dl=None, g=FAKE):
        return lib.dp_balance_loss_backward(None, z, ids, dt, B, T, E, top, c, t, dl, g)

    need = lib.dp_balance_workspace_bytes(1, 2, 5000, 8)
    assert need > 0 and lib.dp_balance_workspace_bytes(1, 2, 8, 8) == 0 and lib.dp_balance_workspace_bytes(1, 0, 8, 8) == 0
    for f in (call, back):
        assert f(z=None) == f(ids=None) == f(c=None) == f(t=None) == NULL
        for bad in (dict(B=0), dict(T=0), dict(E=0), dict(top=0), dict(E=1025), dict(top=1025), dict(B=1 << 31),
                    dict(T=1 << 31), dict(T=1 << 30)):
            assert f(**bad) == SHAPE, bad
        assert f(dt=2) == DTYPE
        assert f(z=FAKE + 1) == f(ids=FAKE + 4) == f(c=FAKE + 4) == f(t=FAKE + 4) == ALIGN
    assert call(loss=None) == call(ws=None) == back(g=None) == NULL
    assert call(n=need - 1) == WORK
    assert call(loss=FAKE + 2) == call(ws=FAKE + 4) == back(g=FAKE + 1) == back(dl=FAKE + 2) == ALIGN


def test_workspace_sizes(lib):
    assert lib.dp_layer_norm_workspace_bytes(1, 5000, 3, 64) == 0  # a workgroup or wave per sample
    assert lib.dp_layer_norm_workspace_bytes(2, 2, 100, 64) == 0   # invalid
    # tokens' values, and one level of tiles for the runs of a sample, two for the words
    N = 32 * 1024
    assert lib.dp_embedding_workspace_bytes(1, 32, 1024, 50257, 1280) >= (N // 16 + N // 256) * 1280 * 4
    # the order: no list longer than a few words per token and the counts of a workgroup's digits
    assert lib.dp_embedding_order_workspace_bytes((1 << 31) - 1, 50257) < (1 << 31) * 20


def test_binding_refuses_host_and_misshapen_tensors():
    x, gain, ids = torch.zeros(2, 4), torch.ones(4), torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError):
        dpc.dp_layer_norm(x, gain, None, 1e-6, torch.empty_like(x))
    with pytest.raises(ValueError):
        dpc.dp_layer_norm(torch.zeros(0, 4), gain, None, 1e-6, torch.zeros(0, 4))
    with pytest.raises(TypeError):
        dpc.dp_layer_norm(x.half(), gain, None, 1e-6, x.half())
    with pytest.raises(ValueError):
        dpc.dp_layer_norm_backward(gain, gain, gain, 1e-6, dx=gain)
    with pytest.raises(ValueError):
        dpc.dp_embedding(ids, x, torch.zeros(2, 3, 4))
    with pytest.raises(ValueError):
        dpc.dp_embedding(ids, gain, torch.zeros(2, 3, 4))
    with pytest.raises(ValueError):
        dpc.dp_embedding_order(ids, 5, torch.zeros(6, dtype=torch.int64), torch.zeros(6, dtype=torch.int64))
    with pytest.raises(ValueError):
        dpc.dp_embedding_norm(torch.zeros(2, 4, 4), ids, ids.view(-1), ids.view(-1), torch.zeros(2))
    z = torch.zeros(2, 3, 7)
    with pytest.raises(ValueError):
        dpc.dp_token_logprob(z, ids[:, :2], 1.0, torch.zeros(2, 2), torch.zeros(2, 2, 2))
    with pytest.raises(ValueError):
        dpc.dp_token_logprob(z, ids, 1.0, torch.zeros(2, 3), torch.zeros(2, 3, 2), top_ids=ids[..., None])
    with pytest.raises(ValueError):
        dpc.dp_token_logprob_backward(z, ids, 1.0, torch.zeros(2, 3, 2), z.clone())
    with pytest.raises(ValueError):
        dpc.dp_token_logprob_backward(z, ids, 1.0, torch.zeros(2, 3, 2), z.clone(), dentropy=torch.zeros(2, 3))
    with pytest.raises(ValueError):
        dpc.dp_balance_loss(z, ids, torch.zeros(2), torch.zeros(2, 7, dtype=torch.int64), torch.zeros(2, dtype=torch.int64))


def test_engine_covers_tables_and_layer_norms():
    model = torch.nn.Sequential(Embedding(10, 8), LayerNorm(8), torch.nn.Embedding(10, 8, padding_idx=3),
                                LayerNorm(8, bias=False), torch.nn.Linear(8, 2))
    e = PrivacyEngine(model, C=1.0, sigma=1.0)
    assert len(e.layers) == 5 and model[0].private and model[1].private and model[3].private
    e.detach()
    assert not model[0].private and not model[1].private
    with pytest.raises(RuntimeError):
        e.step(0)
    frozen = Embedding(10, 8)
    frozen.weight.requires_grad_(False)
    e = PrivacyEngine(torch.nn.Sequential(frozen, torch.nn.Linear(8, 2)), C=1.0, sigma=1.0)
    assert len(e.layers) == 1 and not frozen.private
    e.detach()


def test_engine_refuses_what_it_cannot_clip():
    for m in (torch.nn.Embedding(4, 4, max_norm=1.0), torch.nn.Embedding(4, 4, scale_grad_by_freq=True),
              torch.nn.Embedding(4, 4, sparse=True), torch.nn.LayerNorm(4), torch.nn.LayerNorm((2, 4))):
        with pytest.raises(ValueError):
            PrivacyEngine(torch.nn.Sequential(torch.nn.Linear(4, 4), m), C=1.0, sigma=1.0)
    frozen = LayerNorm(4)
    frozen.weight.requires_grad_(False)  # its bias alone is trainable
    with pytest.raises(ValueError):
        PrivacyEngine(frozen, C=1.0, sigma=1.0)


@pytest.mark.parametrize("make", [lambda: (Embedding(6, 6), torch.nn.Linear(6, 6, bias=False)),
                                  lambda: (torch.nn.Linear(6, 6, bias=False), Embedding(6, 6)),
                                  lambda: (torch.nn.Embedding(6, 6), torch.nn.Linear(6, 6)),
                                  lambda: (Embedding(6, 6), torch.nn.Embedding(6, 6)),
                                  lambda: (LayerNorm(6), LayerNorm(6)), lambda: (LayerNorm(6), RMSNorm(6))])
def test_engine_refuses_shared_tables_and_norms(make):
    """A table tied to the head among them: the two gradients of a sample would
    have to be added before their norm."""
    a, b = make()
    b.weight = a.weight
    with pytest.raises(ValueError):
        PrivacyEngine(torch.nn.Sequential(a, b), C=1.0, sigma=1.0)
    assert not getattr(a, "private", False) and not getattr(b, "private", False)


def test_replace_layer_norms():
    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.ln = torch.nn.LayerNorm(8, eps=3e-4)
            self.again = self.ln
            self.parts = torch.nn.ModuleList([torch.nn.LayerNorm(8, bias=False), torch.nn.Linear(8, 8)])
            self.plain = torch.nn.LayerNorm(8, elementwise_affine=False)
            self.nothing = None

    m = Block()
    before, params = list(m.state_dict()), dict(m.named_parameters())
    assert replace_layer_norms(m) is m
    assert list(m.state_dict()) == before
    assert all(p is params[n] for n, p in m.named_parameters())
    assert isinstance(m.ln, LayerNorm) and m.ln is m.again and m.ln.eps == 3e-4
    assert isinstance(m.parts[0], LayerNorm) and m.parts[0].bias is None
    assert type(m.plain) is torch.nn.LayerNorm
    assert isinstance(replace_layer_norms(torch.nn.LayerNorm(4)), LayerNorm)
    with pytest.raises(ValueError):
        LayerNorm.from_torch(torch.nn.LayerNorm((2, 4)))


def test_layers_refuse_host_tensors():
    ids = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError):
        Embedding(4, 8)(ids)
    with pytest.raises(ValueError):
        LayerNorm(8)(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        token_loss(torch.zeros(2, 3, 5), ids)
