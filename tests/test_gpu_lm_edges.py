"""The distillation loss at values where its statistics could hide or invent
something, against its definition."""
from __future__ import annotations

import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 600])
def test_distill_teachers_that_are_nan(dtype, T):
    """A place whose teacher logit is NaN is used: its sample's loss is NaN,
    and so is the gradient at the token's words, whether NaN is all the teacher
    says, its first word or its last; nothing else of the batch is."""
    dt, g = L.DT[dtype], L.gen(5)
    B, V, K, tau = 6, 700, 300, 1.5
    logits = L.randn(g, B, T, V, scale=2.0, dtype=dt)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(B * T)]).reshape(B, T, K).cuda()
    teacher = L.randn(g, B, T, K, dtype=dt)
    nan = float("nan")
    teacher[1, -1] = nan
    teacher[2, 0, 0] = nan
    teacher[3, -1, K - 1] = nan
    ids[4, 0, 1:] = -1
    teacher[4, 0, 0] = nan         # one used place, NaN
    ids[5, 0, 7] = V
    teacher[5, 0, 7] = nan         # an unused one
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, T, device="cuda")
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse)
    assert torch.isnan(loss).tolist() == [False, True, True, True, True, False]
    grad = torch.empty_like(logits)
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad)
    bad = torch.zeros(B, T, V, dtype=torch.bool, device="cuda")
    for b, t in ((1, T - 1), (2, 0), (3, T - 1), (4, 0)):
        used = ids[b, t][(ids[b, t] >= 0) & (ids[b, t] < V)]
        bad[b, t, used] = True
    assert torch.equal(torch.isnan(grad), bad)
    clean = teacher.masked_fill(torch.isnan(teacher), 0.0)
    want, wlse, bl, _ = L.distill_forward(logits, ids, clean, tau, None)
    for b in (0, 5):
        L.check(loss[b], want[b], bl[b], "loss")
    wg, bg = L.distill_backward(logits, ids, clean, tau, None, None, lse)
    L.check(grad[~bad], wg[~bad], bg[~bad], "grad")
