"""The language-model operators at values and sizes that no model's usual batch
has: teachers of NaN, far more places than words, more tokens or samples than a
grid has workgroups, routings that send everything to one place."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_more_places_than_words(dtype):
    """Every word named many times; each place is a term of its own in the loss."""
    dt, g = L.DT[dtype], L.gen(6)
    B, T, V, K, tau = 2, 4, 53, 2048, 1.3
    logits = L.randn(g, B, T, V, scale=2.0, dtype=dt)
    ids = torch.randint(-1, V + 2, (B, T, K), generator=g).cuda()
    teacher = L.randn(g, B, T, K, dtype=dt)
    loss, lse, grad = torch.empty(B, device="cuda"), torch.empty(B, T, device="cuda"), torch.empty_like(logits)
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse)
    want, wlse, bl, be = L.distill_forward(logits, ids, teacher, tau, None)
    L.check(loss, want, bl, "loss")
    L.check(lse, wlse, be, "lse")
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad)
    L.check(grad, *L.distill_backward(logits, ids, teacher, tau, None, None, lse), "grad")


@pytest.mark.parametrize("B,T", [(3, 400000), (1100000, 2), (1100000, 1)])
def test_distill_more_tokens_than_workgroups(B, T):
    """Workgroups go over more than one token, tokens without weight among
    them, and over more than one sample's sum."""
    dt, g = torch.bfloat16, torch.Generator("cuda").manual_seed(B)
    V, K, tau = 11, 3, 2.0
    logits = (torch.randn(B, T, V, generator=g, device="cuda") * 2).to(dt)
    ids = torch.randint(-1, V, (B, T, K), generator=g, device="cuda")
    teacher = torch.randn(B, T, K, generator=g, device="cuda").to(dt)
    weight = (torch.rand(B, T, generator=g, device="cuda") < 0.7).float()
    loss, lse, grad = torch.empty(B, device="cuda"), torch.empty(B, T, device="cuda"), torch.empty_like(logits)
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse, weight=weight)
    want, wlse, bl, be = L.distill_forward(logits, ids, teacher, tau, weight)
    L.check(loss, want, bl, "loss")
    L.check(lse, wlse, be, "lse")
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad, weight=weight)
    L.check(grad, *L.distill_backward(logits, ids, teacher, tau, weight, None, lse), "grad")


# ---- routings that send everything to one place


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,B,d,p", [(64, 16, 72, 136), (64, 16, 33, 35), (200, 9, 136, 264), (64, 64, 512, 520)])
def test_one_popular_expert(dtype, E, B, d, p):
    """Nearly all rows in one (expert, sample) range, the rest empty or of one
    row: the launch rules go by the average rows per range, which says nothing
    here (thousands of rows on the tiles of short ranges)."""
    dt, g = L.DT[dtype], L.gen(E + d)
    counts = (torch.rand(E, B, generator=g) < 0.05).long()
    counts[E // 2, B // 3] = 3001
    counts[E // 2, B // 3 + 1] = 700
    seg, ends = L.segments_of(counts)
    A, G = L.randn(g, ends[-1], d, scale=d ** -0.5, dtype=dt), L.randn(g, ends[-1], p, dtype=dt)
    sq = torch.empty(B, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, *L.grouped_norm(A, G, ends, B), "sqnorm")
    c = torch.rand(B, generator=g).cuda() + 0.05
    out = torch.empty(E, d, p, device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 4.0, 0, 0, 0, out)
    L.check(out, *L.grouped_sum(A, G, ends, c, 4.0), "sum")
    W = L.randn(g, E, p, d, scale=d ** -0.5, dtype=dt)
    for x, transpose, n in ((A, False, p), (G, True, d)):
        y = torch.empty(ends[-1], n, dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(x, W, seg, y, transpose=transpose)
        L.check(y, *L.grouped_matmul(x, W, ends, B, transpose), f"transpose={transpose}")


def test_norms_of_more_samples_than_workgroups():
    E, B, d = 3, 1100000, 2
    g = torch.Generator("cuda").manual_seed(1)
    counts = torch.randint(0, 2, (E * B,), generator=g, device="cuda")
    seg = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    R = int(seg[-1])
    A, G = (torch.randn(R, d, generator=g, device="cuda") for _ in range(2))
    sq = torch.full((B,), 0.5, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq, accumulate=True)
    row = (A.double() ** 2).sum(1) * (G.double() ** 2).sum(1)  # one row a range at most
    sample = torch.repeat_interleave(torch.arange(E * B, device="cuda"), counts) % B
    want = torch.full((B,), 0.5, dtype=torch.float64, device="cuda").index_add(0, sample, row)
    L.check(sq, want, 64 * L.U * want, "sqnorm")
