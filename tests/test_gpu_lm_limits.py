"""The dp_grouped_* calls at row and range counts near their stated limits, at
widths of a few elements, against sums in 64 bits."""
from __future__ import annotations

import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc

pytestmark = pytest.mark.gpu


def _cuda_gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _inputs(E, B, lo, hi, d, p, dt):
    """Row counts in [lo, hi) of E*B ranges (none where negative), and rows A [R, d], G [R, p]."""
    g = _cuda_gen(E + B)
    counts = torch.randint(lo, hi, (E * B,), generator=g, device="cuda").clamp_(min=0)
    seg = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    R = int(seg[-1])
    A, G = (torch.randn(R, n, generator=g, device="cuda").to(dt) for n in (d, p))
    return counts, seg, A, G


def _range_grads(A, G, counts):
    """Per (expert, sample) range: sum_r a_r g_r^T and the same of magnitudes, in 64 bits."""
    k = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts)
    outer = A.double()[:, :, None] * G.double()[:, None, :]
    zero = torch.zeros(counts.numel(), *outer.shape[1:], dtype=torch.float64, device="cuda")
    return zero.index_add(0, k, outer), zero.index_add(0, k, outer.abs())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ten_million_ranges(dtype):
    """10 experts, a million samples, most ranges empty."""
    E, B, d, p, dt = 10, 1000000, 3, 2, L.DT[dtype]
    counts, seg, A, G = _inputs(E, B, -7, 3, d, p, dt)
    R, g = A.shape[0], _cuda_gen(3)
    grads, mags = _range_grads(A, G, counts)
    grads, mags = grads.view(E, B, d, p), mags.view(E, B, d, p)
    sq = torch.empty(B, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, (grads ** 2).sum((0, 2, 3)), (mags ** 2).sum((0, 2, 3)) * 64 * L.U + 1e-37, "sqnorm")
    c = torch.rand(B, generator=g, device="cuda") * (torch.arange(B, device="cuda") >= B - 500)
    out = torch.empty(E, d, p, device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    cc = c.double()[None, :, None, None]
    rows = int(counts.view(E, B)[:, -500:].sum(1).max())
    L.check(out, (cc * grads).sum(1), (rows + 64) * L.U * (cc * mags).sum(1) + 1e-37, "sum")
    W = torch.randn(E, p, d, generator=g, device="cuda").to(dt)
    e = torch.repeat_interleave(torch.arange(E * B, device="cuda"), counts) // B
    for x, transpose, w in ((A, False, W.double().transpose(1, 2)), (G, True, W.double())):
        y = torch.empty(R, w.shape[2], dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(x, W, seg, y, transpose=transpose)
        prod = x.double()[:, :, None] * w[e]
        want = prod.sum(1)
        L.check(y, want, 16 * L.U * prod.abs().sum(1) + L.half(dt) * want.abs() + 1e-37, f"transpose={transpose}")


def test_three_hundred_million_rows():
    """Two experts, 214000 samples of 700 rows each: whole row tiles with fewer
    workgroups each, 9.8 million pieces, 2.3 million product tiles."""
    E, B, dt = 2, 214000, torch.bfloat16
    counts, seg, A, G = _inputs(E, B, 650, 752, 1, 1, dt)
    R = int(seg[-1])
    assert R > 295000000
    grads, mags = (v.view(E, B) for v in _range_grads(A, G, counts))
    sq = torch.empty(B, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, (grads ** 2).sum(0), (mags ** 2).sum(0) * 514 * L.U, "sqnorm")
    c = torch.zeros(B, device="cuda")
    c[-3:] = torch.tensor([0.3, 1.0, 0.7])
    out = torch.empty(E, 1, 1, device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    cc = c[-3:].double()
    L.check(out.view(E), (cc * grads[:, -3:]).sum(1), (3 * 752 + 64) * L.U * (cc * mags[:, -3:]).sum(1), "sum")
    del grads, mags
    W = torch.tensor([1.5, -0.7], device="cuda").to(dt).view(2, 1, 1)
    half = int(seg[B])
    y = torch.empty(R, 1, dtype=dt, device="cuda")
    for transpose in (False, True):
        dpc.dp_grouped_matmul(A, W, seg, y, transpose=transpose)
        # one product of two bf16 values is exact in fp32: its rounding to bf16 is torch's
        assert torch.equal(y[:half], (A[:half].float() * W[0].float()).to(dt))
        assert torch.equal(y[half:], (A[half:].float() * W[1].float()).to(dt))
        y.fill_(0)


def test_eight_million_experts():
    """As many experts as a sum takes, of 0 to 2 rows and one column."""
    E = (1 << 23) - 1
    counts, seg, A, G = _inputs(E, 1, 0, 3, 1, 1, torch.float32)
    out, sq = torch.empty(E, 1, 1, device="cuda"), torch.empty(1, device="cuda")
    c = torch.tensor([0.37], device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    grads, mags = _range_grads(A, G, counts)
    cc = c.double()
    L.check(out, cc * grads, 8 * L.U * cc * mags + 1e-37, "sum")


def test_the_most_rows_and_ranges():
    """2^30 rows in 2^24 ranges of 64: row tiles would need more workgroups
    than a grid has, so the norms go over packed tiles."""
    B, n, dt = 1 << 24, 64, torch.bfloat16
    R = B * n
    seg = torch.arange(B + 1, device="cuda") * n
    g = _cuda_gen(1)
    A, G = (torch.randn(R, 1, generator=g, device="cuda", dtype=dt) for _ in range(2))
    sq = torch.empty(B, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    for i in range(0, B, B // 8):  # a part of the samples at a time
        rows = slice(i * n, (i + B // 8) * n)
        prod = (A[rows].double() * G[rows].double()).view(-1, n)
        L.check(sq[i:i + B // 8], prod.sum(1) ** 2, prod.abs().sum(1) ** 2 * 514 * L.U + 1e-37, "sqnorm")
    c = torch.zeros(B, device="cuda")
    c[-3:] = torch.tensor([0.3, 1.0, 0.7])
    out = torch.empty(1, 1, 1, device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    terms = (A[-3 * n:].double() * G[-3 * n:].double()).view(3, n) * c[-3:, None].double()
    L.check(out.view(()), terms.sum(), (3 * n + 64) * L.U * terms.abs().sum(), "sum")
    y = torch.empty_like(A)
    dpc.dp_grouped_matmul(A, torch.full((1, 1, 1), 1.5, device="cuda", dtype=dt), seg, y)
    assert torch.equal(y, A * 1.5)  # one product, exact in fp32, rounded once
