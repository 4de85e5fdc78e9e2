"""The language-model operators where a launch rule takes another kernel or a
rarely taken turn inside one: clip factors far apart, many experts, sums split
over K, noise in each epilogue, results at odd addresses, logits of a mask's
value, mixed types, and tensors past 2^31 elements. Sizes are chosen so that
the rules reach the wide kernels; the comments say which."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc
from oracle import noise as N

pytestmark = pytest.mark.gpu


def _counts(g, E, B, lo, hi):
    return torch.randint(lo, hi, (E, B), generator=g)


def _rows(seed, counts, d, p, dt):
    g = L.gen(seed)
    seg, ends = L.segments_of(counts)
    return seg, ends, L.randn(g, ends[-1], d, scale=d ** -0.5, dtype=dt), L.randn(g, ends[-1], p, dtype=dt)


def _sum(A, G, seg, c, shape, denom=4.0, sigma=0.0, noise=(0, 0, 0)):
    out = torch.full(shape, float("nan"), device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, sigma, denom, *noise, out)
    return out


# E, B, rows per (expert, sample) from and to, d, p
WIDE = {
    "pieces": (16, 8, 0, 50, 1016, 1016),         # 256 x 256 tiles, K by pieces of one sample
    "rows": (16, 32, 0, 13, 1016, 1000),          # 256 x 256 tiles, K by rows, factors split over three terms
    "pieces-70": (70, 8, 10, 110, 512, 520),      # more experts than a wave holds
    "rows-70": (70, 64, 0, 10, 520, 768),
    "pieces-split": (1, 8, 1000, 3000, 1024, 1032),   # K split over workgroups
    "rows-split": (1, 2048, 0, 16, 1024, 1032),
    "fold-split": (1, 8, 500, 1500, 128, 136),    # 128 x 128 tiles
    "fold-odd-split": (1, 8, 500, 1500, 129, 131),
    "short-split": (1, 1024, 0, 16, 128, 136),
}


@pytest.mark.parametrize("name", list(WIDE))
def test_wide_sums(name):
    E, B, lo, hi, d, p = WIDE[name]
    g = L.gen(d + p + E)
    counts = _counts(g, E, B, lo, hi)
    if E > 2:
        counts[1] = 0  # an expert without rows
    seg, ends, A, G = _rows(5, counts, d, p, torch.bfloat16)
    c = torch.rand(B, generator=g) + 0.05
    c[torch.rand(B, generator=g) < 0.3] = 1.0
    c[B // 2] = 0.0
    c = c.cuda()
    out = _sum(A, G, seg, c, (E, d, p))
    L.check(out, *L.grouped_sum(A, G, ends, c, 4.0), "sum")
    again = _sum(A, G, seg, c, (E, d, p))
    assert torch.equal(out, again), "the result depends on the order of the work"


@pytest.mark.parametrize("name", ["pieces", "pieces-split", "pieces-70", "rows", "fold-split"])
def test_sums_with_factors_far_apart(name):
    """Factors over 60 binary orders of magnitude within an expert, of both
    signs, and zero: the running sum is held in units of a factor, which must
    neither overflow nor lose the others' parts."""
    E, B, lo, hi, d, p = WIDE[name]
    g = L.gen(9 + d)
    counts = _counts(g, E, B, lo, hi)
    seg, ends, A, G = _rows(6, counts, d, p, torch.bfloat16)
    for k, order in enumerate(([1, 1e-18, 1e-9, -1, 0, 1e9, 1e-18, 0.5], [1e-18, 1e-14, 1e-10, 1e-6, 1e-3, 1, 1e3, 1e9],
                               [1e9, 1e3, 1, 1e-3, 1e-9, 0, 1e-14, 1e-18], [1e-18] * 8, [0] * 8)):
        c = torch.tensor(order, dtype=torch.float32).repeat((B + 7) // 8)[:B].cuda()
        out = _sum(A, G, seg, c, (E, d, p))
        L.check(out, *L.grouped_sum(A, G, ends, c, 4.0), f"order {k}")


@pytest.mark.parametrize("name", list(WIDE))
def test_noise_of_wide_sums_is_the_layers_stream(name):
    """Rows of zeros: the noise alone, bit for bit, from every epilogue."""
    E, B, lo, hi, d, p = WIDE[name]
    g = L.gen(1)
    seg, ends = L.segments_of(_counts(g, E, B, lo, hi))
    A = torch.zeros(ends[-1], d, dtype=torch.bfloat16, device="cuda")
    G = torch.zeros(ends[-1], p, dtype=torch.bfloat16, device="cuda")
    out = _sum(A, G, seg, torch.ones(B, device="cuda"), (E, d, p), 1.0, 1.5, (11, 4, 6))
    rng = np.random.default_rng(d)
    rows = np.concatenate([rng.integers(0, E * d, 20000), np.arange(E * d - 100, E * d)])
    cols = np.concatenate([rng.integers(0, p, 20000), np.full(100, p - 1)])
    z = N.weight_noise_at(rows, cols, p, 11, 4, 6).astype(np.float32)
    np.testing.assert_array_equal(out.cpu().numpy().reshape(E * d, p)[rows, cols], np.float32(1.5) * z)


@pytest.mark.parametrize("name", ["pieces", "rows", "pieces-split", "fold-odd-split"])
@pytest.mark.parametrize("sigma", [0.0, 0.7])
def test_sums_to_an_odd_address(name, sigma):
    E, B, lo, hi, d, p = WIDE[name]
    g = L.gen(2)
    seg, ends, A, G = _rows(7, _counts(g, E, B, lo, hi), d, p, torch.bfloat16)
    c = torch.rand(B, generator=g).cuda()
    want = torch.empty(E, d, p, device="cuda")
    buf = torch.full((E * d * p + 6,), 3.0, device="cuda")
    got = buf[1:1 + E * d * p].view(E, d, p)
    for out in (want, got):
        dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, sigma, 2.0, 1, 2, 3, out)
    assert torch.equal(got, want)
    assert buf[0] == 3.0 and (buf[1 + E * d * p:] == 3.0).all()


# ---- products


@pytest.mark.parametrize("E,lo,hi", [(8, 1500, 2500), (64, 300, 700), (65, 300, 700)])
@pytest.mark.parametrize("transpose", [False, True])
def test_wide_products(E, lo, hi, transpose):
    """256 x 256 tiles (up to 64 experts), K and N no multiples of a chunk or
    a tile, an expert without rows and one of a single row."""
    g = L.gen(E)
    K, Nn = 1032, 1528
    counts = _counts(g, E, 3, lo // 3, hi // 3)
    counts[2] = 0
    counts[3] = torch.tensor([0, 1, 0])
    seg, ends = L.segments_of(counts)
    dt = torch.bfloat16
    X = L.randn(g, ends[-1] + 5, K, dtype=dt)
    W = L.randn(g, E, *((K, Nn) if transpose else (Nn, K)), scale=K ** -0.5, dtype=dt)
    X[ends[-1]:] = float("nan")
    out = torch.full((ends[-1] + 5, Nn), 5.0, dtype=dt, device="cuda")
    dpc.dp_grouped_matmul(X, W, seg, out, transpose=transpose)
    L.check(out[:ends[-1]], *L.grouped_matmul(X[:ends[-1]], W, ends, 3, transpose), "product")
    assert (out[ends[-1]:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[[1]], [[0, 1], [2, 0], [1, 1]], [[3]] * 9])
def test_few_rows_of_wide_experts(dtype, counts):
    """K split over workgroups, its last part short."""
    g = L.gen(len(counts))
    dt, E, B = L.DT[dtype], len(counts), len(counts[0])
    seg, ends = L.segments_of(counts)
    K, Nn = 4104, 136
    X = L.randn(g, ends[-1] + 2, K, dtype=dt)
    for transpose in (False, True):
        W = L.randn(g, E, *((K, Nn) if transpose else (Nn, K)), scale=K ** -0.5, dtype=dt)
        out = torch.full((ends[-1] + 2, Nn), 5.0, dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(X, W, seg, out, transpose=transpose)
        L.check(out[:ends[-1]], *L.grouped_matmul(X[:ends[-1]], W, ends, B, transpose), f"transpose={transpose}")
        assert (out[ends[-1]:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,B,lo,hi,d,p", [(3, 4, 0, 40, 72, 136), (3, 4, 60, 200, 33, 70), (16, 8, 0, 50, 1016, 1016),
                                           (4, 3, 300, 500, 512, 640), (700, 9, 0, 2, 40, 24), (2, 3000, 0, 2, 24, 17)])
def test_rows_ahead_of_and_behind_the_segments(dtype, E, B, lo, hi, d, p):
    """Segments that start behind row 0 and end ahead of row R: the rows
    outside are neither read (they hold NaN) nor written."""
    dt = L.DT[dtype]
    g = L.gen(E * B + d)
    counts = _counts(g, E, B, lo, hi)
    _, ends = L.segments_of(counts)
    head, tail = 37, 130
    n = ends[-1]
    seg = (torch.tensor(ends) + head).cuda()
    A, G = (torch.full((head + n + tail, w), float("nan"), dtype=dt, device="cuda") for w in (d, p))
    a, gr = L.randn(g, n, d, scale=d ** -0.5, dtype=dt), L.randn(g, n, p, dtype=dt)
    A[head:head + n], G[head:head + n] = a, gr
    sq = torch.full((B,), float("nan"), device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, *L.grouped_norm(a, gr, ends, B), "sqnorm")
    c = torch.rand(B, generator=g).cuda()
    out = _sum(A, G, seg, c, (E, d, p))
    L.check(out, *L.grouped_sum(a, gr, ends, c, 4.0), "sum")
    W = L.randn(g, E, p, d, scale=d ** -0.5, dtype=dt)
    for x, part, transpose, w in ((A, a, False, p), (G, gr, True, d)):
        y = torch.full((head + n + tail, w), 5.0, dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(x, W, seg, y, transpose=transpose)
        L.check(y[head:head + n], *L.grouped_matmul(part, W, ends, B, transpose), f"transpose={transpose}")
        assert (y[:head] == 5.0).all() and (y[head + n:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_sample_of_many_rows(dtype):
    """All rows in one segment, over many row tiles and workgroups."""
    dt = L.DT[dtype]
    g = L.gen(4)
    seg, ends, A, G = _rows(3, [[6001]], 136, 72, dt)
    sq = torch.empty(1, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, *L.grouped_norm(A, G, ends, 1), "sqnorm")
    c = torch.tensor([0.37], device="cuda")
    L.check(_sum(A, G, seg, c, (1, 136, 72)), *L.grouped_sum(A, G, ends, c, 4.0), "sum")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,p", [(1, 1), (2, 3), (5, 1), (1, 130), (129, 2)])
def test_rows_narrower_than_a_vector_end_with_their_tensor(dtype, d, p):
    """Widths of a few elements, the tensors' last rows the last of the last
    segment (nothing may be read past them)."""
    dt = L.DT[dtype]
    g = L.gen(d * 10 + p)
    counts = [[70, 3], [0, 41]]
    seg, ends, A, G = _rows(d, counts, d, p, dt)
    c = torch.rand(2, generator=g).cuda()
    L.check(_sum(A, G, seg, c, (2, d, p)), *L.grouped_sum(A, G, ends, c, 4.0), "sum")
    W = L.randn(g, 2, p, d, dtype=dt)
    for x, transpose, w in ((A, False, p), (G, True, d)):
        y = torch.empty(ends[-1], w, dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(x, W, seg, y, transpose=transpose)
        L.check(y, *L.grouped_matmul(x, W, ends, 2, transpose), f"transpose={transpose}")


# ---- distillation


@pytest.mark.parametrize("dtype,teacher_dtype", [("bf16", "f32"), ("f32", "bf16")])
def test_distill_types_of_their_own(dtype, teacher_dtype):
    g = L.gen(31)
    B, T, V, K, tau = 2, 9, 5003, 17, 1.5
    logits = L.randn(g, B, T, V, scale=3.0, dtype=L.DT[dtype])
    ids = torch.randint(0, V, (B, T, K), generator=g).cuda()
    teacher = L.randn(g, B, T, K, scale=2.0, dtype=L.DT[teacher_dtype])
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, T, device="cuda")
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse)
    want, wlse, bl, be = L.distill_forward(logits, ids, teacher, tau, None)
    L.check(loss, want, bl, "loss")
    L.check(lse, wlse, be, "lse")
    grad = torch.empty_like(logits)
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad)
    L.check(grad, *L.distill_backward(logits, ids, teacher, tau, None, None, lse), "grad")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 600])
def test_distill_rows_of_a_masks_value(dtype, T):
    """Tokens whose logits all hold one value of a mask: p = 1/V, though lse
    has no room for log V beside it. At 600 tokens a workgroup holds a whole
    token, at 3 a part of one; in place as well."""
    dt = L.DT[dtype]
    V, K, tau = 6007, 3, 2.0
    low = torch.finfo(dt).min
    values = [low, -1e9, 1e30, -3e4]
    logits = torch.empty(1, T, V, dtype=dt, device="cuda")
    for t in range(T):
        logits[0, t] = values[t % 4]
    logits[0, 2, 5] = low  # one word masked in a row of 1e30
    ids = torch.tensor([7, 9, 7]).expand(1, T, K).contiguous().cuda()
    teacher = torch.tensor([0.5, 1.0, -1.0]).to(dt).expand(1, T, K).contiguous().cuda()
    loss, lse = torch.empty(1, device="cuda"), torch.empty(1, T, device="cuda")
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse)
    q = torch.softmax(teacher[0, 0].double().cpu() / tau, -1)
    n = torch.full((T,), float(V), dtype=torch.float64)
    n[2] = V - 1
    want = tau * tau * ((q * q.log()).sum() * T + n.log().sum())
    # each token: the teacher's K places, two logarithms of one rounding each, values below 16; T tokens added
    assert abs(loss[0].double().cpu() - want) <= (64 + T) * L.U * T * tau * tau * 16
    grad = torch.empty_like(logits)
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad)
    full = torch.zeros(V, dtype=torch.float64).scatter_add_(0, torch.tensor([7, 9, 7]), q)
    p = torch.ones(T, V, dtype=torch.float64) / n[:, None]
    p[2, 5] = 0.0
    wg = (p - full) * tau
    # p = 2^(-log2 V): the logarithm of the sum and its product with log2(e) are of size 13: 16 * 13 u at most
    bound = tau * (p * 256 + full * 64) * L.U + L.half(dt) * wg.abs() + 1e-37
    L.check(grad[0], wg, bound, "grad")
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, logits)
    assert torch.equal(grad, logits)


# ---- past 2^31 elements


def _gpu_randn(seed, *shape):
    return torch.randn(*shape, dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def test_rms_norm_past_32_bits():
    B, T, d = 2, 70000, 16384
    x = _gpu_randn(1, B, T, d)
    gain = _gpu_randn(2, d).float()
    out = torch.empty_like(x)
    dpc.dp_rms_norm(x, gain, 1e-6, out)
    tail = x[1:, -3:]
    y, s = L.rms_forward(tail, None, gain, 1e-6)
    L.check(out[1:, -3:], y, L.rms_forward_bounds(y, s, torch.bfloat16)[0], "out")
    dy = out.zero_()
    dy[1, -3:] = _gpu_randn(3, 3, d)
    dx, rows = torch.empty_like(x), torch.empty(B, d, device="cuda")
    dpc.dp_rms_norm_backward(dy, x, gain, 1e-6, dx=dx, gain_rows=rows)
    wdx, wrows, bdx, brows = L.rms_backward(dy[1:, -3:], tail, None, gain, 1e-6)
    L.check(dx[1:, -3:], wdx, bdx, "dx")
    L.check(rows[1:], wrows, brows, "gain_rows")
    assert (rows[0] == 0).all() and (dx[0] == 0).all()


def test_distill_past_32_bits():
    B, T, V, K, tau = 2, 22000, 50257, 5, 2.0
    logits = _gpu_randn(4, B, T, V)
    g = L.gen(8)
    ids = torch.randint(0, V, (B, T, K), generator=g).cuda()
    teacher = L.randn(g, B, T, K, dtype=torch.bfloat16)
    weight = torch.zeros(B, T, device="cuda")
    weight[1, -2:] = 1.0
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, T, device="cuda")
    dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse, weight=weight)
    tail = [v[1:, -2:] for v in (logits, ids, teacher)]
    want, wlse, bl, be = L.distill_forward(*tail, tau, None)
    L.check(loss[1:], want, bl, "loss")
    assert loss[0] == 0.0
    L.check(lse[1:, -2:], wlse, be, "lse")
    grad = torch.empty_like(logits)
    dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad, weight=weight)
    L.check(grad[1:, -2:], *L.distill_backward(*tail, tau, None, None, lse[1:, -2:]), "grad")
    assert (grad[1, -40:-2] == 0).all() and (grad[0] == 0).all()


@pytest.mark.parametrize("B", [8192, 40000])
def test_grouped_past_32_bits(B):
    """About 1.1 million rows of 2048: the last samples' rows lie past 2^31
    elements. 8192 samples: whole row tiles and pieces; 40000: packed tiles and
    the sums of short ranges."""
    d, p, n = 2048, 256, 3
    g = L.gen(B)
    counts = torch.randint(2200000 // B // 2 - 10, 2200000 // B // 2 + 12, (1, B), generator=g)
    seg, ends = L.segments_of(counts)
    R = ends[-1]
    assert R * d > 2 ** 31
    A, G = _gpu_randn(6, R, d), _gpu_randn(7, R, p)
    first = ends[B - n]
    tail = [v - first for v in ends[B - n:]]
    a, gg = A[first:], G[first:]
    sq = torch.empty(B, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq[-n:], *L.grouped_norm(a, gg, tail, n), "sqnorm")
    c = torch.zeros(B, device="cuda")
    c[-n:] = torch.tensor([0.3, 1.0, 0.7])
    out = _sum(A, G, seg, c, (1, d, p))
    # the rows of factor 0 count in the number of terms added, not in their size
    want, bound = L.grouped_sum(a, gg, tail, c[-n:], 4.0)
    L.check(out, want, bound, "sum")
    W = L.randn(g, 1, p, d, scale=d ** -0.5, dtype=torch.bfloat16)
    Y = torch.empty(R, p, dtype=torch.bfloat16, device="cuda")
    dpc.dp_grouped_matmul(A, W, seg, Y)
    L.check(Y[first:], *L.grouped_matmul(a, W, tail, n, False), "product")
    dX = A.zero_()
    dpc.dp_grouped_matmul(G, W, seg, dX, transpose=True)
    L.check(dX[first:], *L.grouped_matmul(gg, W, tail, n, True), "input gradient")
