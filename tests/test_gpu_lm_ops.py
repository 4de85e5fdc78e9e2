"""The language-model operators' kernels against their plain forms in 64 bits,
at the sizes, types and masks where they can go wrong, through the binding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc
from oracle import noise as N

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f32"]


# ---- root-mean-square norm

# widths: one element, odd ones, each register class and its ends, the largest
WIDTHS = [1, 7, 64, 513, 1001, 1280, 2048, 2056, 4099, 8192, 16384, 16387, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_rms_norm(dtype, d):
    g, dt = L.gen(d), L.DT[dtype]
    rows = 5 if d > 2048 else 11
    x, r = L.randn(g, rows, d, dtype=dt), L.randn(g, rows, d, scale=3.0, dtype=dt)
    x[1] = 0
    r[1] = 0  # an empty row: zeros, not NaN
    gain = 1 + L.randn(g, d, scale=0.3)
    for res, gn in ((r, gain), (None, gain.to(torch.bfloat16))):
        out, s = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
        dpc.dp_rms_norm(x, gn, 1e-6, out, residual=res, sum_out=s)
        y, v = L.rms_forward(x, res, gn, 1e-6)
        by, bv = L.rms_forward_bounds(y, v, dt)
        L.check(out, y, by, "out")
        L.check(s, v, bv, "sum")
        # without the sum, and in place of x
        out2 = x.clone()
        dpc.dp_rms_norm(out2, gn, 1e-6, out2, residual=res)
        assert torch.equal(out2, out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,d", [(1, 1, 64), (3, 1, 1280), (5, 3, 333), (2, 200, 1280), (4, 37, 2048), (3, 19, 2056),
                                   (2, 65, 4099), (2, 7, 8192), (1, 3, 32768), (70, 9, 96), (1, 1500, 17),
                                   (4100, 2, 40), (1030, 40, 24)])
def test_rms_norm_backward(dtype, B, T, d):
    g, dt = L.gen(B + T + d), L.DT[dtype]
    s, dy, dsum = (L.randn(g, B, T, d, scale=c, dtype=dt) for c in (1.5, 0.1, 0.2))
    s[0, 0] = 0
    gain = 1 + L.randn(g, d, scale=0.3)
    dx, rows, bx, br = L.rms_backward(dy, s, dsum, gain, 1e-5)
    got, gr = torch.full_like(s, float("nan")), torch.full((B, d), float("nan"), device="cuda")
    dpc.dp_rms_norm_backward(dy, s, gain, 1e-5, dx=got, dsum=dsum, gain_rows=gr)
    L.check(got, dx, bx, "dx")
    L.check(gr, rows, br, "gain_rows")
    # each output alone; no residual gradient; in place of dy
    gr2 = torch.empty_like(gr)
    dpc.dp_rms_norm_backward(dy, s, gain, 1e-5, gain_rows=gr2)
    assert torch.equal(gr2, gr)
    inplace = dy.clone()
    dpc.dp_rms_norm_backward(inplace, s, gain, 1e-5, dx=inplace)
    dx0, _, bx0, _ = L.rms_backward(dy, s, None, gain, 1e-5)
    L.check(inplace, dx0, bx0, "dx without the residual gradient")


def test_rms_unaligned_rows_and_neighbours():
    """A tensor that starts off a 16-byte boundary takes single-element loads;
    what lies beside the outputs stays."""
    g = L.gen(3)
    flat = L.randn(g, 6 * 128 + 1, dtype=torch.bfloat16)
    x = flat[1:].view(6, 128)
    gain = 1 + L.randn(g, 128, scale=0.3)
    buf = torch.full((6 * 128 + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:-1].view(6, 128)
    dpc.dp_rms_norm(x, gain, 1e-6, out)
    y, v = L.rms_forward(x, None, gain, 1e-6)
    L.check(out, y, L.rms_forward_bounds(y, v, torch.bfloat16)[0], "out")
    assert buf[0] == 7.0 and buf[-1] == 7.0


def test_rms_gain_gradient_by_differences():
    """gain_rows and dx against central differences of the 64-bit forward."""
    g = L.gen(9)
    s, dy = L.randn(g, 2, 3, 6), L.randn(g, 2, 3, 6)
    gain = 1 + L.randn(g, 6, scale=0.3)
    dx, rows = torch.empty_like(s), torch.empty(2, 6, device="cuda")
    dpc.dp_rms_norm_backward(dy, s, gain, 1e-6, dx=dx, gain_rows=rows)
    h = 1e-5

    def f(sv, gv):
        return (L.rms_forward(sv, None, gv, 1e-6)[0] * dy.double()).reshape(2, -1).sum(1)

    for j in range(6):
        e = torch.zeros(6, dtype=torch.float64, device="cuda")
        e[j] = h
        num = (f(s.double(), gain.double() + e) - f(s.double(), gain.double() - e)) / (2 * h)
        assert torch.allclose(rows[:, j].double(), num, rtol=1e-5, atol=1e-5)
        es = torch.zeros_like(s, dtype=torch.float64)
        es[1, 2, j] = h
        num = (f(s.double() + es, gain) - f(s.double() - es, gain))[1] / (2 * h)
        assert torch.allclose(dx[1, 2, j].double(), num, rtol=1e-5, atol=1e-5)


# ---- distillation loss


def _distill_inputs(seed, B, T, V, K, dt):
    g = L.gen(seed)
    logits = L.randn(g, B, T, V, scale=3.0, dtype=dt)
    ids = torch.randint(0, V, (B, T, K), generator=g)
    ids[torch.rand(B, T, K, generator=g) < 0.15] = -1
    ids = ids.cuda()
    teacher = L.randn(g, B, T, K, scale=2.0, dtype=dt)
    weight = (torch.rand(B, T, generator=g) > 0.2).float().cuda() * 0.7
    return logits, ids, teacher, weight


CASES = [(1, 1, 1, 1, 1.0), (2, 3, 5, 2, 2.0), (3, 1, 50257, 64, 2.0), (2, 5, 4099, 300, 0.7), (1, 700, 130, 7, 4.0),
         (5, 1, 8192, 2048, 1.0), (2, 300, 1031, 33, 1.5)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,V,K,tau", CASES)
def test_distill(dtype, B, T, V, K, tau):
    dt = L.DT[dtype]
    logits, ids, teacher, weight = _distill_inputs(V + K, B, T, V, K, dt)
    loss, lse = torch.full((B,), float("nan"), device="cuda"), torch.full((B, T), float("nan"), device="cuda")
    for w in (weight, None):
        dpc.dp_distill_loss(logits, ids, teacher, tau, loss, lse, weight=w)
        want, wlse, bl, be = L.distill_forward(logits, ids, teacher, tau, w)
        L.check(loss, want, bl, "loss")
        L.check(lse, wlse, be, "lse")
        dloss = torch.linspace(-0.5, 2.0, B, device="cuda")
        for dl in (dloss, None):
            grad = torch.full_like(logits, float("nan"))
            dpc.dp_distill_loss_backward(logits, ids, teacher, tau, lse, grad, weight=w, dloss=dl)
            wg, bg = L.distill_backward(logits, ids, teacher, tau, w, dl, lse)
            L.check(grad, wg, bg, "grad")
    over = logits.clone()
    dpc.dp_distill_loss_backward(over, ids, teacher, tau, lse, over, weight=None, dloss=None)
    assert torch.equal(over, grad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_distill_masks_and_repeats(dtype):
    """Tokens without a used place, with weight 0 over NaN and infinite logits,
    a word named twice, words of no probability, the type's lowest value."""
    dt = L.DT[dtype]
    V, K = 1000, 8
    logits, ids, teacher, _ = _distill_inputs(4, 1, 8, V, K, dt)
    weight = torch.ones(1, 8, device="cuda")
    ids[0, 0] = -1                                     # nothing used
    weight[0, 1] = 0
    logits[0, 1, 3:9] = float("nan")                   # masked by its weight
    logits[0, 1, 20] = float("inf")
    ids[0, 2] = torch.tensor([5, 5, 9, 5, -1, 9, V, 11], device="cuda")  # the same words again; a word past V
    teacher[0, 3] = -float("inf")                      # no mass at all
    ids[0, 4] = torch.arange(K, device="cuda")
    teacher[0, 4, 2] = -float("inf")                   # one place without mass, its logit -inf
    logits[0, 4, 2] = -float("inf")
    logits[0, 5, 100:] = torch.finfo(dt).min           # most of the vocabulary masked
    ids[0, 5] = torch.arange(K, device="cuda")
    logits[0, 6, 500:] = -float("inf")
    ids[0, 6] = torch.arange(K, device="cuda") * 3
    ids[0, 7] = torch.tensor([0, V - 1, 0, V - 1, 0, V - 1, 0, V - 1], device="cuda")
    loss, lse = torch.empty(1, device="cuda"), torch.empty(1, 8, device="cuda")
    dpc.dp_distill_loss(logits, ids, teacher, 1.0, loss, lse, weight=weight)
    keep = torch.tensor([0, 2, 3, 4, 5, 6, 7], device="cuda")
    # the bound is that of the token whose logits are finite: the lowest values weigh nothing
    safe = torch.where(logits.double().abs() < 1e6, logits.double(), torch.full_like(logits.double(), -1e4))
    want, _, bl, _ = L.distill_forward(safe[:, keep], ids[:, keep], teacher[:, keep], 1.0, weight[:, keep])
    L.check(loss, want, bl, "loss")
    grad = torch.full_like(logits, float("nan"))
    dpc.dp_distill_loss_backward(logits, ids, teacher, 1.0, lse, grad, weight=weight)
    wg, bg = L.distill_backward(safe[:, keep], ids[:, keep], teacher[:, keep], 1.0, weight[:, keep], None, lse[:, keep])
    L.check(grad[:, keep], wg, bg + L.half(dt) * wg.abs(), "grad")
    for t in (0, 1, 3):
        assert (grad[0, t] == 0).all(), t


def test_distill_gradient_by_differences():
    """The gradient against central differences of the 64-bit loss."""
    logits, ids, teacher, weight = _distill_inputs(2, 2, 2, 11, 3, torch.float32)
    loss, lse, grad = torch.empty(2, device="cuda"), torch.empty(2, 2, device="cuda"), torch.empty_like(logits)
    dpc.dp_distill_loss(logits, ids, teacher, 1.7, loss, lse, weight=weight)
    dpc.dp_distill_loss_backward(logits, ids, teacher, 1.7, lse, grad, weight=weight)
    h = 1e-5
    for t in range(2):
        for j in range(11):
            e = torch.zeros_like(logits, dtype=torch.float64)
            e[:, t, j] = h
            up = L.distill_forward(logits.double() + e, ids, teacher, 1.7, weight)[0]
            dn = L.distill_forward(logits.double() - e, ids, teacher, 1.7, weight)[0]
            assert torch.allclose(grad[:, t, j].double(), (up - dn) / (2 * h), rtol=1e-4, atol=1e-5)


# ---- products grouped by expert

# row counts [E][B]: one row; empty experts and samples; ranges that end inside, at and past tiles; one long range
GROUPS = {
    "one-row": [[1]],
    "empty-experts": [[0, 0, 0], [3, 0, 2], [0, 0, 0], [0, 1, 0]],
    "tile-ends": [[31, 32, 33], [64, 1, 63], [128, 127, 129]],
    "long": [[300, 5], [0, 517]],
    "many-short": [[(3 * e + b) % 4 for b in range(40)] for e in range(70)],
    "single-rows": [[1] * 200, [0] * 100 + [1] * 100],
}
SHAPES = [(1, 1), (8, 16), (64, 64), (33, 70), (136, 264), (200, 129), (320, 96)]


def _rows(name, d, p, dt, tail=3):
    g = L.gen(d * 7 + p)
    counts = GROUPS[name]
    seg, ends = L.segments_of(counts)
    R = ends[-1] + tail  # rows behind the last segment
    return counts, seg, ends, L.randn(g, R, d, dtype=dt), L.randn(g, R, p, scale=0.5, dtype=dt), g


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("d,p", SHAPES)
def test_grouped_matmul(dtype, name, d, p):
    dt = L.DT[dtype]
    counts, seg, ends, X, Y, g = _rows(name, d, p, dt)
    E, B = len(counts), len(counts[0])
    W = L.randn(g, E, p, d, scale=d ** -0.5, dtype=dt)
    X[ends[-1]:] = float("nan")  # not read
    for x, transpose, n in ((X, False, p), (Y, True, d)):
        out = torch.full((x.shape[0], n), 5.0, dtype=dt, device="cuda")
        dpc.dp_grouped_matmul(x, W, seg, out, transpose=transpose)
        want, bound = L.grouped_matmul(x[:ends[-1]], W, ends, B, transpose)
        L.check(out[:ends[-1]], want, bound, f"transpose={transpose}")
        assert (out[ends[-1]:] == 5.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("d,p", SHAPES)
def test_grouped_norm_and_sum(dtype, name, d, p):
    dt = L.DT[dtype]
    counts, seg, ends, A, G, g = _rows(name, d, p, dt)
    E, B = len(counts), len(counts[0])
    A[ends[-1]:] = float("nan")
    G[ends[-1]:] = float("nan")
    sq = torch.full((B,), float("nan"), device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    want, bound = L.grouped_norm(A[:ends[-1]], G[:ends[-1]], ends, B)
    L.check(sq, want, bound, "sqnorm")
    again = torch.full((B,), 2.0, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, again, accumulate=True)
    L.check(again, want + 2.0, bound + 4 * L.U * (want + 2.0), "accumulated")
    c = torch.rand(B, generator=g).cuda() + 0.1
    c[0] = 0.0
    out = torch.full((E, d, p), float("nan"), device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 1.0, 0.0, 4.0, 0, 0, 0, out)
    want, bound = L.grouped_sum(A[:ends[-1]], G[:ends[-1]], ends, c, 4.0)
    L.check(out, want, bound, "sum")


@pytest.mark.parametrize("d,p", [(5, 7), (64, 128), (130, 12)])
def test_grouped_noise_is_the_layers_stream(d, p):
    """The noise of [E, d, p] is the documented stream of a layer of E*d rows,
    bit for bit, also for experts without rows."""
    seg, _ = L.segments_of([[2, 0], [0, 0], [1, 4]])
    A, G = torch.zeros(7, d, device="cuda"), torch.zeros(7, p, device="cuda")
    out = torch.empty(3, d, p, device="cuda")
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, torch.ones(2, device="cuda"), 2.0, 1.5, 1.0, 11, 4, 6, out)
    z = N.weight_noise(3 * d, p, 11, 4, 6).astype(np.float32)
    np.testing.assert_array_equal(out.cpu().numpy().reshape(3 * d, p), (np.float32(3.0) * z).astype(np.float32))


def test_grouped_nan_and_infinite_factors_stay_with_their_sample():
    """A NaN gradient reaches its own sample's norm and nothing else's."""
    seg, ends = L.segments_of([[40, 3, 70], [2, 0, 35]])
    g = L.gen(1)
    A, G = L.randn(g, ends[-1], 64, dtype=torch.bfloat16), L.randn(g, ends[-1], 72, dtype=torch.bfloat16)
    A[41, 5] = float("nan")  # expert 0, sample 1
    sq = torch.empty(3, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    assert torch.isnan(sq[1]) and torch.isfinite(sq[0]) and torch.isfinite(sq[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_grouped_large_ragged(dtype):
    """A size at which every variant of the launch rules is reached."""
    dt = L.DT[dtype]
    g = L.gen(77)
    B, E, d, p = 6, 4, 512, 640
    counts = torch.randint(0, 400, (E, B), generator=g)
    seg, ends = L.segments_of(counts)
    A, G = L.randn(g, ends[-1], d, scale=d ** -0.5, dtype=dt), L.randn(g, ends[-1], p, scale=p ** -0.5, dtype=dt)
    W = L.randn(g, E, p, d, scale=d ** -0.5, dtype=dt)
    out = torch.empty(ends[-1], p, dtype=dt, device="cuda")
    dpc.dp_grouped_matmul(A, W, seg, out)
    L.check(out, *L.grouped_matmul(A, W, ends, B, False), "forward")
    out = torch.empty(ends[-1], d, dtype=dt, device="cuda")
    dpc.dp_grouped_matmul(G, W, seg, out, transpose=True)
    L.check(out, *L.grouped_matmul(G, W, ends, B, True), "input gradient")
    sq, c, S = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty(E, d, p, device="cuda")
    dpc.dp_grouped_norm(A, G, seg, sq)
    L.check(sq, *L.grouped_norm(A, G, ends, B), "sqnorm")
    dpc.dp_clip_factors(sq, 10.0, c)
    dpc.dp_grouped_clipped_sum_noise(A, G, seg, c, 10.0, 0.0, float(B), 0, 0, 0, S)
    L.check(S, *L.grouped_sum(A, G, ends, c, float(B)), "sum")
