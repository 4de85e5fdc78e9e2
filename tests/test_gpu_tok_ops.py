"""The kernels from tokens to a per-sample loss against their plain forms in 64
bits, at the sizes, types and masks where they can go wrong, through the
binding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc
import tok_util as K
from oracle import definitions as D
from oracle import noise as N

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f32"]
NAN, INF = float("nan"), float("inf")


def full(*shape, dtype=torch.float32, value=None):
    value = (NAN if dtype.is_floating_point else -9) if value is None else value
    return torch.full(shape, value, dtype=dtype, device="cuda")


# ---- layer norm

# widths: one element, odd ones, each register class and its ends, the largest
WIDTHS = [1, 7, 64, 513, 1001, 1280, 2048, 2056, 4099, 8192, 8200, 16384, 16387, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_layer_norm(dtype, d):
    g, dt = L.gen(d), L.DT[dtype]
    rows = 5 if d > 2048 else 11
    x, r = L.randn(g, rows, d, dtype=dt), L.randn(g, rows, d, scale=3.0, dtype=dt)
    x[1], r[1] = 0, 0    # one value alone: the bias, not NaN
    x[2], r[2] = 3, 0.5
    x[3] += 100          # far from zero
    gain, bias = 1 + L.randn(g, d, scale=0.3), L.randn(g, d, scale=0.2)
    for res, gn, bs in ((r, gain, bias), (None, gain.bfloat16(), bias.bfloat16()), (r, gain, None)):
        out, s = full(rows, d, dtype=dt), full(rows, d, dtype=dt)
        dpc.dp_layer_norm(x, gn, bs, 1e-5, out, residual=res, sum_out=s)
        y, v, by, bv = K.layer_norm(x, res, gn, bs, 1e-5)
        L.check(out, y, by, "out")
        L.check(s, v, bv, "sum")
        out2 = x.clone()  # without the sum, and in place of x
        dpc.dp_layer_norm(out2, gn, bs, 1e-5, out2, residual=res)
        assert torch.equal(out2, out)


def test_layer_norm_of_rows_far_from_zero():
    """A mean thousands of times the spread: the spread is that of the centred
    row, so only the inputs' own roundings show."""
    g = L.gen(5)
    x = L.randn(g, 9, 1280) + 4096.0
    one, out = torch.ones(1280, device="cuda"), full(9, 1280)
    dpc.dp_layer_norm(x, one, None, 0.0, out)
    y, _, by, _ = K.layer_norm(x, None, one, None, 0.0)
    L.check(out, y, by, "out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,d", [(1, 1, 64), (3, 1, 1280), (5, 3, 333), (2, 200, 1280), (4, 37, 2048), (3, 19, 2056),
                                   (2, 65, 4099), (2, 7, 8192), (2, 9, 10000), (3, 5, 16384), (1, 3, 32768), (70, 9, 96),
                                   (1, 1500, 17), (4100, 2, 40), (1030, 40, 24), (2, 3, 1)])
def test_layer_norm_backward(dtype, B, T, d):
    g, dt = L.gen(B + T + d), L.DT[dtype]
    s, dy, dsum = (L.randn(g, B, T, d, scale=c, dtype=dt) for c in (1.5, 0.1, 0.2))
    s[0, 0] = 2.0
    gain = 1 + L.randn(g, d, scale=0.3)
    dx, rows, brows, bx, br, bb = K.layer_norm_backward(dy, s, dsum, gain, 1e-5)
    got, gr, gb = full(B, T, d, dtype=dt), full(B, d), full(B, d)
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, dx=got, dsum=dsum, gain_rows=gr, bias_rows=gb)
    L.check(got, dx, bx, "dx")
    L.check(gr, rows, br, "gain_rows")
    L.check(gb, brows, bb, "bias_rows")
    # each output alone; no residual gradient; in place of dy and of dsum
    gr2, gb2, got2 = full(B, d), full(B, d), full(B, T, d, dtype=dt)
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, gain_rows=gr2)
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, bias_rows=gb2, dx=got2)
    assert torch.equal(gr2, gr) and torch.equal(gb2, gb)
    dx0, _, _, bx0, _, _ = K.layer_norm_backward(dy, s, None, gain, 1e-5)
    L.check(got2, dx0, bx0, "dx without the residual gradient")
    inplace, onto = dy.clone(), dsum.clone()
    dpc.dp_layer_norm_backward(inplace, s, gain, 1e-5, dx=inplace)
    assert torch.equal(inplace, got2)
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, dx=onto, dsum=onto)
    assert torch.equal(onto, got)


def test_layer_norm_unaligned_rows_and_neighbours():
    g = L.gen(3)
    flat = L.randn(g, 6 * 128 + 1, dtype=torch.bfloat16)
    x = flat[1:].view(6, 128)
    gain, bias = 1 + L.randn(g, 129, scale=0.3)[1:], L.randn(g, 129)[1:]
    buf = full(6 * 128 + 2, dtype=torch.bfloat16, value=7.0)
    out = buf[1:-1].view(6, 128)
    dpc.dp_layer_norm(x, gain, bias, 1e-6, out)
    y, _, by, _ = K.layer_norm(x, None, gain, bias, 1e-6)
    L.check(out, y, by, "out")
    assert buf[0] == 7.0 and buf[-1] == 7.0


def test_layer_norm_gradients_by_differences():
    g = L.gen(9)
    s, dy = L.randn(g, 2, 3, 6), L.randn(g, 2, 3, 6)
    gain, bias = 1 + L.randn(g, 6, scale=0.3), L.randn(g, 6)
    dx, rows, brows = torch.empty_like(s), full(2, 6), full(2, 6)
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-6, dx=dx, gain_rows=rows, bias_rows=brows)
    h = 1e-5

    def f(sv, gv, bv):
        return (K.layer_norm(sv, None, gv, bv, 1e-6)[0] * dy.double()).reshape(2, -1).sum(1)

    sd, gd, bd = s.double(), gain.double(), bias.double()
    for j in range(6):
        e = torch.zeros(6, dtype=torch.float64, device="cuda")
        e[j] = h
        es = torch.zeros_like(sd)
        es[1, 2, j] = h
        for got, num in ((rows[:, j], f(sd, gd + e, bd) - f(sd, gd - e, bd)),
                         (brows[:, j], f(sd, gd, bd + e) - f(sd, gd, bd - e)),
                         (dx[1, 2, j], (f(sd + es, gd, bd) - f(sd - es, gd, bd))[1])):
            assert torch.allclose(got.double(), num / (2 * h), rtol=1e-5, atol=1e-5)


# ---- table of words


def _ids(g, B, T, V, kind="any"):
    ids = torch.randint(0, V, (B, T), generator=g)
    if kind == "few":      # few words: long runs
        ids = torch.randint(0, min(V, 3), (B, T), generator=g)
    drop = torch.rand(B, T, generator=g)
    ids[drop < 0.06] = -1
    ids[drop > 0.98] = V + 7 if kind == "any" else 1 << 40
    return ids.cuda()


def _order(ids, V):
    order, starts = (full(n, dtype=torch.int64) for n in (ids.numel(), V + 1))
    dpc.dp_embedding_order(ids, V, order, starts)
    return order, starts


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wdtype", DTYPES)
@pytest.mark.parametrize("B,T,V,d", [(1, 1, 1, 1), (2, 3, 5, 7), (8, 1, 50257, 1280), (3, 40, 11, 33), (2, 5, 300, 8192),
                                     (1, 2, 9, 20001), (70, 90, 1000, 520)])
def test_embedding(dtype, wdtype, B, T, V, d):
    g = L.gen(V + d)
    ids, w = _ids(g, B, T, V), L.randn(g, V, d, dtype=L.DT[wdtype])
    for scale in (1.0, 11.3):
        out = full(B, T, d, dtype=L.DT[dtype])
        dpc.dp_embedding(ids, w, out, scale=scale)
        y, by = K.embedding(ids, w, float(np.float32(scale)), L.DT[dtype])
        L.check(out, y, by, "out")


def test_embedding_beside_its_neighbours():
    g = L.gen(4)
    w = L.randn(g, 50 * 24 + 1, dtype=torch.bfloat16)[1:].view(50, 24)  # rows off 16 bytes
    ids = _ids(g, 3, 5, 50)
    buf = full(3 * 5 * 24 + 2, dtype=torch.bfloat16, value=7.0)
    out = buf[1:-1].view(3, 5, 24)
    dpc.dp_embedding(ids, w, out)
    y, by = K.embedding(ids, w, 1.0, torch.bfloat16)
    L.check(out, y, by, "out")
    assert buf[0] == 7.0 and buf[-1] == 7.0


# one digit, two, three; one workgroup to many; a full tile and one token more; more workgroups than are summed at once
ORDERS = [(1, 1, 1), (1, 1, 5), (3, 7, 2), (1, 1024, 300), (1, 1025, 511), (5, 700, 512), (2, 2048, 40000),
          (1, 4097, 40000), (32, 1024, 50257),
          (3, 333, 262143), (2, 50, 262144), (2, 9, 1 << 24), (140, 1000, 600), (9, 20000, 70000)]


@pytest.mark.parametrize("B,T,V", ORDERS)
@pytest.mark.parametrize("kind", ["any", "few"])
def test_embedding_order(B, T, V, kind):
    ids = _ids(L.gen(B + T), B, T, V, kind)
    order, starts = _order(ids, V)
    want, wstarts = K.order(ids, V)
    assert torch.equal(order.cpu(), want)
    assert torch.equal(starts.cpu(), wstarts)


@pytest.mark.parametrize("V", [1, 63, 1023, 1024, 1025, 2047, 2048, 5003, (1 << 19) - 1, 1 << 19])
@pytest.mark.parametrize("N", [1, 64, 1001, 4095, 4096, 4097])
def test_embedding_starts_of_few_tokens(N, V):
    """Words spread out, in one place of the table, one alone (at either end), all dropped."""
    g = L.gen(N + V)
    half = max(1, V // 2)
    for ids in (torch.randint(-1, V, (N,), generator=g), torch.randint(V - half, V, (N,), generator=g),
                torch.full((N,), V - 1), torch.zeros(N, dtype=torch.int64), torch.full((N,), V), torch.full((N,), -5)):
        order, starts = _order(ids.cuda(), V)
        want, wstarts = K.order(ids, V)
        assert torch.equal(order.cpu(), want) and torch.equal(starts.cpu(), wstarts)


GRADS = [(1, 1, 1, 1, "any"), (2, 3, 5, 7, "any"), (8, 1, 50257, 64, "any"), (3, 40, 11, 33, "any"),
         (2, 1200, 3, 520, "few"), (1, 5000, 1, 72, "few"), (1, 40000, 2, 24, "few"), (32, 64, 1000, 1280, "any"),
         (4100, 2, 50, 24, "any"), (5, 700, 70000, 40, "any"), (2, 33, 7, 8192, "few"), (1, 300, 4, 2051, "few"),
         (6, 100, 6, 600, "any")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,V,d,kind", GRADS)
def test_embedding_gradient(dtype, B, T, V, d, kind):
    g, dt = L.gen(B + T + V + d), L.DT[dtype]
    ids, G = _ids(g, B, T, V, kind), L.randn(g, B, T, d, dtype=dt)
    order, starts = _order(ids, V)
    scale = 1.7
    sc = float(np.float32(scale))
    sq = full(B)
    dpc.dp_embedding_norm(G, ids, order, starts, sq, scale=scale)
    want, bound = K.embedding_norm(G, ids, V, sc)
    L.check(sq, want, bound, "sqnorm")
    again = sq.clone()
    dpc.dp_embedding_norm(G, ids, order, starts, again, scale=scale, accumulate=True)
    assert torch.equal(again, sq + sq)
    c = torch.rand(B, generator=g).cuda()
    c[0] = 0.0
    out = full(V, d)
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, c, 1.0, 0.0, 4.0, 0, 0, 0, out, scale=scale)
    want, bound = K.embedding_sum(G, ids, V, c, sc, 4.0)
    L.check(out, want, bound, "out")
    # the same bits again
    out2, sq2 = full(V, d), full(B)
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, c, 1.0, 0.0, 4.0, 0, 0, 0, out2, scale=scale)
    dpc.dp_embedding_norm(G, ids, order, starts, sq2, scale=scale)
    assert torch.equal(out2, out) and torch.equal(sq2, sq)


@pytest.mark.parametrize("V,d", [(1, 1), (7, 5), (50, 64), (33, 777)])
def test_embedding_noise_is_the_layers(V, d):
    """Without tokens the sum is the noise of a layer of V rows, bit for bit;
    with them it is added in the order of dp_clipped_sum_noise."""
    g = L.gen(V)
    ids = _ids(g, 2, 6, V)
    G = L.randn(g, 2, 6, d)
    none = torch.full_like(ids, -1)
    z = N.weight_noise(V, d, 77, 3, 9)
    for use in (none, ids):
        order, starts = _order(use, V)
        out, clean = full(V, d), full(V, d)
        c = torch.tensor([0.5, 0.25], device="cuda")
        dpc.dp_embedding_clipped_sum_noise(G, use, order, starts, c, 2.0, 0.75, 2.0, 77, 3, 9, out)
        dpc.dp_embedding_clipped_sum_noise(G, use, order, starts, c, 2.0, 0.0, 1.0, 77, 3, 9, clean)
        want = D.noised_mean_f32(clean.cpu().numpy(), z, 0.75, 2.0, 2.0)
        assert np.array_equal(out.cpu().numpy(), want)


def test_embedding_norm_counts_a_word_once():
    """Two tokens of one word add before the norm is taken; of two samples they do not."""
    G = torch.tensor([[[3.0, 0.0], [0.0, 4.0]], [[3.0, 0.0], [-3.0, 0.0]]], device="cuda")
    ids = torch.tensor([[5, 5], [5, 5]], device="cuda")
    order, starts = _order(ids, 8)
    sq = full(2)
    dpc.dp_embedding_norm(G, ids, order, starts, sq)
    assert sq.tolist() == [25.0, 0.0]


def test_embedding_gradient_by_differences():
    g = L.gen(2)
    V, d = 6, 4
    ids, G, w = _ids(g, 3, 8, V), L.randn(g, 3, 8, d), L.randn(g, V, d).double()
    order, starts = _order(ids, V)
    out, ones = full(V, d), torch.ones(3, device="cuda")
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, ones, 1.0, 0.0, 1.0, 0, 0, 0, out, scale=0.5)

    def f(wv):
        return (K.embedding(ids, wv, 0.5, torch.float32)[0] * G.double()).sum()

    for v in range(V):
        e = torch.zeros_like(w)
        e[v, v % d] = 1e-5
        assert torch.allclose(out[v, v % d].double(), (f(w + e) - f(w - e)) / 2e-5, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [5, 64, 333, 777, 2051])
def test_embedding_norm_of_an_infinite_row(dtype, d):
    """inf in any one column, and a run whose sum overflows: an infinite norm of its sample, as the formula has it."""
    B, T, V, g = 3 + d, 20, 9, L.gen(d)
    ids, G = torch.randint(0, V, (B, T), generator=g).cuda(), L.randn(g, B, T, d, dtype=L.DT[dtype])
    for c in range(d):
        G[2 + c, 3, c] = INF if c % 2 else -INF
    ids[1], G[1] = 4, torch.finfo(torch.bfloat16).max
    sq = full(B)
    dpc.dp_embedding_norm(G, ids, *_order(ids, V), sq)
    assert torch.isinf(sq[1:2 + d]).all() and torch.isfinite(sq[[0, -1]]).all()


def test_embedding_with_a_foreign_order_stays_inside():
    """An order and starts that are not of these ids: no meaning, but nothing outside is touched."""
    g = L.gen(8)
    B, T, V, d = 4, 100, 30, 64
    ids, G = _ids(g, B, T, V), L.randn(g, B, T, d)
    order = torch.randint(-1000, 1000, (B * T,), generator=g).cuda()
    order[7], order[9] = 1 << 62, -(1 << 62)
    starts = torch.randint(-1000, 1000, (V + 1,), generator=g).cuda()
    starts[3], starts[4] = 1 << 62, -(1 << 62)
    buf, sbuf = full(V * d + 2, value=7.0), full(B + 2, value=7.0)
    dpc.dp_embedding_norm(G, ids, order, starts, sbuf[1:-1])
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, torch.ones(B, device="cuda"), 1.0, 0.0, 1.0, 0, 0, 0,
                                       buf[1:-1].view(V, d))
    torch.cuda.synchronize()
    assert buf[0] == buf[-1] == 7.0 and sbuf[0] == sbuf[-1] == 7.0


# ---- log probabilities


def _logits(g, shape, dt, kind):
    z = torch.randn(shape, generator=g) * 3.0
    if kind == "ties":
        z = torch.randint(-3, 4, shape, generator=g).float()
        z[..., ::5] = -0.0
    elif kind == "masked":  # most words at -inf
        z[torch.rand(shape, generator=g) < 0.97] = -INF
    elif kind == "lowest":
        z[torch.rand(shape, generator=g) < 0.5] = torch.finfo(dt).min
    elif kind == "rising":
        z = torch.linspace(-8, 8, shape[-1]).expand(shape).clone()
    return z.to(dt).cuda()


LOGPROBS = [(1, 1, 0, 1.0, "normal"), (1, 1, 1, 2.0, "normal"), (3, 5, 5, 1.0, "normal"), (4, 50257, 20, 0.8, "normal"),
            (300, 4099, 64, 1.0, "normal"), (700, 1031, 32, 1.5, "normal"), (700, 1031, 33, 1.5, "normal"),
            (600, 8191, 100, 0.7, "normal"), (2, 130001, 256, 1.0, "normal"), (5, 257, 256, 1.0, "normal"),
            (5, 257, 257 - 1, 3.0, "ties"), (600, 4097, 50, 1.0, "ties"), (4, 50257, 64, 1.0, "ties"),
            (600, 300, 20, 1.0, "masked"), (6, 9000, 100, 1.0, "masked"), (40, 5001, 40, 1.0, "lowest"),
            (5, 20011, 64, 1.0, "rising"), (513, 2050, 128, 1.0, "rising"), (300, 64, 7, 2.0 ** 40, "normal"),
            (3, 777, 8, 2.0 ** -40, "normal")]


def _check_logprob(logits, targets, tau, top):
    rows = targets.shape
    w = K.logprob(logits, targets, tau, top)
    logp, stats, ent = full(*rows), full(*rows, 2), full(*rows)
    ti, tl = (full(*rows, top, dtype=torch.int64), full(*rows, top)) if top else (None, None)
    dpc.dp_token_logprob(logits, targets, tau, logp, stats, entropy=ent, top_ids=ti, top_logp=tl)

    def near(got, want, bound, what):  # infinities have to be the same ones
        fin = torch.isfinite(want)
        assert torch.equal(got.double()[~fin], want[~fin]), what
        L.check(got[fin], want[fin], bound[fin], what)

    near(logp, w["logp"], w["logp_bound"], "logp")
    assert torch.equal(stats[..., 0].double(), w["m"])
    near(stats[..., 1], w["log_s"], w["log_s_bound"], "log of the sum")
    near(ent, w["entropy"], w["entropy_bound"], "entropy")
    if top:
        assert torch.equal(ti, w["top_ids"])
        near(tl, w["top_logp"], w["top_bound"], "top_logp")
    # without the entropy; without the top words
    logp2, stats2 = full(*rows), full(*rows, 2)
    dpc.dp_token_logprob(logits, targets, tau, logp2, stats2)
    near(logp2, w["logp"], w["logp_bound"], "logp alone")
    return stats, ent


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V,top,tau,kind", LOGPROBS)
def test_token_logprob(dtype, rows, V, top, tau, kind):
    g = L.gen(rows + V)
    logits = _logits(g, (rows, V), L.DT[dtype], kind)
    targets = torch.randint(0, V, (rows,), generator=g)
    targets[torch.rand(rows, generator=g) < 0.1] = -1
    if rows > 4:
        targets[3], logits[4] = V, -INF  # a target past the words; a row without a distribution
    _check_logprob(logits, targets.cuda(), tau, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [(5, 16393), (600, 8205), (600, 16401), (520, 33001)])
@pytest.mark.parametrize("cut", range(0, 17, 3))
def test_top_words_at_the_end_of_a_row(dtype, rows, V, cut):
    """The largest logits in the row's last vectors, which not all lanes have."""
    V -= cut
    g = L.gen(V)
    logits = L.randn(g, rows, V, dtype=L.DT[dtype])
    logits[:, -29:] += 5.0
    targets = torch.randint(0, V, (rows,), generator=g).cuda()
    ti, tl = full(rows, 40, dtype=torch.int64), full(rows, 40)
    dpc.dp_token_logprob(logits, targets, 1.0, full(rows), full(rows, 2), top_ids=ti, top_logp=tl)
    want = torch.sort(logits.float(), dim=-1, descending=True, stable=True)[1][..., :40]
    assert torch.equal(ti, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [3, 8, 64, 67, 256, 257, 300, 511, 512, 513, 1000, 1023, 1024, 1025])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "lowest", "rising"])
def test_top_words_of_short_rows(dtype, V, kind):
    """Few to all words of rows around the ends of what is held by 4 bytes, a row at every alignment."""
    g, rows = L.gen(V), 520
    logits, targets = _logits(g, (rows, V), L.DT[dtype], kind), torch.randint(0, V, (rows,), generator=g).cuda()
    for top in sorted({1, max(1, V // 32), V // 16 + 1, V // 8 + 1, V // 3 + 1, V}):
        if top <= 256:
            _check_logprob(logits, targets, 1.0, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [(6, 3000), (600, 3000), (600, 9000)])
def test_token_logprob_of_nan_and_infinities(dtype, rows, V):
    """A row with NaN or +inf gives NaN, its top words come in order all the
    same; other rows are not touched by it."""
    g = L.gen(rows)
    logits = _logits(g, (rows, V), L.DT[dtype], "normal")
    logits[0, 5], logits[1, 2999], logits[2, 17], logits[2, 4] = NAN, INF, INF, NAN
    targets = torch.randint(0, V, (rows,), generator=g).cuda()
    logp, stats, ent, ti, tl = full(rows), full(rows, 2), full(rows), full(rows, 9, dtype=torch.int64), full(rows, 9)
    dpc.dp_token_logprob(logits, targets, 1.0, logp, stats, entropy=ent, top_ids=ti, top_logp=tl)
    assert torch.isnan(logp[:3]).all() and torch.isnan(ent[:3]).all() and torch.isnan(tl[:3]).all()
    want = torch.sort(logits.float().cpu(), dim=-1, descending=True, stable=True)[1][..., :9]
    assert torch.equal(ti.cpu(), want)
    w = K.logprob(logits[3:], targets[3:], 1.0, 0)
    L.check(logp[3:], w["logp"], w["logp_bound"], "logp")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V,tau,kind", [(1, 1, 1.0, "normal"), (3, 5, 2.0, "normal"), (4, 50257, 0.8, "normal"),
                                             (300, 4099, 1.0, "normal"), (700, 1031, 1.5, "normal"),
                                             (520, 8191, 0.7, "normal"), (2, 130001, 1.0, "normal"),
                                             (600, 300, 1.0, "masked"), (40, 5001, 1.0, "lowest"),
                                             (9, 2048, 1.0, "ties"), (5, 2047, 3.0, "ties")])
def test_token_logprob_backward(dtype, rows, V, tau, kind):
    g, dt = L.gen(rows + V), L.DT[dtype]
    logits = _logits(g, (rows, V), dt, kind)
    targets = torch.randint(0, V, (rows,), generator=g)
    targets[torch.rand(rows, generator=g) < 0.1] = -1
    targets = targets.cuda()
    if rows > 4:
        logits[4] = -INF
    logp, stats, ent = full(rows), full(rows, 2), full(rows)
    dpc.dp_token_logprob(logits, targets, tau, logp, stats, entropy=ent)
    dl, dh = L.randn(g, rows), L.randn(g, rows, scale=0.3)
    if rows > 2:
        dl[2] = dh[2] = 0.0
        logits[2, 0] = NAN  # nothing is passed on: 0 whatever the row holds
    for a, b in ((dl, None), (dl, dh), (None, dh)):
        grad = full(rows, V, dtype=dt)
        dpc.dp_token_logprob_backward(logits, targets, tau, stats, grad, dlogp=a, entropy=ent, dentropy=b)
        z = logits.clone()
        if rows > 2:
            z[2] = 0
        want, bound = K.logprob_backward(z, targets, tau, stats, a, ent, b)
        L.check(grad, want, bound, "grad")
        inplace = logits.clone()
        dpc.dp_token_logprob_backward(inplace, targets, tau, stats, inplace, dlogp=a, entropy=ent, dentropy=b)
        assert torch.equal(inplace, grad)


def test_token_logprob_gradient_by_differences():
    g = L.gen(1)
    z, y = L.randn(g, 3, 7, scale=2.0), torch.tensor([2, -1, 6], device="cuda")
    dl, dh = L.randn(g, 3), L.randn(g, 3)
    logp, stats, ent, grad = full(3), full(3, 2), full(3), full(3, 7)
    dpc.dp_token_logprob(z, y, 1.3, logp, stats, entropy=ent)
    dpc.dp_token_logprob_backward(z, y, 1.3, stats, grad, dlogp=dl, entropy=ent, dentropy=dh)

    def f(zv):
        w = K.logprob(zv, y, 1.3, 0)
        return (w["logp"] * dl.double() + w["entropy"] * dh.double()).sum()

    for i in range(3):
        for j in range(7):
            e = torch.zeros(3, 7, dtype=torch.float64, device="cuda")
            e[i, j] = 1e-5
            num = (f(z.double() + e) - f(z.double() - e)) / 2e-5
            assert torch.allclose(grad[i, j].double(), num, rtol=1e-5, atol=1e-6)


def test_token_logprob_beside_its_neighbours():
    g = L.gen(6)
    rows, V, top = 5, 333, 6
    logits, y = L.randn(g, rows, V, dtype=torch.bfloat16), torch.randint(0, V, (rows,), generator=g).cuda()
    bufs = [full(n + 2, value=7.0) for n in (rows, 2 * rows, rows, rows * top)]
    ti = full(rows * top + 2, dtype=torch.int64, value=7)
    view = [b[1:-1] for b in bufs]
    dpc.dp_token_logprob(logits, y, 1.0, view[0], view[1].view(rows, 2), entropy=view[2],
                         top_ids=ti[1:-1].view(rows, top), top_logp=view[3].view(rows, top))
    gbuf = full(rows * V + 16, dtype=torch.bfloat16, value=7.0)
    dpc.dp_token_logprob_backward(logits, y, 1.0, view[1].view(rows, 2), gbuf[8:8 + rows * V].view(rows, V), dlogp=view[0])
    assert all(b[0] == 7.0 and b[-1] == 7.0 for b in bufs) and ti[0] == ti[-1] == 7
    assert (gbuf[:8] == 7.0).all() and (gbuf[8 + rows * V:] == 7.0).all()


def test_top_words_are_a_teachers():
    """What the distillation loss takes: a student equal to its teacher, whose
    top words are all its words, has loss 0 and gradient 0."""
    g = L.gen(7)
    z = L.randn(g, 2, 3, 40, scale=2.0)
    y = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    ti, tl = full(2, 3, 40, dtype=torch.int64), full(2, 3, 40)
    dpc.dp_token_logprob(z, y, 1.0, full(2, 3), full(2, 3, 2), top_ids=ti, top_logp=tl)
    loss, lse, grad = full(2), full(2, 3), torch.empty_like(z)
    dpc.dp_distill_loss(z, ti, tl, 1.0, loss, lse)
    dpc.dp_distill_loss_backward(z, ti, tl, 1.0, lse, grad)
    # both logarithms and both distributions are off by some 100 roundings of terms of size up to 16
    assert loss.abs().max() <= 3 * 100 * 16 * L.U and grad.abs().max() <= 100 * 16 * L.U


# ---- balance loss


BALANCE = [(1, 1, 1, 1), (2, 3, 4, 2), (3, 33, 8, 2), (2, 200, 9, 3), (4, 100, 16, 2), (2, 50, 31, 4), (32, 130, 64, 2),
           (9, 61, 130, 6), (2, 70, 256, 8), (3, 40, 511, 5), (2, 35, 1024, 9), (1, 3000, 60, 1), (600, 2, 12, 2),
           (1, 65, 700, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T,E,top", BALANCE)
def test_balance(dtype, B, T, E, top):
    g, dt = L.gen(B + T + E), L.DT[dtype]
    logits = L.randn(g, B, T, E, scale=2.0, dtype=dt)
    ids = torch.randint(0, E, (B, T, top), generator=g)
    drop = torch.rand(B, T, top, generator=g)
    ids[drop < 0.1], ids[drop > 0.97] = -1, E + 3
    if T > 2:
        ids[:, T - 1] = -1  # a token without a place
        logits[:, T - 1] = NAN
    if B > 1:
        ids[1] = -1         # a sample without a token
    ids = ids.cuda()
    loss, counts, tokens = full(B), full(B, E, dtype=torch.int64), full(B, dtype=torch.int64)
    dpc.dp_balance_loss(logits, ids, loss, counts, tokens)
    wl, wc, wt, bound = K.balance(logits, ids)
    assert torch.equal(counts, wc) and torch.equal(tokens, wt)
    L.check(loss, wl, bound, "loss")
    dl = torch.linspace(-1.0, 2.0, B, device="cuda") + 0.01
    for d in (dl, None):
        grad = full(B, T, E, dtype=dt)
        dpc.dp_balance_loss_backward(logits, ids, counts, tokens, grad, dloss=d)
        want, gb = K.balance_backward(logits, ids, d)
        L.check(grad, want, gb, "grad")
        inplace = logits.clone()
        dpc.dp_balance_loss_backward(inplace, ids, counts, tokens, inplace, dloss=d)
        assert torch.equal(inplace, grad)


def test_balance_of_even_routing():
    """Every expert named as often: loss 1 and a gradient of exactly 0."""
    E, T = 6, 12
    ids = torch.arange(T, device="cuda").remainder(E).view(1, T, 1)
    logits = L.randn(L.gen(1), 1, T, E)
    loss, counts, tokens, grad = full(1), full(1, E, dtype=torch.int64), full(1, dtype=torch.int64), full(1, T, E)
    dpc.dp_balance_loss(logits, ids, loss, counts, tokens)
    dpc.dp_balance_loss_backward(logits, ids, counts, tokens, grad)
    assert abs(float(loss) - 1.0) <= 256 * L.U and (grad == 0).all()


def test_balance_gradient_by_differences():
    g = L.gen(3)
    z = L.randn(g, 2, 4, 5)
    ids = torch.randint(-1, 5, (2, 4, 2), generator=g).cuda()
    loss, counts, tokens, grad = full(2), full(2, 5, dtype=torch.int64), full(2, dtype=torch.int64), full(2, 4, 5)
    dpc.dp_balance_loss(z, ids, loss, counts, tokens)
    dpc.dp_balance_loss_backward(z, ids, counts, tokens, grad)
    for b in range(2):
        for t in range(4):
            for j in range(5):
                e = torch.zeros(2, 4, 5, dtype=torch.float64, device="cuda")
                e[b, t, j] = 1e-5
                num = (K.balance(z.double() + e, ids)[0] - K.balance(z.double() - e, ids)[0]).sum() / 2e-5
                assert torch.allclose(grad[b, t, j].double(), num, rtol=1e-5, atol=1e-6)
