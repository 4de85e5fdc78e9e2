"""The operators from tokens to a per-sample loss on tensors of more than 2^31
elements: what lies behind that many is checked against sums in 64 bits."""
from __future__ import annotations

import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc
import tok_util as K

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _randn(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=dtype)


def _randint(seed, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def _order(ids, V):
    order = torch.empty(ids.numel(), dtype=torch.int64, device="cuda")
    starts = torch.empty(V + 1, dtype=torch.int64, device="cuda")
    dpc.dp_embedding_order(ids, V, order, starts)
    return order, starts


def test_layer_norm():
    B, T, d = 2, 850000, 1280
    x, gain, bias = _randn(1, B, T, d), 1 + 0.2 * _randn(2, d, dtype=torch.float32), _randn(3, d, dtype=torch.float32)
    assert x.numel() > 1 << 31
    out, s = torch.empty_like(x), torch.empty_like(x)
    dpc.dp_layer_norm(x, gain, bias, 1e-5, out, residual=x, sum_out=s)
    y, v, by, bv = K.layer_norm(x[:, -5:], x[:, -5:], gain, bias, 1e-5)
    L.check(out[:, -5:], y, by, "out")
    L.check(s[:, -5:], v, bv, "sum")
    del out
    n, dy, dx = 1000, torch.zeros_like(x), x
    dy[1, -n:] = _randn(4, n, d)
    rows = [torch.empty(B, d, device="cuda") for _ in range(2)]
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, dx=dx, gain_rows=rows[0], bias_rows=rows[1])
    wx, wg, wb, bx, bg, bb = K.layer_norm_backward(dy[1:, -n:], s[1:, -n:], None, gain, 1e-5)
    L.check(dx[1:, -n:], wx, bx, "dx")
    L.check(rows[0][1:], wg, bg, "gain rows")
    L.check(rows[1][1:], wb, bb, "bias rows")
    assert torch.count_nonzero(dx[0]) == 0 and torch.count_nonzero(rows[0][0]) == 0
    dpc.dp_layer_norm_backward(dy, s, gain, 1e-5, dx=dx)  # the rows as one run
    L.check(dx[1:, -n:], wx, bx, "dx alone")


def test_table_of_many_words():
    V, d = 3400000, 640
    w, ids = _randn(5, V, d), _randint(6, V - 2000, V, 2, 700)
    assert w.numel() > 1 << 31
    rows = torch.empty(2, 700, d, dtype=BF16, device="cuda")
    dpc.dp_embedding(ids, w, rows)
    assert torch.equal(rows, w[ids])
    del w
    order, starts = _order(ids, V)
    c, out = torch.tensor([0.7, 1.0], device="cuda"), torch.empty(V, d, device="cuda")
    dpc.dp_embedding_clipped_sum_noise(rows, ids, order, starts, c, 1.0, 0.0, 2.0, 0, 0, 0, out)
    want, bound = K.embedding_sum(rows, ids - (V - 2000), 2000, c, 1.0, 2.0)
    L.check(out[V - 2000:], want, bound, "out")
    assert torch.count_nonzero(out[:V - 2000]) == 0


@pytest.mark.parametrize("B,T,V", [(3400, 1000, 5003), (2, 1700000, 3)])
def test_table_of_many_tokens(B, T, V):
    """Gradients of -1, 0 and 1, so that sums of a run are exact; runs within a
    thousand tokens and of hundreds of thousands (all levels of tiles)."""
    d, ids = 640, _randint(7, -1, V, B, T)
    w = _randint(8, -1, 2, V, d).to(BF16)
    rows = torch.empty(B, T, d, dtype=BF16, device="cuda")
    assert rows.numel() > 1 << 31
    dpc.dp_embedding(ids, w, rows, scale=1.0)
    last = ids.reshape(-1)[-3000:]
    assert torch.equal(rows.view(-1, d)[-3000:], torch.where(last[:, None] < 0, 0, w[last.clamp(min=0)]))
    sign = _randint(9, 0, 2, B * T).mul_(2).sub_(1).to(BF16)
    G = rows.view(-1, d).mul_(sign[:, None]).view(B, T, d)
    order, starts = _order(ids, V)
    key = torch.where(ids < 0, V, ids).reshape(-1)
    assert torch.equal(starts, torch.bincount(key, minlength=V + 1).cumsum(0).roll(1).index_fill(
        0, torch.tensor([0], device="cuda"), 0))
    places = torch.arange(B * T, device="cuda")
    assert torch.equal(order, ((key << 32) + places).sort()[0])
    sq = torch.empty(B, device="cuda")
    dpc.dp_embedding_norm(G, ids, order, starts, sq)
    c = torch.zeros(B, device="cuda")
    c[-2:] = torch.tensor([0.5, 1.0])
    out = torch.empty(V, d, device="cuda")
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    # the same sums from the signs: exact, as are their halves
    total = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    for b in (B - 2, B - 1):
        of = key.view(B, T)[b]
        n = torch.zeros(V + 1, dtype=torch.float64, device="cuda").index_add_(0, of, sign.view(B, T)[b].double())[:V]
        S = n[:, None] * w.double()
        total += float(c[b]) * S
        want = float((S * S).sum())
        assert abs(float(sq[b]) - want) <= (d / 64 + T / 256 + 96) * L.U * want
    assert torch.equal(out.double(), total)


def test_token_logprob():
    rows, V = 43000, 50257
    z, y = _randn(10, rows, V), _randint(11, 0, V, rows)
    assert z.numel() > 1 << 31
    logp, stats, ent = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda"), torch.empty(rows, device="cuda")
    ti, tl = torch.empty(rows, 9, dtype=torch.int64, device="cuda"), torch.empty(rows, 9, device="cuda")
    dpc.dp_token_logprob(z, y, 1.3, logp, stats, entropy=ent, top_ids=ti, top_logp=tl)
    at = slice(rows - 6, rows)
    w = K.logprob(z[at], y[at], 1.3, 9)
    L.check(logp[at], w["logp"], w["logp_bound"], "logp")
    L.check(ent[at], w["entropy"], w["entropy_bound"], "entropy")
    L.check(tl[at], w["top_logp"], w["top_bound"], "top_logp")
    assert torch.equal(ti[at], w["top_ids"])
    dl = _randn(12, rows, dtype=torch.float32)
    want, bound = K.logprob_backward(z[at], y[at], 1.3, stats[at], dl[at], ent[at], dl[at])
    dpc.dp_token_logprob_backward(z, y, 1.3, stats, z, dlogp=dl, entropy=ent, dentropy=dl)
    L.check(z[at], want, bound, "grad")


@pytest.mark.parametrize("rows,V", [(3, 300007), (2, 2000003)])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_token_logprob_of_many_words(rows, V, dtype):
    """Several parts of a row share a place among the largest ones."""
    z, y = _randn(13, rows, V, dtype=dtype) * 4, _randint(14, 0, V, rows)
    z = z.to(dtype)
    z[1, V - 1], z[1, 17] = 64, 65
    logp, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    ti, tl = torch.empty(rows, 100, dtype=torch.int64, device="cuda"), torch.empty(rows, 100, device="cuda")
    dpc.dp_token_logprob(z, y, 1.0, logp, stats, top_ids=ti, top_logp=tl)
    w = K.logprob(z, y, 1.0, 100)
    L.check(logp, w["logp"], w["logp_bound"], "logp")
    L.check(tl, w["top_logp"], w["top_bound"], "top_logp")
    assert torch.equal(ti, w["top_ids"])


def test_balance():
    B, T, E, n = 2, 1100000, 1024, 500
    z = _randn(15, B, T, E)
    assert z.numel() > 1 << 31
    ids = torch.full((B, T, 2), -1, dtype=torch.int64, device="cuda")
    ids[1, -n:] = _randint(16, -1, E, n, 2)
    loss, counts = torch.empty(B, device="cuda"), torch.empty(B, E, dtype=torch.int64, device="cuda")
    tokens = torch.empty(B, dtype=torch.int64, device="cuda")
    dpc.dp_balance_loss(z, ids, loss, counts, tokens)
    wl, wc, wt, bound = K.balance(z[1:, -n:], ids[1:, -n:])
    assert torch.equal(counts[1:], wc) and torch.equal(tokens[1:], wt) and int(counts[0].sum()) == int(tokens[0]) == 0
    L.check(loss[1:], wl, bound, "loss")
    assert float(loss[0]) == 0
    want, gb = K.balance_backward(z[1:, -n:], ids[1:, -n:], None)
    dpc.dp_balance_loss_backward(z, ids, counts, tokens, z)
    L.check(z[1:, -n:], want, gb, "grad")
    assert torch.count_nonzero(z[0]) == 0 and torch.count_nonzero(z[1, :-n]) == 0


# ---- more work items than a launch has workgroups (2^20): they are looped over


def test_many_short_rows_of_words():
    rows, V = 1200000, 5
    z, y = _randn(17, rows, V), _randint(18, -1, V, rows)
    logp, stats, ent = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda"), torch.empty(rows, device="cuda")
    ti, tl = torch.empty(rows, 3, dtype=torch.int64, device="cuda"), torch.empty(rows, 3, device="cuda")
    dpc.dp_token_logprob(z, y, 1.0, logp, stats, entropy=ent, top_ids=ti, top_logp=tl)
    w = K.logprob(z, y, 1.0, 3)
    L.check(logp, w["logp"], w["logp_bound"], "logp")
    L.check(ent, w["entropy"], w["entropy_bound"], "entropy")
    L.check(tl, w["top_logp"], w["top_bound"], "top_logp")
    assert torch.equal(ti, w["top_ids"])
    dl, grad = _randn(19, rows, dtype=torch.float32), torch.empty_like(z)
    dpc.dp_token_logprob_backward(z, y, 1.0, stats, grad, dlogp=dl)
    want, bound = K.logprob_backward(z, y, 1.0, stats, dl, None, None)
    L.check(grad, want, bound, "grad")


def test_many_samples():
    B, T, V, d, E = 1200000, 2, 7, 8, 4
    ids, z = _randint(20, -1, V, B, T), _randn(21, B, T, E)
    G = _randn(22, B, T, d, dtype=torch.float32)
    sq = torch.empty(B, device="cuda")
    dpc.dp_embedding_norm(G, ids, *_order(ids, V), sq)
    g, on = G.double() * (ids >= 0)[..., None], (ids[:, :1] == ids[:, 1:])
    want = torch.where(on[:, 0], (g[:, 0] + g[:, 1]).square().sum(-1), g.square().sum((1, 2)))
    # a sum of two rows, its square's two roundings, the sum of at most 16 squares
    bound = 64 * L.U * (g[:, 0].abs() + g[:, 1].abs()).square().sum(-1) + 1e-37
    L.check(sq, want, bound, "sqnorm")
    route = ids[..., None].clamp(max=E - 1).contiguous()
    loss, counts = torch.empty(B, device="cuda"), torch.empty(B, E, dtype=torch.int64, device="cuda")
    tokens, grad = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty_like(z)
    dpc.dp_balance_loss(z, route, loss, counts, tokens)
    wl, wc, wt, bl = K.balance(z, route)
    assert torch.equal(counts, wc) and torch.equal(tokens, wt)
    L.check(loss, wl, bl, "loss")
    dpc.dp_balance_loss_backward(z, route, counts, tokens, grad)
    L.check(grad, *K.balance_backward(z, route, None), "grad")
    s, gain = G.view(B, T, d), 1 + 0.1 * _randn(23, d, dtype=torch.float32)
    rows = [torch.empty(B, d, device="cuda") for _ in range(2)]
    dpc.dp_layer_norm_backward(G, s, gain, 1e-5, gain_rows=rows[0], bias_rows=rows[1])
    _, wg, wb, _, bg, bb = K.layer_norm_backward(G, s, None, gain, 1e-5)
    L.check(rows[0], wg, bg, "gain rows")
    L.check(rows[1], wb, bb, "bias rows")


def test_many_words_of_few_tokens():
    ids = _randint(24, -1, 300000000, 3, 333)
    order, starts = _order(ids, 300000000)  # 300 million starts
    key = torch.where(ids < 0, 300000000, ids).reshape(-1)
    sorted_keys, places = torch.sort(key, stable=True)
    assert torch.equal(order, (sorted_keys << 32) + places)
    at = torch.cat([sorted_keys, sorted_keys + 1, _randint(25, 0, 300000000, 10000)]).clamp(max=300000000)
    assert torch.equal(starts[at], torch.searchsorted(sorted_keys, at))
    assert bool((starts[1:] >= starts[:-1]).all())
    V, d = 20000000, 8
    ids = _randint(26, -1, V, 3, 333)
    G, out = _randn(27, 3, 333, d), torch.empty(V, d, device="cuda")
    c = torch.tensor([0.3, 1.0, 0.9], device="cuda")
    dpc.dp_embedding_clipped_sum_noise(G, ids, *_order(ids, V), c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    words, of = torch.unique(ids, return_inverse=True)
    first = int(words[0] < 0)  # the dropped ones' row
    want, bound = K.embedding_sum(G, of - first, words.numel() - first, c, 1.0, 1.0)
    L.check(out[words[first:]], want, bound, "out")
    out[words[first:]] = 0
    assert torch.count_nonzero(out) == 0


def test_many_wide_rows():
    N, V, d = 1100000, 5, 8192
    ids, w = _randint(28, -1, V, N), _randn(29, V, d)
    rows = torch.empty(N, d, dtype=BF16, device="cuda")
    dpc.dp_embedding(ids, w, rows)
    for at in (slice(0, 2000), slice(N - 60000, N)):
        assert torch.equal(rows[at], torch.where(ids[at, None] < 0, 0, w[ids[at].clamp(min=0)]))


# ---- the widest tables, the most experts and places


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("B,T,V,d", [(2, 3, 3, 1 << 20), (1, 70, 2, (1 << 20) - 1), (3, 1, 5, (1 << 20) - 5)])
def test_widest_table(dtype, B, T, V, d):
    ids, w = _randint(30, -1, V, B, T), _randn(31, V, d, dtype=dtype)
    rows = torch.empty(B, T, d, dtype=dtype, device="cuda")
    dpc.dp_embedding(ids, w, rows)
    assert torch.equal(rows, torch.where(ids[..., None] < 0, 0, w[ids.clamp(min=0)]))
    order, starts = _order(ids, V)
    sq, c, out = torch.empty(B, device="cuda"), torch.rand(B, device="cuda"), torch.empty(V, d, device="cuda")
    G = rows.mul_(0.7)
    dpc.dp_embedding_norm(G, ids, order, starts, sq)
    L.check(sq, *K.embedding_norm(G, ids, V, 1.0), "sqnorm")
    dpc.dp_embedding_clipped_sum_noise(G, ids, order, starts, c, 1.0, 0.0, 1.0, 0, 0, 0, out)
    L.check(out, *K.embedding_sum(G, ids, V, c, 1.0, 1.0), "out")


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_most_experts_and_places(dtype):
    B, T, E = 2, 37, 1024
    z, ids = _randn(32, B, T, E, dtype=dtype), _randint(33, -1, E + 1, B, T, 1024)
    loss, counts = torch.empty(B, device="cuda"), torch.empty(B, E, dtype=torch.int64, device="cuda")
    tokens, grad = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty_like(z)
    dpc.dp_balance_loss(z, ids, loss, counts, tokens)
    wl, wc, wt, bound = K.balance(z, ids)
    assert torch.equal(counts, wc) and torch.equal(tokens, wt)
    L.check(loss, wl, bound, "loss")
    dpc.dp_balance_loss_backward(z, ids, counts, tokens, grad)
    L.check(grad, *K.balance_backward(z, ids, None), "grad")
