"""Plain 64-bit forms of the operators from tokens to a per-sample loss and the
error bounds the GPU tests hold the kernels to, counted in roundings as in
lm_util: U is half a step of fp32, half(dtype) half a step of the storage type."""
from __future__ import annotations

import torch

from lm_util import U, half

TINY = 1e-37


# ---- layer norm


def layer_norm(x, residual, gain, bias, eps):
    """(y, s, bound of y, bound of s)."""
    xd, rd = x.double(), torch.zeros_like(x, dtype=torch.float64) if residual is None else residual.double()
    s, g = xd + rd, gain.double()
    b = torch.zeros_like(g) if bias is None else bias.double()
    off = s - s.mean(-1, keepdim=True)
    rstd = torch.rsqrt((off * off).mean(-1, keepdim=True) + eps)
    u = off * rstd
    y = u * g + b
    mean_off = off.abs().mean(-1, keepdim=True)
    add = (xd.abs() + rd.abs()) if residual is not None else torch.zeros_like(s)  # the addition's rounding
    rms_add = add.square().mean(-1, keepdim=True).sqrt()
    # 32 sequential and 10 tree additions in the rest of the mean and in the variance, then the square root, its
    # reciprocal and two products: 64 u of each covers them
    bound = ((64 * U + 2 * U * rms_add * rstd) * (u * g).abs() + g.abs() * rstd * (2 * U * (add + rms_add)
             + 64 * U * mean_off) + 2 * U * (y.abs() + b.abs()) + half(x.dtype) * y.abs() + TINY)
    return y, s, bound, (U + half(x.dtype)) * s.abs() + TINY


def layer_norm_backward(dy, s, dsum, gain, eps):
    """(dx, gain rows, bias rows, their bounds)."""
    B, T = s.shape[0], s[0].numel() // s.shape[-1]
    dyd, v, g = dy.double(), s.double(), gain.double()
    ds = torch.zeros_like(v) if dsum is None else dsum.double()
    off = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt((off * off).mean(-1, keepdim=True) + eps)
    u, h = off * rstd, dyd * g
    dx = ds + rstd * (h - h.mean(-1, keepdim=True) - u * (h * u).mean(-1, keepdim=True))
    # every row sum: 32 sequential and 10 tree additions; u's own error: that of the mean's rest beside its rounding
    um = u.abs() + (off.abs() * rstd).mean(-1, keepdim=True)
    mag = rstd * (h.abs() + h.abs().mean(-1, keepdim=True) + um * (h.abs() * um).mean(-1, keepdim=True))
    bound = 192 * U * mag + 4 * U * ds.abs() + half(s.dtype) * dx.abs() + TINY
    rows = lambda t: t.reshape(B, T, -1).sum(1)
    n = (T + 128) * U
    return dx, rows(dyd * u), rows(dyd), bound, n * rows(dyd.abs() * um) + TINY, n * rows(dyd.abs()) + TINY


# ---- table of words


def embedding(ids, weight, scale, dtype):
    V = weight.shape[0]
    ok = (ids >= 0) & (ids < V)
    y = weight.double()[ids.clamp(0, V - 1)] * scale
    y = torch.where(ok[..., None], y, torch.zeros_like(y))
    return y, (U + half(dtype)) * y.abs() + TINY


def order(ids, V):
    """(order, starts) of ids as host lists' tensors."""
    key = torch.where((ids < 0) | (ids >= V), torch.full_like(ids, V), ids).reshape(-1).cpu()
    key, places = torch.sort(key, stable=True)
    return (key << 32) + places, torch.searchsorted(key, torch.arange(V + 1))


def embedding_norm(G, ids, V, scale):
    B, d = G.shape[0], G.shape[-1]
    G, ids = G.double().reshape(B, -1, d), ids.reshape(B, -1)
    T = ids.shape[1]
    sq, bound = torch.zeros(B, dtype=torch.float64), torch.zeros(B, dtype=torch.float64)
    for b in range(B):
        ok = (ids[b] >= 0) & (ids[b] < V)
        if not ok.any():
            continue
        words, of, n = torch.unique(ids[b][ok], return_inverse=True, return_counts=True)
        S = torch.zeros(words.numel(), d, dtype=torch.float64, device=G.device).index_add_(0, of, G[b][ok])
        M = torch.zeros_like(S).index_add_(0, of, G[b][ok].abs())
        e = (n.double()[:, None] + 8) * U * M  # a run's sum of n rows
        sq[b] = (S * S).sum()
        bound[b] = (2 * S.abs() * e + e * e).sum() + (d / 64 + T / 256 + 96) * U * (S.abs() + e).square().sum()
    return sq * scale ** 2, bound * scale ** 2 * (1 + 1e-6) + TINY


def embedding_sum(G, ids, V, c, scale, denom):
    B, d = G.shape[0], G.shape[-1]
    ok = (ids >= 0) & (ids < V)
    word = torch.where(ok, ids, torch.full_like(ids, V)).reshape(-1)
    rows = (G.double().reshape(B, -1, d) * c.double()[:, None, None]).reshape(-1, d) * scale / denom
    S = torch.zeros(V + 1, d, dtype=torch.float64, device=G.device).index_add_(0, word, rows)
    M = torch.zeros_like(S).index_add_(0, word, rows.abs())
    n = torch.bincount(word, minlength=V + 1)[:, None].double()
    return S[:V], ((n + 16) * U * M)[:V] + TINY


# ---- log probabilities


def logprob(logits, targets, tau, K):
    """A dict of values and bounds; rows of -inf alone have no distribution."""
    z = logits.double()
    V = z.shape[-1]
    m = z.amax(-1, keepdim=True)
    none = (m == -float("inf")).squeeze(-1)
    x = torch.where(none[..., None], torch.zeros_like(z), (z - m) / tau)
    e = torch.exp(x)
    s = e.sum(-1)
    log_s, p = torch.log(s), e / s[..., None]
    far = torch.where(p > 0, x.abs(), torch.zeros_like(x))
    ex, ex2 = (p * far).sum(-1), (p * far * far).sum(-1)
    # the sum: V/256 (or V/64 up to 4096 words) additions a thread, the joins, every exponent's argument off by 4 u
    # of itself, two steps of the exponential
    rel = (V / 256 + 256 + 8 * ex) * U
    out = {"m": m.squeeze(-1), "log_s": torch.where(none, torch.zeros_like(log_s), log_s), "log_s_bound": rel + 4 * U * log_s,
           "entropy": torch.where(none, torch.zeros_like(ex), log_s + ex),
           "entropy_bound": rel * (1 + ex) + (V / 256 + 256) * U * ex + 8 * U * ex2 + 4 * U * (log_s + ex)}
    given = (targets >= 0) & (targets < V)
    xy = torch.gather(x, -1, targets.clamp(0, V - 1)[..., None]).squeeze(-1)
    logp = torch.where(none, torch.full_like(xy, -float("inf")), xy - log_s)
    out["logp"] = torch.where(given, logp, torch.zeros_like(logp))
    out["logp_bound"] = rel + 6 * U * (torch.where(xy.isinf(), torch.zeros_like(xy), xy.abs()) + log_s)
    if K:
        order = torch.sort(logits.float().cpu(), dim=-1, descending=True, stable=True)[1][..., :K].to(logits.device)
        xt = torch.gather(x, -1, order)
        out["top_ids"] = order
        out["top_logp"] = torch.where(none[..., None], torch.full_like(xt, -float("inf")), xt - log_s[..., None])
        out["top_bound"] = rel[..., None] + 6 * U * (torch.where(xt.isinf(), torch.zeros_like(xt), xt.abs())
                                                     + log_s[..., None])
    return out


def logprob_backward(logits, targets, tau, stats, dlogp, entropy, dentropy):
    z, m, log_s = logits.double(), stats[..., :1].double(), stats[..., 1:].double()
    V = z.shape[-1]
    given = (targets >= 0) & (targets < V)
    zero = torch.zeros(targets.shape, dtype=torch.float64, device=z.device)
    dl = (torch.where(given, dlogp.double(), zero) if dlogp is not None else zero)[..., None] / tau
    dh = (zero if dentropy is None else dentropy.double())[..., None] / tau
    h = (zero if entropy is None else entropy.double())[..., None]
    on = ((dl != 0) | (dh != 0)) & (m != -float("inf"))
    x = torch.where(on, (z - m) / tau, torch.zeros_like(z))
    lp = x - log_s
    p = torch.exp(lp)
    far = torch.where(p > 1e-40, x.abs() + lp.abs(), torch.zeros_like(x))
    lp0 = torch.where(p > 0, lp, torch.zeros_like(lp))
    g = -p * (dl + dh * (lp0 + h))
    hit = torch.zeros_like(z).scatter_(-1, targets.clamp(0, V - 1)[..., None], 1.0) * given[..., None]
    g = torch.where(on, g + hit * dl, torch.zeros_like(g))
    mag = p * (dl.abs() + dh.abs() * (lp0.abs() + h.abs()))
    bound = torch.where(on, mag * (4 * far + 24) * U + hit * dl.abs() * 4 * U, torch.zeros_like(g))
    return g, bound + half(logits.dtype) * g.abs() + TINY


# ---- balance loss


def balance(logits, ids):
    """(loss, counts, tokens, bound of the loss)."""
    B, T, E = logits.shape
    ok = (ids >= 0) & (ids < E)
    used = ok.any(-1)
    z = torch.where(used[..., None], logits.double(), torch.zeros_like(logits, dtype=torch.float64))
    p = torch.softmax(z, -1) * used[..., None]
    place = torch.where(ok, ids, torch.full_like(ids, E)).reshape(B, -1)
    counts = torch.zeros(B, E + 1, dtype=torch.int64, device=ids.device).scatter_add_(1, place, torch.ones_like(place))[:, :E]
    tokens = used.sum(1)
    f = counts.double() / counts.sum(1, keepdim=True).clamp(min=1)
    far = (z - z.amax(-1, keepdim=True)).abs()
    n = tokens.clamp(min=1)[:, None]
    loss = E * (f * p.sum(1) / n).sum(1)
    # a probability: its argument's rounding, two steps, its sum over E; then the sums over tokens and experts
    bound = E * (f * (p * (4 * far + T + E / 8 + 128)).sum(1) / n).sum(1) * U
    return loss, counts, tokens, bound + TINY


def balance_backward(logits, ids, dloss):
    B, T, E = logits.shape
    _, counts, tokens, _ = balance(logits, ids)
    used = ((ids >= 0) & (ids < E)).any(-1)[..., None]
    z = torch.where(used, logits.double(), torch.zeros_like(logits, dtype=torch.float64))
    p = torch.softmax(z, -1)
    dl = torch.ones(B, dtype=torch.float64, device=z.device) if dloss is None else dloss.double()
    a = (counts - counts.amin(1, keepdim=True)).double() * (
        E * dl / counts.sum(1).clamp(min=1) / tokens.clamp(min=1))[:, None]
    a = a[:, None, :]
    g = torch.where(used, p * (a - (p * a).sum(-1, keepdim=True)), torch.zeros_like(p))
    far = (z - z.amax(-1, keepdim=True)).abs()
    far = torch.where(p > 1e-40, far, torch.zeros_like(far))
    inner = (p * a.abs() * (4 * far + E / 4 + 64)).sum(-1, keepdim=True)
    bound = U * p * (a.abs() * (4 * far + E / 4 + 64) + inner + (4 * far + E / 4 + 64) * (p * a.abs()).sum(-1, keepdim=True))
    return g, torch.where(used, bound, torch.zeros_like(bound)) + half(logits.dtype) * g.abs() + TINY
