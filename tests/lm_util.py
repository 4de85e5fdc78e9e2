"""Plain 64-bit forms of the language-model operators and the error bounds the
GPU tests hold the kernels to.

Every bound counts roundings: u = 2^-24 is half a step of fp32 (the kernels'
arithmetic), half(dtype) half a step of the storage type. A sum of n products
formed in fp32 in any order is off by at most (n + few) * u times the sum of
the products' magnitudes (products of bf16 are exact in fp32)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half(dtype):
    """Half a storage step, relative; fp32 outputs are the arithmetic's own roundings."""
    return torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    want, bound = want.double().cpu(), bound.double().cpu()
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / bound)[bad].max()):.3g} "
                           f"of the bound, first at {bad.nonzero()[0].tolist()}")


# ---- root-mean-square norm


def rms_forward(x, residual, gain, eps):
    s = x.double() + (0 if residual is None else residual.double())
    return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + eps) * gain.double(), s


def rms_forward_bounds(y, s, dtype):
    # sum of squares: 32 sequential and 10 tree additions, halved by the square root; then sqrt, 1/x, two
    # products, the sum's own rounding: 40 u covers them
    return (40 * U + half(dtype)) * y.abs() + 1e-37, (U + half(dtype)) * s.abs() + 1e-37


def rms_backward(dy, s, dsum, gain, eps):
    dy, v, gain = dy.double(), s.double(), gain.double()
    rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    u, h = v * rstd, dy * gain
    along = (h * u).mean(-1, keepdim=True)
    dx = rstd * (h - u * along) + (0 if dsum is None else dsum.double())
    mag = rstd * (h.abs() + u.abs() * (h * u).abs().mean(-1, keepdim=True)) + (0 if dsum is None else dsum.double().abs())
    T = s[0].numel() // s.shape[-1]
    rows = (dy * u).reshape(s.shape[0], T, -1)
    # 32 sequential, 10 tree additions in each row sum, rstd to the third power: 128 u of the terms' magnitudes
    dx_bound = 128 * U * mag + half(s.dtype) * dx.abs() + 1e-37
    return dx, rows.sum(1), dx_bound, (T + 128) * U * rows.abs().sum(1) + 1e-37


# ---- distillation loss


def teacher_dist(ids, teacher, V, tau):
    used = (ids >= 0) & (ids < V) & (teacher.double() > -float("inf"))
    t = (teacher.double() / tau).masked_fill(~used, -float("inf"))
    some = used.any(-1)
    q = torch.softmax(t.masked_fill(~some[..., None], 0.0), -1)
    return torch.where(used, q, torch.zeros_like(q)), some


def distill_forward(logits, ids, teacher, tau, weight):
    V = logits.shape[-1]
    z = logits.double() / tau
    lse = torch.logsumexp(z, -1)
    q, some = teacher_dist(ids, teacher, V, tau)
    w = torch.ones_like(lse) if weight is None else weight.double()
    at = torch.gather(z, -1, ids.clamp(0, V - 1)) - lse[..., None]
    term = torch.where(q > 0, torch.special.xlogy(q, q) - q * at, torch.zeros_like(q))
    count = some & (w != 0)
    tok = torch.where(count, term.sum(-1) * w * tau ** 2, torch.zeros_like(lse))
    # per token: the student's sum (V/256 additions a thread, the joins, two roundings of each exponent's
    # argument, weighted by the exponentials themselves: at most 64 u), the places' sums and logarithms
    big = z.abs().amax(-1) + lse.abs() + torch.where(q > 0, at.abs(), torch.zeros_like(q)).amax(-1)
    tok_bound = torch.where(count, (V / 256 + 128 + ids.shape[-1] / 32 + 8 * big) * U * w.abs() * tau ** 2
                            * (1 + 0 * lse), torch.zeros_like(lse))
    T = logits.shape[1]
    loss_bound = tok_bound.sum(1) + (T + 8) * U * tok.abs().sum(1) + 1e-37
    return tok.sum(1), lse, loss_bound, (V / 256 + 128) * U + 4 * U * (z.abs().amax(-1) + lse.abs())


def distill_backward(logits, ids, teacher, tau, weight, dloss, lse):
    V = logits.shape[-1]
    z = logits.double() / tau
    q, some = teacher_dist(ids, teacher, V, tau)
    f = torch.full_like(lse, tau, dtype=torch.float64)
    if weight is not None:
        f = f * weight.double()
    if dloss is not None:
        f = f * dloss.double()[:, None]
    on = (some & (f != 0))[..., None]
    arg = z - lse.double()[..., None]
    p = torch.where(on, arg.exp(), torch.zeros_like(z))
    full = torch.zeros_like(z).scatter_add_(-1, ids.clamp(0, V - 1), q)
    grad = torch.where(on, (p - full) * f[..., None], torch.zeros_like(z))
    # the exponent's argument: three roundings of it and of z / tau; q: its exponential and its sum over K
    bound = f.abs()[..., None] * U * torch.where(on, p * (4 * arg.abs() + 4 * z.abs() + 16) + full * (64 + ids.shape[-1]),
                                                 torch.zeros_like(z))
    return grad, bound + half(logits.dtype) * grad.abs() + 1e-37


# ---- products grouped by expert


def segments_of(counts):
    """[E, B] row counts -> segments [E*B + 1] on the GPU and the host list."""
    flat = torch.as_tensor(counts, dtype=torch.int64).reshape(-1)
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), flat.cumsum(0)])
    return ends.cuda(), ends.tolist()


def grouped_matmul(X, W, ends, B, transpose):
    E = W.shape[0]
    x, w = X.double(), W.double()
    n = w.shape[2] if transpose else w.shape[1]
    y = torch.zeros(X.shape[0], n, dtype=torch.float64, device=X.device)
    mag = torch.zeros_like(y)
    for e in range(E):
        i, j = ends[e * B], ends[(e + 1) * B]
        if j > i:
            we = w[e] if transpose else w[e].T.contiguous()
            y[i:j] = x[i:j] @ we
            mag[i:j] = x[i:j].abs() @ we.abs()
    return y, (X.shape[1] + 8) * U * mag + half(X.dtype) * y.abs() + 1e-37


def grouped_norm(A, G, ends, B):
    E = (len(ends) - 1) // B
    a, g = A.double(), G.double()
    sq = torch.zeros(B, dtype=torch.float64, device=A.device)
    bound = torch.zeros_like(sq)
    for k in range(E * B):
        i, j = ends[k], ends[k + 1]
        if j > i:
            sq[k % B] += ((a[i:j].T @ g[i:j]) ** 2).sum()
            gram = (a[i:j].abs() @ a[i:j].abs().T) * (g[i:j].abs() @ g[i:j].abs().T)
            bound[k % B] += gram.sum() * U * (A.shape[1] + G.shape[1] + 512)
    return sq, bound + 1e-37


def grouped_sum(A, G, ends, c, denom):
    B = c.numel()
    E = (len(ends) - 1) // B
    a, g = A.double(), G.double()
    out = torch.zeros(E, A.shape[1], G.shape[1], dtype=torch.float64, device=A.device)
    mag = torch.zeros_like(out)
    for k in range(E * B):
        i, j = ends[k], ends[k + 1]
        if j > i:
            out[k // B] += c[k % B].double() * (a[i:j].T @ g[i:j])
            mag[k // B] += c[k % B].double().abs() * (a[i:j].abs().T @ g[i:j].abs())
    rows = max(ends[(e + 1) * B] - ends[e * B] for e in range(E))
    return out / denom, (rows + 2 * B + 64) * U * mag / denom + 1e-37
