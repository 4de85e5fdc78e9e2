"""What the operators of private language-model training are measured on: the
cases, their inputs, the operators' plain forms in elementary torch
operations, and their values in 64 bits.

Operators and their directions (``case["op"]``):

  rms-forward       y = s / rms(s) * gain and s = x + residual
  rms-backward      ds of it (the residual stream's gradient joined in), and
                    the gain's gradient of every sample, [B, d]
  distill-forward   per-sample distillation loss from a teacher's top logits,
                    and each token's log-sum-exp
  distill-backward  its gradient over the whole vocabulary
  experts-forward   rows sorted by expert times their expert's weight
  experts-input     the gradient of those products' rows
  experts-clip      an expert layer's clipping pass: every sample's squared
                    gradient norm over all experts, the clip factors, and
                    every expert's clipped weight-gradient mean
"""
import math

import torch

own = False  # True: run() calls the library; False: the plain forms

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 8 sequences at GPT-2-large width: a launch's latency
        {"name": "rms-forward-tokens", "op": "rms-forward", "dtype": "bf16", "B": 8, "T": 1, "d": 1280},
        # a training batch of the GPT-2-large workload
        {"name": "rms-forward-batch", "op": "rms-forward", "dtype": "bf16", "B": 32, "T": 1024, "d": 1280},
        {"name": "rms-backward-batch", "op": "rms-backward", "dtype": "bf16", "B": 32, "T": 1024, "d": 1280},
        # an odd width and ragged row count in 32 bits
        {"name": "rms-backward-odd", "op": "rms-backward", "dtype": "f32", "B": 13, "T": 77, "d": 1001},
        # scoring the last token of 4 sequences over GPT-2's vocabulary
        {"name": "distill-forward-tokens", "op": "distill-forward", "dtype": "bf16", "B": 4, "T": 1, "V": 50257,
         "K": 64, "tau": 2.0},
        # an evaluation batch in 32 bits
        {"name": "distill-forward-batch", "op": "distill-forward", "dtype": "f32", "B": 8, "T": 256, "V": 32003,
         "K": 100, "tau": 1.0},
        # a physical training batch over GPT-2's vocabulary
        {"name": "distill-backward-batch", "op": "distill-backward", "dtype": "bf16", "B": 8, "T": 512, "V": 50257,
         "K": 64, "tau": 2.0},
        # one token of 4 sequences through 8 experts: the active experts' weights are the traffic
        {"name": "experts-forward-tokens", "op": "experts-forward", "dtype": "bf16", "B": 4, "T": 1, "top": 2, "E": 8,
         "d": 1280, "p": 5120},
        # a training batch through the up projection of 8 experts
        {"name": "experts-forward-batch", "op": "experts-forward", "dtype": "bf16", "B": 32, "T": 512, "top": 2,
         "E": 8, "d": 1280, "p": 5120},
        # the same layer's gradient of its rows, more and shorter experts
        {"name": "experts-input-batch", "op": "experts-input", "dtype": "bf16", "B": 8, "T": 512, "top": 2, "E": 16,
         "d": 1280, "p": 5120},
        # the clipping pass of an expert layer
        {"name": "experts-clip-batch", "op": "experts-clip", "dtype": "bf16", "B": 32, "T": 512, "top": 2, "E": 8,
         "d": 1280, "p": 5120},
        # odd sizes, short ragged segments, 32 bits
        {"name": "experts-clip-odd", "op": "experts-clip", "dtype": "f32", "B": 9, "T": 131, "top": 2, "E": 5,
         "d": 333, "p": 517},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms-forward", "rms-backward", "distill-forward", "distill-backward", "experts-forward",
                     "experts-input", "experts-clip"])
    case = {"op": op, "dtype": rng.choice(["bf16", "f32"])}
    size = 2 if case["dtype"] == "bf16" else 4
    while True:
        case["B"] = _log_int(rng, 1, 64)
        case["T"] = 1 if rng.random() < 0.15 else _log_int(rng, 1, 2048)
        rows = case["B"] * case["T"]
        if op.startswith("rms"):
            case["d"] = _log_int(rng, 32, 8192)
            if rng.random() < 0.6:
                case["d"] = max(8, case["d"] // 8 * 8)
            if rows * case["d"] * size <= 84e6:
                return case
        elif op.startswith("distill"):
            case["V"] = _log_int(rng, 500, 130000)
            case["K"] = _log_int(rng, 1, 256)
            case["tau"] = rng.choice([1.0, 1.5, 2.0, 4.0])
            if rows * case["V"] * size <= 400e6:
                return case
        else:
            case["E"] = _log_int(rng, 1, 64)
            case["top"] = rng.randint(1, min(4, case["E"]))
            case["d"] = _log_int(rng, 64, 2560)
            case["p"] = _log_int(rng, 64, 5120)
            if rng.random() < 0.6:
                case["d"], case["p"] = max(16, case["d"] // 16 * 16), max(16, case["p"] // 16 * 16)
            r = rows * case["top"]
            if 2 * r * case["d"] * case["p"] <= (2e11 if size == 2 else 5e10) and r <= 40000 and \
                    case["E"] * case["d"] * case["p"] <= 120e6 and case["E"] * case["B"] <= 512:
                return case


def work(case):
    B, T = case["B"], case["T"]
    size, rows = (2 if case["dtype"] == "bf16" else 4), B * T
    op = case["op"]
    if op == "rms-forward":
        return {"bytes": 4 * rows * case["d"] * size + 4 * case["d"], "flops": 5 * rows * case["d"]}
    if op == "rms-backward":
        return {"bytes": 4 * rows * case["d"] * size + 4 * case["d"] + 4 * B * case["d"],
                "flops": 12 * rows * case["d"]}
    if op.startswith("distill"):
        small = rows * case["K"] * (8 + size) + 8 * rows + 4 * B
        if op == "distill-forward":
            return {"bytes": rows * case["V"] * size + small, "flops": 4 * rows * case["V"]}
        return {"bytes": 2 * rows * case["V"] * size + small, "flops": 4 * rows * case["V"]}
    E, d, p, r = case["E"], case["d"], case["p"], rows * case["top"]
    if op in ("experts-forward", "experts-input"):
        active = E * (1.0 - (1.0 - 1.0 / E) ** r) if E > 1 else 1.0  # experts that get a row, on average
        return {"bytes": int(r * (d + p) * size + active * d * p * size), "flops": 2 * r * d * p}
    per = r / float(E * B)  # rows of one sample in one expert, on average
    return {"bytes": r * (d + p) * size + 4 * E * d * p + 8 * B,
            "flops": int(2 * r * d * p + r * (per + 1) * (d + p))}


def _normal(g, shape, scale, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, B, T = TYPES[case["dtype"]], case["B"], case["T"]
    s = {"case": dict(case)}
    if case["op"].startswith("rms"):
        d = case["d"]
        s["gain"] = 1.0 + _normal(g, (d,), 0.2, torch.float32)
        # rows of uneven size, as a residual stream has them
        size = torch.exp(_normal(g, (B, T, 1), 0.5, torch.float32))
        x = (_normal(g, (B, T, d), 1.0, torch.float32) * size).to(dt)
        s["out"] = torch.empty(B, T, d, device="cuda", dtype=dt)
        if case["op"] == "rms-forward":
            s["x"], s["residual"] = x, (_normal(g, (B, T, d), 1.0, torch.float32) * size).to(dt)
            s["sum"] = torch.empty_like(x)
        else:
            s["s"], s["dy"], s["dsum"] = x, _normal(g, (B, T, d), 0.02, dt), _normal(g, (B, T, d), 0.02, dt)
            s["rows"] = torch.empty(B, d, device="cuda", dtype=torch.float32)
            if own:
                s["ws"] = _scratch(_library().dp_rms_norm_workspace_bytes(_code(dt), B, T, d))
    elif case["op"].startswith("distill"):
        V, K = case["V"], min(case["K"], case["V"])
        s["logits"] = _normal(g, (B, T, V), 2.5, dt)
        # K different words a token, at places that depend on the token; a tenth of the places unused
        step = 1 + torch.randint(0, max(1, V // K), (B, T, 1), generator=g, device="cuda")
        ids = (torch.randint(0, V, (B, T, 1), generator=g, device="cuda")
               + step * torch.arange(K, device="cuda")) % V
        unused = torch.rand((B, T, K), generator=g, device="cuda") < 0.1
        s["ids"] = torch.where(unused, torch.full_like(ids, -1), ids)
        s["teacher"] = torch.sort(_normal(g, (B, T, K), 2.0, torch.float32), dim=-1, descending=True)[0].to(dt)
        # prompt tokens carry no loss
        s["weight"] = (torch.rand((B, T), generator=g, device="cuda") > 0.05).float()
        s["loss"] = torch.empty(B, device="cuda", dtype=torch.float32)
        s["lse"] = torch.empty(B, T, device="cuda", dtype=torch.float32)
        if case["op"] == "distill-backward":
            z = s["logits"].double() / case["tau"]
            s["lse"] = torch.logsumexp(z, dim=-1).float()
            del z
            s["dloss"] = 0.5 + torch.rand(B, generator=g, device="cuda")
            s["grad"] = torch.empty_like(s["logits"])
        elif own:
            s["ws"] = _scratch(_library().dp_distill_workspace_bytes(_code(dt), B, T, V, K))
    else:
        E, d, p = case["E"], case["d"], case["p"]
        # routing: every token goes to `top` different experts, some experts being more popular
        popular = 0.5 * torch.randn((E,), generator=g, device="cuda")
        noise = torch.rand((B * T, E), generator=g, device="cuda").clamp_(1e-6, 1.0)
        expert = torch.topk(popular - torch.log(-torch.log(noise * 0.999999)), case["top"], dim=-1)[1]
        sample = torch.arange(B * T, device="cuda")[:, None] // T
        counts = torch.bincount((expert * B + sample).reshape(-1), minlength=E * B)
        # segments[e * B + b] .. segments[e * B + b + 1]: the rows of sample b in expert e
        s["segments"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(counts, 0)])
        s["ends"] = s["segments"].tolist()
        r = B * T * case["top"]
        if case["op"] == "experts-clip":
            s["A"], s["G"] = _normal(g, (r, d), d ** -0.5, dt), _normal(g, (r, p), p ** -0.5, dt)
            s["C"] = math.sqrt(T * case["top"])  # about half of the samples clip
            s["sq"], s["c"] = (torch.empty(B, device="cuda", dtype=torch.float32) for _ in range(2))
            s["out"] = torch.empty(E, d, p, device="cuda", dtype=torch.float32)
            if own:
                s["ws"] = _scratch(_library().dp_grouped_workspace_bytes(_code(dt), r, E, B, d, p))
        else:
            forward = case["op"] == "experts-forward"
            s["w"] = _normal(g, (E, p, d), d ** -0.5, dt)
            s["x"] = _normal(g, (r, d if forward else p), 1.0 if forward else 0.05, dt)
            s["out"] = torch.empty(r, p if forward else d, device="cuda", dtype=dt)
            if own:
                s["ws"] = _scratch(_library().dp_grouped_workspace_bytes(_code(dt), r, E, B, d, p))
    return s


def _library():
    import sample_gradient_clipping_layer_amd as dpc
    return dpc


def _code(dt):
    return _library().DP_BF16 if dt == torch.bfloat16 else _library().DP_F32


def _scratch(nbytes):
    return torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    dpc, case = _library(), s["case"]
    op = case["op"]
    if op == "rms-forward":
        dpc.dp_rms_norm(s["x"], s["gain"], EPS, s["out"], residual=s["residual"], sum_out=s["sum"])
        return s["out"], s["sum"]
    if op == "rms-backward":
        dpc.dp_rms_norm_backward(s["dy"], s["s"], s["gain"], EPS, dx=s["out"], dsum=s["dsum"], gain_rows=s["rows"],
                                 workspace=s["ws"])
        return s["out"], s["rows"]
    if op == "distill-forward":
        dpc.dp_distill_loss(s["logits"], s["ids"], s["teacher"], case["tau"], s["loss"], s["lse"],
                            weight=s["weight"], workspace=s["ws"])
        return s["loss"], s["lse"]
    if op == "distill-backward":
        dpc.dp_distill_loss_backward(s["logits"], s["ids"], s["teacher"], case["tau"], s["lse"], s["grad"],
                                     weight=s["weight"], dloss=s["dloss"])
        return s["grad"]
    if op == "experts-clip":
        dpc.dp_grouped_norm(s["A"], s["G"], s["segments"], s["sq"], workspace=s["ws"])
        dpc.dp_clip_factors(s["sq"], s["C"], s["c"])
        dpc.dp_grouped_clipped_sum_noise(s["A"], s["G"], s["segments"], s["c"], s["C"], 0.0, float(case["B"]), 0, 0, 0,
                                         s["out"], workspace=s["ws"])
        return s["sq"], s["c"], s["out"]
    dpc.dp_grouped_matmul(s["x"], s["w"], s["segments"], s["out"], transpose=op == "experts-input",
                          workspace=s["ws"])
    return s["out"]


def _teacher_plain(s, tau):
    """The teacher's distribution over its listed words: probabilities and
    their logarithms, zero where a place is unused."""
    used = s["ids"] >= 0
    t = torch.where(used, s["teacher"].float() / tau, torch.full_like(s["teacher"], -1e30, dtype=torch.float32))
    top = t.amax(-1, keepdim=True)
    e = torch.where(used, torch.exp(t - top), torch.zeros_like(t))
    total = e.sum(-1, keepdim=True)
    some = total > 0
    q = torch.where(some, e / torch.where(some, total, torch.ones_like(total)), torch.zeros_like(e))
    logq = torch.where(used & some, t - top - torch.log(torch.where(some, total, torch.ones_like(total))),
                       torch.zeros_like(t))
    return q, logq, some.squeeze(-1), torch.where(used, s["ids"], torch.zeros_like(s["ids"]))


def _run_plain(s):
    case = s["case"]
    op, B, T = case["op"], case["B"], case["T"]
    if op == "rms-forward":
        v = s["x"].float() + s["residual"].float()
        y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["gain"]
        return y.to(s["x"].dtype), v.to(s["x"].dtype)
    if op == "rms-backward":
        v, dy = s["s"].float(), s["dy"].float()
        rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        unit, h = v * rstd, dy * s["gain"]
        dx = s["dsum"].float() + rstd * (h - unit * (h * unit).mean(-1, keepdim=True))
        return dx.to(s["s"].dtype), (dy * unit).sum(1)
    if op == "distill-forward":
        tau = case["tau"]
        z = s["logits"].float() / tau
        top = z.amax(-1, keepdim=True)
        lse = (top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))).squeeze(-1)
        q, logq, some, at = _teacher_plain(s, tau)
        token = (q * (logq - torch.gather(z, -1, at) + lse[..., None])).sum(-1)
        return (torch.where(some, token, torch.zeros_like(token)) * s["weight"] * tau * tau).sum(1), lse
    if op == "distill-backward":
        tau = case["tau"]
        g = torch.exp(s["logits"].float() / tau - s["lse"][..., None])
        q, _, some, at = _teacher_plain(s, tau)
        g = g * some[..., None]
        g.scatter_add_(-1, at, -q)
        return (g * (s["weight"] * s["dloss"][:, None] * tau)[..., None]).to(s["logits"].dtype)
    E, ends = case["E"], s["ends"]
    if op == "experts-clip":
        A, G = s["A"].float(), s["G"].float()
        norms = []
        for b in range(B):
            total = torch.zeros((), device="cuda")
            for e in range(E):
                i, j = ends[e * B + b], ends[e * B + b + 1]
                if j > i:
                    total = total + ((A[i:j] @ A[i:j].T) * (G[i:j] @ G[i:j].T)).sum()
            norms.append(total)
        sq = torch.stack(norms)
        norm = torch.sqrt(sq)
        c = torch.where(norm > s["C"], s["C"] / norm, torch.ones_like(norm))
        row_sample = (torch.searchsorted(s["segments"], torch.arange(A.shape[0], device="cuda"), right=True) - 1) % B
        A = A * c[row_sample][:, None]
        out = torch.stack([A[ends[e * B]:ends[(e + 1) * B]].T @ G[ends[e * B]:ends[(e + 1) * B]] for e in range(E)])
        return sq, c, out / float(B)
    x, w = s["x"], s["w"]
    parts = []
    for e in range(E):
        i, j = ends[e * B], ends[(e + 1) * B]
        if j > i:
            we = w[e].float()
            parts.append(x[i:j].float() @ (we.T if op == "experts-forward" else we))
    return torch.cat(parts).to(x.dtype)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits: norms from explicit
    sums, the loss from probabilities, products row block by row block."""
    s = prepare(case, seed)
    op, B, T = case["op"], case["B"], case["T"]
    f64 = torch.float64
    if op == "rms-forward":
        v = s["x"].to(f64).add(s["residual"].to(f64))
        rms = torch.linalg.vector_norm(v, dim=-1, keepdim=True).square().div(case["d"]).add(EPS).sqrt()
        return v / rms * s["gain"].to(f64), v
    if op == "rms-backward":
        # column by column of the Jacobian's action: d(s/rms)/ds = (I - s s^T / (d rms^2)) / rms
        v, dy = s["s"].to(f64), s["dy"].to(f64)
        ms = torch.einsum("btd,btd->bt", v, v) / case["d"] + EPS
        h = dy * s["gain"].to(f64)
        along = torch.einsum("btd,btd->bt", h, v) / (case["d"] * ms)
        dx = (h - along[..., None] * v) / ms.sqrt()[..., None] + s["dsum"].to(f64)
        return dx, torch.einsum("btd,btd,bt->bd", dy, v, ms.rsqrt())
    if op.startswith("distill"):
        tau, V = case["tau"], case["V"]
        used = s["ids"] >= 0
        q = torch.softmax((s["teacher"].to(f64) / tau).masked_fill(~used, -math.inf), dim=-1)
        q = torch.nan_to_num(q, nan=0.0)
        some = used.any(-1)
        if op == "distill-backward":
            p = torch.softmax(s["logits"].to(f64) / tau, dim=-1)
            full = torch.zeros(B, T, V, dtype=f64, device="cuda")
            full.scatter_add_(-1, s["ids"].clamp(min=0), q)
            return (p * some[..., None] - full) * (tau * s["weight"].to(f64) * s["dloss"].to(f64)[:, None])[..., None]
        logp = torch.log_softmax(s["logits"].to(f64) / tau, dim=-1)
        at = torch.gather(logp, -1, s["ids"].clamp(min=0))
        token = (torch.special.xlogy(q, q) - q * at).sum(-1)
        loss = (token * some * s["weight"].to(f64)).sum(1) * tau ** 2
        return loss, torch.logsumexp(s["logits"].to(f64) / tau, dim=-1)
    E, ends = case["E"], s["ends"]
    if op == "experts-clip":
        if 6 * s["A"].shape[0] * case["d"] * case["p"] > 3e12:
            return None
        A, G = s["A"].to(f64), s["G"].to(f64)
        held = [k for k in range(E * B) if ends[k + 1] > ends[k]]  # (expert, sample) pairs with rows

        def gradient(k):
            return A[ends[k]:ends[k + 1]].T @ G[ends[k]:ends[k + 1]]

        sq = torch.zeros(B, dtype=f64, device="cuda")
        for k in held:
            sq[k % B] += torch.linalg.vector_norm(gradient(k)).square()
        c = (s["C"] / sq.sqrt()).clamp(max=1.0)
        sums = torch.zeros(E, case["d"], case["p"], dtype=f64, device="cuda")
        for k in held:
            sums[k // B].add_(gradient(k) * c[k % B])
        return sq, c, sums / B
    x, w = s["x"].to(f64), s["w"].to(f64)
    out = torch.zeros(x.shape[0], s["out"].shape[1], dtype=f64, device="cuda")
    for e in range(E):
        i, j = ends[e * B], ends[(e + 1) * B]
        if j > i:
            out[i:j] = torch.matmul(x[i:j], w[e].T if op == "experts-forward" else w[e])
    return out
