"""What the operators of private language-model training from tokens to a
per-sample loss are measured on: the cases, their inputs, the operators' plain
forms in elementary torch operations, and their values in 64 bits.

Operators and their directions (``case["op"]``):

  embed-forward     rows of a table of words, scaled; a dropped token's row is 0
  embed-clip        the table's clipping pass: the tokens sorted by word, every
                    sample's squared gradient norm, the clip factors, and the
                    clipped mean gradient of the whole table
  ln-forward        layer norm of s = x + residual, and s
  ln-backward       ds of it (the residual stream's gradient joined in), and
                    the gain's and the bias's gradient of every sample, [B, d]
  logprob-forward   log probabilities of given tokens, the distribution's
                    entropy and its top alternatives (and what the gradient
                    takes: the largest logit and the log of the sum beside it)
  logprob-backward  the gradient of the first two over the whole vocabulary
  balance-forward   a router's balance loss per sample, its rows per expert and its tokens
  balance-backward  its gradient
"""
import math

import numpy as np
import torch

own = False  # True: run() calls the library; False: the plain forms

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 8 sequences over GPT-2's vocabulary at GPT-2-large width: a launch's latency
        {"name": "embed-forward-tokens", "op": "embed-forward", "dtype": "bf16", "B": 8, "T": 1, "V": 50257, "d": 1280,
         "scale": 1.0},
        # the clipping pass of that table over a training batch
        {"name": "embed-clip-batch", "op": "embed-clip", "dtype": "bf16", "B": 32, "T": 1024, "V": 50257, "d": 1280,
         "scale": 1.0},
        # a small vocabulary of odd sizes in 32 bits, rows scaled by the root of the width
        {"name": "embed-clip-odd", "op": "embed-clip", "dtype": "f32", "B": 13, "T": 77, "V": 5003, "d": 333,
         "scale": 18.248287590894657},
        # a training batch of the GPT-2-large workload
        {"name": "ln-forward-batch", "op": "ln-forward", "dtype": "bf16", "B": 32, "T": 1024, "d": 1280},
        {"name": "ln-backward-batch", "op": "ln-backward", "dtype": "bf16", "B": 32, "T": 1024, "d": 1280},
        # an odd width and ragged row count in 32 bits
        {"name": "ln-backward-odd", "op": "ln-backward", "dtype": "f32", "B": 13, "T": 77, "d": 1001},
        # the next token of 4 sequences over GPT-2's vocabulary, with alternatives
        {"name": "logprob-forward-tokens", "op": "logprob-forward", "dtype": "bf16", "B": 4, "T": 1, "V": 50257,
         "K": 20, "tau": 0.8},
        # scoring a batch and keeping its top words, as a teacher does for distillation
        {"name": "logprob-forward-batch", "op": "logprob-forward", "dtype": "bf16", "B": 8, "T": 512, "V": 50257,
         "K": 64, "tau": 1.0},
        # the loss of a physical training batch, gradient of the logits
        {"name": "logprob-backward-batch", "op": "logprob-backward", "dtype": "bf16", "B": 8, "T": 512, "V": 50257,
         "tau": 1.0, "entropy": False},
        # the same with an entropy bonus in 32 bits, an odd vocabulary
        {"name": "logprob-backward-odd", "op": "logprob-backward", "dtype": "f32", "B": 3, "T": 101, "V": 32003,
         "tau": 1.5, "entropy": True},
        # the router of a training batch
        {"name": "balance-forward-batch", "op": "balance-forward", "dtype": "f32", "B": 32, "T": 1024, "E": 64,
         "top": 2},
        # the same direction back, more and oddly many experts
        {"name": "balance-backward-odd", "op": "balance-backward", "dtype": "bf16", "B": 9, "T": 611, "E": 130,
         "top": 6},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed-forward", "embed-clip", "ln-forward", "ln-backward", "logprob-forward", "logprob-backward",
                     "balance-forward", "balance-backward"])
    case = {"op": op, "dtype": rng.choice(["bf16", "f32"])}
    size = 2 if case["dtype"] == "bf16" else 4
    while True:
        case["B"] = _log_int(rng, 1, 128)
        case["T"] = 1 if rng.random() < 0.15 else _log_int(rng, 1, 4096)
        rows = case["B"] * case["T"]
        if op.startswith("balance"):
            case["E"] = _log_int(rng, 4, 512)
            case["top"] = rng.randint(1, min(8, case["E"] // 2))
            if rows * case["E"] * 4 <= 60e6:
                return case
        elif op.startswith("logprob"):
            case["V"] = _log_int(rng, 300, 130000)
            case["tau"] = rng.choice([0.7, 1.0, 1.0, 1.5])
            if op == "logprob-forward":
                case["K"] = rng.choice([0, 0, 1, 5, 20, 50, 64, 100])
            else:
                case["entropy"] = rng.random() < 0.4
            if rows * case["V"] * size <= 400e6:
                return case
        else:
            case["d"] = _log_int(rng, 32, 8192)
            if rng.random() < 0.6:
                case["d"] = max(8, case["d"] // 8 * 8)
            if op.startswith("embed"):
                case["V"] = _log_int(rng, 250, 130000)
                case["scale"] = rng.choice([1.0, math.sqrt(case["d"])])
            if rows * case["d"] * size <= 84e6 and (not op.startswith("embed") or case["V"] * case["d"] <= 64e6):
                return case


def _words_met(V, n):
    """How many of V words n tokens of Zipf's law name, on average."""
    k = np.arange(1, V + 1, dtype=np.float64)
    return float((1.0 - (1.0 - np.log1p(1.0 / k) / math.log(V + 1.0)) ** n).sum())


def work(case):
    B, T = case["B"], case["T"]
    size, rows = (2 if case["dtype"] == "bf16" else 4), B * T
    op = case["op"]
    if op == "embed-forward":
        return {"bytes": int(8 * rows + (rows + _words_met(case["V"], rows)) * case["d"] * size),
                "flops": rows * case["d"]}
    if op == "embed-clip":
        return {"bytes": 8 * rows + rows * case["d"] * size + 4 * case["V"] * case["d"] + 8 * B,
                "flops": 5 * rows * case["d"]}
    if op == "ln-forward":
        return {"bytes": 4 * rows * case["d"] * size + 8 * case["d"], "flops": 8 * rows * case["d"]}
    if op == "ln-backward":
        return {"bytes": 4 * rows * case["d"] * size + 4 * case["d"] + 8 * B * case["d"],
                "flops": 16 * rows * case["d"]}
    if op == "logprob-forward":
        return {"bytes": rows * case["V"] * size + rows * (8 + 8 + 12 * min(case["K"], case["V"])),
                "flops": 5 * rows * case["V"]}
    if op == "logprob-backward":
        return {"bytes": 2 * rows * case["V"] * size + rows * 28, "flops": 5 * rows * case["V"]}
    E, top = case["E"], case["top"]
    if op == "balance-forward":
        return {"bytes": rows * E * size + 8 * rows * top + 8 * B * E + 4 * B, "flops": 6 * rows * E}
    return {"bytes": 2 * rows * E * size + 8 * rows * top + 8 * B * E + 4 * B, "flops": 8 * rows * E}


def _normal(g, shape, scale, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _tokens(g, B, T, V):
    """Word ids of B ragged sequences of up to T tokens: Zipf's law, the words
    of one rank anywhere in the table; -1 behind a sequence's end."""
    u = torch.rand((B, T), generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank]
    length = torch.randint((3 * T + 3) // 4, T + 1, (B, 1), generator=g, device="cuda")
    return torch.where(torch.arange(T, device="cuda") < length, ids, torch.full_like(ids, -1))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, B, T = TYPES[case["dtype"]], case["B"], case["T"]
    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("embed"):
        V, d = case["V"], case["d"]
        s["ids"] = _tokens(g, B, T, V)
        if op == "embed-forward":
            s["weight"] = _normal(g, (V, d), 0.02, dt)
            s["out"] = torch.empty(B, T, d, device="cuda", dtype=dt)
            return s
        # tokens' gradients of uneven size
        size = torch.exp(_normal(g, (B, T, 1), 0.5, torch.float32))
        s["G"] = (_normal(g, (B, T, d), d ** -0.5, torch.float32) * size).to(dt)
        s["C"] = case["scale"] * 1.3 * math.sqrt(T)  # about half of the samples clip
        s["sq"], s["c"] = (torch.empty(B, device="cuda", dtype=torch.float32) for _ in range(2))
        s["out"] = torch.empty(V, d, device="cuda", dtype=torch.float32)
        if own:
            s["order"] = torch.empty(B * T, device="cuda", dtype=torch.int64)
            s["starts"] = torch.empty(V + 1, device="cuda", dtype=torch.int64)
            lib = _library()
            s["ws"] = _scratch(max(lib.dp_embedding_order_workspace_bytes(B * T, V),
                                   lib.dp_embedding_workspace_bytes(_code(dt), B, T, V, d)))
    elif op.startswith("ln"):
        d = case["d"]
        s["gain"], s["bias"] = 1.0 + _normal(g, (d,), 0.2, torch.float32), _normal(g, (d,), 0.1, torch.float32)
        # rows of uneven size and mean, as a residual stream has them
        size = torch.exp(_normal(g, (B, T, 1), 0.5, torch.float32))
        x = ((_normal(g, (B, T, d), 1.0, torch.float32) + _normal(g, (B, T, 1), 0.5, torch.float32)) * size).to(dt)
        s["out"] = torch.empty(B, T, d, device="cuda", dtype=dt)
        if op == "ln-forward":
            s["x"], s["residual"] = x, (_normal(g, (B, T, d), 1.0, torch.float32) * size).to(dt)
            s["sum"] = torch.empty_like(x)
        else:
            s["s"], s["dy"], s["dsum"] = x, _normal(g, (B, T, d), 0.02, dt), _normal(g, (B, T, d), 0.02, dt)
            s["gain_rows"], s["bias_rows"] = (torch.empty(B, d, device="cuda", dtype=torch.float32) for _ in range(2))
            if own:
                s["ws"] = _scratch(_library().dp_layer_norm_workspace_bytes(_code(dt), B, T, d))
    elif op.startswith("logprob"):
        V, tau = case["V"], case["tau"]
        s["logits"] = _normal(g, (B, T, V), 2.5, dt)
        s["targets"] = _tokens(g, B, T, V)
        if op == "logprob-forward":
            K = min(case["K"], V)
            s["logp"], s["entropy"] = (torch.empty(B, T, device="cuda", dtype=torch.float32) for _ in range(2))
            s["stats"] = torch.empty(B, T, 2, device="cuda", dtype=torch.float32)
            s["top_ids"] = torch.empty(B, T, K, device="cuda", dtype=torch.int64) if K else None
            s["top_logp"] = torch.empty(B, T, K, device="cuda", dtype=torch.float32) if K else None
        else:
            z = s["logits"].double() / tau
            top = z.amax(-1)
            lse = torch.logsumexp(z - top[..., None], dim=-1)
            # a forward pass's own: the largest logit and the logarithm of the sum beside it
            s["stats"] = torch.stack([s["logits"].float().amax(-1), lse.float()], dim=-1)
            z = z.sub_((top + lse)[..., None])
            s["entropy"] = -(torch.exp(z) * z).sum(-1).float()
            del z
            s["dlogp"] = -(0.5 + torch.rand((B, T), generator=g, device="cuda"))
            s["dentropy"] = _normal(g, (B, T), 0.1, torch.float32) if case["entropy"] else None
            s["grad"] = torch.empty_like(s["logits"])
    else:
        E, top = case["E"], case["top"]
        # some experts are more popular
        s["logits"] = (_normal(g, (B, T, E), 1.0, torch.float32) + _normal(g, (E,), 0.7, torch.float32)).to(dt)
        ids = torch.topk(s["logits"].float() + _normal(g, (B, T, E), 1e-3, torch.float32), top, dim=-1)[1]
        length = torch.randint((3 * T + 3) // 4, T + 1, (B, 1, 1), generator=g, device="cuda")
        used = torch.arange(T, device="cuda")[:, None] < length
        s["ids"] = torch.where(used, ids, torch.full_like(ids, -1))
        s["loss"] = torch.empty(B, device="cuda", dtype=torch.float32)
        if op == "balance-forward":
            s["counts"] = torch.empty(B, E, device="cuda", dtype=torch.int64)
            s["tokens"] = torch.empty(B, device="cuda", dtype=torch.int64)
            if own:
                s["ws"] = _scratch(_library().dp_balance_workspace_bytes(_code(dt), B, T, E))
        else:
            s["counts"] = torch.zeros(B, E + 1, device="cuda", dtype=torch.int64).scatter_add_(
                1, torch.where(used, ids, torch.full_like(ids, E)).view(B, -1),
                torch.ones(B, T * top, device="cuda", dtype=torch.int64))[:, :E].contiguous()
            s["tokens"] = used[..., 0].sum(1)
            s["dloss"] = 0.01 * (0.5 + torch.rand(B, generator=g, device="cuda"))
            s["grad"] = torch.empty_like(s["logits"])
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
    if op == "embed-forward":
        dpc.dp_embedding(s["ids"], s["weight"], s["out"], scale=case["scale"])
        return s["out"]
    if op == "embed-clip":
        dpc.dp_embedding_order(s["ids"], case["V"], s["order"], s["starts"], workspace=s["ws"])
        dpc.dp_embedding_norm(s["G"], s["ids"], s["order"], s["starts"], s["sq"], scale=case["scale"],
                              workspace=s["ws"])
        dpc.dp_clip_factors(s["sq"], s["C"], s["c"])
        dpc.dp_embedding_clipped_sum_noise(s["G"], s["ids"], s["order"], s["starts"], s["c"], s["C"], 0.0,
                                           float(case["B"]), 0, 0, 0, s["out"], scale=case["scale"], workspace=s["ws"])
        return s["sq"], s["c"], s["out"]
    if op == "ln-forward":
        dpc.dp_layer_norm(s["x"], s["gain"], s["bias"], EPS, s["out"], residual=s["residual"], sum_out=s["sum"])
        return s["out"], s["sum"]
    if op == "ln-backward":
        dpc.dp_layer_norm_backward(s["dy"], s["s"], s["gain"], EPS, dx=s["out"], dsum=s["dsum"],
                                   gain_rows=s["gain_rows"], bias_rows=s["bias_rows"], workspace=s["ws"])
        return s["out"], s["gain_rows"], s["bias_rows"]
    if op == "logprob-forward":
        dpc.dp_token_logprob(s["logits"], s["targets"], case["tau"], s["logp"], s["stats"], entropy=s["entropy"],
                             top_ids=s["top_ids"], top_logp=s["top_logp"])
        made = (s["logp"], s["entropy"], s["stats"])
        return made if s["top_ids"] is None else made + (s["top_ids"], s["top_logp"])
    if op == "logprob-backward":
        dpc.dp_token_logprob_backward(s["logits"], s["targets"], case["tau"], s["stats"], s["grad"], dlogp=s["dlogp"],
                                      entropy=s["entropy"], dentropy=s["dentropy"])
        return s["grad"]
    if op == "balance-forward":
        dpc.dp_balance_loss(s["logits"], s["ids"], s["loss"], s["counts"], s["tokens"], workspace=s["ws"])
        return s["loss"], s["counts"], s["tokens"]
    dpc.dp_balance_loss_backward(s["logits"], s["ids"], s["counts"], s["tokens"], s["grad"], dloss=s["dloss"])
    return s["grad"]


def _run_plain(s):
    case = s["case"]
    op, B, T = case["op"], case["B"], case["T"]
    if op == "embed-forward":
        ids = s["ids"]
        rows = s["weight"][ids.clamp(min=0)].float() * case["scale"]
        return torch.where((ids >= 0)[..., None], rows, torch.zeros_like(rows)).to(s["weight"].dtype)
    if op == "embed-clip":
        V, d = case["V"], case["d"]
        G = s["G"].float().view(B * T, d) * case["scale"]
        sample = torch.arange(B, device="cuda").repeat_interleave(T)
        key = torch.where(s["ids"] >= 0, s["ids"] + V * torch.arange(B, device="cuda")[:, None],
                          torch.full_like(s["ids"], B * V)).view(-1)
        pairs, of = torch.unique(key, return_inverse=True)
        sums = torch.zeros(pairs.numel(), d, device="cuda").index_add_(0, of, G)
        each = torch.where(pairs < B * V, (sums * sums).sum(1), torch.zeros(pairs.numel(), device="cuda"))
        sq = torch.zeros(B + 1, device="cuda").index_add_(0, pairs // V, each)[:B]
        norm = torch.sqrt(sq)
        c = torch.where(norm > s["C"], s["C"] / norm, torch.ones_like(norm))
        word = torch.where(s["ids"] >= 0, s["ids"], torch.full_like(s["ids"], V)).view(-1)
        out = torch.zeros(V + 1, d, device="cuda").index_add_(0, word, G * c[sample][:, None])
        return sq, c, out[:V] / float(B)
    if op == "ln-forward":
        v = s["x"].float() + s["residual"].float()
        off = v - v.mean(-1, keepdim=True)
        y = off * torch.rsqrt((off * off).mean(-1, keepdim=True) + EPS) * s["gain"] + s["bias"]
        return y.to(s["x"].dtype), v.to(s["x"].dtype)
    if op == "ln-backward":
        v, dy = s["s"].float(), s["dy"].float()
        off = v - v.mean(-1, keepdim=True)
        rstd = torch.rsqrt((off * off).mean(-1, keepdim=True) + EPS)
        unit, h = off * rstd, dy * s["gain"]
        dx = s["dsum"].float() + rstd * (h - h.mean(-1, keepdim=True) - unit * (h * unit).mean(-1, keepdim=True))
        return dx.to(s["s"].dtype), (dy * unit).sum(1), dy.sum(1)
    if op == "logprob-forward":
        z = s["logits"].float()
        top = z.amax(-1, keepdim=True)
        x = (z - top) / case["tau"]
        e = torch.exp(x)
        total = e.sum(-1, keepdim=True)
        entropy = torch.log(total).squeeze(-1) - (e * x).sum(-1) / total.squeeze(-1)
        del e
        at = s["targets"]
        logp = torch.gather(x, -1, at.clamp(min=0)[..., None]) - torch.log(total)
        logp = torch.where(at >= 0, logp.squeeze(-1), torch.zeros_like(entropy))
        stats = torch.cat([top, torch.log(total)], dim=-1)
        K = min(case["K"], case["V"])
        if not K:
            return logp, entropy, stats
        # the largest first, of equal ones the lowest word first
        words = torch.sort(z, dim=-1, descending=True, stable=True)[1][..., :K].contiguous()
        return logp, entropy, stats, words, torch.gather(x, -1, words) - torch.log(total)
    if op == "logprob-backward":
        log_p = (s["logits"].float() - s["stats"][..., :1]) / case["tau"] - s["stats"][..., 1:]
        p = torch.exp(log_p)
        dl = torch.where(s["targets"] >= 0, s["dlogp"], torch.zeros_like(s["dlogp"]))[..., None]
        g = -dl * p
        if s["dentropy"] is not None:
            g = g - s["dentropy"][..., None] * p * (log_p + s["entropy"][..., None])
        g.scatter_add_(-1, s["targets"].clamp(min=0)[..., None], dl)
        return (g / case["tau"]).to(s["logits"].dtype)
    E = case["E"]
    z = s["logits"].float()
    e = torch.exp(z - z.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    used = (s["ids"] >= 0).any(-1)
    tokens = used.float().sum(1, keepdim=True)
    if op == "balance-forward":
        place = torch.where(s["ids"] >= 0, s["ids"], torch.full_like(s["ids"], E)).view(B, -1)
        counts = torch.zeros(B, E + 1, dtype=torch.int64, device="cuda")
        counts = counts.scatter_add_(1, place, torch.ones_like(place))[:, :E]
        mean = (p * used[..., None]).sum(1) / tokens
        share = counts.float() / counts.sum(1, keepdim=True).float()
        return E * (share * mean).sum(1), counts, used.sum(1)
    # a share more for all experts changes nothing: where they are nearly even only the differences are left
    above = s["counts"] - s["counts"].amin(1, keepdim=True)
    share = above.float() / s["counts"].sum(1, keepdim=True).float()
    a = (E * s["dloss"][:, None] * share / tokens)[:, None, :]
    g = p * (a - (p * a).sum(-1, keepdim=True))
    return (g * used[..., None]).to(s["logits"].dtype)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, B, T = case["op"], case["B"], case["T"]
    f64 = torch.float64
    if op == "embed-forward":
        table = torch.cat([s["weight"].to(f64) * case["scale"], torch.zeros(1, case["d"], dtype=f64, device="cuda")])
        return table.index_select(0, s["ids"].view(-1)
                                  .where(s["ids"].view(-1) >= 0, torch.tensor(case["V"], device="cuda"))
                                  ).view(B, T, case["d"])
    if op == "embed-clip":
        V, d = case["V"], case["d"]
        G = s["G"].to(f64).view(B, T, d) * case["scale"]

        def runs(keys, rows):
            """(the different keys, the sums of their rows): running sums of the sorted rows, differences at the ends."""
            keys, order = torch.sort(keys, stable=True)
            run = torch.cumsum(rows[order], 0)
            last = torch.cat([keys[1:] != keys[:-1], torch.ones(1, dtype=torch.bool, device="cuda")])
            total = run[last]
            return keys[last], torch.cat([total[:1], total[1:] - total[:-1]])

        sq = torch.zeros(B, dtype=f64, device="cuda")
        for b in range(B):
            words, sums = runs(s["ids"][b], G[b])
            sq[b] = torch.linalg.vector_norm(sums[words >= 0]).square()
        c = (s["C"] / sq.sqrt()).clamp(max=1.0)
        words, sums = runs(s["ids"].view(-1), (G * c[:, None, None]).view(B * T, d))
        out = torch.zeros(V, d, dtype=f64, device="cuda")
        out[words[words >= 0]] = sums[words >= 0]
        return sq, c, out / B
    if op == "ln-forward":
        v = s["x"].to(f64).add(s["residual"].to(f64))
        var, mean = torch.var_mean(v, dim=-1, correction=0, keepdim=True)
        return (v - mean) / (var + EPS).sqrt() * s["gain"].to(f64) + s["bias"].to(f64), v
    if op == "ln-backward":
        # the Jacobian's action: d((s - mean)/r)/ds = (I - 1 1^T / d - o o^T / (d r^2)) / r, o = s - mean
        v, dy, d = s["s"].to(f64), s["dy"].to(f64), case["d"]
        var, mean = torch.var_mean(v, dim=-1, correction=0, keepdim=True)
        r, o = (var + EPS).sqrt(), v - mean
        h = dy * s["gain"].to(f64)
        along = torch.matmul(h[..., None, :], o[..., None])[..., 0] / (d * r * r)
        dx = (h - h.sum(-1, keepdim=True) / d - along * o) / r + s["dsum"].to(f64)
        return dx, (dy * o / r).sum(1), dy.sum(1)
    if op.startswith("logprob"):
        tau, at = case["tau"], s["targets"]
        logp = torch.log_softmax(s["logits"].to(f64) / tau, dim=-1)
        if op == "logprob-forward":
            p = torch.exp(logp)
            entropy = -torch.special.xlogy(p, p).sum(-1)
            del p
            here = torch.gather(logp, -1, at.clamp(min=0)[..., None]).squeeze(-1) * (at >= 0)
            top = s["logits"].to(f64).amax(-1)
            stats = torch.stack([top, torch.logsumexp((s["logits"].to(f64) - top[..., None]) / tau, dim=-1)], dim=-1)
            K = min(case["K"], case["V"])
            if not K:
                return here, entropy, stats
            # the whole numbers of (value, word) in one order: words of equal value ascending
            _, rank = torch.unique(s["logits"], return_inverse=True)
            best = torch.topk(rank * case["V"] + (case["V"] - 1 - torch.arange(case["V"], device="cuda")), K, dim=-1)[0]
            words = case["V"] - 1 - best % case["V"]
            return here, entropy, stats, words, torch.gather(logp, -1, words)
        p = torch.exp(logp)
        dl = (s["dlogp"].to(f64) * (at >= 0))[..., None]
        g = torch.zeros_like(p).scatter_(-1, at.clamp(min=0)[..., None], dl).sub_(dl * p)
        if s["dentropy"] is not None:
            entropy = -torch.special.xlogy(p, p).sum(-1, keepdim=True)
            g.sub_(s["dentropy"].to(f64)[..., None] * p * (logp + entropy))
        return g / tau
    E = case["E"]
    p = torch.softmax(s["logits"].to(f64), dim=-1)
    used = (s["ids"] >= 0).any(-1)
    place = torch.where(s["ids"] >= 0, s["ids"], torch.full_like(s["ids"], E)).view(B, -1)
    counts = torch.stack([torch.bincount(place[b], minlength=E + 1)[:E] for b in range(B)])
    rows = counts.sum(1, keepdim=True)
    if op == "balance-forward":
        share = counts.to(f64) / rows
        loss = [E * torch.dot(share[b], p[b][used[b]].mean(0)) for b in range(B)]
        return torch.stack(loss), counts, torch.tensor([used[b].nonzero().numel() for b in range(B)], device="cuda")
    # differences to the rarest expert: the gradient does not change with a share that all experts have more
    a = (counts - counts.amin(1, keepdim=True)).to(f64) / rows * (E * s["dloss"].to(f64) / used.sum(1))[:, None]
    inner = torch.matmul(p, a[..., None])
    return p * (a[:, None, :] - inner) * used[..., None]
