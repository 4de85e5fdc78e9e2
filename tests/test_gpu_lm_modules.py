"""The language-model layers and the loss as a user's module calls them, and
the engine over them, where an argument, a type or an address is not the usual
one."""
from __future__ import annotations

import pytest
import torch

import lm_util as L
import sample_gradient_clipping_layer_amd as dpc
from sample_gradient_clipping_layer_amd.engine import PrivacyEngine
from sample_gradient_clipping_layer_amd.layers import ExpertLinear, RMSNorm, distillation_loss

pytestmark = pytest.mark.gpu

DT = {**L.DT, "f16": torch.float16}


def _check_gain_step(engine, m, s, dy, eps, C):
    """step() of a model that is one norm layer, from its rows s and output
    gradients dy: norms and clipped mean in 64 bits."""
    B, d = s.shape[0], s.shape[-1]
    _, rows, _, br = L.rms_backward(dy, s, None, torch.ones(d, device="cuda"), eps)
    norms = engine.step(0)
    want = rows.norm(dim=1)
    # a norm moves by the length of its rows' error at most; d products added, and a root
    bn = br.norm(dim=1) + (d + 16) * L.U * want
    L.check(norms, want, bn, "norms")
    c = torch.clamp(C / want, max=1.0)
    grad = (c[:, None] * rows).sum(0) / B
    # c is off by the norm's relative error; then the rows' own, B products added, and the gradient's type
    bound = (c[:, None] * (br + (bn / want)[:, None] * rows.abs() + (B + 16) * L.U * rows.abs())).sum(0) / B
    half = torch.finfo(m.weight.dtype).eps / 2
    L.check(m.weight.grad, grad, bound * (1 + half) + half * grad.abs() + torch.finfo(m.weight.dtype).tiny, "gradient")


@pytest.mark.parametrize("dtype,weight_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "f32")])
def test_engine_takes_torchs_default_eps(dtype, weight_dtype):
    """torch.nn.RMSNorm with eps=None over rows far below 1: torch adds
    float32's epsilon whatever the rows' type (one type for both takes torch's
    fused kernel, two do not)."""
    dt, g = DT[dtype], L.gen(17)
    B, T, d = 4, 6, 96
    x = L.randn(g, B, T, d, scale=1e-2 if dt != torch.float32 else 1e-4).to(dt).requires_grad_()
    t = L.randn(g, B, T, d, scale=0.1).to(dt)
    m = torch.nn.RMSNorm(d, dtype=DT[weight_dtype]).cuda()
    eps = torch.finfo(torch.float32).eps
    y = m(x)
    want = L.rms_forward(x.detach(), None, m.weight.detach(), eps)[0]
    assert ((y.double() - want).abs() <= (torch.finfo(dt).eps / 2 + 64 * L.U) * want.abs() + 1e-30).all()
    rows = L.rms_backward(t, x.detach(), None, m.weight.detach(), eps)[1]
    C = float(rows.norm(dim=1).median())
    engine = PrivacyEngine(m, C=C, sigma=0.0)
    (m(x) * t).sum().backward()
    _check_gain_step(engine, m, x.detach(), t, eps, C)
    engine.detach()


@pytest.mark.parametrize("weight_dtype", [torch.float16, torch.float64])
def test_engine_takes_gains_of_other_types(weight_dtype):
    """Gains of a type the library does not read: they enter it in float32."""
    g = L.gen(18)
    x = L.randn(g, 3, 5, 40).to(weight_dtype)
    t = L.randn(g, 3, 5, 40, scale=0.1).to(weight_dtype)
    m = torch.nn.RMSNorm(40, eps=1e-6, dtype=weight_dtype).cuda()
    engine = PrivacyEngine(m, C=0.3, sigma=0.0)
    (m(x) * t).sum().backward()
    _check_gain_step(engine, m, x.float(), t.float(), 1e-6, 0.3)  # fp64 rows enter in fp32 too (values of fp32 here)
    engine.detach()


# ---- contiguous views that start off a 16-byte boundary


def _off(t):
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape).copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expert_layer_over_offset_views(dtype):
    """A microbatch's slice, the gradient that torch.cat hands to a part, and
    weights of a flat buffer: the bits of the same values at an aligned start,
    with and without an engine."""
    dt, g = L.DT[dtype], L.gen(21)
    d, p = 33, 35
    seg = torch.tensor([0, 2, 5, 5, 9], device="cuda")
    w, x = L.randn(g, 2, p, d, scale=d ** -0.5, dtype=dt), L.randn(g, 9, d, dtype=dt)
    dy, head = L.randn(g, 9, p, dtype=dt), L.randn(g, 3, p, dtype=dt)
    results = []
    for place in (lambda t: t.clone(), _off):
        for with_engine in (False, True):
            m = ExpertLinear(2, d, p, device="cuda", dtype=dt)
            m.weight = torch.nn.Parameter(place(w))
            engine = PrivacyEngine(m, C=1.0, sigma=0.0) if with_engine else None
            xx = place(x).requires_grad_()
            # the part's gradient is a narrowed view of the concatenation's, 3 rows in
            out = torch.cat([head, m(xx, segments=seg)])
            out.backward(torch.cat([head, dy]) if place is _off else torch.cat([head, dy]).clone())
            norms = engine.step(0) if with_engine else torch.zeros(2)
            results.append((out.detach(), xx.grad, m.weight.grad, norms))
            if with_engine:
                engine.detach()
    for a, b in ((results[0], results[2]), (results[1], results[3])):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distillation_loss_of_a_slice(dtype):
    """Samples from the second on, of an odd number of logits each."""
    dt, g = L.DT[dtype], L.gen(22)
    B, T, V, K = 4, 3, 101, 5
    z = L.randn(g, B, T, V, scale=3.0, dtype=dt)
    ids, teacher = torch.randint(-1, V, (B, T, K), generator=g).cuda(), L.randn(g, B, T, K, dtype=dt)
    assert z[1:].data_ptr() % 16
    got = []
    for part in (z[1:], z[1:].clone()):
        part = part.detach().requires_grad_()
        loss = distillation_loss(part, ids[1:], teacher[1:], 2.0)
        loss.sum().backward()
        got.append((loss.detach(), part.grad))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    want, _, bl, _ = L.distill_forward(z[1:], ids[1:], teacher[1:], 2.0, None)
    L.check(got[0][0], want, bl, "loss")


def test_norm_over_an_offset_view():
    """RMSNorm takes rows at any element as they are."""
    g = L.gen(23)
    x, r = L.randn(g, 3, 7, 33, dtype=torch.bfloat16), L.randn(g, 3, 7, 33, dtype=torch.bfloat16)
    got = []
    for place in (lambda t: t.clone(), _off):
        m = RMSNorm(33).cuda()
        xx = place(x).requires_grad_()
        y, s = m(xx, residual=place(r))
        (y.float() * 0.5 + s.float()).sum().backward()
        got.append((y.detach(), s.detach(), xx.grad, m.weight.grad))
    for u, v in zip(*got):
        assert torch.equal(u, v)


# ---- the norm's outputs over its inputs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [96, 333, 1280, 4099, 20000])
def test_norm_outputs_over_inputs(dtype, d):
    """Every alias that the header allows: out and sum_out over x and residual
    each way round, dx over dy and over dsum."""
    dt, g = L.DT[dtype], L.gen(d)
    rows = 9
    x, r = L.randn(g, rows, d, dtype=dt), L.randn(g, rows, d, scale=2.0, dtype=dt)
    gain = 1 + L.randn(g, d, scale=0.3)
    out, s = torch.empty_like(x), torch.empty_like(x)
    dpc.dp_rms_norm(x, gain, 1e-6, out, residual=r, sum_out=s)
    for o, k in ((None, "x"), (None, "r"), ("x", None), ("r", None), ("x", "r"), ("r", "x")):
        t = {"x": x.clone(), "r": r.clone(), None: torch.empty_like(x)}
        o_t, s_t = (torch.empty_like(x) if o is None else t[o]), (torch.empty_like(x) if k is None else t[k])
        dpc.dp_rms_norm(t["x"], gain, 1e-6, o_t, residual=t["r"], sum_out=s_t)
        assert torch.equal(o_t, out) and torch.equal(s_t, s), (o, k)
        for n in {"x", "r"} - {o, k}:
            assert torch.equal(t[n], x if n == "x" else r)
    dy, dsum = L.randn(g, 3, 3, d, scale=0.1, dtype=dt), L.randn(g, 3, 3, d, scale=0.2, dtype=dt)
    s3 = s.view(3, 3, d)
    dx, gr = torch.empty_like(s3), torch.empty(3, d, device="cuda")
    dpc.dp_rms_norm_backward(dy, s3, gain, 1e-6, dx=dx, dsum=dsum, gain_rows=gr)
    for over in ("dy", "dsum"):
        t = {"dy": dy.clone(), "dsum": dsum.clone()}
        gr2 = torch.empty_like(gr)
        dpc.dp_rms_norm_backward(t["dy"], s3, gain, 1e-6, dx=t[over], dsum=t["dsum"], gain_rows=gr2)
        assert torch.equal(t[over], dx) and torch.equal(gr2, gr), over


# ---- a bf16 model's step from the operands it kept


def test_bf16_model_against_gradients_of_its_own_operands():
    """Norms and clipped gradients of every layer of a bf16 language model,
    from its layers' inputs and output gradients in 64 bits; the norms' gains
    from the sums that their forward passes gave, not from the library's rows."""
    from test_gpu_lm_engine import B, E, _data, _Model
    data = _data(6)
    model = _Model(7, dtype=torch.bfloat16).cuda()
    x, expert_ids, ids, teacher, weight = (t.cuda() for t in data)
    sums = {}
    for m in (model.norm, model.norm2):
        m.register_forward_hook(lambda m, args, out: sums.__setitem__(m, (out[1] if isinstance(out, tuple) else args[0])
                                                                      .detach().clone()))
    engine = PrivacyEngine(model, C=0.7, sigma=0.0)
    distillation_loss(model(x.bfloat16(), expert_ids), ids, teacher, 2.0, weight).sum().backward()
    names = {id(p): n for n, p in model.named_parameters()}
    per, err = {}, {}  # parameter -> per-sample gradients [B, ...] and their error bounds
    for layer in engine.layers:
        m, a, g = layer.module, layer.a.double(), layer.g.double()
        if isinstance(m, RMSNorm):
            _, rows, _, bound = L.rms_backward(layer.g, sums[m], None, m.weight.detach(), m.eps)
            per[names[id(m.weight)]], err[names[id(m.weight)]] = rows, bound
        elif isinstance(m, ExpertLinear):
            ends = layer.segments.tolist()
            full = torch.zeros(B, *m.weight.shape, dtype=torch.float64, device="cuda")
            mag = torch.zeros_like(full)
            for k in range(E * B):
                i, j = ends[k], ends[k + 1]
                full[k % B, k // B] = g[i:j].T @ a[i:j]
                mag[k % B, k // B] = g[i:j].abs().T @ a[i:j].abs()
            per[names[id(m.weight)]], err[names[id(m.weight)]] = full, 64 * L.U * mag
        else:
            gt = g.transpose(1, 2).contiguous()
            per[names[id(m.weight)]] = torch.matmul(gt, a)
            err[names[id(m.weight)]] = 64 * L.U * torch.matmul(gt.abs(), a.abs())
            if m.bias is not None:
                per[names[id(m.bias)]], err[names[id(m.bias)]] = g.sum(1), 64 * L.U * g.abs().sum(1)
    assert set(per) == set(names.values())
    want = torch.sqrt(sum((v ** 2).flatten(1).sum(1) for v in per.values()))
    # a sample's norm moves by the length of its gradients' errors at most; the ghost sums add up to d + p = 64 products
    # and 36 pairs of positions of each layer: 512 u of what they add, which the layers' magnitudes bound
    mags = torch.sqrt(sum(((err[n] / (64 * L.U)) ** 2).flatten(1).sum(1) for n in per if "norm" not in n))
    bn = torch.sqrt(sum((v ** 2).flatten(1).sum(1) for v in err.values())) + 512 * L.U * (mags ** 2 / want + want)
    norms = engine.step(0)
    L.check(norms, want, bn, "norms")
    c = torch.clamp(0.7 / want, max=1.0)
    assert (c < 1).any()
    for n, p in model.named_parameters():
        cc = c.view(B, *[1] * p.dim())
        grad = (cc * per[n]).sum(0) / B
        rel = (bn / want).view(B, *[1] * p.dim())
        bound = (cc * (err[n] + (rel + (B + 16) * L.U) * (per[n].abs() + err[n] / (64 * L.U)))).sum(0) / B
        half = L.half(p.dtype)
        L.check(p.grad, grad, (1 + half) * bound + half * grad.abs() + 1e-37, n)
    engine.detach()


# ---- norms beside convolutions


@pytest.mark.parametrize("conv_input", ["library-unfold", "folded", "unfolded"])
def test_norms_share_the_clipping_of_convolutions(conv_input):
    """A convolution (by each of its routes), a norm over its channels and a
    linear layer: one norm per sample over all three, against one backward pass
    per example in 64 bits."""
    torch.manual_seed(4)
    B, C = 4, 8

    class Net(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.conv = torch.nn.Conv2d(3, C, 3, padding=1)
            self.norm = torch.nn.RMSNorm(C)
            self.own = RMSNorm(C)
            self.head = torch.nn.Linear(C, 5)

        def forward(self, x):
            h = self.norm(self.conv(x).flatten(2).transpose(1, 2))
            if h.is_cuda:
                y, s = self.own(torch.tanh(h), h)
            else:
                s = torch.tanh(h) + h
                y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + self.own.eps) * self.own.weight
            return self.head(y + s).square().mean((1, 2))

    model = Net()
    x = torch.randn(B, 3, 6, 5)
    ref = Net().double()
    ref.load_state_dict(model.state_dict())
    ref.norm.eps = torch.finfo(torch.float32).eps
    per = []
    for i in range(B):
        per.append(torch.autograd.grad(ref(x[i:i + 1].double()).sum(), list(ref.parameters())))
    norms = torch.stack([torch.sqrt(sum((v ** 2).sum() for v in gs)) for gs in per])
    bound = float(norms.median())
    c = torch.clamp(bound / norms, max=1.0)
    model.cuda()
    engine = PrivacyEngine(model, C=bound, sigma=0.0, conv_input=conv_input)
    model(x.cuda()).sum().backward()
    got = engine.step(0)
    # fp32 through the forward and backward pass, against 64 bits: the tolerances of the engine's other tests
    assert torch.allclose(got.double().cpu(), norms, rtol=1e-4)
    for k, p in enumerate(model.parameters()):
        want = sum(c[i] * per[i][k] for i in range(B)) / B
        assert (p.grad.double().cpu() - want).abs().max() <= 1e-3 * want.abs().max() + 1e-7, k
    engine.detach()


# ---- modules in a captured graph


def test_modules_captured_and_replayed():
    """Norm, experts and loss, forward and backward, captured once and replayed
    over changed inputs and another routing: the eager bits, with eager work in
    between."""
    from sample_gradient_clipping_layer_amd.layers import route
    g = L.gen(31)
    B, T, D, H, E, V, K = 3, 5, 40, 72, 4, 61, 6
    norm, up, head = RMSNorm(D).cuda(), ExpertLinear(E, D, H, device="cuda"), L.randn(g, H, V, scale=0.2)
    params = [norm.weight, up.weight]
    teacher = L.randn(g, B, T, K)

    def fresh(seed):
        h = L.gen(seed)
        experts = torch.randint(-1, E, (B, T, 1), generator=h)
        return L.randn(h, B, T, D), L.randn(h, B, T, D), experts.cuda(), torch.randint(-1, V, (B, T, K), generator=h).cuda()

    x, r, experts, ids = fresh(0)

    def work():
        y, s = norm(x, residual=r)
        order, seg = route(experts, E)
        rows = up(y.reshape(-1, D)[order], seg)
        back = torch.empty_like(order).scatter_(0, order, torch.arange(B * T, device="cuda"))
        logits = torch.matmul(torch.tanh(rows[back]), head).view(B, T, V)
        loss = distillation_loss(logits, ids, teacher, 1.5)
        return [loss.detach(), s.detach(), *torch.autograd.grad(loss.sum() + s.square().sum() * 0.01, params)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for seed in (1, 2, 3, 0):
        for static, new in zip((x, r, experts, ids), fresh(seed)):
            static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = work()
        torch.cuda.synchronize()
        for k, (u, v) in enumerate(zip(kept, want)):
            assert torch.equal(u, v), k
