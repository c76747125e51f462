"""The pieces of a linear-attention layer together, as a model uses them: the gated norm before the block,
linear attention over a prompt and then token by token, the heads' gated output norm, and the norm between
two blocks; and a training step's gradients through all of them, against autograd in 64 bits."""
import pytest
import torch

import _linear as ref
from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu

T, H_QK, H, D, HIDDEN = 150, 2, 4, 128, 512
EPS = 1e-6


def make(dtype):
    g = torch.Generator().manual_seed(0)
    r = lambda *s, std=1.0: std * torch.randn(s, generator=g)  # noqa: E731
    p = {"wq": r(HIDDEN, H_QK * D, std=HIDDEN ** -0.5), "wk": r(HIDDEN, H_QK * D, std=HIDDEN ** -0.5),
         "wv": r(HIDDEN, H * D, std=HIDDEN ** -0.5), "wz": r(HIDDEN, H * D, std=HIDDEN ** -0.5),
         "wo": r(H * D, HIDDEN, std=(H * D) ** -0.5)}
    norms = {"before": 1 + 0.1 * r(HIDDEN), "heads": 1 + 0.1 * r(D), "behind": 1 + 0.1 * r(HIDDEN), "next": 1 + 0.1 * r(HIDDEN)}
    return ({n: w.to(dtype) for n, w in p.items()}, norms, r(T, HIDDEN).to(dtype), r(T, HIDDEN).to(dtype), r(T, HIDDEN).to(dtype))


def decays():
    return -0.5 * torch.exp2(-2.0 * torch.arange(H))


def layer(p, norms, x, decay, norm_gate, attend):
    """The residual stream and its norm behind one layer (what the next block reads)."""
    h, _ = norm_gate(x, norms["before"])
    q, k, v, z = (h @ p[n] for n in ("wq", "wk", "wv", "wz"))
    rows = x.shape[0]
    o = attend(q.view(rows, H_QK, D) / D ** 0.25, k.view(rows, H_QK, D) / D ** 0.25, v.view(rows, H, D))
    y, _ = norm_gate(o, norms["heads"], gate=z.view(rows, H, D))
    return norm_gate((y.reshape(rows, H * D)) @ p["wo"], norms["behind"], residual=x, next_weight=norms["next"], scale=0.5)


def plain_norm(x, weight, gate=None, residual=None, next_weight=None, scale=1.0):
    return ref.norm_gate(x, weight, gate, residual, next_weight, scale, EPS, "silu")


def plain_attend(q, k, v):
    g, n = decays().double(), torch.arange(q.shape[0], dtype=torch.float64)
    apart = n[:, None] - n
    mask = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0)
    q, k = (t.repeat_interleave(H // H_QK, 1).transpose(0, 1) for t in (q, k))
    return (((q @ k.transpose(1, 2)) * mask) @ v.transpose(0, 1)).transpose(0, 1)


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, gate, residual, next_weight, scale):
        ctx.save_for_backward(x, weight, gate, residual, next_weight)
        ctx.scale = scale
        return gdr.gdr_norm_gate(x, weight, gate, residual, next_weight, scale=scale, eps=EPS)

    @staticmethod
    def backward(ctx, dy, dn):
        x, weight, gate, residual, next_weight = ctx.saved_tensors
        dn = dn.contiguous() if next_weight is not None else None
        return (*gdr.gdr_norm_gate_backward(x, dy.contiguous(), dn, weight, gate, residual, next_weight, scale=ctx.scale,
                                            eps=EPS), None)


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay):
        ctx.save_for_backward(q, k, v, decay)
        return gdr.gdr_linear_prefill(q, k, v, decay, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, decay = ctx.saved_tensors
        return (*gdr.gdr_linear_backward(q, k, v, decay, d_o=d_o.contiguous(), want_d_initial_state=False)[:3], None)


def own_norm(x, weight, gate=None, residual=None, next_weight=None, scale=1.0):
    return Norm.apply(x.contiguous(), weight, None if gate is None else gate.contiguous(), residual, next_weight, scale)


def relative(a, b):
    return float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())


def run(dtype):
    p, norms, x, dy, dn = make(dtype)
    want_in = {**{n: w.double().requires_grad_() for n, w in {**p, **norms}.items()}, "x": x.double().requires_grad_()}
    y, n = layer(want_in, want_in, want_in["x"], decays(), plain_norm, plain_attend)
    want = torch.autograd.grad((y * dy.double()).sum() + (n * dn.double()).sum(), list(want_in.values()))
    own_in = {m: w.detach().cuda().requires_grad_() for m, w in {**p, **norms, "x": x}.items()}
    decay = decays().cuda()
    oy, on = layer(own_in, own_in, own_in["x"], decay, own_norm,
                   lambda q, k, v: Attend.apply(q.contiguous(), k.contiguous(), v.contiguous(), decay))
    got = torch.autograd.grad((oy.float() * dy.cuda().float()).sum() + (on.float() * dn.cuda().float()).sum(), list(own_in.values()))
    return relative(oy, y), relative(on, n), {m: relative(a, b) for m, a, b in zip(want_in, got, want)}


def test_training_step_single_precision():
    """fp32 throughout: about forty roundings and sums in sequence, each at most 2^-24 sqrt(512) in the
    2-norm (the products' accumulation), amplified by the norms' gradients at most ten times: 6e-4."""
    ey, en, grads = run(torch.float32)
    assert ey <= 6e-5 and en <= 6e-5
    assert max(grads.values()) <= 6e-4, grads


def test_training_step_bf16():
    """bf16 tensors between the operators: each of the twenty on the longest path through the layer and
    back is rounded by at most 2^-8 in the 2-norm, the scores' and the state's copy included: 20 * 2^-8."""
    ey, en, grads = run(torch.bfloat16)
    assert ey <= 20 * 2.0 ** -8 and en <= 20 * 2.0 ** -8
    assert max(grads.values()) <= 20 * 2.0 ** -8, grads


def test_serving_prompt_then_tokens():
    """A prompt and then single tokens give the layer's outputs over the whole text."""
    p, norms, x, _, _ = make(torch.bfloat16)
    p, norms, x, decay = ({n: w.cuda() for n, w in p.items()}, {n: w.cuda() for n, w in norms.items()}, x.cuda(), decays().cuda())
    norm = lambda t, weight, **kw: gdr.gdr_norm_gate(t, weight, eps=EPS, **kw)  # noqa: E731
    state = {}

    def prompt(q, k, v):
        o, state["S"] = gdr.gdr_linear_prefill(q.contiguous(), k.contiguous(), v.contiguous(), decay)
        return o

    def step(q, k, v):
        return gdr.gdr_linear_decode(q.contiguous(), k.contiguous(), v.contiguous(), decay, state["S"])

    whole, _ = layer(p, norms, x, decay, norm, prompt)
    end = state["S"]
    first, _ = layer(p, norms, x[:140].contiguous(), decay, norm, prompt)
    rest = [layer(p, norms, x[t:t + 1].contiguous(), decay, norm, step)[0] for t in range(140, T)]
    both = torch.cat([first] + rest)
    assert float((both.double() - whole.double()).norm() / whole.double().norm()) <= 6 * 2.0 ** -8
    # the same tokens through other tiles of the same products: q, k, v may round the other way (2^-8)
    assert float((state["S"] - end).double().norm() / end.double().norm()) <= 2 * 2.0 ** -8


def test_prologue_feeds_linear_attention():
    """The library's own prologue (convolution, SiLU, norms) in front, at the shapes it hands on."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    xq, xk, xv = (r(100, 2, 128).to(torch.bfloat16).cuda() for _ in range(3))
    taps = [0.5 * r(256, 4).cuda() for _ in range(3)]
    q, k, v, _, _ = gdr.gdr_prologue(xq, xk, xv, *taps, r(100, 2).cuda(), torch.full((2,), 0.05).cuda(), r(100, 2).cuda(), silu=True)
    decay = torch.tensor([-0.3, -0.01])
    o, s = gdr.gdr_linear_prefill(q, k, v, decay.cuda())
    want = ref.prefill(q, k, v, decay, None, None, 1, True)
    ref.check("o", o, want[0], want[1])
    ref.check("state", s, want[2], want[3])
    y, _ = gdr.gdr_norm_gate(o, torch.ones(128).cuda(), gate=xv)
    n, _ = ref.norm_gate(o.double().cpu(), torch.ones(128).double(), xv.double().cpu(), None, None, 1.0, EPS, "silu")
    assert relative(y, n) <= 2.0 ** -8 + 1e-5
