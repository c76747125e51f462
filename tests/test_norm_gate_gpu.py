"""The gated norm and its gradient on the GPU against their definitions in 64 bits."""
import itertools

import pytest
import torch

import _linear as ref
from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu

EPS = 1e-6
DIMS = [8, 16, 24, 64, 128, 136, 512, 1000, 2048, 4096, 4104, 8192, 16384]


def make(rows, dim, dtype, parts, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = {"x": r(rows, dim).to(dtype), "weight": 1 + 0.3 * r(dim), "gate": (2 * r(rows, dim)).to(dtype),
         "residual": r(rows, dim).to(dtype), "next_weight": 1 + 0.3 * r(dim), "dy": r(rows, dim).to(dtype),
         "dn": r(rows, dim).to(dtype)}
    return {n: v if n in parts or n == "x" else None for n, v in t.items()}


def gpu(t):
    return {n: None if v is None else v.cuda() for n, v in t.items()}


def relative(got, want):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def step(dtype):
    """Relative 2-norm a result in this type may be off: half a step at its rounding, and what fp32 gives.
    A row's fp32 sums of d products and the dozen operations behind them stay below 2^-24 (sqrt(d) + 32)
    in the 2-norm, d <= 16384: 1e-5."""
    return (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) + 1e-5


FULL = ("weight", "gate", "residual", "next_weight")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows", [1, 5, 67])
def test_forward_sizes(rows, dim, dtype):
    c = make(rows, dim, dtype, FULL)
    y, n = gdr.gdr_norm_gate(*(gpu(c)[k] for k in ("x",) + FULL), scale=0.5, eps=EPS)
    want = ref.norm_gate(*(c[k].double() for k in ("x",) + FULL), 0.5, EPS, "silu")
    assert relative(y, want[0]) <= step(dtype) and relative(n, want[1]) <= step(dtype)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("parts", [p for k in range(5) for p in itertools.combinations(FULL, k)],
                         ids=lambda p: "+".join(p) or "plain")
def test_parts(parts, act):
    """Every combination of what may be left out, forward and backward, with dy and dn given or not."""
    for rows, dim, dtype in ((37, 128, torch.bfloat16), (19, 264, torch.float32)):
        c = make(rows, dim, dtype, parts + ("dy", "dn"), seed=1)
        d = gpu(c)
        y, n = gdr.gdr_norm_gate(*(d[k] for k in ("x",) + FULL), scale=-0.75, eps=EPS, activation=act)
        leaves = {k: None if c[k] is None else c[k].double().requires_grad_() for k in ("x",) + FULL}
        want = ref.norm_gate(*leaves.values(), -0.75, EPS, act)
        assert relative(y, want[0].detach()) <= step(dtype)
        assert (n is None) == ("next_weight" not in parts)
        if n is not None:
            assert relative(n, want[1].detach()) <= step(dtype)
        for dy, dn in ((True, False), (False, True), (True, True)):
            if dn and "next_weight" not in parts:
                continue
            loss = (want[0] * c["dy"].double()).sum() if dy else 0
            if dn:
                loss = loss + (want[1] * c["dn"].double()).sum()
            names = [k for k in leaves if leaves[k] is not None and (k != "next_weight" or dn)]
            grads = dict(zip(names, torch.autograd.grad(loss, [leaves[k] for k in names], retain_graph=True)))
            got = gdr.gdr_norm_gate_backward(d["x"], d["dy"] if dy else None, d["dn"] if dn else None,
                                             *(d[k] for k in FULL), scale=-0.75, eps=EPS, activation=act)
            for k, r in zip(("x", "weight", "gate", "residual", "next_weight"), got):
                assert (r is None) == (k not in grads), k
                if r is not None:
                    # a gradient is a difference of terms: its fp32 error is relative to them, up to ten times its size
                    tol = step(r.dtype) if r.dtype == torch.bfloat16 else 1e-5
                    assert relative(r, grads[k]) <= tol, (k, dy, dn)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 16384), (9, 8192), (600, 4096), (1237, 1000), (5003, 128), (40000, 16), (2, 4104)])
def test_backward_sizes(rows, dim, dtype):
    c = make(rows, dim, dtype, FULL + ("dy", "dn"), seed=2)
    d = gpu(c)
    got = gdr.gdr_norm_gate_backward(d["x"], d["dy"], d["dn"], *(d[k] for k in FULL), scale=0.5, eps=EPS,
                                     activation="sigmoid")
    again = gdr.gdr_norm_gate_backward(d["x"], d["dy"], d["dn"], *(d[k] for k in FULL), scale=0.5, eps=EPS,
                                       activation="sigmoid")
    leaves = [c[k].double().requires_grad_() for k in ("x",) + FULL]
    y, n = ref.norm_gate(*leaves, 0.5, EPS, "sigmoid")
    want = torch.autograd.grad((y * c["dy"].double()).sum() + (n * c["dn"].double()).sum(), leaves)
    for k, r, a, w in zip(("dx", "dweight", "dgate", "dresidual", "dnext_weight"), got, again, want):
        assert relative(r, w) <= (step(dtype) if r.dtype == torch.bfloat16 else 1e-5), k
        assert torch.equal(r, a), k


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_gradient_against_differences(act):
    """Along random directions of every input, against central differences of the 64-bit definition."""
    c = make(13, 72, torch.float32, FULL + ("dy", "dn"), seed=5)
    d = gpu(c)
    got = gdr.gdr_norm_gate_backward(d["x"], d["dy"], d["dn"], *(d[k] for k in FULL), scale=0.5, eps=EPS, activation=act)
    g = torch.Generator().manual_seed(6)

    def loss(**over):
        a = {k: over.get(k, c[k].double()) for k in ("x",) + FULL}
        y, n = ref.norm_gate(*a.values(), 0.5, EPS, act)
        return float((y * c["dy"].double()).sum() + (n * c["dn"].double()).sum())

    for k, r in zip(("x",) + FULL, got):
        way, h = torch.randn(c[k].shape, generator=g).double(), 1e-4
        diff = (loss(**{k: c[k].double() + h * way}) - loss(**{k: c[k].double() - h * way})) / (2 * h)
        along = (r.double().cpu() * way)
        # the difference's own error is h^2 times a third derivative of order one; fp32 gradients 1e-5
        assert abs(float(along.sum()) - diff) <= 1e-5 * float(along.abs().sum()), k


def test_extreme_rows():
    """A row of zeros, huge and tiny rows, and gates far out: finite, and as the definition."""
    x = torch.zeros(6, 128)
    x[1], x[2], x[3] = 1e18, 1e-18, torch.linspace(-1, 1, 128)
    x[4:] = torch.randn(2, 128, generator=torch.Generator().manual_seed(0))
    gate = torch.zeros(6, 128)
    gate[3], gate[4], gate[5] = -80.0, 80.0, -1e4
    w = torch.ones(128)
    y, _ = gdr.gdr_norm_gate(x.cuda(), w.cuda(), gate.cuda(), eps=EPS)
    want, _ = ref.norm_gate(x.double(), w.double(), gate.double(), None, None, 1.0, EPS, "silu")
    assert torch.isfinite(y).all()
    # a gate at -80 and below gives a denormal or zero, which is 0 to the next norm
    assert (y.double().cpu() - want).abs().max() <= 1e-5 * want.abs().max()
    got = gdr.gdr_norm_gate_backward(x.cuda(), torch.ones(6, 128).cuda(), None, w.cuda(), gate.cuda(), eps=EPS)
    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_rows_stay_apart():
    c = gpu(make(50, 264, torch.bfloat16, FULL, seed=3))
    y, n = gdr.gdr_norm_gate(*(c[k] for k in ("x",) + FULL))
    c["x"][7], c["gate"][21], c["residual"][33] = float("nan"), float("inf"), float("-inf")
    y2, n2 = gdr.gdr_norm_gate(*(c[k] for k in ("x",) + FULL))
    keep = [r for r in range(50) if r not in (7, 21, 33)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(n[keep], n2[keep])


def test_residual_in_place_stream_and_graph():
    c = gpu(make(300, 1000, torch.bfloat16, FULL + ("dy", "dn"), seed=4))
    args = [c[k] for k in FULL]
    y, n = gdr.gdr_norm_gate(c["x"], *args, scale=0.5)
    res = c["residual"].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, n2 = gdr.gdr_norm_gate(c["x"], c["weight"], c["gate"], res, c["next_weight"], scale=0.5, y=res, stream=s)
    torch.cuda.synchronize()
    assert y2 is res and torch.equal(y, y2) and torch.equal(n, n2)
    want = gdr.gdr_norm_gate_backward(c["x"], c["dy"], c["dn"], *args)
    x = torch.zeros_like(c["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdr.gdr_norm_gate_backward(x, c["dy"], c["dn"], *args)
    x.copy_(c["x"])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows():
    c = gpu(make(0, 128, torch.bfloat16, FULL + ("dy", "dn")))
    y, n = gdr.gdr_norm_gate(*(c[k] for k in ("x",) + FULL))
    assert y.shape == n.shape == (0, 128)
    got = gdr.gdr_norm_gate_backward(c["x"], c["dy"], c["dn"], *(c[k] for k in FULL))
    assert (got[1] == 0).all() and (got[4] == 0).all() and got[0].shape == (0, 128)


@pytest.mark.parametrize("second", [True, False], ids=["next", "alone"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(700, 8192), (1500, 4096), (4001, 2048), (50000, 128)])
def test_blocks_of_many_rows(rows, dim, dtype, second):
    """Four row groups and more for each block, so that every place of its ring is used again."""
    parts = FULL if second else FULL[:2]
    c = make(rows, dim, dtype, parts + ("dy", "dn"), seed=7)
    d = gpu(c)
    arg = {k: d[k] for k in parts}
    out = gdr.gdr_norm_gate(d["x"], **arg, scale=0.5, eps=EPS)
    got = gdr.gdr_norm_gate_backward(d["x"], d["dy"], d["dn"] if second else None, **arg, scale=0.5, eps=EPS)
    leaves = {k: d[k].double().requires_grad_() for k in ("x",) + parts}
    y, n = ref.norm_gate(leaves["x"], *(leaves.get(k) for k in FULL), 0.5, EPS, "silu")
    loss = (y * d["dy"].double()).sum() + ((n * d["dn"].double()).sum() if second else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    tol = step(dtype) if dtype == torch.bfloat16 else 1e-5
    assert relative(out[0], y.detach().cpu()) <= tol
    assert not second or relative(out[1], n.detach().cpu()) <= tol
    for k, r in zip(("x", "weight", "gate", "residual", "next_weight"), got):
        assert (r is None) == (k not in want), k
        if r is not None:
            assert relative(r, want[k].cpu()) <= (step(dtype) if r.dtype == torch.bfloat16 else 1e-5), k
