"""The gated norm's activations and norms element by element, over the range of their arguments."""
import pytest
import torch

import _linear as ref
from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gates(dtype, reach):
    z = torch.linspace(-reach, reach, 128 * 512).to(dtype).view(-1, 128)
    z[0, :4] = torch.tensor([0.0, -0.0, 1e-30, -1e-30], dtype=dtype)
    return z


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_activation(dtype, act):
    """y = act(z) where x = 1 is not normed.  In fp32: the exponential's and the reciprocal's two half
    steps, the sum's and the product's one each, 2^-24 times 6; 8 are allowed.  In bf16 the rounding, 2^-8, and
    2^-20 (1 + |z| / 8) < 2^-16.  z from -80, where the sigmoid is a normal number."""
    z = gates(dtype, 80.0)
    y, _ = gdr.gdr_norm_gate(torch.ones_like(z).cuda(), gate=z.cuda(), activation=act)
    z = z.double()
    want = torch.sigmoid(z) * (z if act == "silu" else 1)
    tol = 8 * 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -16 * (1 + 2.0 ** -8)
    # (a product below the type's normal numbers is a step of those off: 2^-126 2^-7 in bf16, 2^-149 in fp32)
    off = (y.double().cpu() - want).abs()
    assert (off <= tol * want.abs() + 2.0 ** -126).all(), float((off / want.abs().clamp(min=1e-37)).max())


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_slope(dtype, act):
    """dgate = act'(z) where x = dy = 1, at both ends of the gate.  With s the sigmoid, s' = s (1 - s) and
    silu' = s (1 + z (1 - s)): relative to its terms' magnitudes either is off, in fp32, by the exponential (2),
    the sum (1) and the reciprocal (2) in s, the exponential's and the product's 3 in 1 - s besides, of which the
    exponential's in s and in 1 - s sum to 2, and by three more operations: 2^-24 times 14; 16 are allowed.  In bf16 twice the approximations' 2^-16 and the rounding."""
    z = gates(dtype, 60.0)
    one = torch.ones_like(z).cuda()
    dz = gdr.gdr_norm_gate_backward(one, one, gate=z.cuda(), activation=act)[2]
    z = z.double()
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    want = s * rest if act == "sigmoid" else s * (1 + z * rest)
    terms = s * rest if act == "sigmoid" else s * (1 + z.abs() * rest)
    off = (dz.double().cpu() - want).abs()
    tol = 16 * 2.0 ** -24 * terms if dtype == torch.float32 else 2.0 ** -8 * want.abs() + 2.0 ** -14 * terms
    assert (off <= tol + 2.0 ** -126).all(), float((off / terms).max())


@pytest.mark.parametrize("gate", [None, "gate"], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rows_of_every_size(dtype, gate):
    """Rows of zeros, of 1e-18 to 1e17, and one with a single large element, each row held to its own size, and
    their gradients to autograd in 64 bits.

    fp32 sums of 128 squares, the root and at most a dozen products in each direction, 2^-24 times 2 sqrt(128) and
    a term each: 1e-5 as for the other sizes, of the row's 2-norm; the gradient is a difference of terms that a row
    along one direction cancels: 1e-5 of |t| r.  bf16: 2^-8 besides."""
    g = torch.Generator().manual_seed(40)
    size = 10.0 ** torch.tensor([-18, -12, -6, -3, 0, 3, 9, 15, 17.0])
    x = torch.cat([torch.zeros(1, 128), size[:, None] * torch.randn(9, 128, generator=g)])
    x = torch.cat([x, x[4:5] * 1e-3])
    x[-1, 77] = 1e6
    rows = x.shape[0]
    z = torch.randn(rows, 128, generator=g) if gate else None
    w, dy = 1 + 0.3 * torch.randn(128, generator=g), torch.randn(rows, 128, generator=g)
    x, z, dy = (None if t is None else t.to(dtype) for t in (x, z, dy))
    dev = [None if t is None else t.cuda() for t in (x, dy, w, z)]
    y, _ = gdr.gdr_norm_gate(dev[0], dev[2], dev[3], eps=EPS)
    got = gdr.gdr_norm_gate_backward(dev[0], dev[1], None, dev[2], dev[3], eps=EPS)
    leaves = [None if t is None else t.double().requires_grad_() for t in (x, w, z)]
    want, _ = ref.norm_gate(leaves[0], leaves[1], leaves[2], None, None, 1.0, EPS, "silu")
    (want * dy.double()).sum().backward()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24

    def held(name, r, w, extra=None):
        r, size = r.double().cpu(), w.norm(dim=-1)
        assert torch.isfinite(r).all(), name
        over = (r - w).norm(dim=-1) - (half * size + 1e-5 * (size if extra is None else extra))
        assert (over <= 1e-30).all(), (name, over)

    held("y", y, want.detach())
    t = dy.double() * leaves[1].detach()
    if gate:
        t = t * torch.nn.functional.silu(z.double())
    root = torch.sqrt((x.double() ** 2).mean(-1) + EPS)
    held("dx", got[0], leaves[0].grad, t.norm(dim=-1) / root)
    held("dweight", got[1][None], leaves[1].grad[None])
    if gate:
        held("dgate", got[2], leaves[2].grad)
