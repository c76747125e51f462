"""Linear attention with a decay for each head over lengths that are cut into segments and calls with many
outputs, where the kernels' passes follow one another and every rounding counts."""
import os
import subprocess
import sys

import pytest
import torch

from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu

KINDS = [(torch.float32, 32), (torch.bfloat16, 128)]
KIND_IDS = ["f32", "bf16"]


def make(T, Hqk, H, d, dtype, N=1, cu=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    t = {"q": unit(r(T, Hqk, d)).to(dtype), "k": unit(r(T, Hqk, d)).to(dtype), "v": r(T, H, d).to(dtype),
         "decay": -0.7 * torch.exp2(-7.0 * torch.arange(H) / H), "state": 0.3 * r(N, H, d, d),
         "cu": None if cu is None else torch.tensor(cu, dtype=torch.int32), "d_o": r(T, H, d).to(dtype),
         "d_final": 0.3 * r(N, H, d, d)}
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def backward(x, **kw):
    return gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], d_o=x["d_o"],
                                   d_final_state=x["d_final"], **kw)


@pytest.mark.parametrize("heads", [(3, 3), (1, 3)], ids=["own", "shared"])
@pytest.mark.parametrize("cu", [None, [0, 2000, 2001, 5000]], ids=["one", "packed"])
@pytest.mark.parametrize("dtype,d", KINDS, ids=KIND_IDS)
def test_passes_read_this_calls_states(dtype, d, cu, heads):
    """Two inputs in turn through one workspace, call behind call: the states between segments that a pass
    reads are those that the same call has joined, never what the call before left there."""
    T, N = 5000, 1 if cu is None else 3
    x, y = (make(T, *heads, d, dtype, N, cu, seed=s) for s in (1, 2))
    need = gdr.gdr_linear_workspace_size(N, T, *heads, d, d, gdr._io_code(dtype), True)
    want = []
    for t in (x, y):
        want.append(backward(t, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda")))
        torch.cuda.synchronize()
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = [backward(t, workspace=ws) for _ in range(8) for t in (x, y)]
    gdr.gdr_linear_check_workspace(ws)
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2])), i


def scan(a, b, v, g, state, reverse):
    """One head of one sequence in 64 bits, from every pair of its tokens: o_p = sum x^|p - j| (a_p . b_j) v_j over
    the tokens up to p (from p on if reverse) and x^(p + 1) S a_p (x^(L - 1 - p)), the state behind the last token,
    and both again with every product's magnitude."""
    L = a.shape[0]
    p = torch.arange(L, device=a.device, dtype=torch.float64)
    apart = p - p[:, None] if reverse else p[:, None] - p
    x = torch.where(apart >= 0, torch.exp(g * apart.clamp(min=0)), 0.0)
    lead = torch.exp(g * ((L - 1 - p) if reverse else p + 1))[:, None]
    left = torch.exp(g * ((p + 1) if reverse else L - 1 - p))[:, None]

    def both(a, b, v, S):
        return ((a @ b.T) * x) @ v + lead * (a @ S.T), (v * left).T @ b + torch.exp(g * L) * S

    return both(a, b, v, state) + both(a.abs(), b.abs(), v.abs(), state.abs())


def definition(x, back):
    """What the call returns, in 64 bits, and per element the sum of its products' magnitudes: the output and the
    last state, or the four gradients."""
    q, k, v, do, S, dF = (x[n].double() for n in ("q", "k", "v", "d_o", "state", "d_final"))
    T, Hqk, _ = q.shape
    N, H = S.shape[:2]
    cuts = [0, T] if x["cu"] is None else x["cu"].tolist()
    new = [torch.zeros_like(t) for t in ((q, k, v, S) if back else (v, S))]
    mag = [torch.zeros_like(t) for t in new]
    for n in range(N):
        t = slice(cuts[n], cuts[n + 1])
        for h in range(H):
            j, g = h // (H // Hqk), x["decay"][h].double()
            if not back:
                runs = [((q[t, j], k[t, j], v[t, h], g, S[n, h], False), 0, (t, h), 1)]
            else:
                runs = [((do[t, h], v[t, h], k[t, j], g, S[n, h].T, False), 0, (t, j), None),
                        ((v[t, h], do[t, h], q[t, j], g, dF[n, h].T, True), 1, (t, j), None),
                        ((k[t, j], q[t, j], do[t, h], g, dF[n, h], True), 2, (t, h), 3)]
            for args, i, at, s in runs:
                o, end, o_mag, end_mag = scan(*args)
                new[i][at] += o
                mag[i][at] += o_mag
                if s is not None:
                    new[s][n, h], mag[s][n, h] = end, end_mag
    return new, mag


@pytest.mark.parametrize("T,Hqk,H,cu", [(77, 16, 16, None), (2500, 3, 3, None), (2500, 1, 3, None), (2500, 2, 4, [0, 700, 701, 2500]),
                                        (2501, 4, 4, [0, 64, 64, 2440, 2501])],
                         ids=["short", "one", "one-shared", "packed-shared", "packed"])
@pytest.mark.parametrize("back", [False, True], ids=["forward", "gradient"])
def test_bf16_results_carry_one_rounding(T, Hqk, H, cu, back):
    """A bf16 result is off by the rounding of its own type and by nothing of that size besides, whether a call has
    few outputs or many, one segment or several, and heads of their own or shared.

    In the 2-norm: the operands' copies keep 16 bits, 2^-8 of a bf16 rounding each, and a sum of n products in
    fp32 adds 2^-24 sqrt(n) of its terms' 2-norm, n < 1500, about 2^-18 of a result with random signs; in
    quadrature the rounding alone is exceeded by less than a thousandth.  2 % are allowed; one operand's copy in
    8 bits gives up to 22 %, two give 41 %.
    Each element: half a bf16 step, 2^-8 of it; 2^-16 of the products' magnitudes for either copy (half a step of
    its second term, 2^-8 2^-8); in fp32 the decay's power and the state's update of each of L / 64 blocks (four
    roundings), and the sums over d channels (of a score, of S a) and 64 tokens (three terms of each in the state's
    product, two in the output's)."""
    d, N = 128, 1 if cu is None else len(cu) - 1
    x = make(T, Hqk, H, d, torch.bfloat16, N, cu, seed=20)
    if back:
        got = backward(x)
    else:
        got = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    fp32 = (4 * -(-T // 64) + 3 * d + 5 * 64 + 32) * 2.0 ** -24
    for i, (r, want, mag) in enumerate(zip(got, *definition(x, back))):
        off = (r.double() - want).abs()
        extra = fp32 * mag + (2 * 2.0 ** -16 * mag if r.dtype == torch.bfloat16 else 0)
        half = 2.0 ** -8 if r.dtype == torch.bfloat16 else 2.0 ** -24
        assert (off <= half * (want.abs() + extra) + extra).all(), (i, float(off.max()))
        if r.dtype == torch.bfloat16:
            alone = (want.float().to(r.dtype).double() - want).norm()
            assert off.norm() <= 1.02 * alone, (i, float(off.norm() / alone))
        else:
            assert off.norm() <= 1e-5 * want.norm(), i


def test_bf16_results_do_not_depend_on_the_batch():
    """A prompt alone and among many others: the same to fp32 sums, so that only elements at a rounding border move.

    Both differ from the exact value by less than 2^-16 of it in the 2-norm (two copies of 16 bits, their fp32 sums
    far below).  An element moves by a step, at most 2^-7 of it, where its border lies between, with a probability of
    the difference over the step: in the 2-norm sqrt(2 2^-16 / 2^-8) 2^-8 = 2^-11.5 for steps of 2^-8, 2^-11 for 2^-7."""
    L, N, H, d = 60, 70, 2, 128
    x = make(L * N, H, H, d, torch.bfloat16, N, list(range(0, L * N + 1, L)), seed=21)
    o, _ = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    grads = backward(x)
    for n in (0, 33, N - 1):
        t = slice(n * L, n * L + L)
        y = {**{m: x[m][t].contiguous() for m in ("q", "k", "v", "d_o")}, "decay": x["decay"], "cu": None,
             "state": x["state"][n:n + 1].contiguous(), "d_final": x["d_final"][n:n + 1].contiguous()}
        alone, _ = gdr.gdr_linear_prefill(y["q"], y["k"], y["v"], y["decay"], y["state"])
        for a, b in zip((o, *grads[:3]), (alone, *backward(y)[:3])):
            assert (a[t].double() - b.double()).norm() <= 2.0 ** -11 * b.double().norm()


FIRST_CALLS = """
import sys, threading, torch
from gated_delta_rule_151_b200 import gdr
torch.manual_seed(0)
n = int(sys.argv[1])
q = torch.nn.functional.normalize(torch.randn(300, 2, 128, device="cuda"), dim=-1).bfloat16()
v, decay, beta = torch.randn_like(q), torch.tensor([-0.1, -0.01], device="cuda"), torch.rand(300, 2, device="cuda")
calls = [lambda: gdr.gdr_linear_prefill(q, q, v, decay), lambda: gdr.gdr_linear_backward(q, q, v, decay, d_o=v),
         lambda: gdr.gdr_prefill_chunked(q, q, v, -beta, beta)]
warm = [[torch.empty_like(v) for _ in range(64)], torch.empty(1 << 26, device="cuda")]
del warm                     # (memory at hand: the threads' first CUDA call is the library's)
torch.cuda.synchronize()
for call in calls:
    start, out = threading.Barrier(n), [None] * n
    def run(i):
        start.wait()
        out[i] = call()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert all(o is not None and all(torch.equal(a, b) for a, b in zip(o, call())) for o in out)
"""


@pytest.mark.parametrize("threads", [1, 16])
def test_first_calls_of_threads(threads):
    """The first calls of a process come from new threads, one or many at the same time: none finds the library
    half set up or is refused for want of a context."""
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(threads)], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0, run.stderr[-2000:]
