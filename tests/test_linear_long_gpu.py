"""Linear attention with a decay for each head over lengths that are cut into segments and calls with many
outputs, where the kernels' passes follow one another and every rounding counts."""
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
