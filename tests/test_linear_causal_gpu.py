"""Linear attention with a decay for each head: which results an infinity or NaN of one input element reaches,
inside blocks and segments as across them."""
import pytest
import torch

from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu

HEAD, CHANNEL = 2, 5


def make(T, dtype, d, N, cu):
    g = torch.Generator().manual_seed(30)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    t = {"q": unit(r(T, 2, d)).to(dtype), "k": unit(r(T, 2, d)).to(dtype), "v": r(T, 4, d).to(dtype),
         "decay": torch.tensor([-0.5, -0.1, -0.02, -0.004]), "state": 0.3 * r(N, 4, d, d),
         "cu": torch.tensor(cu, dtype=torch.int32), "d_o": r(T, 4, d).to(dtype), "d_final": 0.3 * r(N, 4, d, d)}
    return {n: x.cuda() for n, x in t.items()}


def run(x):
    o, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    grads = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], d_o=x["d_o"],
                                    d_final_state=x["d_final"])
    return dict(zip(("o", "fin", "dq", "dk", "dv", "dS"), (o, fin, *grads)))


# Of each input: the results it enters, from or up to its token (or that one alone), and whether in its own
# channel or in all of them.  o_i = sum_{j <= i} (q_i k_j) v_j; dq_i = sum_{j <= i} (do_i v_j) k_j;
# dk_j = sum_{i >= j} (v_j do_i) q_i; dv_j = sum_{i >= j} (k_j q_i) do_i.
REACHES = {
    "q": {"o": ("at", "all"), "dk": ("upto", "own"), "dv": ("upto", "all")},
    "k": {"o": ("from", "all"), "dq": ("from", "own"), "dv": ("at", "all")},
    "v": {"o": ("from", "own"), "dq": ("from", "all"), "dk": ("at", "all")},
    "d_o": {"dq": ("at", "all"), "dk": ("upto", "all"), "dv": ("upto", "own")},
}
PER_HEAD = ("o", "dv")      # the others belong to the head's group


@pytest.mark.parametrize("name", list(REACHES))
@pytest.mark.parametrize("T,cu", [(230, [0, 29, 230]), (3000, [0, 100, 3000])], ids=["short", "segments"])
@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_one_element_reaches_what_the_formulas_say(dtype, d, T, cu, name):
    """Everything else keeps its bits; what is reached is not finite.  The tokens lie at both ends and inside of
    blocks, the last one in a block that is not full."""
    x = make(T, dtype, d, len(cu) - 1, cu)
    clean = run(x)
    own_head = name in ("v", "d_o")
    for place, value in ((0, float("nan")), (37, float("inf")), (63, float("-inf")), (64 + 20, float("nan")),
                         (cu[2] - cu[1] - 1, float("inf")), (cu[2] - cu[1] - 5, float("nan"))):
        t = cu[1] + place
        y = dict(x)
        y[name] = x[name].clone()
        y[name][t, HEAD if own_head else HEAD // 2, CHANNEL] = value
        got = run(y)
        for out in ("o", "dq", "dk", "dv"):
            hit = torch.zeros_like(clean[out], dtype=torch.bool)
            if out in REACHES[name]:
                where, which = REACHES[name][out]
                rows = {"at": slice(t, t + 1), "from": slice(t, cu[2]), "upto": slice(cu[1], t + 1)}[where]
                heads = slice(HEAD // 2, HEAD // 2 + 1) if out not in PER_HEAD else \
                    slice(HEAD, HEAD + 1) if own_head else slice(HEAD // 2 * 2, HEAD // 2 * 2 + 2)
                hit[rows, heads, slice(CHANNEL, CHANNEL + 1) if which == "own" else slice(None)] = True
            assert torch.equal(got[out][~hit], clean[out][~hit]), (out, place, value)
            assert not torch.isfinite(got[out][hit]).any(), (out, place, value)
        for out in ("fin", "dS"):        # the other sequence's states
            assert torch.equal(got[out][0], clean[out][0]), (out, place, value)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_several_elements_of_one_block(dtype, d):
    """Of a channel's elements in one block the first one counts (for the gradients the last), and channels and
    heads each have their own."""
    T = 150
    x = make(T, dtype, d, 1, [0, T])
    clean = run(x)
    at = {(3, 0): [10, 11, 50], (3, 9): [40], (1, 0): [70, 127], (0, d - 1): [31, 32], (2, 17): [T - 1]}
    for name, out, reverse in (("v", "o", False), ("d_o", "dv", True)):
        y = dict(x)
        y[name] = x[name].clone()
        hit = torch.zeros_like(clean[out], dtype=torch.bool)
        for (h, c), tokens in at.items():
            y[name][tokens, h, c] = float("nan")
            hit[slice(0, max(tokens) + 1) if reverse else slice(min(tokens), T), h, c] = True
        got = run(y)
        assert torch.equal(got[out][~hit], clean[out][~hit])
        assert not torch.isfinite(got[out][hit]).any()
