"""Linear attention with a decay for each head on the GPU against its definition in 64 bits."""
import pytest
import torch

import _linear as ref
from gated_delta_rule_151_b200 import gdr

pytestmark = pytest.mark.gpu


def make(T, Hqk, H, dk, dv, dtype, N=1, cu=None, state=True, seed=0, strong=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    decay = -0.7 * torch.exp2(-7.0 * torch.arange(H) / H)
    if strong:   # no memory, a reset, none lost, far beyond what a product of decays can hold
        decay = torch.tensor([0.0, -float("inf"), -30.0, -3.0, -1e-4, -12.0])[torch.arange(H) % 6]
    t = {"q": unit(r(T, Hqk, dk)).to(dtype), "k": unit(r(T, Hqk, dk)).to(dtype), "v": r(T, H, dv).to(dtype),
         "decay": decay, "state": 0.3 * r(N, H, dv, dk) if state else None,
         "cu": None if cu is None else torch.tensor(cu, dtype=torch.int32),
         "d_o": r(T, H, dv).to(dtype), "d_final": 0.3 * r(N, H, dv, dk) if state else None}
    return t, {n: None if x is None else x.cuda() for n, x in t.items()}


CASES = [
    # T, Hqk, H, dk, dv, dtype, cu
    (1, 1, 1, 16, 16, torch.float32, None),
    (7, 2, 2, 16, 32, torch.float32, None),
    (63, 1, 2, 32, 16, torch.float32, None),
    (64, 2, 2, 64, 128, torch.float32, None),
    (65, 2, 2, 128, 64, torch.bfloat16, None),
    (130, 2, 4, 128, 128, torch.float32, [0, 1, 1, 65, 130]),
    (97, 1, 3, 64, 64, torch.bfloat16, [0, 0, 97, 97]),
    (50, 2, 2, 32, 128, torch.bfloat16, [0, 20, 50]),
    (1, 2, 2, 128, 128, torch.bfloat16, None),
    (3, 2, 2, 128, 128, torch.bfloat16, None),
    (63, 2, 2, 128, 128, torch.bfloat16, None),
    (64, 2, 2, 128, 128, torch.bfloat16, None),
    (65, 2, 2, 128, 128, torch.bfloat16, None),
    (129, 1, 3, 128, 128, torch.bfloat16, None),
    (200, 2, 2, 128, 128, torch.bfloat16, [0, 1, 1, 66, 200]),
    (255, 2, 6, 128, 128, torch.bfloat16, [0, 0, 128, 255, 255]),
    (321, 1, 1, 128, 128, torch.bfloat16, None),
    (700, 1, 2, 128, 128, torch.bfloat16, [0, 640, 700]),
]
ids = [f"T{c[0]}-H{c[1]}.{c[2]}-d{c[3]}.{c[4]}-{'bf16' if c[5] == torch.bfloat16 else 'f32'}{'-packed' if c[6] else ''}"
       for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=ids)
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_prefill(case, state):
    T, Hqk, H, dk, dv, dtype, cu = case
    N = 1 if cu is None else len(cu) - 1
    c, d = make(T, Hqk, H, dk, dv, dtype, N, cu, state)
    o, fin = gdr.gdr_linear_prefill(d["q"], d["k"], d["v"], d["decay"], d["state"], d["cu"])
    want = ref.prefill(c["q"], c["k"], c["v"], c["decay"], c["state"], c["cu"], N, dtype == torch.bfloat16)
    ref.check("o", o, want[0], want[1])
    ref.check("final state", fin, want[2], want[3])


@pytest.mark.parametrize("case", CASES, ids=ids)
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_backward(case, state):
    T, Hqk, H, dk, dv, dtype, cu = case
    N = 1 if cu is None else len(cu) - 1
    c, d = make(T, Hqk, H, dk, dv, dtype, N, cu, state, seed=1)
    got = gdr.gdr_linear_backward(d["q"], d["k"], d["v"], d["decay"], d["state"], d["cu"], d_o=d["d_o"],
                                  d_final_state=d["d_final"])
    want = ref.backward(c["q"], c["k"], c["v"], c["decay"], c["state"], c["cu"], N, c["d_o"], c["d_final"],
                        dtype == torch.bfloat16)
    for name, g, (w, tol) in zip(("dq", "dk", "dv", "d_initial_state"), got, want):
        ref.check(name, g, w, tol)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_extreme_decays(dtype, d):
    c, x = make(140, 6, 6, d, d, dtype, 2, [0, 70, 140], True, seed=2, strong=True)
    o, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    bf16 = dtype == torch.bfloat16
    want = ref.prefill(c["q"], c["k"], c["v"], c["decay"], c["state"], c["cu"], 2, bf16)
    ref.check("o", o, want[0], want[1])
    ref.check("final state", fin, want[2], want[3])
    got = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], d_o=x["d_o"],
                                  d_final_state=x["d_final"])
    want = ref.backward(c["q"], c["k"], c["v"], c["decay"], c["state"], c["cu"], 2, c["d_o"], c["d_final"], bf16)
    for name, g, (w, tol) in zip(("dq", "dk", "dv", "d_initial_state"), got, want):
        ref.check(name, g, w, tol)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_equal_lengths_are_packed_lengths(dtype, d):
    """num_seqs equal sequences give what cu_seqlens with the same cuts gives, however each is cut."""
    T, N, H = 6 * 704, 6, 2
    _, x = make(T, H, H, d, d, dtype, N, None, True, seed=3)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * (T // N)
    o1, s1 = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], num_seqs=N)
    o2, s2 = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], cu)
    # two orders of the same fp32 sums; in bf16 a rounding of the state's copy may go the other way
    tol = 2.0 ** -7 if dtype == torch.bfloat16 else 1e-5
    assert (o1.double() - o2.double()).norm() <= tol * o1.double().norm()
    assert (s1 - s2).double().norm() <= 1e-5 * s1.double().norm()


@pytest.mark.parametrize("dtype,d", [(torch.float32, 16), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_long_sequence_in_segments(dtype, d):
    """One long sequence (which is cut) equals its pieces run one after another, in both directions."""
    T, H = 5 * 1024 + 37, 2
    _, x = make(T, 1, H, d, d, dtype, 1, None, True, seed=4)
    o, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"])
    s, parts = x["state"], []
    for t0 in range(0, T, 512):
        t = slice(t0, min(T, t0 + 512))
        p, s = gdr.gdr_linear_prefill(x["q"][t].contiguous(), x["k"][t].contiguous(), x["v"][t].contiguous(),
                                      x["decay"], s)
        parts.append(p)
    tol = 2.0 ** -7 if dtype == torch.bfloat16 else 1e-5
    assert (o.double() - torch.cat(parts).double()).norm() <= tol * o.double().norm()
    assert (fin - s).double().norm() <= 1e-5 * s.double().norm()
    got = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], d_o=x["d_o"], d_final_state=x["d_final"])
    G, dv = x["d_final"], []
    for t0 in range(T // 512 * 512, -1, -512):
        t = slice(t0, min(T, t0 + 512))
        r = gdr.gdr_linear_backward(*(x[n][t].contiguous() for n in ("q", "k", "v")), x["decay"], None,
                                    d_o=x["d_o"][t].contiguous(), d_final_state=G)
        G = r[3]
        dv.insert(0, r[2])
    assert (got[2].double() - torch.cat(dv).double()).norm() <= tol * got[2].double().norm()
    assert (got[3] - G).double().norm() <= 1e-5 * G.double().norm()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,N,Hqk,H", [(16, 16, 1, 1, 1), (32, 128, 3, 2, 4), (64, 16, 5, 1, 3), (128, 128, 1, 2, 2),
                                           (128, 128, 40, 4, 8), (128, 32, 2, 3, 3), (16, 128, 7, 2, 2)])
def test_decode(dtype, dk, dv, N, Hqk, H):
    c, x = make(N, Hqk, H, dk, dv, dtype, N, None, True, seed=5)
    cu = torch.arange(N + 1, dtype=torch.int32)
    want = ref.prefill(c["q"], c["k"], c["v"], c["decay"], c["state"], cu, N, False)
    s = x["state"].clone()
    o = gdr.gdr_linear_decode(x["q"], x["k"], x["v"], x["decay"], s)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    ref.check("o", o, want[0], want[1] + half * (want[0].abs() + want[1]))
    ref.check("state", s, want[2], want[3])


def test_decode_continues_prefill():
    c, x = make(90, 2, 4, 128, 128, torch.bfloat16, 1, None, True, seed=6)
    o, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"])
    _, s = gdr.gdr_linear_prefill(x["q"][:80], x["k"][:80], x["v"][:80], x["decay"], x["state"])
    tail = [gdr.gdr_linear_decode(x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1], x["decay"], s) for t in range(80, 90)]
    want = ref.prefill(c["q"], c["k"], c["v"], c["decay"], c["state"], None, 1, True)
    ref.check("o", torch.cat(tail), want[0][80:], want[1][80:])
    ref.check("state", s, want[2], want[3])
    ref.check("state", fin, want[2], want[3])


@pytest.mark.parametrize("T", [100, 4097, 20000])
def test_state_in_place_and_repeatable(T):
    _, x = make(T, 2, 2, 128, 128, torch.bfloat16, 1, None, True, seed=7)
    o1, s1 = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"])
    s = x["state"].clone()
    o2, s2 = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], s, final_state=s)
    assert s2 is s and torch.equal(o1, o2) and torch.equal(s1, s2)
    a = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], d_o=x["d_o"], d_final_state=x["d_final"])
    b = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], d_o=x["d_o"], d_final_state=x["d_final"])
    assert all(torch.equal(u, w) for u, w in zip(a, b))


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_sequences_do_not_touch_each_other(dtype, d):
    """Infinities and NaN of one packed sequence stay in it, in every place of a block."""
    cu = [0, 70, 71, 135, 200]
    _, x = make(200, 2, 2, d, d, dtype, 4, cu, True, seed=8)
    clean = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    grads = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], d_o=x["d_o"],
                                    d_final_state=x["d_final"])
    for bad in (1, 2):
        y = {n: (t.clone() if t is not None else None) for n, t in x.items()}
        for n in ("q", "k", "v", "d_o"):
            y[n][cu[bad]:cu[bad + 1]] = float("inf") if bad == 1 else float("nan")
        o, s = gdr.gdr_linear_prefill(y["q"], y["k"], y["v"], y["decay"], y["state"], y["cu"])
        r = gdr.gdr_linear_backward(y["q"], y["k"], y["v"], y["decay"], y["state"], y["cu"], d_o=y["d_o"],
                                    d_final_state=y["d_final"])
        for n in range(4):
            if n == bad:
                continue
            t = slice(cu[n], cu[n + 1])
            assert torch.equal(o[t], clean[0][t]) and torch.equal(s[n], clean[1][n])
            assert all(torch.equal(u[t], w[t]) for u, w in zip(r[:3], grads[:3]))
            assert torch.equal(r[3][n], grads[3][n])


@pytest.mark.parametrize("dtype,d", [(torch.float32, 16), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_later_tokens_reach_no_earlier_output(dtype, d):
    """An infinity or NaN behind a token leaves that token's output as it was."""
    _, x = make(100, 2, 2, d, d, dtype, 1, None, True, seed=9)
    clean, _ = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"])
    for name, value in (("k", float("inf")), ("v", float("nan"))):
        y = dict(x)
        y[name] = x[name].clone()
        y[name][64:] = value
        o, _ = gdr.gdr_linear_prefill(y["q"], y["k"], y["v"], y["decay"], y["state"])
        assert torch.equal(o[:64], clean[:64])


def test_gradient_against_differences():
    """The gradient of q, k, v and the state against central differences of the forward pass (fp32)."""
    c, x = make(40, 1, 2, 16, 16, torch.float32, 2, [0, 13, 40], True, seed=10)
    got = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], d_o=x["d_o"],
                                  d_final_state=x["d_final"])

    def loss(**over):
        a = {**c, **over}
        o, _, s, _ = ref.prefill(a["q"], a["k"], a["v"], a["decay"], a["state"], a["cu"], 2, False)
        return float((o * c["d_o"].double()).sum() + (s * c["d_final"].double()).sum())

    g = torch.Generator().manual_seed(0)
    for name, grad in zip(("q", "k", "v", "state"), got):
        way = torch.randn(c[name].shape, generator=g).double()
        # the loss is a polynomial of degree at most 1 in each input alone: the difference is exact
        diff = (loss(**{name: c[name].double() + 0.5 * way}) - loss(**{name: c[name].double() - 0.5 * way}))
        along = float((grad.double().cpu() * way).sum())
        assert abs(along - diff) <= 2e-5 * float((grad.double().cpu() * way).abs().sum())


def test_streams_and_graph():
    """On a stream of its own, twice at once, and captured and replayed with new inputs in place."""
    _, x = make(1500, 2, 2, 128, 128, torch.bfloat16, 1, None, True, seed=11)
    _, y = make(1500, 2, 2, 128, 128, torch.bfloat16, 1, None, True, seed=12)
    run = lambda t, **kw: gdr.gdr_linear_prefill(t["q"], t["k"], t["v"], t["decay"], t["state"], **kw)  # noqa: E731
    back = lambda t: gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["decay"], t["state"], d_o=t["d_o"],  # noqa: E731
                                             d_final_state=t["d_final"])
    want_x, want_y, want_b = run(x), run(y), back(y)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got_x, got_y = run(x, stream=s1), run(y, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run(x, stream=0), want_x))     # the legacy stream's handle
    assert all(torch.equal(a, b) for a, b in zip(got_x + got_y, want_x + want_y))
    graph = torch.cuda.CUDAGraph()
    held = {n: t.clone() for n, t in x.items() if t is not None}
    with torch.cuda.graph(graph):
        out, grads = run(held), back(held)
    for n in held:
        held[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + grads, want_y + want_b))


@pytest.mark.parametrize("dtype,d", [(torch.float32, 16), (torch.bfloat16, 128)], ids=["f32", "bf16"])
def test_rows_behind_the_last_sequence_stay(dtype, d):
    """A batch padded behind its last sequence: what lies there is neither read into a result nor written."""
    T, end, Hqk, H = 200, 131, 2, 4
    _, x = make(T, Hqk, H, d, d, dtype, 2, [0, 60, end], True, seed=14)
    short = {n: (t[:end].contiguous() if n in ("q", "k", "v", "d_o") else t) for n, t in x.items()}
    want = gdr.gdr_linear_prefill(short["q"], short["k"], short["v"], short["decay"], short["state"], short["cu"])
    want_g = gdr.gdr_linear_backward(short["q"], short["k"], short["v"], short["decay"], short["state"], short["cu"],
                                     d_o=short["d_o"], d_final_state=short["d_final"])
    for n in ("q", "k", "v", "d_o"):
        x[n][end:] = float("nan")
    o = torch.full((T, H, d), 7.0, dtype=dtype, device="cuda")
    _, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"], o=o)
    assert (o[end:] == 7.0).all()
    tol = 2.0 ** -7 if dtype == torch.bfloat16 else 1e-5     # (the lengths are cut elsewhere: another order of sums)
    assert (o[:end].double() - want[0].double()).norm() <= tol * want[0].double().norm()
    assert (fin - want[1]).double().norm() <= 1e-5 * want[1].double().norm()
    # the gradients' tensors come from the binding: what lies behind is whatever the memory held
    lib = gdr.load_library()
    dq, dk, dv = (torch.full_like(t, 7.0) for t in (x["q"], x["k"], x["v"]))
    dS = torch.empty_like(x["state"])
    need = gdr.gdr_linear_workspace_size(2, T, Hqk, H, d, d, gdr._io_code(dtype), True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")       # NaN wherever it is read unwritten
    status = lib.gdr_linear_backward(
        x["q"].data_ptr(), x["k"].data_ptr(), x["v"].data_ptr(), x["decay"].data_ptr(), x["state"].data_ptr(),
        x["cu"].data_ptr(), 2, T, Hqk, H, d, d, gdr._io_code(dtype), x["d_o"].data_ptr(), x["d_final"].data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dS.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert status == gdr.GDR_OK
    for g, w in zip((dq, dk, dv), want_g):
        assert (g[end:] == 7.0).all()
        assert (g[:end].double() - w.double()).norm() <= tol * w.double().norm()
    assert (dS - want_g[3]).double().norm() <= 1e-5 * want_g[3].double().norm()


def test_malformed_cu_seqlens_stays_in_bounds():
    """Cuts that are no partition give wrong values, but write nothing outside the outputs."""
    T, H, d = 2500, 2, 128
    _, x = make(T, H, H, d, d, torch.bfloat16, 5, None, True, seed=13)
    guard = 4096
    for cu in ([0, T, 0, T, 0, T], [-5, 900, 10 ** 6, 3, 2 ** 31 - 1, T], [7, 7, 7, 7, 7, 7]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o = torch.full((T * H * d + 2 * guard,), 3.0, dtype=torch.bfloat16, device="cuda")
        need = gdr.gdr_linear_workspace_size(5, T, H, H, d, d, gdr.GDR_BF16)
        ws = torch.full((need + 2 * guard,), 77, dtype=torch.uint8, device="cuda")
        fin = torch.full((5 * H * d * d + 2 * guard,), 3.0, device="cuda")
        gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], cu, o=o[guard:-guard].view(T, H, d),
                               final_state=fin[guard:-guard].view(5, H, d, d), workspace=ws[guard:-guard])
        torch.cuda.synchronize()
        for t, value in ((o, 3.0), (fin, 3.0), (ws, 77)):
            assert (t[:guard] == value).all() and (t[-guard:] == value).all()


def test_check_workspace():
    _, x = make(300, 2, 2, 128, 128, torch.bfloat16, 1, None, False)
    need = gdr.gdr_linear_workspace_size(1, 300, 2, 2, 128, 128, gdr.GDR_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], workspace=ws)
    gdr.gdr_linear_check_workspace(ws)
    need = gdr.gdr_linear_workspace_size(1, 300, 2, 2, 128, 128, gdr.GDR_BF16, True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], d_o=x["d_o"], workspace=ws)
    gdr.gdr_linear_check_workspace(ws)


def test_empty():
    _, x = make(0, 2, 2, 128, 128, torch.bfloat16, 2, [0, 0, 0], True)
    o, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], x["cu"])
    assert o.shape == (0, 2, 128) and torch.equal(fin, x["state"])
    _, fin = gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["decay"], None, x["cu"])
    assert (fin == 0).all()
    *_, dS = gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["decay"], None, x["cu"], d_o=x["d_o"], d_final_state=x["d_final"])
    assert torch.equal(dS, x["d_final"])
