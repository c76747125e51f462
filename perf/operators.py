"""What is measured of the operators that stand around the recurrence: linear attention with a decay for each
head (chunked prefill, one decode step, gradient) and the gated norm with its residual (forward, gradient).

    S_t = e^{g_h} S_{t-1} + v_t k_t^T,    o_t = S_t q_t                                   (linear attention)
    u = act(z) * norm(x) * w,   y = residual + scale * u,   n = norm(y) * w_next           (gated norm)

`listed()` gives the cases, `run()` one pass: the plain form in elementary torch operations where `own` is false,
the library's entry points where it is true.  `exact()` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64      # tokens per block of the plain form


# ------------------------------------------------------------------ cases ----

def _linear(name, op, N, T, H_qk, H, d_k, d_v, dtype, ragged, state):
    return {"name": name, "op": op, "N": N, "T": T, "H_qk": H_qk, "H": H, "d_k": d_k, "d_v": d_v, "dtype": dtype,
            "ragged": ragged, "state": state}


def _norm(name, op, rows, dim, dtype, gate, residual, scale):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "gate": gate, "residual": residual,
            "scale": scale}


def listed():
    return [
        # one layer over one prompt, at the scalar-gate prefill workload's shape
        _linear("prefill_prompt", "prefill", 1, 8192, 16, 16, 128, 128, "bf16", False, False),
        # packed prompts of unequal lengths continuing from states, three value heads to a query/key head
        _linear("prefill_packed", "prefill", 8, 16384, 16, 48, 128, 128, "bf16", True, True),
        # single precision, unequal d_k and d_v, odd lengths: the form a model is debugged in
        _linear("prefill_single", "prefill", 3, 2011, 8, 8, 64, 128, "f32", True, True),
        # a short prompt, where latency counts
        _linear("prefill_short", "prefill", 1, 77, 16, 16, 128, 128, "bf16", False, False),
        # a serving batch's step, at the decode workload's shape
        _linear("decode_batch", "decode", 256, 256, 32, 32, 128, 128, "bf16", False, True),
        # one user's step, where latency counts
        _linear("decode_one", "decode", 1, 1, 16, 16, 128, 128, "bf16", False, True),
        # training: one layer's gradient at the gradient workload's shape
        _linear("backward_long", "backward", 1, 8192, 16, 16, 128, 128, "bf16", False, True),
        # training on packed documents with shared query/key heads
        _linear("backward_packed", "backward", 5, 3001, 4, 12, 128, 128, "bf16", True, True),
        # the output norm of every head with its SiLU gate, behind a prompt of the first case
        _norm("norm_heads", "norm", 131072, 128, "bf16", "silu", False, 1.0),
        # between two blocks while decoding: norm, residual, next block's norm, a few rows
        _norm("norm_block_step", "norm", 7, 4096, "bf16", "none", True, 0.5),
        # training: the output norm's gradient
        _norm("norm_heads_backward", "norm_backward", 131072, 128, "bf16", "silu", False, 1.0),
        # training: the gradient between two blocks, gated, in single precision, an odd number of rows
        _norm("norm_block_backward", "norm_backward", 8191, 2048, "f32", "sigmoid", True, 0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "backward", "norm", "norm_backward"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        dim = 128 if rng.random() < 0.4 else 8 * _log(rng, 2, 1024)
        rows = _log(rng, 1, max(2, (1 << 24) // dim))
        residual = dim != 128 and rng.random() < 0.7
        return _norm("", op, rows, dim, dtype, rng.choice(["none", "silu", "sigmoid"]), residual,
                     rng.choice([1.0, 0.5, 0.25])) | {"name": "%s_%d_%d" % (op, rows, dim)}
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if dtype == "bf16" and rng.random() < 0.75:
        d_k = d_v = 128
    else:
        d_k, d_v = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    H_qk = rng.choice([1, 2, 3, 4, 8, 16])
    H = H_qk * rng.choice([1, 1, 1, 2, 3])
    if op == "decode":
        N = _log(rng, 1, 256)
        return _linear("decode_%d_%d" % (N, H), op, N, N, H_qk, H, d_k, d_v, dtype, False, True)
    most = (8192 if dtype == "bf16" and d_k == d_v == 128 else 2048) * 16 // max(H, 16)
    T = _log(rng, 1, most)
    N = min(T, rng.choice([1, 1, 2, 3, 5, 8]))
    return _linear("%s_%d_%d_%d" % (op, N, T, H), op, N, T, H_qk, H, d_k, d_v, dtype, N > 1, rng.random() < 0.6)


# ----------------------------------------------------------------- inputs ----

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    io = _type(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    if case["op"] in ("norm", "norm_backward"):
        shape = (case["rows"], case["dim"])
        s = {"case": case, "x": (normal(*shape) * 0.7).to(io), "weight": 1 + 0.2 * normal(case["dim"]),
             "gate": normal(*shape, dtype=io) if case["gate"] != "none" else None,
             "residual": (normal(*shape) * 1.5).to(io) if case["residual"] else None,
             "next_weight": 1 + 0.2 * normal(case["dim"]) if case["residual"] else None}
        if case["op"] == "norm_backward":
            s["dy"] = normal(*shape, dtype=io)
            s["dn"] = normal(*shape, dtype=io) if case["residual"] else None
        return s

    N, T, H_qk, H, d_k, d_v = (case[n] for n in ("N", "T", "H_qk", "H", "d_k", "d_v"))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    # decays from e^-0.7 (a window of a token or two) to e^-0.004 (hundreds of tokens), spread over the heads
    decay = -0.7 * torch.exp2(-7.5 * (torch.arange(H, device="cuda") + torch.rand(1, generator=g, device="cuda")) / H)
    s = {"case": case, "q": unit(normal(T, H_qk, d_k)).to(io), "k": unit(normal(T, H_qk, d_k)).to(io),
         "v": normal(T, H, d_v, dtype=io), "decay": decay.float(),
         "S": 0.1 * normal(N, H, d_v, d_k) if case["state"] else None}
    if case["op"] == "decode":
        return s
    # the lengths of the packed sequences, and where each token lies in a batch padded to whole blocks
    if case["ragged"]:
        cpu = torch.Generator()
        cpu.manual_seed(seed)
        share = torch.rand(N, generator=cpu) * 1.6 + 0.2
        cuts = [0] + [round(float(c) * T) for c in (share.cumsum(0) / share.sum())[:-1]] + [T]
        s["cu_seqlens"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    else:
        cuts = [T // N * n for n in range(N + 1)]
        s["cu_seqlens"] = None
    lens = torch.tensor([b - a for a, b in zip(cuts, cuts[1:])], device="cuda")
    blocks = max(1, -(-int(lens.max()) // CHUNK))
    at = torch.arange(blocks * CHUNK, device="cuda")
    inside = at < lens[:, None]
    first = torch.tensor(cuts[:-1], device="cuda")[:, None]
    s |= {"lens": lens, "blocks": blocks, "inside": inside, "cuts": cuts,
          "forward": torch.where(inside, first + at, T), "reverse": torch.where(inside, first + lens[:, None] - 1 - at, T)}
    if case["op"] == "backward":
        s["d_o"] = normal(T, H, d_v, dtype=io)
        s["d_final"] = 0.1 * normal(N, H, d_v, d_k) if case["state"] else None
    return s


# ------------------------------------------------------------- plain forms ----

def _scan(s, a, b, v, state, reverse):
    """o_p = e^{g(p + 1 - r)} S a_p + sum_{j <= p} e^{g(p - j)} (a_p . b_j) v_j over each sequence's positions p, taken
    from the last token to the first if `reverse` (r = 1), and the state e^{g L} S + sum_j e^{g(L - 1 + r - j)} v_j b_j^T
    behind the last.  a, b [T, H, d_b] and v [T, H, d_v] in 32 bits, state [N, H, d_v, d_b] or None."""
    index, inside, lens, n = s["reverse" if reverse else "forward"], s["inside"], s["lens"], s["blocks"]
    N, H, g, r = len(lens), a.shape[1], s["decay"], int(reverse)

    def padded(x):
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[index]
        return x.view(N, n, CHUNK, H, x.shape[-1]).permute(0, 3, 1, 2, 4)       # [N, H, block, token, d]

    A, B, V = padded(a), padded(b), padded(v)
    i = torch.arange(CHUNK, device=a.device)
    apart = (i[:, None] - i)
    mask = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0)
    o = ((A @ B.transpose(-1, -2)) * mask[:, None]) @ V
    # each block's own state, and what all earlier blocks' hand on to each
    local = (V * torch.exp(g[:, None] * (CHUNK - 1 - i))[:, None, :, None]).transpose(-1, -2) @ B
    c = torch.arange(n, device=a.device)
    gap = c[:, None] - 1 - c
    hand = torch.where(gap >= 0, torch.exp(g[:, None, None] * CHUNK * gap.clamp(min=0)), 0.0)
    before = torch.matmul(hand, local.flatten(-2)).view_as(local)
    o = o + torch.exp(g[:, None] * (i + 1))[:, None, :, None] * (A @ before.transpose(-1, -2))
    at = torch.arange(n * CHUNK, device=a.device)
    left = (lens[:, None] - 1 + r - at).clamp(min=0)
    w = torch.exp(g[None, :, None] * left[:, None]) * inside[:, None]
    end = (V.flatten(2, 3) * w[..., None]).transpose(-1, -2) @ B.flatten(2, 3)
    if state is not None:
        lead = torch.exp(g[:, None] * (at + 1 - r)).view(H, n, CHUNK, 1)
        o = o + lead * (A @ state[:, :, None].transpose(-1, -2))
        end = end + torch.exp(g * lens[:, None])[..., None, None] * state
    out = o.new_empty(a.shape[0] + 1, H, v.shape[-1])
    out[index] = o.permute(0, 2, 3, 1, 4).reshape(N, n * CHUNK, H, -1)
    return out[:-1], end


def _spread(x, H):
    return x.float().repeat_interleave(H // x.shape[1], 1)


def _gather(x, H_qk):
    return x.view(x.shape[0], H_qk, -1, x.shape[-1]).sum(2)


def _plain_prefill(s):
    H = s["v"].shape[1]
    o, end = _scan(s, _spread(s["q"], H), _spread(s["k"], H), s["v"].float(), s["S"], False)
    return o.to(s["v"].dtype), end


def _plain_decode(s):
    H = s["v"].shape[1]
    q, k = _spread(s["q"], H), _spread(s["k"], H)
    s["S"].mul_(torch.exp(s["decay"])[:, None, None]).add_(s["v"].float()[..., None] * k[..., None, :])
    return (s["S"] * q[..., None, :]).sum(-1).to(s["v"].dtype), s["S"]


def _plain_backward(s):
    H_qk, H, io = s["q"].shape[1], s["v"].shape[1], s["v"].dtype
    q, k, v, do = _spread(s["q"], H), _spread(s["k"], H), s["v"].float(), s["d_o"].float()
    turned = lambda S: None if S is None else S.transpose(-1, -2)  # noqa: E731
    dq, _ = _scan(s, do, v, k, turned(s["S"]), False)
    dk, _ = _scan(s, v, do, q, turned(s["d_final"]), True)
    dv, dS = _scan(s, k, q, do, s["d_final"], True)
    return _gather(dq, H_qk).to(io), _gather(dk, H_qk).to(io), dv.to(io), dS


EPS = 1e-6


def _act(z, kind):
    sig = 1 / (1 + torch.exp(-z))
    return (z * sig, sig * (1 + z * (1 - sig))) if kind == "silu" else (sig, sig * (1 - sig))


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    u = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["gate"] is not None:
        u = u * _act(s["gate"].float(), case["gate"])[0]
    if s["residual"] is None:
        return (u * case["scale"]).to(s["x"].dtype)
    y = s["residual"].float() + case["scale"] * u
    n = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["next_weight"]
    return y.to(s["x"].dtype), n.to(s["x"].dtype)


def _plain_norm_backward(s):
    case, x, io, dy = s["case"], s["x"].float(), s["x"].dtype, s["dy"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, w = x * r, s["weight"]
    a, da = _act(s["gate"].float(), case["gate"]) if s["gate"] is not None else (1.0, None)
    out = {}
    if s["residual"] is not None:
        y = s["residual"].float() + case["scale"] * a * xh * w
        r2 = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        yh, dn = y * r2, s["dn"].float()
        t = dn * s["next_weight"]
        dy = dy + r2 * (t - yh * (t * yh).mean(-1, keepdim=True))
        out |= {"dnext_weight": (dn * yh).sum(0), "dresidual": dy.to(io)}
    du = case["scale"] * dy
    if da is not None:
        out["dgate"] = (du * xh * w * da).to(io)
    out["dweight"] = (du * a * xh).sum(0)
    t = du * a * w
    return out | {"dx": (r * (t - xh * (t * xh).mean(-1, keepdim=True))).to(io)}


# --------------------------------------------------------------- one pass ----

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"prefill": _plain_prefill, "decode": _plain_decode, "backward": _plain_backward, "norm": _plain_norm,
                "norm_backward": _plain_norm_backward}[op](s)
    from gated_delta_rule_151_b200 import gdr
    if op == "prefill":
        return gdr.gdr_linear_prefill(s["q"], s["k"], s["v"], s["decay"], s["S"], s["cu_seqlens"], num_seqs=case["N"])
    if op == "decode":
        return gdr.gdr_linear_decode(s["q"], s["k"], s["v"], s["decay"], s["S"]), s["S"]
    if op == "backward":
        return gdr.gdr_linear_backward(s["q"], s["k"], s["v"], s["decay"], s["S"], s["cu_seqlens"], d_o=s["d_o"],
                                       d_final_state=s["d_final"], num_seqs=case["N"])
    named = {"weight": s["weight"], "gate": s["gate"], "residual": s["residual"], "next_weight": s["next_weight"],
             "scale": case["scale"], "eps": EPS, "activation": case["gate"]}
    if op == "norm":
        y, n = gdr.gdr_norm_gate(s["x"], **named)
        return y if n is None else (y, n)
    got = gdr.gdr_norm_gate_backward(s["x"], s["dy"], s["dn"], **named)
    return {name: t for name, t in zip(("dx", "dweight", "dgate", "dresidual", "dnext_weight"), got) if t is not None}


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_backward"):
        n, res, gate = case["rows"] * case["dim"], int(case["residual"]), int(case["gate"] != "none")
        if case["op"] == "norm":
            return {"bytes": n * b * (2 + gate + 2 * res) + 4 * case["dim"] * (1 + res), "flops": n * (6 + 4 * gate + 6 * res)}
        return {"bytes": n * b * (3 + 2 * gate + 3 * res) + 8 * case["dim"] * (1 + res), "flops": n * (12 + 8 * gate + 12 * res)}
    N, T, H_qk, H, d_k, d_v = (case[n] for n in ("N", "T", "H_qk", "H", "d_k", "d_v"))
    qk, vo, S = T * H_qk * d_k * b, T * H * d_v * b, N * H * d_k * d_v * 4
    if case["op"] == "decode":
        return {"bytes": 2 * qk + 2 * vo + 2 * S + 4 * H, "flops": 5 * T * H * d_k * d_v}
    # a token's products with the state and its update, and half of its block's
    fwd = T * H * (4 * d_k * d_v + CHUNK * (d_k + d_v))
    if case["op"] == "prefill":
        return {"bytes": 2 * qk + 2 * vo + S * (1 + case["state"]) + 4 * H, "flops": fwd}
    # the two states and their updates, three more products with them, and the block's
    return {"bytes": 4 * qk + 3 * vo + S * (1 + 2 * case["state"]) + 4 * H,
            "flops": T * H * (10 * d_k * d_v + CHUNK * (3 * d_k + 2 * d_v))}


# ------------------------------------------------- the definition, 64 bits ----

def _pairs(a, b, v, g, state, reverse):
    """One sequence and one head in 64 bits, from every pair of its tokens: a, b [L, d_b], v [L, d_v], state [d_v, d_b]."""
    L = a.shape[0]
    p = torch.arange(L, device=a.device, dtype=torch.float64)
    o = torch.empty(L, v.shape[1], device=a.device, dtype=torch.float64)
    for at in range(0, L, 2048):
        rows = slice(at, min(L, at + 2048))
        apart = (p - p[rows, None]) if reverse else (p[rows, None] - p)
        o[rows] = torch.where(apart >= 0, (a[rows] @ b.T) * torch.exp(g * apart.clamp(min=0)), 0.0) @ v
    steps = (L - 1 - p) if reverse else p + 1
    end = (v * torch.exp(g * (p + 1 if reverse else L - 1 - p))[:, None]).T @ b
    if state is not None:
        o += torch.exp(g * steps)[:, None] * (a @ state.T)
        end = end + torch.exp(g * L) * state
    return o, end


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda name: None if s[name] is None else s[name].double()  # noqa: E731
    if case["op"] in ("norm", "norm_backward"):
        x, w, z, res, w2 = f("x"), f("weight"), f("gate"), f("residual"), f("next_weight")
        c, D = case["scale"], case["dim"]
        root = torch.sqrt((x * x).sum(1) / D + EPS)[:, None]
        gate = torch.ones_like(x) if z is None else torch.sigmoid(z) * (z if case["gate"] == "silu" else 1)
        y = c * gate * w * x / root + (0 if res is None else res)
        root2 = torch.sqrt((y * y).sum(1) / D + EPS)[:, None]
        if case["op"] == "norm":
            return y if res is None else (y, y / root2 * w2)
        e, out = f("dy"), {}
        if res is not None:
            h = f("dn") * w2
            out["dnext_weight"] = (f("dn") * y / root2).sum(0)
            e = e + h / root2 - y * ((h * y).sum(1, keepdim=True) / (D * root2 ** 3))
            out["dresidual"] = e
        if z is not None:
            t = torch.sigmoid(z)
            slope = t * (1 - t) if case["gate"] == "sigmoid" else t + z * t * (1 - t)
            out["dgate"] = c * e * slope * w * x / root
        out["dweight"] = (c * e * gate * x / root).sum(0)
        h = c * e * gate * w
        out["dx"] = h / root - x * ((h * x).sum(1, keepdim=True) / (D * root ** 3))
        return out
    q, k, v, S, g = f("q"), f("k"), f("v"), f("S"), f("decay")
    N, H_qk, H, d_k, d_v = (case[n] for n in ("N", "H_qk", "H", "d_k", "d_v"))
    T, per = case["T"], H // H_qk
    new = lambda *shape: torch.zeros(shape, device="cuda", dtype=torch.float64)  # noqa: E731
    end = new(N, H, d_v, d_k)
    if case["op"] == "decode":
        o = new(N, H, d_v)
        for h in range(H):
            end[:, h] = torch.exp(g[h]) * S[:, h] + torch.einsum("nv,nk->nvk", v[:, h], k[:, h // per])
            o[:, h] = torch.einsum("nvk,nk->nv", end[:, h], q[:, h // per])
        return o, end
    o, dq, dk, dv = new(T, H, d_v), new(T, H_qk, d_k), new(T, H_qk, d_k), new(T, H, d_v)
    if case["op"] == "backward":
        do, dF = f("d_o"), f("d_final")
    for n, (a, b) in enumerate(zip(s["cuts"], s["cuts"][1:])):
        for h in range(H):
            j, t = h // per, slice(a, b)
            S0 = None if S is None else S[n, h]
            if case["op"] == "prefill":
                o[t, h], end[n, h] = _pairs(q[t, j], k[t, j], v[t, h], g[h], S0, False)
                continue
            G = None if dF is None else dF[n, h]
            dq[t, j] += _pairs(do[t, h], v[t, h], k[t, j], g[h], None if S0 is None else S0.T, False)[0]
            dk[t, j] += _pairs(v[t, h], do[t, h], q[t, j], g[h], None if G is None else G.T, True)[0]
            dv[t, h], end[n, h] = _pairs(k[t, j], q[t, j], do[t, h], g[h], G, True)
    return (o, end) if case["op"] == "prefill" else (dq, dk, dv, end)
