"""Linear attention with a decay for each head and the gated norm from their
definitions in 64 bits, and the error bounds the kernels are held to.

`scan` walks the tokens of one sequence and head:

    o_p = S_p a_p,  S_p = e^g S_{p-1} + v_p b_p^T        (last to first token if reverse:
                                                          S_p = S' + v_p b_p^T, S' = e^g S_p)

Beside o and the last state it returns, per element, two sums of magnitudes:
`near` = what a rounding of each product a.b and of each element of the state at
the start of a 64-token block scales (sum of |x^{p-j} (a.b) v| and |S||a|), and
`far` = the same of the inputs' magnitudes, which bounds fp32 rounding.
"""
import torch

BLOCK = 64


def scan(a, b, v, g, state, reverse):
    L, dv, db = a.shape[0], v.shape[1], a.shape[1]
    x = torch.exp(torch.clamp(torch.as_tensor(g, dtype=torch.float64), min=-20.0))
    S = torch.zeros(dv, db, dtype=torch.float64) if state is None else state.clone()
    A = S.abs()
    o, near, far = (torch.zeros(L, dv, dtype=torch.float64) for _ in range(3))
    order = range(L - 1, -1, -1) if reverse else range(L)
    at_block = S.clone()
    for p in order:
        if (p % BLOCK == BLOCK - 1 or p == L - 1) if reverse else p % BLOCK == 0:
            at_block, inside = S.clone(), []
            lead = torch.tensor(1.0, dtype=torch.float64)
        if not reverse:
            S, A, lead = x * S, x * A, lead * x
            inside = [x * y for y in inside]
        S = S + torch.outer(v[p], b[p])
        A = A + torch.outer(v[p].abs(), b[p].abs())
        inside.append(torch.ones((), dtype=torch.float64))
        o[p] = S @ a[p]
        far[p] = A @ a[p].abs()
        first = p - len(inside) + 1 if not reverse else p + len(inside) - 1
        rows = slice(first, p + 1) if not reverse else slice(p, first + 1)
        w = torch.stack(inside if not reverse else inside[::-1])
        near[p] = (w * (b[rows] @ a[p]).abs()) @ v[rows].abs() + lead * (at_block.abs() @ a[p].abs())
        if reverse:
            S, A, lead = x * S, x * A, lead * x
            inside = [x * y for y in inside]
    return o, S, near, far, A


def fp32_terms(L, d):
    """Rounding errors that reach one output in units of 2^-24 of `far`: a decay's power (two each
    token), the token's update, the sums over d channels and over the tokens of a block."""
    return (4 * L + 2 * d + 4 * BLOCK + 16) * 2.0 ** -24


def bounds(o, near, far, L, d, bf16, rounded=True):
    """|kernel - o|: fp32 rounding, and in bf16 half a step (2^-8) of the score, of the state's copy and
    of the result."""
    fp32 = fp32_terms(L, d) * far
    if not bf16:
        return fp32 + 2.0 ** -24 * o.abs()
    return fp32 + 2.0 ** -8 * (1 + 2.0 ** -7) * near + (2.0 ** -8 * (o.abs() + fp32 + 2.0 ** -7 * near) if rounded else 0)


def lengths(cu, N, T):
    if cu is None:
        return [(T // N * n, T // N * (n + 1)) for n in range(N)]
    return list(zip(cu.tolist(), cu.tolist()[1:]))


def prefill(q, k, v, decay, state, cu, N, bf16):
    """(o, bound of o, final state, bound) of the whole batch, on the CPU in 64 bits."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    state = None if state is None else state.double().cpu()
    T, Hqk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    o, tol = torch.zeros(T, H, dv, dtype=torch.float64), torch.zeros(T, H, dv, dtype=torch.float64)
    end, end_tol = (torch.zeros(N, H, dv, dk, dtype=torch.float64) for _ in range(2))
    for n, (t0, t1) in enumerate(lengths(cu, N, T)):
        for h in range(H):
            j = h // (H // Hqk)
            r, S, near, far, A = scan(q[t0:t1, j], k[t0:t1, j], v[t0:t1, h], float(decay[h]),
                                      None if state is None else state[n, h], False)
            o[t0:t1, h], end[n, h] = r, S
            tol[t0:t1, h] = bounds(r, near, far, t1 - t0, dk, bf16)
            end_tol[n, h] = fp32_terms(t1 - t0, 0) * A
    return o, tol, end, end_tol


def backward(q, k, v, decay, state, cu, N, d_o, d_final, bf16):
    """((gradient, bound), ...) of q, k, v and the initial state."""
    q, k, v, d_o = (t.double().cpu() for t in (q, k, v, d_o))
    state = None if state is None else state.double().cpu()
    d_final = None if d_final is None else d_final.double().cpu()
    T, Hqk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    new = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    out = {n: [new(*s), new(*s)] for n, s in (("q", (T, Hqk, dk)), ("k", (T, Hqk, dk)), ("v", (T, H, dv)),
                                              ("s", (N, H, dv, dk)))}
    group = H // Hqk
    for n, (t0, t1) in enumerate(lengths(cu, N, T)):
        t, L = slice(t0, t1), t1 - t0
        for h in range(H):
            j, g = h // group, float(decay[h])
            S = None if state is None else state[n, h]
            G = None if d_final is None else d_final[n, h]
            turned = lambda x: None if x is None else x.T  # noqa: E731
            for name, args, at, d in (("q", (d_o[t, h], v[t, h], k[t, j], g, turned(S), False), (t, j), dv),
                                      ("k", (v[t, h], d_o[t, h], q[t, j], g, turned(G), True), (t, j), dv),
                                      ("v", (k[t, j], q[t, j], d_o[t, h], g, G, True), (t, h), dk)):
                r, X, near, far, A = scan(*args)
                out[name][0][at] += r
                # dv belongs to its value head alone and is rounded at once, dq and dk of a group after the sum
                out[name][1][at] += bounds(r, near, far, L, d, bf16, rounded=group == 1 or name == "v")
                if name == "v":
                    out["s"][0][n, h], out["s"][1][n, h] = X, fp32_terms(L, 0) * A
    if group > 1:   # the heads' sum, then the one rounding of dq and dk
        for name in "qk":
            r, b = out[name]
            out[name][1] = (b + 2.0 ** -23 * group * r.abs()) * (1 + 2.0 ** -8) + (2.0 ** -8 if bf16 else 2.0 ** -24) * r.abs()
    return tuple(tuple(out[n]) for n in "qkvs")


def check(name, got, want, tol):
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{name}: off by {(got - want).abs().max():.3g}, {int((over > 0).sum())} over the bound"


# ------------------------------------------------------------- gated norm ----

def norm_gate(x, weight, gate, residual, next_weight, scale, eps, act):
    """(y, y_norm or None) in 64 bits; differentiable."""
    u = x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    if gate is not None:
        s = torch.sigmoid(gate)
        u = u * {"silu": gate * s, "sigmoid": s, "none": gate}[act]
    y = scale * u if residual is None else residual + scale * u
    if next_weight is None:
        return y, None
    return y, y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * next_weight
