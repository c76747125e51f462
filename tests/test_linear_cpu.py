"""What the linear-attention and gated-norm entry points refuse, on a machine without a GPU: every check
runs on the host before anything is launched."""
import ctypes

import pytest
import torch

from gated_delta_rule_151_b200 import gdr

A = 0x7f0000000000          # 16-byte aligned addresses, far apart, never dereferenced
FAR = 1 << 32
MIS = A + 8
BIG = 1 << 40
P = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


def at(i):
    return A + i * FAR


def prefill(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), decay=at(3), h0=at(4), cu=None, N=1, T=64, Hqk=2, H=2, dk=16, dv=16, io=0,
             o=at(5), fin=at(6), ws=at(7), wsb=BIG)
    a.update(kw)
    return gdr.load_library().gdr_linear_prefill(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["decay"]), P(a["h0"]), P(a["cu"]), a["N"], a["T"], a["Hqk"], a["H"],
        a["dk"], a["dv"], a["io"], P(a["o"]), P(a["fin"]), P(a["ws"]), a["wsb"], None)


def backward(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), decay=at(3), h0=at(4), cu=None, N=1, T=64, Hqk=2, H=2, dk=16, dv=16, io=0,
             do=at(5), df=at(6), dq=at(7), dk_=at(8), dv_=at(9), dh0=at(10), ws=at(11), wsb=BIG)
    a.update(kw)
    return gdr.load_library().gdr_linear_backward(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["decay"]), P(a["h0"]), P(a["cu"]), a["N"], a["T"], a["Hqk"], a["H"],
        a["dk"], a["dv"], a["io"], P(a["do"]), P(a["df"]), P(a["dq"]), P(a["dk_"]), P(a["dv_"]), P(a["dh0"]),
        P(a["ws"]), a["wsb"], None)


SHAPES = [dict(dk=48), dict(dv=256), dict(dk=0), dict(H=0), dict(Hqk=0), dict(H=3), dict(T=-1), dict(N=-1),
          dict(N=3, T=64), dict(N=0, T=64), dict(io=2), dict(H=1 << 20, Hqk=1, T=1 << 20), dict(N=1 << 30, T=1 << 30, H=1, Hqk=1)]


@pytest.mark.parametrize("kw", SHAPES + [
    dict(q=None), dict(k=None), dict(v=None), dict(decay=None), dict(o=None), dict(q=MIS), dict(k=MIS), dict(v=MIS),
    dict(decay=at(3) + 2), dict(h0=MIS), dict(o=MIS), dict(fin=MIS), dict(cu=at(8) + 2),
    dict(o=at(2)), dict(o=at(0)), dict(fin=at(4) + 16), dict(fin=at(5)), dict(ws=at(0) + 16), dict(ws=at(5))])
def test_prefill_refuses(kw):
    assert prefill(**kw) == gdr.GDR_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SHAPES + [
    dict(q=None), dict(k=None), dict(v=None), dict(decay=None), dict(do=None), dict(dq=None), dict(dk_=None), dict(dv_=None),
    dict(do=MIS), dict(dq=MIS), dict(df=MIS), dict(dh0=MIS), dict(dq=at(0)), dict(dk_=at(7)), dict(dv_=at(5)),
    dict(dh0=at(6)), dict(dh0=at(4)), dict(ws=at(9))])
def test_backward_refuses(kw):
    assert backward(**kw) == gdr.GDR_ERR_INVALID_ARG


@pytest.mark.parametrize("io,d", [(0, 16), (1, 128)])
def test_workspace(io, d):
    for call, back in ((prefill, False), (backward, True)):
        need = gdr.gdr_linear_workspace_size(1, 5000, 2, 4, d, d, io, back)
        assert need > 0
        kw = dict(T=5000, H=4, io=io, dk=d, dv=d)
        assert call(ws=None, wsb=0, **kw) == gdr.GDR_ERR_WORKSPACE
        assert call(wsb=16, **kw) == gdr.GDR_ERR_WORKSPACE
        assert call(ws=at(11) + 8, **kw) == gdr.GDR_ERR_WORKSPACE
    # no tokens, no sequences: nothing to run, and no workspace
    assert gdr.gdr_linear_workspace_size(0, 0, 2, 4, d, d, io) == 0
    assert prefill(N=0, T=0, q=None, k=None, v=None, o=None, ws=None, wsb=0) == gdr.GDR_OK
    with pytest.raises(gdr.GdrError):
        gdr.gdr_linear_workspace_size(1, 64, 3, 4, d, d, io)


def test_workspace_stays_small_however_many_sequences():
    """The states between segments are bounded by the tokens, not by the number of sequences."""
    for N in (1, 64, 100000):
        need = gdr.gdr_linear_workspace_size(N, 1 << 18, 16, 16, 128, 128, gdr.GDR_BF16)
        # beside them: a copy of the incoming states, and a status word per segment
        assert need <= N * 16 * (128 * 128 * 4 + 16) + (256 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), 0), (dict(N=-1), 1), (dict(H=3), 1), (dict(dk=24), 1), (dict(io=3), 1), (dict(q=None), 1), (dict(k=MIS), 1),
    (dict(state=None), 1), (dict(state=MIS), 1), (dict(o=at(4)), 1), (dict(decay=at(3) + 1), 1), (dict(state=at(0)), 1)])
def test_decode_refuses(kw, status):
    a = dict(q=at(0), k=at(1), v=at(2), decay=at(3), state=at(4), N=2, Hqk=2, H=2, dk=16, dv=16, io=0, o=at(5))
    a.update(kw)
    assert gdr.load_library().gdr_linear_decode(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["decay"]), P(a["state"]), a["N"], a["Hqk"], a["H"], a["dk"], a["dv"],
        a["io"], P(a["o"]), None) == status


def test_check_workspace_refuses():
    lib = gdr.load_library()
    assert lib.gdr_linear_check_workspace(None, 256, None) == gdr.GDR_ERR_WORKSPACE
    assert lib.gdr_linear_check_workspace(P(A), 16, None) == gdr.GDR_ERR_WORKSPACE


NORM = dict(x=at(0), w=at(1), z=at(2), res=at(3), w2=at(4), rows=4, dim=128, scale=1.0, eps=1e-6, act=1, io=1)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=MIS), dict(w=MIS), dict(z=MIS), dict(res=MIS), dict(w2=MIS), dict(y=None), dict(y=MIS), dict(n=MIS),
    dict(w2=None), dict(n=None), dict(rows=-1), dict(dim=12), dict(dim=0), dict(dim=16392), dict(scale=float("nan")),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")), dict(act=3), dict(io=2), dict(y=at(0)), dict(y=at(2)),
    dict(n=at(5)), dict(y=at(3) + 16), dict(n=at(3)), dict(rows=1 << 31)])
def test_norm_refuses(kw):
    a = {**NORM, "y": at(5), "n": at(6), **kw}
    assert gdr.load_library().gdr_norm_gate(
        P(a["x"]), P(a["w"]), P(a["z"]), P(a["res"]), P(a["w2"]), a["rows"], a["dim"], a["scale"], a["eps"], a["act"],
        a["io"], P(a["y"]), P(a["n"]), None) == gdr.GDR_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None, dn=None, dw2=None), 1), (dict(dw=None), 1), (dict(dz=None), 1), (dict(z=None), 1), (dict(dw2=None), 1),
    (dict(w2=None), 1), (dict(res=None), 1), (dict(dx=None), 1), (dict(dx=at(5)), 1), (dict(dz=at(7)), 1), (dict(dw=MIS), 1),
    (dict(ws=None), 3), (dict(wsb=64), 3), (dict(ws=at(12) + 8), 3), (dict(ws=at(7)), 1)])
def test_norm_backward_refuses(kw, status):
    a = {**NORM, "dy": at(5), "dn": at(6), "dx": at(7), "dw": at(8), "dz": at(9), "dres": at(10), "dw2": at(11), "ws": at(12),
         "wsb": BIG, **kw}
    assert gdr.load_library().gdr_norm_gate_backward(
        P(a["x"]), P(a["w"]), P(a["z"]), P(a["res"]), P(a["w2"]), a["rows"], a["dim"], a["scale"], a["eps"], a["act"],
        a["io"], P(a["dy"]), P(a["dn"]), P(a["dx"]), P(a["dw"]), P(a["dz"]), P(a["dres"]), P(a["dw2"]), P(a["ws"]),
        a["wsb"], None) == status


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 2, 16)
    with pytest.raises(ValueError):
        gdr.gdr_linear_prefill(x, x, x, torch.zeros(2))        # not on a GPU
    with pytest.raises(ValueError):
        gdr.gdr_norm_gate(x)


@pytest.mark.parametrize("size", [
    lambda n: gdr.gdr_linear_workspace_size(n + 1, 64, 2, 2, 16, 16, 0), lambda n: gdr.gdr_linear_workspace_size(1, n + 64, 2, 2, 16, 16, 0),
    lambda n: gdr.gdr_linear_workspace_size(1, 64, 2, n + 2, 16, 16, 0), lambda n: gdr.gdr_norm_gate_workspace_size(4, n + 128)])
def test_binding_refuses_sizes_beyond_32_bits(size):
    """Whole multiples of 2^32 beside a good size: cut to 32 bits they would pass for it."""
    assert size(0) >= 0
    with pytest.raises(ValueError):
        size(1 << 32)


@pytest.mark.parametrize("sizes", [dict(N=1 << 32), dict(T=1 << 32), dict(H=1 << 32), dict(d=1 << 32), dict(num_seqs=(1 << 32) + 1)],
                         ids=lambda s: next(iter(s)))
def test_tensors_beyond_32_bits_are_refused(sizes, monkeypatch):
    """Tensors without storage whose sizes, cut to 32 bits, are those of a good call."""
    monkeypatch.setattr(gdr, "_need", lambda *a, **kw: None)
    s = dict(N=0, T=0, H=0, d=0, num_seqs=None) | sizes
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    q, v = new(64 + s["T"], 2, 16 + s["d"]), new(64 + s["T"], 2 + s["H"], 16)
    cu = None if s["num_seqs"] else new(2 + s["N"], dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        gdr._linear_args(q, q, v, new(2 + s["H"]), cu, s["num_seqs"])
