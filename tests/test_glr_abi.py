"""Argument checks of the gated linear recurrence and the block norm on the
host: every call fails a check before anything is launched; the pointers are
fake addresses that no code dereferences, and each case breaks one rule."""
import ctypes

import pytest

from bidirectional_mamba_denoiser_b200 import bimamba as bm

F = 0x7F0000000000
INV, UNS, MIS, WS = (bm.BIMAMBA_ERR_INVALID_ARG, bm.BIMAMBA_ERR_UNSUPPORTED, bm.BIMAMBA_ERR_MISALIGNED,
                     bm.BIMAMBA_ERR_WORKSPACE)
B, L, D = 2, 100, 32


def _row(k, **kw):
    return bm.Rows(kw.get("ptr", F + (k << 16)), kw.get("bs", L * D), kw.get("ts", D))


def _glr(bwd=False, inp=None, par=None, rows=None, grads=None, broken=True, **a):
    assert broken, "a validation case must break some argument"
    i = bm.GlrInputs(_row(0), _row(1), _row(2), _row(3), _row(4), F + (5 << 16), bm.BIMAMBA_BF16)
    for k, v in (inp or {}).items():
        setattr(i, k, v)
    p = bm.GlrParams(F + (6 << 16), F + (7 << 16), F + (8 << 16))
    for k, v in (par or {}).items():
        setattr(p, k, v)
    r = rows or _row(9)
    b, l, d = a.get("b", B), a.get("L", L), a.get("D", D)
    need = bm.bimamba_glr_workspace_bytes(B, L, D, bwd)
    flags, ws, wsb = a.get("flags", 0), a.get("ws", F + (10 << 16)), a.get("wsb", need)
    null = a.get("null", ())
    ref = lambda name, s: None if name in null else ctypes.byref(s)  # noqa: E731
    if not bwd:
        return bm.lib.bimamba_glr_fwd(ref("in", i), ref("p", p), a.get("h_in", F), ref("rows", r), a.get("h_out", F),
                                      a.get("chunk", F), b, l, d, flags, ws, wsb, None)
    g = bm.GlrGrads(_row(11), _row(12), _row(13), _row(14), _row(15), F, F, F, F)
    for k, v in (grads or {}).items():
        setattr(g, k, v)
    return bm.lib.bimamba_glr_bwd(ref("in", i), ref("p", p), ref("rows", r), a.get("chunk", F), a.get("dh_out", F),
                                  ref("grads", g), b, l, d, flags, ws, wsb, None)


COMMON = [
    (dict(null=("in",)), INV), (dict(null=("p",)), INV), (dict(null=("rows",)), INV),
    (dict(b=0), INV), (dict(b=65536), INV), (dict(L=0), INV), (dict(L=-1), INV), (dict(L=2 ** 31), INV), (dict(D=0), INV),
    (dict(flags=1), UNS), (dict(flags=0x18), UNS), (dict(inp={"dtype": 7}), UNS),
    (dict(inp={"x": _row(0, ptr=None)}), INV), (dict(inp={"r": _row(0, ptr=None)}), INV),
    (dict(inp={"i": _row(0, ptr=None)}), INV), (dict(inp={"x": _row(0, ts=-1)}), INV),
    (dict(inp={"z": _row(0, bs=-1)}), INV), (dict(inp={"add": _row(0, ptr=F + 1)}), MIS),
    (dict(inp={"x": _row(0, ptr=F + 1)}), MIS), (dict(inp={"lengths": F + 2}), MIS),
    (dict(par={"A": None}), INV), (dict(par={"A": F + 2}), MIS), (dict(par={"r_bias": F + 1}), MIS),
    (dict(ws=None), WS), (dict(ws=F + 16), WS), (dict(wsb=8), WS), (dict(chunk=F + 2), MIS),
]


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", COMMON)
def test_both_refuse(bwd, kw, status):
    assert _glr(bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=_row(9, ptr=None)), INV), (dict(rows=_row(9, ptr=F + 1)), MIS), (dict(h_in=F + 1), MIS),
    (dict(h_out=F + 2), MIS),
    # rows of the output that overlap one another
    (dict(rows=_row(9, ts=D - 1)), INV), (dict(rows=_row(9, ts=0)), INV), (dict(rows=_row(9, bs=0)), INV),
    (dict(rows=_row(9, bs=(L - 1) * D)), INV), (dict(rows=_row(9, bs=D, ts=2 * D - 1)), INV),
])
def test_forward_refuses(kw, status):
    assert _glr(False, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(chunk=None), INV), (dict(null=("grads",)), INV), (dict(rows=_row(9, ptr=None)), INV),
    (dict(grads={"dx": _row(1, ptr=None)}), INV), (dict(grads={"dr": _row(1, ts=3)}), INV),
    (dict(grads={"di": _row(1, ptr=F + 1)}), MIS), (dict(grads={"dadd": _row(1, ptr=None)}), INV),
    (dict(grads={"dz": _row(1, ptr=None)}), INV), (dict(grads={"dA": F + 1}), MIS),
    (dict(grads={"dh_in": F + 2}), MIS), (dict(dh_out=F + 3), MIS),
])
def test_backward_refuses(kw, status):
    assert _glr(True, **kw) == status


def test_workspace_sizes():
    for f in (lambda *a: bm.bimamba_glr_workspace_bytes(*a), lambda *a: bm.bimamba_glr_workspace_bytes(*a, True),
              bm.bimamba_block_norm_workspace_bytes):
        assert f(2, 100, 32) > 0
        assert f(0, 100, 32) == f(2, 0, 32) == f(2, 100, 0) == f(70000, 1, 1) == 0


def _norm(bwd=False, par=None, grads=None, broken=True, **a):
    assert broken
    p = bm.BlockNormParams(F, F, F, F, 1.0, 1e-5)
    for k, v in (par or {}).items():
        setattr(p, k, v)
    ref = lambda name, s: None if name in a.get("null", ()) else ctypes.byref(s)  # noqa: E731
    ts, tu = a.get("ts", bm.BIMAMBA_BF16), a.get("tu", bm.BIMAMBA_BF16)
    b, l, d, flags = a.get("b", B), a.get("L", L), a.get("d", D), a.get("flags", 0)
    if not bwd:
        return bm.lib.bimamba_block_norm_fwd(a.get("x", F), a.get("u", F), ref("p", p), a.get("x_out", F),
                                             a.get("y", F), a.get("stats", F), ts, tu, b, l, d, flags, None)
    g = bm.BlockNormGrads(F, F, F, F, F, F)
    for k, v in (grads or {}).items():
        setattr(g, k, v)
    return bm.lib.bimamba_block_norm_bwd(a.get("dy", F), a.get("dx_out", F), a.get("x", F), a.get("u", F),
                                         a.get("stats", F), ref("p", p), ref("g", g), ts, tu, b, l, d, flags,
                                         a.get("ws", F), a.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(null=("p",)), INV), (dict(b=0), INV), (dict(b=65536), INV), (dict(L=0), INV), (dict(L=2 ** 31), INV),
    (dict(d=0), INV), (dict(d=16385), UNS), (dict(flags=1), UNS), (dict(ts=9), UNS), (dict(tu=9), UNS),
    (dict(tu=bm.BIMAMBA_F32), UNS), (dict(x=None), INV), (dict(x=F + 1), MIS), (dict(u=F + 1), MIS),
    (dict(stats=F + 2), MIS), (dict(par={"gate": F + 1}), MIS), (dict(par={"post_w": F + 2}), MIS),
    (dict(par={"gamma": F + 3}), MIS),
])
def test_norm_both_refuse(bwd, kw, status):
    assert _norm(bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x_out=None, y=None), INV), (dict(par={"eps": 0.0}), INV), (dict(par={"eps": -1.0}), INV),
    (dict(par={"eps": float("nan")}), INV), (dict(u=None), INV), (dict(y=F + 1), MIS), (dict(x_out=F + 1), MIS),
    (dict(par={"beta": F + 1}), MIS),
])
def test_norm_forward_refuses(kw, status):
    assert _norm(False, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None, dx_out=None), INV), (dict(stats=None), INV), (dict(null=("g",)), INV),
    (dict(grads={"dx": None}), INV), (dict(grads={"du": None}), INV), (dict(u=None), INV), (dict(dy=None), INV),
    (dict(par={"gate": None}), INV), (dict(par={"post_w": None}), INV), (dict(par={"gamma": None}), INV),
    (dict(grads={"du": F + 1}), MIS), (dict(grads={"dgamma": F + 1}), MIS), (dict(ws=None), WS), (dict(ws=F + 8), WS),
    (dict(wsb=16), WS),
])
def test_norm_backward_refuses(kw, status):
    assert _norm(True, **kw) == status
