"""Inputs and bounds of the recurrence's tests.

Bounds against the fp64 oracle, fixed before the first run.  A step's decay a
= exp(A rg) carries at most 2^-22 relative error (ex2.approx 2^-22.5 plus the
rounding of its argument |A rg| log2 e <= 1.2), and a state remembers at most M
= 1 / (1 - max a) steps, so that error grows to M 2^-22 of the state; the gates,
beta and the products add a dozen roundings (16 x 2^-22).  So a state is within
E = 2^-22 (M + 16) of the largest, and so is G, the same scan of dout.  Each
gradient multiplies up to three such factors: 3 E.  The parameters' sums add
the same relative error to each summand: 3 E of the sum of magnitudes.
The drawn A in [-0.8, -0.02] with gates near one half gives M up to 100, taken
here with all errors of one sign; channels whose gates stay nearly closed
remember longer, but over more steps the errors' signs mix and add like the
root of M, which M = 100 covers up to 10,000 steps.  A bf16 store
adds half a step, 2^-8 relative.
"""
from __future__ import annotations

import numpy as np
import torch

from tests import parity_util as U

E = 2.0 ** -22 * (100 + 16)
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def case(b, L, D, dtype="fp32", seed=0, gated=False, state=False, lengths=None, fused=False, bias=True):
    """Everything a forward and a backward call take, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = {}
    if fused:
        c["x"], c["r"], c["i"] = rn(b, L, 3 * D).to(t).split(D, dim=-1)
    else:
        c["x"], c["r"], c["i"] = (rn(b, L, D).to(t) for _ in range(3))
    c["params"] = {"A": -torch.exp(torch.rand(D, generator=g) * 3.7 - 3.9)}
    if bias:
        c["params"].update(r_bias=torch.rand(D, generator=g) - 0.5, i_bias=torch.rand(D, generator=g) - 0.5)
    c["add"], c["z"] = (rn(b, L, D).to(t), rn(b, L, D).to(t)) if gated else (None, None)
    c["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    c["h_in"], c["dh_out"] = (rn(b, D), rn(b, D)) if state else (None, None)
    c["dout"] = rn(b, L, D).to(t)
    return c


def to_gpu(c):
    """On the GPU, column slices of one buffer staying that."""
    out = {}
    for k, v in c.items():
        if isinstance(v, dict):
            out[k] = {n: w.cuda() for n, w in v.items()}
        elif v is None:
            out[k] = None
        else:
            out[k] = v.cuda()
    if not c["x"].is_contiguous():
        D = c["x"].shape[-1]
        out["x"], out["r"], out["i"] = torch.cat([out["x"], out["r"], out["i"]], -1).split(D, dim=-1)
    return out


def forward(bm, g, reverse=False, **kw):
    """(out, h_out, chunk_states) of one call; what is written is pre-filled with NaN."""
    b, L, D = g["x"].shape
    h_out = torch.full((b, D), float("nan"), device="cuda")
    states = torch.full((b, (L + bm.GLR_CHUNK - 1) // bm.GLR_CHUNK, D), float("nan"), device="cuda")
    out = torch.full((b, L, D), float("nan"), device="cuda", dtype=g["x"].dtype)
    got = bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], reverse=reverse, add=g["add"], z=g["z"],
                             lengths=g["lengths"], h_in=g["h_in"], h_out=h_out, chunk_states=states, out=out, **kw)
    assert got is out
    return out, h_out, states


def backward(bm, g, states, reverse=False, **kw):
    b, L, D = g["x"].shape
    dh_in = torch.full((b, D), float("nan"), device="cuda")
    res = bm.bimamba_glr_bwd(g["dout"], g["x"], g["r"], g["i"], g["params"], states, reverse=reverse, add=g["add"],
                             z=g["z"], lengths=g["lengths"], dh_out=g["dh_out"], dh_in=dh_in, **kw)
    return dict(res, dh_in=dh_in)


def close(got, want, tol, name, scale=None):
    """Within tol of the largest value (or of `scale`), plus half a step of a bf16 result."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    got = U.to_cpu64(got)
    assert got.shape == want.shape, name
    top = np.max(np.abs(want)) if scale is None else scale
    bad = ~(np.abs(got - want) <= half * np.abs(want) + tol * top + 1e-30)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want)):.3e} of {np.max(top):.3e}"


def check_forward(got, ref):
    out, h_out, states = got
    close(out, ref["out"], 2 * E, "out")
    close(h_out, ref["h_out"], E, "h_out")
    written = ~np.isnan(ref["chunk_states"])
    s = U.to_cpu64(states)
    assert np.isnan(s[~written]).all(), "chunk states past the length were written"
    if written.any():
        top = max(np.max(np.abs(ref["chunk_states"][written])), np.max(np.abs(ref["h_out"])), 1.0)
        assert np.max(np.abs(s[written] - ref["chunk_states"][written])) <= E * top


def check_backward(res, ref):
    for k in ("dx", "dr", "di", "dadd", "dz"):
        if k in res:
            close(res[k], ref[k], 3 * E, k)
    close(res["dh_in"], ref["dh_in"], 3 * E, "dh_in")
    for k in ("dA", "dr_bias", "di_bias"):
        if k in res:
            close(res[k], ref[k], 3 * E, k, scale=ref[k + "_abs"])


def oracle_of(c, reverse=False, grads=False):
    from oracle import glr as G
    kw = dict(dout=c["dout"], dh_out=c["dh_out"]) if grads else {}
    return G.glr(c["x"], c["r"], c["i"], c["params"], reverse=reverse, add=c["add"], z=c["z"], lengths=c["lengths"],
                 h_in=c["h_in"], **kw)
