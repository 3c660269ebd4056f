"""The gated linear recurrence on a B200 where a step forgets strongly: A down
to -64 with gates nearly open, so that a decay is anything down to e^-64.  What
carries a factor a has to keep its relative accuracy, channel by channel and
step by step; the whole tensor's largest value is no scale for it.

Bounds, fixed before the first run, from the roundings of a step, with e = 2^-22
(what ex2.approx, rcp.approx and rsqrt.approx are good to) and u = 2^-24.  For
gates whose argument stays below 14:
  rg    relative error R = e (1 + 6 (1 - rg)): the argument's error of at most
        20 u and ex2's reach rg only through 1 - rg
  a     its logarithm A rg is off by R + e of itself, so a by
        rho = e (2 + |A| rg (2 + 6 (1 - rg))) <= e (2 + 3.5 |A|), relative
  beta  6 e, ig 7 e, w = beta ig x 16 e, dh = dout silu(z) 16 e
  h     dH = M (rho am H + 16 e W + 2 u H) with H = max |h|, W = max |w|, am = max a
        over the channel and M = 1 / (1 - am); G the same with dh in w's place: dG
  v = h_{s-1} - (a / beta^2) w and dla = G a v:
        d(dla) = |G| a (dH + (rho + 28 e)(|h_{s-1}| + a |w| / beta^2)) + dG a |v| + 2 u |dla|
  dr = A dla rg (1 - rg): |A| rg (1 - rg) d(dla) + |dr| (R / (1 - rg) + R + 4 u)
A sum over n partial rows adds at most 64 + n / 32 terms one after another.
"""
import numpy as np
import pytest
import torch

from tests import glr_util as T
from tests import parity_util as U

pytestmark = pytest.mark.gpu

e, u = 2.0 ** -22, 2.0 ** -24


@pytest.fixture(scope="module")
def bm():
    from bidirectional_mamba_denoiser_b200 import bimamba
    return bimamba


def _case(b, L, D, dtype, seed, gated):
    c = T.case(b, L, D, dtype, seed=seed, gated=gated, state=True)
    c["params"]["A"] = torch.tensor([-8.0, -16.0, -24.0, -64.0]).repeat((D + 3) // 4)[:D].contiguous()
    c["params"]["r_bias"] += 4.0
    return c


def _bounds(c, ref, reverse):
    """Absolute bounds of out, dr, dA and dr_bias; [b, L, D] in fp64."""
    f = {k: v.double().numpy() for k, v in c.items() if torch.is_tensor(v)}
    p = {k: v.double().numpy() for k, v in c["params"].items()}
    turn = (lambda v: v[:, ::-1]) if reverse else (lambda v: v)
    rg, ig = 1 / (1 + np.exp(-turn(f["r"]) - p["r_bias"])), 1 / (1 + np.exp(-turn(f["i"]) - p["i_bias"]))
    assert np.max(np.abs(f["r"])) + 4.5 < 14 and np.max(np.abs(f["i"])) + 0.5 < 14
    A = np.abs(p["A"])
    a, beta = np.exp(-A * rg), np.sqrt(-np.expm1(-2 * A * rg))
    w = beta * ig * turn(f["x"])
    dh = turn(f["dout"])
    if c["z"] is not None:
        z = turn(f["z"])
        dh = dh * z / (1 + np.exp(-z))
    b, L, _ = a.shape
    h, G = np.empty_like(a), np.empty_like(a)
    s, q = f["h_in"], f["dh_out"]
    for t in range(L):
        s = a[:, t] * s + w[:, t]
        h[:, t] = s
    for t in range(L - 1, -1, -1):
        G[:, t] = q + dh[:, t]
        q = a[:, t] * G[:, t]
    prev = np.concatenate([f["h_in"][:, None], h[:, :-1]], 1)
    top = lambda v: np.max(np.abs(v), axis=(0, 1))  # noqa: E731
    am, H, Gm, rho = a.max(axis=(0, 1)), top(prev), top(G), e * (2 + 3.5 * A)
    H, Gm = np.maximum(H, top(h)), np.maximum(Gm, top(f["dh_out"][:, None]))
    dH = (rho * am * H + 16 * e * top(w) + 2 * u * H) / (1 - am)
    dG = (rho * am * Gm + 16 * e * top(dh) + 2 * u * Gm) / (1 - am)
    v = prev - a / beta ** 2 * w
    dla = G * a * v
    ddla = np.abs(G) * a * (dH + (rho + 28 * e) * (np.abs(prev) + a * np.abs(w) / beta ** 2)) + dG * a * np.abs(v) \
        + 2 * u * np.abs(dla)
    R, shut = e * (1 + 6 * (1 - rg)), 1 / (1 + np.exp(turn(f["r"]) + p["r_bias"]))  # 1 - rg
    dr = A * rg * shut * np.abs(dla)
    ddr = A * rg * shut * ddla + dr * (R / shut + R + 4 * u)
    sums = (64 + b * L / 64 / 32) * u
    assert np.allclose(np.abs(ref["dr"]), turn(dr), rtol=1e-6, atol=0)  # the same quantities as the oracle's
    return {"state": dH, "dr": turn(ddr), "dA": (rg * ddla + rg * np.abs(dla) * (R + sums)).sum((0, 1)),
            "dr_bias": (ddr + dr * sums).sum((0, 1))}


def _within(got, want, bound, name):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    off = np.abs(U.to_cpu64(got) - want)
    bad = ~(off <= half * np.abs(want) + bound + 1e-36)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(off / (bound + 1e-36)):.3g} bounds"


def _check(bm, c, reverse):
    g = T.to_gpu(c)
    ref = T.oracle_of(c, reverse, True)
    bound = _bounds(c, ref, reverse)
    out, h_out, states = T.forward(bm, g, reverse)
    T.check_forward((out, h_out, states), ref)
    res = T.backward(bm, g, states, reverse)
    T.check_backward(res, ref)
    _within(h_out, ref["h_out"], bound["state"], "h_out")
    if c["z"] is None:
        _within(out, ref["out"], bound["state"], "out")
    for k in ("dr", "dA", "dr_bias"):
        _within(res[k], ref[k], bound[k], k)
    assert bm.bimamba_device_error() == 0


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_of_strong_decays(bm, reverse, dtype, gated):
    _check(bm, _case(2, 300, 68, dtype, 1, gated), reverse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_of_strong_decays_by_maps(bm, dtype, gated):
    _check(bm, _case(10, 150, 4096, dtype, 2, gated), gated)


def _relative(got, want, bound, name):
    off = np.abs(U.to_cpu64(got) - want)
    bad = ~(off <= bound * np.abs(want) + 1e-36)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(off / np.abs(want)):.3e} of {np.max(bound):.3e}"


# (A, steps): products of decays down to about e^-65, in one warp's steps and over several tiles
@pytest.mark.parametrize("A,L", [(-8.0, 4), (-16.0, 3), (-24.0, 2), (-0.5, 120), (-0.3, 200)])
@pytest.mark.parametrize("reverse", [False, True])
def test_a_state_that_only_decays(bm, A, L, reverse):
    """x = 0 and a gradient of the last state alone: every state, its gradient and every dr is a product of decays,
    and each is right to its own size: rho and 2 u a step, and the factors beside them."""
    c = T.case(2, L, 70, "fp32", seed=3, state=True)
    c["x"] *= 0.0
    c["dout"] *= 0.0
    c["params"]["A"] = torch.full((70,), A)
    c["params"]["r_bias"] += 4.0
    g = T.to_gpu(c)
    ref = T.oracle_of(c, reverse, True)
    out, h_out, states = T.forward(bm, g, reverse)
    res = T.backward(bm, g, states, reverse)
    bound = L * (e * (2 + 3.5 * abs(A)) + 2 * u)
    _relative(out, ref["out"], bound, "out")
    _relative(h_out, ref["h_out"], bound, "h_out")
    _relative(res["dh_in"], ref["dh_in"], bound, "dh_in")
    _relative(res["dx"], ref["dx"], bound + 16 * e, "dx")
    rg = 1 / (1 + np.exp(-c["r"].double().numpy() - c["params"]["r_bias"].double().numpy()))
    _relative(res["dr"], ref["dr"], bound + 8 * e + e * (1 + 6 * (1 - rg)) / (1 - rg), "dr")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_with_infinite_parameters(bm, dtype, gated):
    """A = -inf forgets at every step: A e^(A rg) goes to 0, and with it the channel's dr and dA; a gate that is closed
    there keeps the state.  r_bias = inf opens and i_bias = -inf closes a gate.  In a padded batch, whose closed steps are no
    part of it.  (In fp64 -1e30 is as good as -inf, and leaves 0 times it 0.)"""
    c = T.case(3, 150, 16, dtype, seed=4, gated=gated, state=True, lengths=[150, 0, 77])
    c["params"]["A"][3] = c["params"]["A"][9] = -float("inf")
    c["params"]["r_bias"][5], c["params"]["i_bias"][7] = float("inf"), -float("inf")
    c["r"][:, 20:30, 9] = -float("inf")
    g = T.to_gpu(c)
    c["params"]["A"][3] = c["params"]["A"][9] = -1e30
    ref = T.oracle_of(c, False, True)
    fwd = T.forward(bm, g)
    T.check_forward(fwd, ref)
    res = T.backward(bm, g, fwd[2])
    T.check_backward(res, ref)
    for k in ("dr", "dA", "dr_bias"):
        assert bool((res[k][..., [3, 9]] == 0).all()), k
