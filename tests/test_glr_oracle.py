"""The oracle of the gated linear recurrence and of the block norm, pinned on
the CPU: closed forms, invariants, and gradients against central differences
of the forward (step 1e-6, so the difference is good to about 1e-9 relative)."""
import numpy as np
import pytest
import torch

from oracle import glr as G
from tests import glr_util as T


def test_constant_gates_give_the_geometric_series():
    D, L = 3, 40
    A, r, i, x = -0.5, 0.3, -0.2, 1.7
    full = lambda v: np.full((1, L, D), v)  # noqa: E731
    res = G.glr(full(x), full(r), full(i), {"A": np.full(D, A)}, h_in=np.full((1, D), 2.0))
    rg, ig = 1 / (1 + np.exp(-r)), 1 / (1 + np.exp(-i))
    a = np.exp(A * rg)
    n = np.arange(1, L + 1)
    want = 2.0 * a ** n + np.sqrt(1 - a * a) * ig * x * (1 - a ** n) / (1 - a)
    assert np.allclose(res["out"][0, :, 0], want, rtol=1e-12)
    assert np.allclose(res["h_out"], want[-1], rtol=1e-12)


def test_reverse_is_the_flipped_forward():
    c = T.case(2, 17, 5, seed=1, gated=True, state=True)
    f = {k: (v.flip(1) if k in ("x", "r", "i", "add", "z", "dout") else v) for k, v in c.items()}
    a, b = T.oracle_of(c, True, True), T.oracle_of(f, False, True)
    for k in ("out", "dx", "dr", "di", "dadd", "dz"):
        assert np.allclose(a[k], b[k][:, ::-1], rtol=1e-12, atol=1e-14), k
    for k in ("h_out", "dA", "dh_in"):
        assert np.allclose(a[k], b[k], rtol=1e-12), k


@pytest.mark.parametrize("reverse", [False, True])
def test_padded_rows_are_rows_of_their_own(reverse):
    c = T.case(3, 12, 4, seed=2, state=True, lengths=[12, 0, 7])
    full = T.oracle_of(c, reverse, True)
    assert np.all(full["out"][1] == 0) and np.all(full["dx"][2, 7:] == 0)
    assert np.array_equal(full["h_out"][1], c["h_in"][1].double().numpy())
    row = {k: (v[2:3, :7] if k in ("x", "r", "i", "dout") else v) for k, v in c.items()}
    row.update(h_in=c["h_in"][2:3], dh_out=c["dh_out"][2:3], lengths=None)
    own = T.oracle_of(row, reverse, True)
    assert np.allclose(own["out"][0], full["out"][2, :7]) and np.allclose(own["dh_in"][0], full["dh_in"][2])


def _differences(f, v, want, picks, rng):
    """Central differences of the scalar f at some entries of v against want."""
    flat = v.reshape(-1)
    for e in rng.choice(flat.size, min(picks, flat.size), replace=False):
        at, step = flat[e], 1e-6
        flat[e] = at + step
        up = f()
        flat[e] = at - step
        down = f()
        flat[e] = at
        assert (up - down) / (2 * step) == pytest.approx(want.reshape(-1)[e], rel=2e-6, abs=2e-7)


@pytest.mark.parametrize("reverse,gated,ragged", [(False, False, False), (True, True, True), (False, True, True)])
def test_recurrence_gradients_against_differences(reverse, gated, ragged):
    rng = np.random.default_rng(3)
    c = T.case(2, 9, 3, seed=3, gated=gated, state=True, lengths=[9, 4] if ragged else None)
    n = {k: v.double().numpy() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in c.items()}
    n["params"] = {k: v.double().numpy() for k, v in c["params"].items()}
    ref = G.glr(n["x"], n["r"], n["i"], n["params"], reverse, n["add"], n["z"], n["lengths"], n["h_in"], n["dout"],
                n["dh_out"])

    def f():
        o = G.glr(n["x"], n["r"], n["i"], n["params"], reverse, n["add"], n["z"], n["lengths"], n["h_in"])
        return float((o["out"] * n["dout"]).sum() + (o["h_out"] * n["dh_out"]).sum())

    pairs = [("x", "dx"), ("r", "dr"), ("i", "di"), ("h_in", "dh_in")] + ([("add", "dadd"), ("z", "dz")] if gated else [])
    for k, d in pairs:
        _differences(f, n[k], ref[d], 12, rng)
    for k in ("A", "r_bias", "i_bias"):
        _differences(f, n["params"][k], ref["d" + k], 3, rng)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_block_norm_gradients_against_differences(rms, post, shared):
    rng = np.random.default_rng(4)
    b, L, d = 2, 3, 6
    rn = lambda *s: rng.standard_normal(s)  # noqa: E731
    vec = (lambda: rn(d)) if shared else (lambda: rn(b, d))
    v = {"x": rn(b, L, d), "u": rn(b, L, d), "gate": vec(), "gamma": vec(), "beta": vec(),
         "post_w": rn(d) if post else None}
    dy, dxo = rn(b, L, d), rn(b, L, d)
    x_out, _, _ = G.block_norm(**v, res_scale=0.7, rms=rms)
    ref = G.block_norm_bwd(dy, dxo, x_out, v["u"], v["gate"], v["post_w"], v["gamma"], 0.7, rms=rms)

    def f():
        xo, y, _ = G.block_norm(**v, res_scale=0.7, rms=rms)
        return float((xo * dxo).sum() + (y * dy).sum())

    for k in v:
        if v[k] is not None:
            _differences(f, v[k], ref["d" + k], 12, rng)


def test_block_norm_without_a_branch_is_the_layer_norm():
    from oracle import proj
    rng = np.random.default_rng(5)
    x, g, be = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 8)), rng.standard_normal((2, 8))
    _, y, stats = G.block_norm(x, gamma=g, beta=be)
    assert np.allclose(y, proj.adaln(x, g, be), rtol=1e-12)
    assert np.allclose(stats[..., 0], x.mean(-1)) and np.all(stats[..., 2] == 0) and np.all(stats[..., 3] == 1)
