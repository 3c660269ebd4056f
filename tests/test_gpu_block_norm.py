"""The block norm on a B200 against the fp64 oracle, through the C ABI.

Bounds, fixed before the first run: a row's mean and variance are fp32 sums of
d terms in a tree of depth log2(d) + the terms a thread adds in a row (32 at
most), so they carry at most 50 x 2^-24 of the sums of magnitudes; a normed
value multiplies that with a few roundings: 2^-24 x 64 = 4e-6 of the row's
largest, doubled where two norms follow one another and again through the
gradient's three terms: TOL = 1.6e-5 normwise.  Column sums over n rows add
2^-24 x (rows a segment adds in turn): the same bound of the sum of magnitudes.
A bf16 store adds half a step (2^-8 relative).  y, the statistics and the
gradients are compared with the oracle's for the stream as the kernel stored
it, whose rounding x_out's own bound covers.
"""
import numpy as np
import pytest
import torch

from oracle import glr as G
from tests import parity_util as U
from tests.glr_util import TYPES, close

pytestmark = pytest.mark.gpu
TOL = 1.6e-5


@pytest.fixture(scope="module")
def bm():
    from bidirectional_mamba_denoiser_b200 import bimamba
    return bimamba


def case(b, L, d, stream, dtype, seed, branch=True, post=False, gate=True, gamma=True, beta=True, gate_shared=False,
         gamma_shared=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gs, ms = (() if gate_shared else (b,)), (() if gamma_shared else (b,))
    v = {"x": (rn(b, L, d) + 0.5).to(TYPES[stream]), "u": (rn(b, L, d) - 0.3).to(TYPES[dtype]) if branch else None,
         "gate": rn(*gs, d) if gate and branch else None, "post_w": 1 + 0.1 * rn(d) if post and branch else None,
         "gamma": 1 + 0.1 * rn(*ms, d) if gamma else None, "beta": 0.1 * rn(*ms, d) if beta else None}
    return v, rn(b, L, d).to(TYPES[dtype]), rn(b, L, d).to(TYPES[stream])


def dev(v):
    return {k: (None if t is None else t.cuda()) for k, t in v.items()}


def _store(t):
    return (lambda v: torch.from_numpy(v).to(t).double().numpy()) if t == torch.bfloat16 else None


def check(bm, v, dy, dxo, res_scale=1.0, rms=False, ty=None):
    b, L, d = v["x"].shape
    g = dev(v)
    ty = ty or (v["u"].dtype if v["u"] is not None else dy.dtype)
    stats = torch.full((b, L, 4), float("nan"), device="cuda")
    x_out, y = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], g["post_w"], g["gamma"], g["beta"], res_scale,
                                         rms=rms, dtype=ty, stats=stats)
    torch.cuda.synchronize()
    want_x, _, _ = G.block_norm(**v, res_scale=res_scale, rms=rms)
    close(x_out, want_x, TOL, "x_out")
    # y and the statistics: of the stream as the kernel stored it
    stored = x_out.cpu()
    _, want_y, want_s = G.block_norm(stored, None, None, None, v["gamma"], v["beta"], rms=rms)
    close(y, want_y, TOL, "y")
    s = U.to_cpu64(stats)
    assert np.all(np.abs(s[..., :2] - want_s[..., :2]) <= TOL * np.maximum(1.0, np.abs(want_s[..., :2])))
    _, _, su = G.block_norm(v["x"], v["u"], v["gate"], v["post_w"], rms=rms)
    assert np.all(np.abs(s[..., 2:] - su[..., 2:]) <= TOL * np.maximum(1.0, np.abs(su[..., 2:])))
    res = bm.bimamba_block_norm_bwd(dy.cuda(), dxo.cuda(), x_out, stats, g["u"], g["gate"], g["post_w"], g["gamma"],
                                    res_scale, rms, want_dbeta=v["beta"] is not None,
                                    dbeta_shared=None if v["beta"] is None else v["beta"].dim() == 1)
    torch.cuda.synchronize()
    check_bwd(res, v, dy, dxo, stored, res_scale, rms)
    return x_out, y, stats, res


def check_bwd(res, v, dy, dxo, stored, res_scale, rms):
    shared = v["beta"] is not None and v["beta"].dim() == 1
    kw = dict(gate=v["gate"], post_w=v["post_w"], gamma=v["gamma"], res_scale=res_scale, rms=rms)
    ref = G.block_norm_bwd(dy, dxo, stored, v["u"], beta_shared=shared, **kw)
    n = (dy if dy is not None else dxo)
    n = n.shape[1] * (n.shape[0] if any(t is not None and t.dim() == 1 for t in (v["gate"], v["gamma"], v["beta"])) else 1)
    for k, t in res.items():
        # a sum of n products: the bound is of the sum of magnitudes, n times a typical product of two N(0, 1)'s and
        # the vectors' O(1) entries
        summed = k not in ("dx", "du")
        many = n if k != "dpost_w" else stored.shape[0] * stored.shape[1]
        # dx and du: the row's gradient is rs (dn - n mean(dn n) - mean(dn)), each term good to TOL of rs max|dn|; of
        # one or two columns n = +-1 and they cancel to eps / sigma^2 of that, so the bound is of the terms
        # dgate and dpost_w: one summand holds D times a factor, and D is such a row's gradient, so the worst row adds
        # TOL of its terms times that factor
        scale = max(np.max(np.abs(ref[k])), 2.0 * many + ref.get(k + "_term", 0.0) if summed else ref.get(k + "_terms", 0.0))
        close(t, ref[k], TOL, k, scale=scale)
    return ref


# one value to the widest, the borders of the warp form and odd widths
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 33, 64, 129, 256, 264, 513, 1000, 1024, 1025, 1032, 1920, 2049, 4096, 8200,
                               16384, 16383])
@pytest.mark.parametrize("rms", [False, True])
def test_widths(bm, d, rms):
    v, dy, dxo = case(2, 3, d, "fp32", "fp32", d, post=True)
    check(bm, v, dy, dxo, rms=rms)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_shared,gamma_shared", [(False, False), (True, True), (False, True)])
def test_forms(bm, types, rms, post, gate_shared, gamma_shared):
    v, dy, dxo = case(3, 37, 192, *types, 3, post=post, beta=not rms, gate_shared=gate_shared,
                      gamma_shared=gamma_shared)
    check(bm, v, dy, dxo, res_scale=0.5, rms=rms)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 17, 600, 1201])
def test_row_counts(bm, L):
    v, dy, dxo = case(2, L, 136, "bf16", "bf16", L, post=True, gamma_shared=True)
    check(bm, v, dy, dxo)


def test_many_batch_rows(bm):
    v, dy, dxo = case(700, 1, 72, "bf16", "bf16", 5)
    check(bm, v, dy, dxo)


@pytest.mark.parametrize("left_out", ["gate", "gamma", "beta"])
def test_vectors_left_out(bm, left_out):
    v, dy, dxo = case(2, 9, 80, "bf16", "bf16", 6, **{left_out: False})
    check(bm, v, dy, dxo)


def test_no_branch_matches_adaln(bm):
    """The norm alone is the framework's AdaLN: equal up to one bf16 step (the same formula, sums in another order)."""
    v, dy, dxo = case(2, 21, 256, "bf16", "bf16", 7, branch=False)
    x_out, y, _, _ = check(bm, v, dy, dxo)
    g = dev(v)
    a = bm.bimamba_adaln(g["x"], g["gamma"], g["beta"])
    assert torch.allclose(y.float(), a.float(), rtol=2.0 ** -7, atol=1e-6)
    assert bm.bimamba_block_norm_fwd(g["x"], None, gamma=g["gamma"])[0] is g["x"]


def test_no_branch_of_an_fp32_stream(bm):
    v, dy, dxo = case(2, 5, 96, "fp32", "bf16", 8, branch=False)
    check(bm, v, dy, dxo, res_scale=0.25, ty=torch.bfloat16)


def test_sum_alone_and_unused_outputs(bm):
    v, dy, dxo = case(2, 9, 96, "bf16", "bf16", 9, post=True)
    g = dev(v)
    b, L, d = v["x"].shape
    stats = torch.empty(b, L, 4, device="cuda")
    x_out, y = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], g["post_w"], norm=False, stats=stats)
    assert y is None
    close(x_out, G.block_norm(v["x"], v["u"], v["gate"], v["post_w"])[0], TOL, "x_out")
    res = bm.bimamba_block_norm_bwd(None, dxo.cuda(), x_out, stats, g["u"], g["gate"], g["post_w"])
    assert set(res) == {"dx", "du", "dgate", "dpost_w"}
    check_bwd(res, dict(v, gamma=None, beta=None), None, dxo, x_out.cpu(), 1.0, False)
    stats2 = torch.empty_like(stats)
    x_out, y = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], None, g["gamma"], g["beta"], stats=stats2)
    res = bm.bimamba_block_norm_bwd(dy.cuda(), None, x_out, stats2, g["u"], g["gate"], None, g["gamma"])
    assert set(res) == {"dx", "du", "dgate", "dgamma"}
    check_bwd(res, dict(v, post_w=None, beta=None), dy, None, x_out.cpu(), 1.0, False)


def test_in_place(bm):
    v, dy, dxo = case(2, 40, 1928, "bf16", "bf16", 10)
    g = dev(v)
    want_x, want_y, stats, want = check(bm, v, dy, dxo)
    x = g["x"].clone()
    got_x, got_y = bm.bimamba_block_norm_fwd(x, g["u"], g["gate"], None, g["gamma"], g["beta"], x_out=x)
    assert got_x is x and torch.equal(x, want_x) and torch.equal(got_y, want_y)
    dx = dxo.cuda()
    res = bm.bimamba_block_norm_bwd(dy.cuda(), dx, want_x, stats, g["u"], g["gate"], None, g["gamma"], dx=dx)
    assert res["dx"] is dx and torch.equal(dx, want["dx"]) and torch.equal(res["dgate"], want["dgate"])


def test_misaligned_rows_take_the_scalar_path(bm):
    """A view one element into its storage: 2-byte aligned only."""
    v, dy, dxo = case(2, 6, 64, "bf16", "bf16", 11, post=True)
    g = dev(v)
    want = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], g["post_w"], g["gamma"], g["beta"])
    shifted = torch.empty(g["u"].numel() + 1, device="cuda", dtype=torch.bfloat16)[1:].view_as(g["u"])
    shifted.copy_(g["u"])
    got = bm.bimamba_block_norm_fwd(g["x"], shifted, g["gate"], g["post_w"], g["gamma"], g["beta"])
    for p, q in zip(got, want):
        assert torch.allclose(p.float(), q.float(), rtol=2.0 ** -7, atol=1e-5)


def test_rows_far_from_zero(bm):
    """A mean 1000 times the spread: the centred sum of squares keeps the variance."""
    v, dy, dxo = case(1, 5, 512, "fp32", "fp32", 12, branch=False)
    v["x"] = v["x"] + 1000.0
    g = dev(v)
    stats = torch.empty(1, 5, 4, device="cuda")
    _, y = bm.bimamba_block_norm_fwd(g["x"], gamma=g["gamma"], beta=g["beta"], stats=stats)
    _, want, ws = G.block_norm(v["x"], gamma=v["gamma"], beta=v["beta"])
    # the mean is good to half a step of 1000 (3e-5) plus its sum's 2^-20 of 1000; y moves by as much over sigma
    close(y, want, 1e-3, "y")
    assert np.allclose(stats[..., 1].cpu().numpy(), ws[..., 1], rtol=1e-5)


def test_constant_and_zero_rows(bm):
    x = torch.zeros(1, 2, 64, device="cuda")
    x[0, 1] = 3.0
    _, y = bm.bimamba_block_norm_fwd(x, beta=torch.full((64,), 0.5, device="cuda"))
    assert bool((y == 0.5).all())


def test_repeatable_captured_and_on_a_stream(bm):
    v, dy, dxo = case(3, 500, 264, "fp32", "bf16", 13, post=True, gate_shared=True)
    g, gy, gx = dev(v), dy.cuda(), dxo.cuda()
    stats = torch.empty(3, 500, 4, device="cuda")

    def run(stream=None):
        xo, y = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], g["post_w"], g["gamma"], g["beta"], stats=stats,
                                          stream=stream)
        r = bm.bimamba_block_norm_bwd(gy, gx, xo, stats, g["u"], g["gate"], g["post_w"], g["gamma"], stream=stream)
        return [xo, y] + [r[k] for k in sorted(r)]

    first = run()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    second = run(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        third = run()
    graph.replay()
    torch.cuda.synchronize()
    for p, q, r in zip(first, second, third):
        assert torch.equal(p, q) and torch.equal(p, r)


def test_refuses(bm):
    v, dy, dxo = case(2, 4, 16, "bf16", "bf16", 14)
    g = dev(v)
    with pytest.raises(ValueError):
        bm.bimamba_block_norm_fwd(g["x"], g["u"][:, :3])
    with pytest.raises(ValueError):
        bm.bimamba_block_norm_fwd(g["x"], g["u"], gate=g["gate"][:1])
    with pytest.raises(TypeError):
        bm.bimamba_block_norm_fwd(g["x"], g["u"], gate=g["gate"].bfloat16())
    with pytest.raises(ValueError):
        bm.bimamba_block_norm_fwd(g["x"].transpose(1, 2), None)
    with pytest.raises(ValueError):
        bm.bimamba_block_norm_bwd(None, None, g["x"], torch.empty(2, 4, 4, device="cuda"))
    with pytest.raises(bm.BimambaError) as e:
        bm.bimamba_block_norm_fwd(g["x"], g["u"].float())
    assert e.value.status == bm.BIMAMBA_ERR_UNSUPPORTED
    with pytest.raises(bm.BimambaError) as e:
        bm.bimamba_block_norm_fwd(g["x"], None, gate=g["gate"])
    assert e.value.status == bm.BIMAMBA_ERR_INVALID_ARG
    with pytest.raises(bm.BimambaError) as e:
        bm.bimamba_block_norm_fwd(torch.empty(1, 1, 16385, device="cuda"))
    assert e.value.status == bm.BIMAMBA_ERR_UNSUPPORTED
