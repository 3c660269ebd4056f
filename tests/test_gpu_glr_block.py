"""The recurrence and the block norm together, as a denoiser block uses them:
norm -> projection -> both directions (the second summed and gated) -> output
projection -> gated residual sum and the next norm, forward and backward,
against the same block in torch's fp64 with its own autograd.

The projections are plain fp64 products on both sides (rounded to fp32 for the
kernels), so the difference is the kernels': the bounds of tests/glr_util.py and of
the block norm, times the number of operators a value passes (five).
"""
import pytest
import torch

from tests import glr_util as T

pytestmark = pytest.mark.gpu


def _norm(v, eps=1e-5):
    return (v - v.mean(-1, keepdim=True)) / (v.var(-1, unbiased=False, keepdim=True) + eps).sqrt()


def _scan(x, r, i, A, lengths, reverse):
    b, L, D = x.shape
    rows = []
    for k in range(b):
        n = int(lengths[k])
        h, hs = torch.zeros(D, dtype=torch.float64), [None] * L
        for t in (range(n - 1, -1, -1) if reverse else range(n)):
            la = A * torch.sigmoid(r[k, t])
            h = torch.exp(la) * h + torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i[k, t]) * x[k, t]
            hs[t] = h
        rows.append(torch.stack([torch.zeros(D, dtype=torch.float64) if v is None else v for v in hs]))
    return torch.stack(rows)


def test_block_forward_and_backward():
    from bidirectional_mamba_denoiser_b200 import bimamba as bm
    b, L, d, D = 2, 70, 24, 40
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    lengths = [70, 41]
    keep = (torch.arange(L)[None] < torch.tensor(lengths)[:, None])[..., None]
    leaf = {"x": rn(b, L, d), "gamma0": 1 + 0.1 * rn(b, d), "beta0": 0.1 * rn(b, d), "w_in": rn(6 * D, d) / d ** 0.5,
            "Af": -torch.rand(D, generator=g).double() * 0.5 - 0.05, "Ab": -torch.rand(D, generator=g).double() * 0.5 - 0.05,
            "w_out": rn(d, D) / D ** 0.5, "gate": rn(b, d), "gamma1": 1 + 0.1 * rn(b, d), "beta1": 0.1 * rn(b, d)}
    dy, dxo = rn(b, L, d), rn(b, L, d)
    leaf = {k: v.float().double() for k, v in leaf.items()}
    dy, dxo = dy.float().double(), dxo.float().double()

    # fp64 with autograd
    q = {k: v.clone().requires_grad_(True) for k, v in leaf.items()}
    n0 = _norm(q["x"]) * q["gamma0"][:, None] + q["beta0"][:, None]
    x, z, rf, fi, rb, bi = (n0 @ q["w_in"].T).split(D, dim=-1)
    hf = _scan(x, rf, fi, q["Af"], lengths, False)
    y = (hf + _scan(x, rb, bi, q["Ab"], lengths, True)) * torch.nn.functional.silu(z)
    y = torch.where(keep, y, torch.zeros_like(y))
    stream = q["x"] + q["gate"][:, None] * (y @ q["w_out"].T)
    out = _norm(stream) * q["gamma1"][:, None] + q["beta1"][:, None]
    ((out * dy).sum() + (stream * dxo).sum()).backward()

    # the framework's calls, in fp32 with the products in fp64
    f = {k: v.float().cuda() for k, v in leaf.items()}
    mm = lambda a, w: (a.double() @ w.double()).float()  # noqa: E731
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    st0, st1 = (torch.empty(b, L, 4, device="cuda") for _ in range(2))
    _, k0 = bm.bimamba_block_norm_fwd(f["x"], gamma=f["gamma0"], beta=f["beta0"], stats=st0)
    p = mm(k0, f["w_in"].T)
    x, z, rf, fi, rb, bi = p.split(D, dim=-1)
    sf, sb = (torch.empty(b, (L + bm.GLR_CHUNK - 1) // bm.GLR_CHUNK, D, device="cuda") for _ in range(2))
    kh = bm.bimamba_glr_fwd(x, rf, fi, {"A": f["Af"]}, lengths=lens, chunk_states=sf)
    back = dict(reverse=True, add=kh, z=z, lengths=lens)
    ky = bm.bimamba_glr_fwd(x, rb, bi, {"A": f["Ab"]}, chunk_states=sb, **back)
    ko = mm(ky, f["w_out"].T)
    ks, kout = bm.bimamba_block_norm_fwd(f["x"], ko, f["gate"], None, f["gamma1"], f["beta1"], stats=st1)
    dyk, dxk = dy.float().cuda(), dxo.float().cuda()
    r1 = bm.bimamba_block_norm_bwd(dyk, dxk, ks, st1, ko, f["gate"], None, f["gamma1"], want_dbeta=True)
    dky = mm(r1["du"], f["w_out"])
    gb = bm.bimamba_glr_bwd(dky, x, rb, bi, {"A": f["Ab"]}, sb, **back)
    dp = torch.empty_like(p)  # the projection's gradient, written in place by the forward direction's call
    gf = bm.bimamba_glr_bwd(gb["dadd"], x, rf, fi, {"A": f["Af"]}, sf, lengths=lens, dx=dp[..., :D],
                            dr=dp[..., 2 * D:3 * D], di=dp[..., 3 * D:4 * D])
    dp[..., :D] += gb["dx"]
    dp[..., D:2 * D], dp[..., 4 * D:5 * D], dp[..., 5 * D:] = gb["dz"], gb["dr"], gb["di"]
    r0 = bm.bimamba_block_norm_bwd(mm(dp, f["w_in"]), r1["dx"], f["x"], st0, None, None, None, f["gamma0"],
                                   want_dbeta=True)
    flat = lambda v: v.reshape(-1, v.shape[-1]).double()  # noqa: E731
    got = {"x": r0["dx"], "gamma0": r0["dgamma"], "beta0": r0["dbeta"], "w_in": flat(dp).T @ flat(k0),
           "Af": gf["dA"], "Ab": gb["dA"], "w_out": flat(r1["du"]).T @ flat(ky), "gate": r1["dgate"],
           "gamma1": r1["dgamma"], "beta1": r1["dbeta"]}
    torch.cuda.synchronize()
    assert torch.equal(gf["dx"][1, 41:], torch.zeros_like(gf["dx"][1, 41:]))
    tol = 5 * 3 * T.E
    for name, a, w in [("stream", ks, stream), ("out", kout, out)] + [(k, got[k], q[k].grad) for k in got]:
        a, w = a.double().cpu(), w.detach()
        assert (a - w).abs().max() <= tol * w.abs().max(), name
    assert bm.bimamba_device_error() == 0


def test_serving_a_block_bidirectionally():
    """An active block: the forward direction continues the cached state, the reverse sees the block alone."""
    from bidirectional_mamba_denoiser_b200 import bimamba as bm
    b, P, G, D = 2, 90, 32, 64
    c = T.case(b, P + G, D, "fp32", seed=2, gated=True)
    g = T.to_gpu(c)
    blk = slice(P, P + G)
    h = torch.zeros(b, D, device="cuda")
    bm.bimamba_glr_fwd(g["x"][:, :P], g["r"][:, :P], g["i"][:, :P], g["params"], h_out=h)
    cut = {k: g[k][:, blk] for k in ("x", "r", "i", "z")}
    hf = bm.bimamba_glr_fwd(cut["x"], cut["r"], cut["i"], g["params"], h_in=h)
    out = bm.bimamba_glr_fwd(cut["x"], cut["r"], cut["i"], g["params"], reverse=True, add=hf, z=cut["z"])
    torch.cuda.synchronize()
    import numpy as np
    from oracle import glr as O
    full = O.glr(c["x"], c["r"], c["i"], c["params"])["out"][:, blk]
    n = {k: c[k][:, blk] for k in ("x", "r", "i", "z")}
    want = O.glr(n["x"], n["r"], n["i"], c["params"], reverse=True, add=full, z=n["z"])["out"]
    assert np.max(np.abs(out.double().cpu().numpy() - want)) <= 3 * T.E * np.max(np.abs(want))
