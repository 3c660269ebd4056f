"""fp64 oracle of the gated linear recurrence and of the block norm (test
infrastructure; only the test suite and ``__graft_entry__.smoke()`` may use
it).  Plain numpy in double precision, one step after another, written from
the formulas; shares no code with the CUDA library.

Gated linear recurrence, per batch row and channel over the row's tokens in
scan order (reverse: last token first):
  rg = sigmoid(r + r_bias), ig = sigmoid(i + i_bias), a = exp(A rg),
  h <- a h + sqrt(1 - a^2) ig x,   out = (h + add) silu(z)
Block norm, per token row:
  x_out = res_scale x + gate N(u) post_w,   y = gamma N(x_out) + beta
("DiffuMamba: High-Throughput Diffusion LMs with Mamba Backbone", App. A.1
Eq. (10)-(12)).  The gradients are the chain rule through the same steps.
"""
from __future__ import annotations

import numpy as np


def _f64(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().to("cpu").double().numpy()
    return np.asarray(t, dtype=np.float64)


def _sig(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _rows_of(x, lengths):
    b, L, _ = x.shape
    return [L] * b if lengths is None else [int(min(max(n, 0), L)) for n in np.asarray(lengths)]


def glr(x, r, i, params, reverse=False, add=None, z=None, lengths=None, h_in=None, dout=None, dh_out=None, chunk=64):
    """Forward; with dout also the gradients.  Returns a dict: out, h_out,
    chunk_states [b, ceil(L/chunk), D] (NaN where no step starts) and, with
    dout, dx, dr, di, dA, dr_bias, di_bias, dh_in, dadd, dz, and the sums of the
    magnitudes behind dA, dr_bias, di_bias (dA_abs, ...)."""
    x, r, i, add, z, h_in, dout, dh_out = map(_f64, (x, r, i, add, z, h_in, dout, dh_out))
    A = _f64(params["A"])
    rb = _f64(params["r_bias"]) if params.get("r_bias") is not None else 0.0
    ib = _f64(params["i_bias"]) if params.get("i_bias") is not None else 0.0
    b, L, D = x.shape
    res = {"out": np.zeros((b, L, D)), "h_out": np.zeros((b, D)),
           "chunk_states": np.full((b, (L + chunk - 1) // chunk, D), np.nan)}
    if dout is not None:
        for k in ("dx", "dr", "di", "dadd", "dz"):
            res[k] = np.zeros((b, L, D))
        for k in ("dA", "dr_bias", "di_bias", "dA_abs"):
            res[k] = np.zeros(D)
        res["dh_in"] = np.zeros((b, D))
    for row, n in enumerate(_rows_of(x, lengths)):
        order = range(n - 1, -1, -1) if reverse else range(n)
        h = np.zeros(D) if h_in is None else h_in[row].copy()
        before = {}
        for s, t in enumerate(order):
            if s % chunk == 0:
                res["chunk_states"][row, s // chunk] = h
            rg, ig = _sig(r[row, t] + rb), _sig(i[row, t] + ib)
            a = np.exp(A * rg)
            before[t] = h
            h = a * h + np.sqrt(-np.expm1(2 * A * rg)) * ig * x[row, t]
            y = h if add is None else h + add[row, t]
            res["out"][row, t] = y if z is None else y * z[row, t] * _sig(z[row, t])
        res["h_out"][row] = h
        if dout is None:
            continue
        q = np.zeros(D) if dh_out is None else dh_out[row].copy()  # gradient of the state after step t
        for t in reversed(order):
            rg, ig = _sig(r[row, t] + rb), _sig(i[row, t] + ib)
            a, beta = np.exp(A * rg), np.sqrt(-np.expm1(2 * A * rg))
            dh = dout[row, t]
            if z is not None:
                h = a * before[t] + beta * ig * x[row, t] + (0.0 if add is None else add[row, t])
                sz = _sig(z[row, t])
                res["dz"][row, t] = dh * h * (sz + z[row, t] * sz * (1 - sz))
                dh = dh * z[row, t] * sz
            res["dadd"][row, t] = dh
            q = q + dh
            dbeta = q * ig * x[row, t]
            dig = q * beta * x[row, t]
            # beta = sqrt(1 - a^2): d beta / d a = -a / beta, taken as 0 where beta is 0
            with np.errstate(divide="ignore", invalid="ignore"):
                dda = q * before[t] + np.where(beta > 0, -a / beta, 0.0) * dbeta
            drg = dda * a * A
            res["dA"] += dda * a * rg
            res["dA_abs"] += np.abs(dda * a * rg)
            res["dx"][row, t] = q * beta * ig
            res["dr"][row, t] = drg * rg * (1 - rg)
            res["di"][row, t] = dig * ig * (1 - ig)
            q = q * a
        res["dh_in"][row] = q
    if dout is not None:
        for k in ("r", "i"):
            res[f"d{k}_bias"], res[f"d{k}_bias_abs"] = res[f"d{k}"].sum((0, 1)), np.abs(res[f"d{k}"]).sum((0, 1))
    return res


def _per_row(v, b):
    return None if v is None else (np.broadcast_to(v, (b,) + v.shape) if v.ndim == 1 else v)[:, None, :]


def _norm(v, eps, rms):
    """(normed, mean, 1/sigma) of the rows."""
    mu = np.zeros(v.shape[:-1] + (1,)) if rms else v.mean(-1, keepdims=True)
    rs = 1.0 / np.sqrt(((v - mu) ** 2).mean(-1, keepdims=True) + eps)
    return (v - mu) * rs, mu, rs


def block_norm(x, u=None, gate=None, post_w=None, gamma=None, beta=None, res_scale=1.0, eps=1e-5, rms=False,
               store=None):
    """Returns (x_out, y, stats).  `store` rounds x_out as the stream's type does."""
    x, u, gate, post_w, gamma, beta = map(_f64, (x, u, gate, post_w, gamma, beta))
    b = x.shape[0]
    x_out = res_scale * x
    one, zero = np.ones(x.shape[:-1] + (1,)), np.zeros(x.shape[:-1] + (1,))
    mu_u, rs_u = zero, one
    if u is not None:
        un = u
        if post_w is not None:
            un, mu_u, rs_u = _norm(u, eps, rms)
            un = un * post_w
        x_out = x_out + (un if gate is None else _per_row(gate, b) * un)
    if store is not None:
        x_out = store(x_out)
    y, mu, rs = _norm(x_out, eps, rms)
    if gamma is not None:
        y = y * _per_row(gamma, b)
    if beta is not None:
        y = y + _per_row(beta, b)
    return x_out, y, np.concatenate([mu, rs, mu_u, rs_u], axis=-1)


def block_norm_bwd(dy, dx_out, x_out, u=None, gate=None, post_w=None, gamma=None, res_scale=1.0, eps=1e-5, rms=False,
                   beta_shared=False):
    """Gradients for the stored x_out, through each row's Jacobian of v / sigma.
    "dx_terms", "du_terms": the largest term whose sum dx (du) is -- a row's
    Jacobian subtracts projections, so the sum may cancel far below them."""
    dy, dx_out, x_out, u = map(_f64, (dy, dx_out, x_out, u))
    gate, post_w, gamma = map(_f64, (gate, post_w, gamma))
    b = x_out.shape[0]

    def back(v, dn):
        n, _, rs = _norm(v, eps, rms)
        c = n / rs
        dv = dn * rs - c * rs ** 3 * (dn * c).mean(-1, keepdims=True)
        return dv if rms else dv - dv.mean(-1, keepdims=True)

    def total(v, like_shared):
        return v.sum((0, 1)) if like_shared else v.sum(1)

    res = {}
    d = np.zeros_like(x_out) if dx_out is None else dx_out
    if dy is not None:
        n = _norm(x_out, eps, rms)[0]
        d = d + back(x_out, dy if gamma is None else dy * _per_row(gamma, b))
        shared = beta_shared if gamma is None else gamma.ndim == 1
        res["dgamma"], res["dbeta"] = total(dy * n, shared), total(dy, shared)
        res["dx_terms"] = np.max(np.abs(res_scale * (0.0 if dx_out is None else dx_out))) + abs(res_scale) * np.max(
            np.abs(dy if gamma is None else dy * _per_row(gamma, b)) * _norm(x_out, eps, rms)[2])
    res["dx"] = res_scale * d
    if u is not None:
        g = d if gate is None else d * _per_row(gate, b)
        un = u
        if post_w is not None:
            m = _norm(u, eps, rms)[0]
            res["dpost_w"] = (g * m).sum((0, 1))
            un = m * post_w
            res["du_terms"] = np.max(np.abs(g * post_w) * _norm(u, eps, rms)[2])
            g = back(u, g * post_w)
        if gate is not None:
            res["dgate"] = total(d * un, gate.ndim == 1)
        # the largest summand of dgate or dpost_w that the terms of D alone would make
        terms = res.get("dx_terms", np.max(np.abs(res["dx"]))) / abs(res_scale)
        res["dgate_term"] = terms * np.max(np.abs(un))
        res["dpost_w_term"] = terms * (1.0 if gate is None else np.max(np.abs(gate))) * np.max(
            np.abs(un if post_w is None else m))
        res["du"] = g
    return res
