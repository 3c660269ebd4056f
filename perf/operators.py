"""The cases that the gated linear recurrence and the block norm are measured on.

The gated linear recurrence is one direction of a mixer: gates from raw
activations, a decay per token and channel, a scan over the sequence, and the
sum with the other direction and the SiLU(z) gate where the caller has them.
The block norm is what stands between two blocks of a denoiser: the branch's
norm, its gate and the residual sum, then the next block's norm.

A case's "op" says which call it is: "glr" (the recurrence forward), "glr_train"
(forward, then backward), "norm" (the block norm forward), "norm_bwd" (its
backward).
"""
import math

import torch

own = False

_SIZES = {"bf16": 2, "fp32": 4}
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _glr(name, op, b, L, D, dtype, reverse=False, gated=False, state=False, ragged=False, fused=False):
    # reverse: right to left; gated: summed with the other direction's states and gated by silu(z);
    # state: a state enters and the final one is returned; ragged: lengths[b], one row empty;
    # fused: x, r, i are column slices of one projection's output
    c = {"op": op, "b": b, "L": L, "D": D, "dtype": dtype, "reverse": reverse, "gated": gated, "state": state,
         "ragged": ragged, "fused": fused}
    return dict(c, name=name) if name else c


def _norm(name, op, b, L, d, dtype, stream, rms=False, post=False, shared=False, res_scale=1.0):
    # dtype: of the branch and the norm's output; stream: of the residual stream; post: the branch is normed too;
    # shared: gate, gamma and beta are one vector for all rows instead of one per batch row (no beta with rms)
    c = {"op": op, "b": b, "L": L, "d": d, "dtype": dtype, "stream": stream, "rms": rms, "post": post,
         "shared": shared, "res_scale": res_scale}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of 16 requests, the state kept in place: latency
        _glr("glr_token", "glr", 16, 1, 4096, "bf16", state=True),
        # one denoising step on the active block of 16 requests, continuing from their states
        _glr("glr_block", "glr", 16, 32, 4096, "bf16", state=True, fused=True),
        # the layer's ordinary size
        _glr("glr_layer", "glr", 8, 2048, 4096, "bf16"),
        # one long sequence, the second direction: right to left, summed and gated
        _glr("glr_long_gated", "glr", 1, 65536, 4096, "bf16", reverse=True, gated=True),
        # a padded batch in fp32, one row empty, odd length
        _glr("glr_ragged_fp32", "glr", 5, 1537, 1920, "fp32", state=True, ragged=True),
        # a training step of one direction
        _glr("glr_train", "glr_train", 8, 2048, 4096, "bf16"),
        # a training step of the second direction on a padded batch, from one projection's output
        _glr("glr_train_ragged", "glr_train", 3, 4099, 1920, "bf16", reverse=True, gated=True, state=True, ragged=True,
             fused=True),
        # between two blocks while decoding 16 requests: latency
        _norm("norm_token", "norm", 16, 1, 2048, "bf16", "bf16"),
        # between two blocks of a denoiser, modulated per batch row
        _norm("norm_layer", "norm", 8, 2048, 2048, "bf16", "bf16"),
        # a long sequence with the residual stream in fp32, the branch normed before its gate
        _norm("norm_long_post", "norm", 1, 65536, 1920, "bf16", "fp32", rms=True, post=True, shared=True),
        # backward of the modulated form
        _norm("norm_bwd_layer", "norm_bwd", 8, 2048, 2048, "bf16", "bf16"),
        # backward with the branch normed, vectors shared by all rows, an odd number of tokens
        _norm("norm_bwd_post", "norm_bwd", 3, 2731, 1920, "bf16", "fp32", rms=True, post=True, shared=True,
              res_scale=0.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["glr", "glr", "glr_train", "norm", "norm_bwd"])
    cap = {"glr": 1 << 27, "glr_train": 1 << 25, "norm": 1 << 27, "norm_bwd": 1 << 26}[op]
    L = _log_int(rng, 1, 65536)
    b = _log_int(rng, 1, 32)
    # widths: whole multiples of eight as projections have them, and odd ones
    w = _log_int(rng, 24, 4096)
    if rng.random() < 0.7:
        w = max(8, w // 8 * 8)
    L = max(1, min(L, cap // (b * w)))
    dtype = "bf16" if rng.random() < 0.7 else "fp32"
    flag = lambda p=0.5: rng.random() < p  # noqa: E731
    if op.startswith("glr"):
        return _glr(None, op, b, L, w, dtype, flag(), flag(), flag(), flag(0.4), flag(0.3))
    stream = "fp32" if dtype == "fp32" or flag() else "bf16"
    return _norm(None, op, b, L, w, dtype, stream, flag(), flag(), flag(), rng.choice([1.0, 0.5, 1.25]))


def _lengths(case):
    """The rows' lengths of a case: the whole length first, then an empty row, then what a golden-section
    sequence gives, so that work() knows them too."""
    b, L = case["b"], case["L"]
    if not case["ragged"]:
        return [L] * b
    out = [1 + int((L - 1) * ((j * 0.6180339887498949) % 1.0)) for j in range(b)]
    out[0] = L
    if b > 1:
        out[1] = 0
    return out


def work(case):
    if case["op"].startswith("glr"):
        e, D = _SIZES[case["dtype"]], case["D"]
        used, all_ = sum(_lengths(case)) * D, case["b"] * case["L"] * D
        rows = case["b"] * D * 4
        gated, st = case["gated"], case["state"]
        by = (3 + 2 * gated) * used * e + all_ * e + 12 * D + 2 * st * rows
        fl = (30 + 8 * gated) * used
        if case["op"] == "glr_train":
            # the backward is a call of its own: its dout exists only after out has gone through the rest of the
            # network, so it reads the inputs again
            by += (4 + 2 * gated) * used * e + (3 + 2 * gated) * all_ * e + 24 * D + 2 * st * rows
            fl += (60 + 16 * gated) * used
        return {"bytes": by, "flops": fl}
    e, s = _SIZES[case["dtype"]], _SIZES[case["stream"]]
    n, vec = case["b"] * case["L"] * case["d"], (1 if case["shared"] else case["b"]) * case["d"] * 4
    vecs = (2 if case["rms"] else 3) * vec + case["post"] * case["d"] * 4
    if case["op"] == "norm":
        return {"bytes": n * (2 * s + 2 * e) + vecs, "flops": (12 + 6 * case["post"]) * n}
    return {"bytes": n * (3 * s + 3 * e) + 2 * vecs, "flops": (22 + 12 * case["post"]) * n}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = _TYPES[case["dtype"]]

    def rn(*shape, kind=torch.float32, scale=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).add_(mean).to(kind)

    s = dict(case)
    if case["op"].startswith("glr"):
        b, L, D = case["b"], case["L"], case["D"]
        if case["fused"]:
            s["x"], s["r"], s["i"] = rn(b, L, 3 * D, kind=t).split(D, dim=-1)
        else:
            s["x"], s["r"], s["i"] = (rn(b, L, D, kind=t) for _ in range(3))
        # the decay of a whole-open gate, exp(A), between about 0.45 and 0.99
        lo, hi = math.log(8e-3), math.log(8e-1)
        s["params"] = {"A": -torch.exp(torch.rand(D, generator=g, device="cuda") * (hi - lo) + lo),
                       "r_bias": torch.rand(D, generator=g, device="cuda") - 0.5,
                       "i_bias": torch.rand(D, generator=g, device="cuda") - 0.5}
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["add"] = rn(b, L, D, kind=t) if case["gated"] else None
        s["z"] = rn(b, L, D, kind=t) if case["gated"] else None
        s["h_in"] = rn(b, D) if case["state"] else None
        if case["op"] == "glr_train":
            s["dout"] = rn(b, L, D, kind=t)
            s["dh_out"] = rn(b, D) if case["state"] else None
        return s
    b, L, d = case["b"], case["L"], case["d"]
    ts, vb = _TYPES[case["stream"]], () if case["shared"] else (b,)
    s["u"] = rn(b, L, d, kind=t)
    s["gate"] = rn(*vb, d, scale=0.5)
    s["gamma"] = rn(*vb, d, scale=0.1, mean=1.0)
    s["beta"] = None if case["rms"] else rn(*vb, d, scale=0.1)
    s["post_w"] = rn(d, scale=0.1, mean=1.0) if case["post"] else None
    if case["op"] == "norm":
        s["x"] = rn(b, L, d, kind=ts)
        return s
    # what the forward left: the stored stream, and the mean and 1/sigma of its rows and of the branch's
    s["x_out"] = rn(b, L, d, kind=ts, mean=0.1)
    s["stats"] = torch.stack(_stats(s["x_out"].float(), case["rms"]) + _stats(s["u"].float(), case["rms"]), dim=-1)
    s["dy"], s["dx_out"] = rn(b, L, d, kind=t), rn(b, L, d, kind=ts)
    return s


def _stats(v, rms):
    """Mean (0 for the root-mean-square norm) and 1/sigma of each row."""
    mu = torch.zeros_like(v[..., 0]) if rms else v.mean(-1)
    return mu, torch.rsqrt(((v - mu[..., None]) ** 2).mean(-1) + 1e-5)


# ---------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _scan(a, b, h0):
    """h[s] = a[s] h[s-1] + b[s] over dim 1 from h0, by doubling: after each round every position holds the
    affine map of twice as many steps."""
    b = b.clone()
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], dim=1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], dim=1)
        k *= 2
    return b


def _glr_parts(s):
    """Everything in scan order, padded tokens as steps that keep the state (a = 1, b = 0)."""
    turn = (lambda v: v.flip(1)) if s["reverse"] else (lambda v: v)
    p, b, L = s["params"], s["b"], s["L"]
    x = turn(s["x"].float())
    rg = _sigmoid(turn(s["r"].float()) + p["r_bias"])
    ig = _sigmoid(turn(s["i"].float()) + p["i_bias"])
    la = p["A"] * rg
    a, beta = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    w = beta * ig * x
    keep = None
    if s["ragged"]:
        keep = turn(torch.arange(L, device=x.device)[None, :, None] < s["lengths"][:, None, None])
        a, w = torch.where(keep, a, torch.ones_like(a)), torch.where(keep, w, torch.zeros_like(w))
    return turn, keep, x, rg, ig, a, beta, w


def _plain_glr(s):
    turn, keep, x, rg, ig, a, beta, w = _glr_parts(s)
    t = s["x"].dtype
    h = _scan(a, w, s["h_in"])
    y = turn(h)
    if s["gated"]:
        z = s["z"].float()
        y = (y + s["add"].float()) * (z * _sigmoid(z))
    zero = lambda v: v if keep is None else torch.where(turn(keep), v, torch.zeros_like(v))  # noqa: E731
    out = {"out": zero(y).to(t)}
    if s["state"]:
        out["h_out"] = h[:, -1]
    if s["op"] == "glr":
        return out
    dh = turn(s["dout"].float())
    if s["gated"]:
        z, add, dout = turn(s["z"].float()), turn(s["add"].float()), dh
        sz = _sigmoid(z)
        out["dz"] = zero(turn(dout * (h + add) * (sz * (1.0 + z * (1.0 - sz))))).to(t)
        dh = dout * (z * sz)
        out["dadd"] = zero(turn(dh)).to(t)
    if keep is not None:
        dh = torch.where(keep, dh, torch.zeros_like(dh))
    G = _scan(torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1).flip(1), dh.flip(1), s["dh_out"]).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["h_in"] is None else s["h_in"][:, None], h[:, :-1]], dim=1)
    b2 = beta * beta
    dla = G * (a * before - torch.where(b2 > 0, a * a / b2, torch.zeros_like(b2)) * w)
    dr = s["params"]["A"] * dla * rg * (1.0 - rg)
    di = G * w * (1.0 - ig)
    dx = G * beta * ig
    if keep is not None:
        dr, di, dx, dla = (torch.where(keep, v, torch.zeros_like(v)) for v in (dr, di, dx, dla))
    total = lambda v: v.sum((0, 1), dtype=torch.float64).float()  # noqa: E731
    out.update(dx=turn(dx).to(t), dr=turn(dr).to(t), di=turn(di).to(t), dA=total(dla * rg), dr_bias=total(dr),
               di_bias=total(di))
    if s["state"]:
        out["dh_in"] = a[:, 0] * G[:, 0]
    return out


def _rows(v, case):
    """A vector per batch row, or one for all, as it multiplies [b, L, d]."""
    return v if case["shared"] else v[:, None, :]


def _plain_norm(s):
    x, u = s["x"].float(), s["u"].float()
    if s["post"]:
        mu, rs = _stats(u, s["rms"])
        u = (u - mu[..., None]) * rs[..., None] * s["post_w"]
    stored = (s["res_scale"] * x + _rows(s["gate"], s) * u).to(s["x"].dtype)
    v = stored.float()
    mu, rs = _stats(v, s["rms"])
    y = _rows(s["gamma"], s) * ((v - mu[..., None]) * rs[..., None])
    if s["beta"] is not None:
        y = y + _rows(s["beta"], s)
    return {"x_out": stored, "y": y.to(s["u"].dtype)}


def _through(dn, n, rs, rms):
    """The gradient of the rows behind n = (v - mean) rs from the gradient dn of n."""
    out = dn - n * (dn * n).mean(-1, keepdim=True)
    if not rms:
        out = out - dn.mean(-1, keepdim=True)
    return out * rs[..., None]


def _plain_norm_bwd(s):
    v, u, dy, dxo = (s[k].float() for k in ("x_out", "u", "dy", "dx_out"))
    mu, rs, mu_u, rs_u = s["stats"].unbind(-1)
    n = (v - mu[..., None]) * rs[..., None]
    dim = (0, 1) if s["shared"] else (1,)
    total = lambda q, over=dim: q.sum(over, dtype=torch.float64).float()  # noqa: E731
    d = dxo + _through(_rows(s["gamma"], s) * dy, n, rs, s["rms"])
    g = _rows(s["gate"], s) * d
    out = {"dx": (s["res_scale"] * d).to(s["x_out"].dtype), "dgamma": total(dy * n)}
    if s["beta"] is not None:
        out["dbeta"] = total(dy)
    if s["post"]:
        m = (u - mu_u[..., None]) * rs_u[..., None]
        out["dgate"] = total(d * (m * s["post_w"]))
        out["dpost_w"] = total(g * m, (0, 1))
        g = _through(g * s["post_w"], m, rs_u, s["rms"])
    else:
        out["dgate"] = total(d * u)
    out["du"] = g.to(s["u"].dtype)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own_glr(bm, s):
    b, L, D = s["b"], s["L"], s["D"]
    kw = dict(reverse=s["reverse"], add=s["add"], z=s["z"], lengths=s["lengths"])
    h_out = torch.empty(b, D, device="cuda") if s["state"] else None
    if s["op"] == "glr":
        out = {"out": bm.bimamba_glr_fwd(s["x"], s["r"], s["i"], s["params"], h_in=s["h_in"], h_out=h_out, **kw)}
        return dict(out, h_out=h_out) if s["state"] else out
    chunks = (L + bm.GLR_CHUNK - 1) // bm.GLR_CHUNK
    states = torch.empty(b, chunks, D, device="cuda")
    out = {"out": bm.bimamba_glr_fwd(s["x"], s["r"], s["i"], s["params"], h_in=s["h_in"], h_out=h_out,
                                     chunk_states=states, **kw)}
    dh_in = torch.empty(b, D, device="cuda") if s["state"] else None
    out.update(bm.bimamba_glr_bwd(s["dout"], s["x"], s["r"], s["i"], s["params"], states, dh_out=s["dh_out"],
                                  dh_in=dh_in, **kw))
    if s["state"]:
        out.update(h_out=h_out, dh_in=dh_in)
    return out


def _own_norm(bm, s):
    kw = dict(gate=s["gate"], post_w=s["post_w"], gamma=s["gamma"], res_scale=s["res_scale"], rms=s["rms"])
    if s["op"] == "norm":
        x_out, y = bm.bimamba_block_norm_fwd(s["x"], s["u"], beta=s["beta"], **kw)
        return {"x_out": x_out, "y": y}
    return bm.bimamba_block_norm_bwd(s["dy"], s["dx_out"], s["x_out"], s["stats"], s["u"],
                                     want_dbeta=s["beta"] is not None, **kw)


def run(state):
    if own:
        from bidirectional_mamba_denoiser_b200 import bimamba as bm
        return _own_glr(bm, state) if state["op"].startswith("glr") else _own_norm(bm, state)
    return {"glr": _plain_glr, "glr_train": _plain_glr, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[state["op"]](state)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definition, one step after another in 64 bits; the gradients of the recurrence by differentiating
    each step by hand, those of the norms through their rows' Jacobian."""
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"].startswith("glr"):
        return _exact_glr(case, f, {k: v.double() for k, v in s["params"].items()})
    return _exact_norm(case, f, s)


def _exact_glr(case, f, p):
    b, L, D = case["b"], case["L"], case["D"]
    dev = f["x"].device
    lens = f["lengths"].long() if case["ragged"] else torch.full((b,), L, device=dev)
    pos = torch.arange(L, device=dev)[None]
    inside = (pos < lens[:, None])[..., None]
    rg = torch.sigmoid(f["r"] + p["r_bias"]).masked_fill_(~inside, 0.0)   # a closed gate keeps the state
    ig = torch.sigmoid(f["i"] + p["i_bias"]).masked_fill_(~inside, 0.0)
    a = (p["A"] * rg).exp_()
    one_less = -torch.expm1(2.0 * p["A"] * rg)
    h = torch.zeros(b, D, dtype=torch.float64, device=dev) if f["h_in"] is None else f["h_in"].clone()
    add = one_less.sqrt().mul_(ig).mul_(f["x"])
    add.masked_fill_(~inside, 0.0)
    order = range(L - 1, -1, -1) if case["reverse"] else range(L)
    after = torch.empty_like(a)
    for t in order:
        h = torch.addcmul(add[:, t], a[:, t], h)
        after[:, t] = h
    out = {}
    if case["gated"]:
        sz = torch.sigmoid(f["z"])
        out["out"] = ((after + f["add"]) * f["z"] * sz).masked_fill_(~inside, 0.0)
    else:
        out["out"] = after.masked_fill(~inside, 0.0)
    if case["state"]:
        out["h_out"] = h
    if case["op"] == "glr":
        return out
    up = f["dout"].masked_fill(~inside, 0.0)
    if case["gated"]:
        out["dz"] = up * (after + f["add"]) * sz * (1.0 + f["z"] * (1.0 - sz))
        up = up * f["z"] * sz
        out["dadd"] = up
    q = torch.zeros(b, D, dtype=torch.float64, device=dev) if f["dh_out"] is None else f["dh_out"].clone()
    G = torch.empty_like(a)
    for t in reversed(order):
        q = q + up[:, t]
        G[:, t] = q
        q = q * a[:, t]
    first = torch.zeros(b, 1, D, dtype=torch.float64, device=dev) if f["h_in"] is None else f["h_in"][:, None]
    prev = torch.cat([after[:, 1:], first], 1) if case["reverse"] else torch.cat([first, after[:, :-1]], 1)
    root = one_less.sqrt()
    dla = G * (a * prev - torch.where(root > 0, a * a / root, torch.zeros_like(root)) * ig * f["x"])
    dla.masked_fill_(~inside, 0.0)
    drg = dla * p["A"]
    out["dx"] = (G * root * ig).masked_fill_(~inside, 0.0)
    out["dr"] = (drg * rg * (1.0 - rg)).masked_fill_(~inside, 0.0)
    out["di"] = (G * root * f["x"] * ig * (1.0 - ig)).masked_fill_(~inside, 0.0)
    out["dA"] = (dla * rg).sum((0, 1))
    out["dr_bias"], out["di_bias"] = out["dr"].sum((0, 1)), out["di"].sum((0, 1))
    if case["state"]:
        out["dh_in"] = q
    return out


def _exact_norm(case, f, s):
    spread = (lambda v: v) if case["shared"] else (lambda v: v.unsqueeze(1))
    center = (lambda v: v) if case["rms"] else (lambda v: v - v.mean(-1, keepdim=True))
    unit = lambda v: center(v) / (center(v).square().mean(-1, keepdim=True) + 1e-5).sqrt()  # noqa: E731
    u = f["u"]
    if case["op"] == "norm":
        un = unit(u) * f["post_w"] if case["post"] else u
        x_out = f["x"] * case["res_scale"] + un * spread(f["gate"])
        y = unit(x_out.to(s["x"].dtype).double()) * spread(f["gamma"])  # of the stream as it is stored
        return {"x_out": x_out, "y": y if f["beta"] is None else y + spread(f["beta"])}
    over = [0, 1] if case["shared"] else [1]

    def back(v, dn):
        c = center(v)
        sig = (c.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        return center(dn / sig - c * (c * dn).mean(-1, keepdim=True) / sig ** 3)

    d = f["dx_out"] + back(f["x_out"], f["dy"] * spread(f["gamma"]))
    g = d * spread(f["gate"])
    un = unit(u)
    out = {"dx": d * case["res_scale"], "dgamma": (f["dy"] * unit(f["x_out"])).sum(over)}
    if f["beta"] is not None:
        out["dbeta"] = f["dy"].sum(over)
    if case["post"]:
        out["dgate"] = (d * un * f["post_w"]).sum(over)
        out["dpost_w"] = (g * un).sum([0, 1])
        out["du"] = back(u, g * f["post_w"])
    else:
        out["dgate"], out["du"] = (d * u).sum(over), g
    return out
