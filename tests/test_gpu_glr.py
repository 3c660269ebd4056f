"""The gated linear recurrence on a B200 against the fp64 oracle, through the
C ABI.  Bounds: tests/glr_util.py."""
import numpy as np
import pytest
import torch

from tests import glr_util as T
from tests import parity_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    from bidirectional_mamba_denoiser_b200 import bimamba
    return bimamba


def _check(bm, c, reverse):
    g = T.to_gpu(c)
    ref = T.oracle_of(c, reverse, True)
    fwd = T.forward(bm, g, reverse)
    torch.cuda.synchronize()
    T.check_forward(fwd, ref)
    res = T.backward(bm, g, fwd[2], reverse)
    torch.cuda.synchronize()
    T.check_backward(res, ref)
    assert bm.bimamba_device_error() == 0


# one token to several tiles, the borders of every tile and chunk among them
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lengths(bm, L, dtype):
    _check(bm, T.case(2, L, 66, dtype, seed=L, state=True), False)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 63, 64, 65, 127, 128, 130, 200])
@pytest.mark.parametrize("reverse", [False, True])
def test_widths(bm, D, reverse):
    _check(bm, T.case(2, 150, D, "bf16" if D % 2 else "fp32", seed=D, gated=D % 4 < 2, state=True), reverse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("fused", [False, True])
def test_forms(bm, dtype, reverse, gated, state, fused):
    _check(bm, T.case(3, 333, 72, dtype, seed=5, gated=gated, state=state, fused=fused), reverse)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [68, 33])
def test_padded_batch(bm, reverse, dtype, D):
    """Lengths of none, one, all, ends inside a tile and on its border, and out of range (clamped)."""
    lens = [300, 0, 1, 64, 65, 128, 129, 256, 17, 1000, -3]
    _check(bm, T.case(len(lens), 300, D, dtype, seed=6, gated=True, state=True, lengths=lens), reverse)


def test_all_rows_empty(bm):
    _check(bm, T.case(2, 200, 40, "bf16", seed=7, gated=True, state=True, lengths=[0, 0]), True)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), torch.finfo(torch.float32).min])
def test_padding_is_never_read(bm, reverse, what):
    lens = [200, 0, 63, 130]
    c = T.case(4, 200, 64, "bf16", seed=8, gated=True, state=True, lengths=lens)
    clean = T.oracle_of(c, reverse, True)
    for row, n in enumerate(lens):
        for k in ("x", "r", "i", "add", "z", "dout"):
            c[k][row, n:] = what
    g = T.to_gpu(c)
    fwd = T.forward(bm, g, reverse)
    res = T.backward(bm, g, fwd[2], reverse)
    torch.cuda.synchronize()
    T.check_forward(fwd, clean)
    T.check_backward(res, clean)
    for row, n in enumerate(lens):
        for v in (fwd[0], res["dx"], res["dr"], res["di"], res["dadd"], res["dz"]):
            assert bool((v[row, n:] == 0).all())


def test_add_or_z_alone(bm):
    for drop in ("add", "z"):
        c = T.case(2, 140, 48, "bf16", seed=9, gated=True)
        c[drop] = None
        _check(bm, c, True)


def test_without_biases(bm):
    c = T.case(2, 100, 34, "fp32", seed=10, bias=False)
    _check(bm, c, False)
    g = T.to_gpu(c)
    assert set(T.backward(bm, g, T.forward(bm, g)[2])) == {"dx", "dr", "di", "dA", "dh_in"}


def test_closed_and_open_gates(bm):
    """Gates at both ends: r = -inf keeps the state exactly, i = -inf adds nothing, r = +inf decays by exp(A); and
    A = 0 keeps the state with beta = 0, whose derivative is taken as 0."""
    c = T.case(1, 130, 8, "fp32", seed=11, state=True, bias=False)
    c["r"][..., 0], c["i"][..., 1], c["r"][..., 2], c["r"][..., 3] = -float("inf"), -float("inf"), float("inf"), 90.0
    c["r"][..., 4], c["i"][..., 5] = -60.0, 60.0
    c["params"]["A"][6] = 0.0
    g = T.to_gpu(c)
    out, h_out, states = T.forward(bm, g)
    res = T.backward(bm, g, states)
    torch.cuda.synchronize()
    ref = T.oracle_of(c, False, True)
    T.check_forward((out, h_out, states), ref)
    assert torch.equal(h_out[:, 0], g["h_in"][:, 0]) and torch.equal(h_out[:, 6], g["h_in"][:, 6])
    for k in ("dx", "dr", "di", "dA", "dh_in"):
        assert bool(torch.isfinite(res[k]).all()), k
        T.close(res[k], ref[k], 3 * T.E, k, scale=ref["dA_abs"].max() if k == "dA" else None)
    assert bool((res["dr"][..., [0, 6]] == 0).all())


def test_large_inputs_stay_finite(bm):
    c = T.case(2, 150, 40, "fp32", seed=12, gated=True, state=True)
    for k in ("r", "i", "z"):
        c[k] *= 40.0
    c["x"] *= 1e4
    _check(bm, c, False)


def test_transposed_layout_and_grads_in_one_buffer(bm):
    """[L, b, D] storage in, and dx, dr, di written as column slices of one buffer."""
    c = T.case(3, 150, 40, "bf16", seed=13, gated=True, state=True)
    g = T.to_gpu(c)
    ref = T.oracle_of(c, True, True)
    for k in ("x", "r", "i", "z", "dout"):
        g[k] = g[k].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(150, 3, 40, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    h_out, states = torch.empty(3, 40, device="cuda"), torch.empty(3, 3, 40, device="cuda")
    kw = dict(reverse=True, add=g["add"], z=g["z"])
    bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], h_in=g["h_in"], h_out=h_out, chunk_states=states, out=out,
                       **kw)
    buf = torch.full((3, 150, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    dx, dr, di = buf[..., :40], buf[..., 40:80], buf[..., 80:120]
    dh_in = torch.empty(3, 40, device="cuda")
    res = bm.bimamba_glr_bwd(g["dout"], g["x"], g["r"], g["i"], g["params"], states, dh_out=g["dh_out"], dh_in=dh_in,
                             dx=dx, dr=dr, di=di, **kw)
    torch.cuda.synchronize()
    T.check_forward((out, h_out, states), ref)
    T.check_backward(dict(res, dh_in=dh_in), ref)
    assert bool((buf[..., 120:] == 7.0).all())


def test_odd_strides_and_offsets(bm):
    """Rows that start at odd elements and have odd strides (no paired access is possible)."""
    c = T.case(2, 90, 20, "bf16", seed=14, state=True)
    g = T.to_gpu(c)
    for k in ("x", "r", "i", "dout"):
        buf = torch.full((2, 90, 23), float("nan"), device="cuda", dtype=torch.bfloat16)
        buf[..., 1:21] = g[k]
        g[k] = buf[..., 1:21]
    out = torch.full((2, 90, 21), 5.0, device="cuda", dtype=torch.bfloat16)
    h_out, states = torch.empty(2, 20, device="cuda"), torch.empty(2, 2, 20, device="cuda")
    bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], h_in=g["h_in"], h_out=h_out, chunk_states=states,
                       out=out[..., 1:])
    res = T.backward(bm, g, states)
    torch.cuda.synchronize()
    ref = T.oracle_of(c, False, True)
    T.check_forward((out[..., 1:], h_out, states), ref)
    T.check_backward(res, ref)
    assert bool((out[..., 0] == 5.0).all())


def test_broadcast_inputs(bm):
    """Rows shared by the batch (stride 0) are read as they are; their gradient is per row."""
    c = T.case(3, 70, 24, "fp32", seed=15)
    for k in ("x", "r", "i"):
        c[k] = c[k][:1].expand(3, -1, -1)
    g = T.to_gpu({k: (v if k not in ("x", "r", "i") else v.contiguous()) for k, v in c.items()})
    ref = T.oracle_of(c, False, True)
    for k in ("x", "r", "i"):
        g[k] = g[k][:1].expand(3, -1, -1)
    fwd = T.forward(bm, g)
    T.check_forward(fwd, ref)
    T.check_backward(T.backward(bm, g, fwd[2]), ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_token_by_token(bm, dtype):
    """One token at a time with the state in place is the whole sequence."""
    c = T.case(4, 20, 130, dtype, seed=16, state=True)
    g = T.to_gpu(c)
    whole, h_out, _ = T.forward(bm, g)
    h = g["h_in"].clone()
    for t in range(20):
        y = bm.bimamba_glr_fwd(g["x"][:, t:t + 1], g["r"][:, t:t + 1], g["i"][:, t:t + 1], g["params"], h_in=h, h_out=h)
        half = 2.0 ** -7 if dtype == "bf16" else 4 * T.E   # two roundings of nearly the same value
        assert torch.allclose(y[:, 0].float(), whole[:, t].float(), rtol=half, atol=4 * T.E)
    assert torch.allclose(h, h_out, rtol=2 * T.E, atol=2 * T.E)


@pytest.mark.parametrize("cut", [1, 64, 130, 500])
def test_a_sequence_in_two_calls(bm, cut):
    c = T.case(2, 600, 64, "bf16", seed=17, state=True)
    g = T.to_gpu(c)
    ref = T.oracle_of(c)
    h = g["h_in"].clone()
    parts = [bm.bimamba_glr_fwd(g["x"][:, s], g["r"][:, s], g["i"][:, s], g["params"], h_in=h, h_out=h)
             for s in (slice(0, cut), slice(cut, 600))]
    torch.cuda.synchronize()
    T.close(torch.cat(parts, 1), ref["out"], 2 * T.E, "out")
    T.close(h, ref["h_out"], T.E, "h_out")


def test_long_sequence(bm):
    """Many tiles in a row; sampled channels against the oracle."""
    L, D = 20000, 256
    c = T.case(1, L, D, "bf16", seed=18, gated=True, state=True)
    g = T.to_gpu(c)
    for reverse in (False, True):
        out, h_out, states = T.forward(bm, g, reverse)
        res = T.backward(bm, g, states, reverse)
        torch.cuda.synchronize()
        pick = [0, 1, 63, 64, 130, 255]
        sub = {k: (v[..., pick] if torch.is_tensor(v) and v.dim() >= 2 else v) for k, v in c.items()}
        sub["params"] = {k: v[pick] for k, v in c["params"].items()}
        ref = T.oracle_of(sub, reverse, True)
        T.check_forward((out[..., pick], h_out[..., pick], states[..., pick]), ref)
        T.check_backward({k: v[..., pick] for k, v in res.items()}, ref)
    assert bm.bimamba_device_error() == 0


def test_offsets_past_32_bits(bm):
    """More than 2^32 bytes and 2^31 elements of output: constant inputs shared by all tokens, so the state follows
    the geometric series wherever the row lies."""
    L, D = 540000, 4096
    assert L * D > 2 ** 31
    one = torch.ones(1, 1, D, device="cuda", dtype=torch.bfloat16)
    x, r, i = one.expand(1, L, D), (one * 0.5).expand(1, L, D), (one * -0.25).expand(1, L, D)
    A = torch.full((D,), -0.3, device="cuda")
    for reverse in (False, True):
        out = bm.bimamba_glr_fwd(x, r, i, {"A": A}, reverse=reverse)
        torch.cuda.synchronize()
        rg, ig = 1 / (1 + np.exp(-0.5)), 1 / (1 + np.exp(0.25))
        a = np.exp(-0.3 * rg)
        drive = np.sqrt(1 - a * a) * ig
        for s in (0, 1, 5, 1000, L // 2, L - 2, L - 1):
            want = drive * (1 - a ** (s + 1)) / (1 - a)
            got = out[0, L - 1 - s if reverse else s].double().cpu().numpy()
            assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2 * T.E) * want), s
        del out


def test_runs_are_bitwise_repeatable(bm):
    c = T.case(3, 2000, 136, "bf16", seed=19, gated=True, state=True, lengths=[2000, 1999, 700])
    g = T.to_gpu(c)
    first = None
    for _ in range(4):
        fwd = T.forward(bm, g, True)
        res = T.backward(bm, g, fwd[2], True)
        now = [torch.nan_to_num(v) for v in fwd] + [res[k] for k in sorted(res)]
        if first is not None:
            assert all(torch.equal(p, q) for p, q in zip(first, now))
        first = now


def test_captured_and_replayed_with_new_inputs(bm):
    """Forward and backward in one graph, replayed on changed inputs, while an eager call runs between."""
    c = T.case(2, 700, 64, "bf16", seed=20, gated=True, state=True)
    g = T.to_gpu(c)
    T.backward(bm, g, T.forward(bm, g)[2])
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fwd = T.forward(bm, g)
        res = T.backward(bm, g, fwd[2])
    for seed in (21, 22):
        c2 = T.case(2, 700, 64, "bf16", seed=seed, gated=True, state=True)
        c2["params"] = c["params"]
        for k in ("x", "r", "i", "add", "z", "dout", "h_in", "dh_out"):
            g[k].copy_(c2[k])
        eager = T.forward(bm, g)[0]
        graph.replay()
        torch.cuda.synchronize()
        ref = T.oracle_of(c2, False, True)
        T.check_forward(fwd, ref)
        T.check_backward(res, ref)
        assert torch.equal(eager, fwd[0])


def test_two_calls_at_once(bm):
    """Overlapping calls on two streams, each with its own workspace."""
    cs = [T.case(2, 3000, 128, "bf16", seed=s, state=True) for s in (23, 24)]
    gs = [T.to_gpu(c) for c in cs]
    want = [T.forward(bm, g) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for g, s in zip(gs, streams):
            s.wait_stream(torch.cuda.current_stream())
            h = torch.empty(2, 128, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            got.append((bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], h_in=g["h_in"], h_out=h, stream=s), h))
    torch.cuda.synchronize()
    for k, (o, h) in enumerate(got):
        assert torch.equal(o, want[k % 2][0]) and torch.equal(h, want[k % 2][1])


def test_refuses_overlapping_output_rows(bm):
    c = T.to_gpu(T.case(2, 10, 8, "fp32", seed=25))
    for bad in (torch.empty(2, 1, 8, device="cuda").expand(2, 10, 8), torch.empty(10, 8, device="cuda").expand(2, 10, 8)):
        with pytest.raises(bm.BimambaError) as e:
            bm.bimamba_glr_fwd(c["x"], c["r"], c["i"], c["params"], out=bad)
        assert e.value.status == bm.BIMAMBA_ERR_INVALID_ARG


def test_refuses_mismatched_tensors(bm):
    g = T.to_gpu(T.case(2, 10, 8, "fp32", seed=26, state=True))
    x, r, i, p = g["x"], g["r"], g["i"], g["params"]
    bad = [dict(r=r[:, :9]), dict(i=i.bfloat16()), dict(add=x.cpu()), dict(h_in=g["h_in"].double()),
           dict(lengths=torch.tensor([10, 10], device="cuda")), dict(params={"A": p["A"][:4].contiguous()}),
           dict(chunk_states=torch.empty(2, 2, 8, device="cuda")), dict(x=x.transpose(1, 2))]
    for kw in bad:
        a = dict(dict(x=x, r=r, i=i, params=p), **kw)
        with pytest.raises((ValueError, TypeError)):
            bm.bimamba_glr_fwd(a.pop("x"), a.pop("r"), a.pop("i"), a.pop("params"), **a)
