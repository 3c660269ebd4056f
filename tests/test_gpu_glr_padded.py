"""Padded batches of the gated linear recurrence, its waits and its short calls
on a B200.  Bounds: tests/glr_util.py."""
import pytest
import torch

from tests import glr_util as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    from bidirectional_mamba_denoiser_b200 import bimamba
    return bimamba


def _check(bm, c, reverse):
    g = T.to_gpu(c)
    ref = T.oracle_of(c, reverse, True)
    fwd = T.forward(bm, g, reverse)
    T.check_forward(fwd, ref)
    T.check_backward(T.backward(bm, g, fwd[2], reverse), ref)
    assert bm.bimamba_device_error() == 0


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
def test_many_rows_of_any_length(bm, reverse, dtype, gated):
    gen = torch.Generator().manual_seed(1)
    lens = [int(v) for v in torch.randint(0, 701, (37,), generator=gen)]
    for k in (0, 5, 6, 36):
        lens[k] = 0
    lens[7] = 700
    _check(bm, T.case(37, 700, 66, dtype, seed=2, gated=gated, state=True, lengths=lens), reverse)


@pytest.mark.parametrize("lens", [[0, 0, 0], [64, 0, 1], [0, 63, 64], [5, 64, 0]])
def test_short_padded_rows(bm, lens):
    _check(bm, T.case(3, 64, 72, "bf16", seed=3, gated=True, state=True, lengths=lens), True)
    _check(bm, T.case(3, 64, 33, "fp32", seed=3, state=True, lengths=lens), False)


@pytest.mark.parametrize("only", [0, 2])
def test_one_row_has_tokens(bm, only):
    lens = [0, 0, 0]
    lens[only] = 500
    _check(bm, T.case(3, 500, 130, "bf16", seed=4, gated=True, lengths=lens), False)


def test_gaps_beside_rows_are_left_alone(bm):
    """Outputs that are column slices of wider rows: zeros behind a length, nothing between the slices."""
    lens = [150, 0, 70]
    c = T.case(3, 150, 40, "bf16", seed=5, state=True, lengths=lens)
    g = T.to_gpu(c)
    wide = torch.full((3, 150, 56), 7.0, device="cuda", dtype=torch.bfloat16)
    bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], lengths=g["lengths"], h_in=g["h_in"], out=wide[..., 8:48])
    T.close(wide[..., 8:48], T.oracle_of(c)["out"], 2 * T.E, "out")
    assert bool((wide[..., :8] == 7.0).all()) and bool((wide[..., 48:] == 7.0).all())
    for row, n in enumerate(lens):
        assert bool((wide[row, n:, 8:48] == 0).all())


def test_replayed_with_other_lengths(bm):
    """The lengths are read on the device: a captured call follows them."""
    c = T.case(4, 400, 64, "bf16", seed=6, gated=True, state=True, lengths=[400, 10, 0, 129])
    g = T.to_gpu(c)
    T.backward(bm, g, T.forward(bm, g)[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        fwd = T.forward(bm, g)
        res = T.backward(bm, g, fwd[2])
    for lens in ([400, 10, 0, 129], [0, 400, 399, 1], [0, 0, 0, 0], [400] * 4):
        g["lengths"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = T.oracle_of(dict(c, lengths=torch.tensor(lens)), False, True)
        T.check_forward(fwd, ref)
        T.check_backward(res, ref)


@pytest.mark.parametrize("L", [1, 64, 65, 128, 129])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_around_the_border_without_a_workspace(bm, L, dtype):
    c = T.case(5, L, 96, dtype, seed=L, state=True)
    g = T.to_gpu(c)
    h = g["h_in"].clone()
    out = bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], h_in=h, h_out=h)
    ref = T.oracle_of(c)
    T.close(out, ref["out"], 2 * T.E, "out")
    T.close(h, ref["h_out"], T.E, "h_out")


@pytest.mark.parametrize("k", ["x", "r", "i"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_channel(bm, k, what):
    c = T.case(1, 300, 128, "fp32", seed=8)
    g = T.to_gpu(c)
    clean = bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"])
    g[k][0, 140, 5] = what
    out = bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"])
    if k == "x" or what != what:
        assert not bool(torch.isfinite(out[0, 140:, 5]).any())
    else:  # an open or a closed gate
        assert bool(torch.isfinite(out[0, :, 5]).all())
    assert torch.equal(out[0, :140], clean[0, :140])
    out[0, :, 5] = clean[0, :, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_that_runs_out_is_reported(bm, backward):
    """With BIMAMBA_TEST_STARVE nothing is handed over: the waits end, the error word says so, and the next call is
    as ever."""
    c = T.case(2, 1000, 64, "bf16", seed=9, state=True)
    g = T.to_gpu(c)
    ref = T.oracle_of(c, False, True)
    fwd = T.forward(bm, g)
    assert bm.bimamba_device_error() == 0
    if backward:
        T.backward(bm, g, fwd[2], flags=bm.BIMAMBA_TEST_STARVE)
    else:
        T.forward(bm, g, flags=bm.BIMAMBA_TEST_STARVE)
    assert bm.bimamba_device_error() & 4
    assert bm.bimamba_device_error() == 0
    fwd = T.forward(bm, g)
    T.check_forward(fwd, ref)
    T.check_backward(T.backward(bm, g, fwd[2]), ref)


def test_infinite_parameters(bm):
    """A = -inf forgets at every step, r_bias = inf opens and i_bias = -inf closes a gate, in padded rows too."""
    c = T.case(3, 150, 16, "fp32", seed=10, state=True, lengths=[150, 0, 77])
    c["params"]["A"][3] = -float("inf")
    c["params"]["r_bias"][5] = float("inf")
    c["params"]["i_bias"][7] = -float("inf")
    T.check_forward(T.forward(bm, T.to_gpu(c)), T.oracle_of(c))
