"""The gated linear recurrence on a B200 where inputs come by tensor maps: chains
of many tiles that hand over states alone, and rows of one tile.  Sampled
channels against the oracle.  Bounds: tests/glr_util.py."""
import pytest
import torch

from tests import glr_util as T

pytestmark = pytest.mark.gpu
D = 4096
PICK = [0, 1, 62, 63, 64, 127, 2050, 4031, 4032, 4095]


@pytest.fixture(scope="module")
def bm():
    from bidirectional_mamba_denoiser_b200 import bimamba
    return bimamba


def _picked(c):
    sub = {k: (v[..., PICK] if torch.is_tensor(v) and v.dim() >= 2 else v) for k, v in c.items()}
    sub["params"] = {k: v[PICK] for k, v in c["params"].items()}
    return sub


def _check(bm, c, reverse):
    g = T.to_gpu(c)
    ref = T.oracle_of(_picked(c), reverse, True)
    fwd = T.forward(bm, g, reverse)
    T.check_forward(tuple(v[..., PICK] for v in fwd), ref)
    res = T.backward(bm, g, fwd[2], reverse)
    T.check_backward({k: v[..., PICK] for k, v in res.items()}, ref)
    assert bm.bimamba_device_error() == 0
    return g, fwd


# 11 tiles a chain in a bf16 forward, 22 in an fp32 one and in every backward; 8 x 64 chains are more than 1.5 times the
# blocks that stay, so a group is one tile
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
def test_long_chains(bm, reverse, dtype, gated):
    _check(bm, T.case(8, 1400, D, dtype, seed=1, gated=gated, state=True), reverse)


@pytest.mark.parametrize("L", [2, 20, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_one_tile(bm, L, dtype, reverse, gated):
    """4096 tiles, one a row and slab, without a ticket; the state in place as well, and the same bits."""
    c = T.case(64, L, D, dtype, seed=L, gated=gated, state=True, fused=gated)
    g, (out, h_out, _) = _check(bm, c, reverse)
    h = g["h_in"].clone()
    again = bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], reverse=reverse, add=g["add"], z=g["z"], h_in=h, h_out=h)
    assert torch.equal(again, out) and torch.equal(h, h_out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_padded_rows_of_one_tile(bm, dtype, reverse):
    gen = torch.Generator().manual_seed(3)
    lens = [int(v) for v in torch.randint(0, 41, (64,), generator=gen)]
    lens[0], lens[1], lens[63] = 40, 0, 0
    c = T.case(64, 40, D, dtype, seed=4, gated=True, state=True, lengths=lens)
    for row, n in enumerate(lens):
        for k in ("x", "r", "i", "add", "z", "dout"):
            c[k][row, n:] = float("nan")
    _check(bm, c, reverse)
