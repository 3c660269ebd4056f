"""The gated linear recurrence on a B200 at sizes where every block has several
tiles and inputs come by tensor maps.  Bounds: tests/glr_util.py."""
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
@pytest.mark.parametrize("D", [4096, 4104])
def test_many_tiles(bm, reverse, dtype, gated, D):
    _check(bm, T.case(10, 150, D, dtype, seed=1, gated=gated, state=True, fused=gated), reverse)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_tiles_of_a_padded_batch(bm, reverse, dtype):
    gen = torch.Generator().manual_seed(2)
    lens = [int(v) for v in torch.randint(0, 201, (12,), generator=gen)]
    lens[3] = lens[11] = 0
    lens[4] = 200
    c = T.case(12, 200, 4104, dtype, seed=3, gated=True, state=True, lengths=lens)
    for row, n in enumerate(lens):
        for k in ("x", "r", "i", "add", "z", "dout"):
            c[k][row, n:] = float("nan")
    _check(bm, c, reverse)


def test_add_alone(bm):
    c = T.case(10, 150, 4096, "bf16", seed=4, gated=True)
    c["z"] = None
    _check(bm, c, True)


def test_z_alone(bm):
    c = T.case(10, 150, 4096, "bf16", seed=5, gated=True)
    c["add"] = None
    _check(bm, c, False)


def test_shared_rows_are_copied_without_a_map(bm):
    """Rows that the batch shares (stride 0)."""
    c = T.case(10, 150, 4096, "bf16", seed=6)
    c["r"] = c["r"][:1].expand(10, -1, -1)
    g = T.to_gpu(dict(c, r=c["r"].contiguous()))
    g["r"] = g["r"][:1].expand(10, -1, -1)
    fwd = T.forward(bm, g)
    ref = T.oracle_of(c, False, True)
    T.check_forward(fwd, ref)
    T.check_backward(T.backward(bm, g, fwd[2]), ref)


def test_token_major_layout_and_repeatable(bm):
    """[L, b, D] storage, twice the same bits, and from a captured graph."""
    c = T.case(10, 150, 4096, "bf16", seed=7, gated=True, state=True)
    g = T.to_gpu(c)
    for k in ("x", "r", "i", "add", "z", "dout"):
        g[k] = g[k].transpose(0, 1).contiguous().transpose(0, 1)
    first = T.forward(bm, g, True)
    grads = T.backward(bm, g, first[2], True)
    ref = T.oracle_of(c, True, True)
    T.check_forward(first, ref)
    T.check_backward(grads, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        again = T.forward(bm, g, True)
        more = T.backward(bm, g, again[2], True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    assert all(torch.equal(grads[k], more[k]) for k in grads)
