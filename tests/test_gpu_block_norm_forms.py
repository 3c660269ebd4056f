"""The block norm's forms on a B200: rows copied ahead (256 to 8192 columns in
whole eights), packed rows (odd and narrow widths), and the plain one, at the
borders between them, against the fp64 oracle.  Bounds: tests/test_gpu_block_norm.py."""
import pytest
import torch

from tests.test_gpu_block_norm import bm, case, check, dev  # noqa: F401

pytestmark = pytest.mark.gpu
PAIRS = [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")]


@pytest.mark.parametrize("d", [256, 264, 504, 512, 520, 1928, 4096, 4104, 8192])
@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("post", [False, True])
def test_copied_rows(bm, d, types, post):  # noqa: F811
    v, dy, dxo = case(2, 45, d, *types, d, post=post, gamma_shared=post)
    check(bm, v, dy, dxo, rms=d % 16 == 8)


@pytest.mark.parametrize("d", [3, 24, 57, 96, 130, 249, 250, 255, 514, 1001, 2050, 4093])
@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("post", [False, True])
def test_packed_rows(bm, d, types, post):  # noqa: F811
    v, dy, dxo = case(2, 45, d, *types, d, post=post, gate_shared=post)
    check(bm, v, dy, dxo, rms=d % 4 == 1)


@pytest.mark.parametrize("d", [33, 88, 129, 352])
def test_many_tiles_a_block(bm, d):  # noqa: F811
    v, dy, dxo = case(1, 9001, d, "bf16", "bf16", d, post=True, gate_shared=True, gamma_shared=True)
    check(bm, v, dy, dxo)


@pytest.mark.parametrize("d", [130, 264, 77])
@pytest.mark.parametrize("shared", [False, True])
def test_batch_rows_of_a_few_tokens(bm, d, shared):  # noqa: F811
    v, dy, dxo = case(40, 3, d, "fp32", "bf16", d, gate_shared=shared, gamma_shared=shared)
    check(bm, v, dy, dxo)


@pytest.mark.parametrize("d", [131, 98, 520])
def test_in_place_and_nothing_beside(bm, d):  # noqa: F811
    """In place, inside a larger buffer: the same values, and not a byte before or behind."""
    v, dy, dxo = case(2, 40, d, "bf16", "bf16", d)
    g = dev(v)
    want_x, want_y, stats, want = check(bm, v, dy, dxo)
    n = 2 * 40 * d
    store = [torch.full((n + 128,), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    x, y, dx = (s[64:64 + n].view(2, 40, d) for s in store)
    x.copy_(v["x"])
    dx.copy_(dxo)
    bm.bimamba_block_norm_fwd(x, g["u"], g["gate"], None, g["gamma"], g["beta"], x_out=x, y=y)
    res = bm.bimamba_block_norm_bwd(dy.cuda(), dx, x, stats, g["u"], g["gate"], None, g["gamma"], dx=dx)
    assert torch.equal(x, want_x) and torch.equal(y, want_y) and torch.equal(dx, want["dx"])
    for k in ("du", "dgate", "dgamma"):
        assert torch.equal(res[k], want[k]), k
    for s in store:
        assert bool((s[:64] == 7.0).all()) and bool((s[64 + n:] == 7.0).all())


@pytest.mark.parametrize("d", [64, 129, 264, 1024])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_bad_row_stays_alone(bm, d, what):  # noqa: F811
    v, _, _ = case(2, 50, d, "fp32", "bf16", d, post=True)
    g = dev(v)
    kw = dict(gate=g["gate"], post_w=g["post_w"], gamma=g["gamma"], beta=g["beta"])
    clean = bm.bimamba_block_norm_fwd(g["x"], g["u"], **kw)
    g["u"][1, 7, d // 2] = what
    bad = bm.bimamba_block_norm_fwd(g["x"], g["u"], **kw)
    for p, q in zip(clean, bad):
        assert not bool(torch.isfinite(q[1, 7]).all())
        q[1, 7] = p[1, 7]
        assert torch.equal(p, q)


def test_odd_rows_of_a_misaligned_view(bm):  # noqa: F811
    """Bytes that no 16-byte access can use: the plain form, the same bounds."""
    v, dy, dxo = case(2, 20, 129, "fp32", "fp32", 4)
    store = torch.empty(v["u"].numel() + 1, device="cuda")
    shifted = store[1:].view_as(v["u"])
    shifted.copy_(v["u"])
    g = dev(v)
    want = bm.bimamba_block_norm_fwd(g["x"], g["u"], g["gate"], None, g["gamma"], g["beta"])
    got = bm.bimamba_block_norm_fwd(g["x"], shifted, g["gate"], None, g["gamma"], g["beta"])
    for p, q in zip(want, got):
        # both within 1.6e-5 of the row's largest (an N(0, 1) row of 129, below 8)
        assert torch.allclose(p, q, rtol=0, atol=2 * 1.6e-5 * 8)
