"""Limits of the gated linear recurrence that the host checks: the token stride, and the workspace that a short
forward call does not need."""
import ctypes

from bidirectional_mamba_denoiser_b200 import bimamba as bm

F = 0x7F0000000000


def _fwd(L, ts, ws=None):
    rows = lambda k: bm.Rows(F + (k << 20), 0, ts)  # noqa: E731
    none = bm.Rows(None, 0, 0)
    i = bm.GlrInputs(rows(0), rows(1), rows(2), none, none, None, bm.BIMAMBA_BF16)
    p = bm.GlrParams(F, None, None)
    out = bm.Rows(F + (9 << 20), 0, 32)
    # the rows' addresses are fake: every call here fails a check before anything is launched
    return bm.lib.bimamba_glr_fwd(ctypes.byref(i), ctypes.byref(p), None, ctypes.byref(out), F + 1, None, 1, L, 32, 0, ws,
                                  0, None)


def test_token_strides_of_many_tokens_are_bounded():
    assert _fwd(2, 0x20000000) == bm.BIMAMBA_ERR_UNSUPPORTED
    # within the limit, or a single token: on to the next check (h_out is misaligned)
    assert _fwd(2, 0x1fffffff) == bm.BIMAMBA_ERR_MISALIGNED
    assert _fwd(1, 1 << 40) == bm.BIMAMBA_ERR_MISALIGNED


def test_workspace_bytes_of_short_and_long_calls():
    short, long_ = bm.bimamba_glr_workspace_bytes(1, 64, 32), bm.bimamba_glr_workspace_bytes(1, 65536, 32)
    assert 0 < short < long_ < bm.bimamba_glr_workspace_bytes(1, 65536, 32, True)
