"""bimamba_device_error waits for all of the device's work: a call on a stream
of its own, which the legacy stream does not wait for, is reported as well."""
import pytest
import torch

from tests import glr_util as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reset", [False, True])
def test_a_call_still_running_on_a_side_stream_is_reported(reset):
    from bidirectional_mamba_denoiser_b200 import bimamba as bm
    g = T.to_gpu(T.case(2, 1000, 64, "bf16", seed=1))
    torch.cuda.synchronize()
    assert bm.bimamba_device_error() == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some 20 ms: the call behind it has not begun when the word is read
        # nothing is handed over, so a wait runs out after 0.1 ms
        bm.bimamba_glr_fwd(g["x"], g["r"], g["i"], g["params"], flags=bm.BIMAMBA_TEST_STARVE)
    assert bm.bimamba_device_error(reset) == 4
    torch.cuda.synchronize()
    assert bm.bimamba_device_error() == (0 if reset else 4)
    assert bm.bimamba_device_error() == 0
