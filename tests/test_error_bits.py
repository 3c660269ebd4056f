"""The bits of the device error word: those that the kernels set are those that the header names, one a cause."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bidirectional_mamba_denoiser_b200", "csrc")


def test_the_header_names_every_bit_that_a_kernel_sets():
    bits = {}
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for k, v in re.findall(r"constexpr unsigned (k\w*Err\w+) = (\d+)u;", f.read()):
                bits[k] = int(v)
    assert len(bits) >= 3 and len(set(bits.values())) == len(bits)
    assert all(v & (v - 1) == 0 for v in bits.values())
    with open(os.path.join(ROOT, "include", "bimamba.h")) as f:
        doc = re.search(r"/\*([^/]*?)\*/\s*int bimamba_device_error\(", f.read(), re.S).group(1)
    named = {int(v) for v in re.findall(r"bit (\d+)", doc)}
    assert named == {v.bit_length() - 1 for v in bits.values()}
