"""A rule of the operators' kernels that their sources show (CPU only)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_routed_sqrt_b200", "csrc")


@pytest.mark.parametrize("name", ["mxfp4.cuh", "mxfp4_product.cuh", "combine.cuh", "scored_router.cuh", "scan.cuh"])
def test_kernels_launched_ahead_use_no_read_only_loads(name):
    """These kernels are resident while the kernel before them writes their inputs, so the read-only path, which is
    for data that nothing writes during the kernel's life, is closed to them."""
    src = open(os.path.join(CSRC, name)).read()
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)
    assert re.findall(r"\.nc\b|__ldg|__restrict__|ld_stream_\w+|tex\w+\(", code) == []
