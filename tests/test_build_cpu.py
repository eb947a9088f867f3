"""CPU checks of the built library's own symbols."""
import re
import shutil
import subprocess

import pytest

from expert_routed_grouped_amd import moe


@pytest.mark.parametrize("kernel", ["decode_route_gate_up_kernel", "decode_layer_kernel"])
def test_resident_workgroups_are_counted_per_kernel_instance(kernel):
    """The instances of a persistent kernel share one pointer type but not their registers: how many workgroups fit on the
    device is remembered for each of them."""
    if shutil.which("nm") is None:
        pytest.skip("no nm here")
    names = subprocess.run(["nm", "-j", moe.LIB_PATH], capture_output=True, text=True, check=True).stdout.split()
    stubs = [s for s in names if re.search(r"__device_stub__" + kernel, s)]
    kept = [s for s in names if re.search(r"resident_blocks.*" + kernel + r".*5cache$", s)]
    assert len(stubs) > 1 and len(kept) == len(stubs)
