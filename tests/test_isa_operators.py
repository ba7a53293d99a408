"""Checks of the compiled gfx950 kernels of the selective scan, the conv1d and the group norm (CPU): no vector memory
instruction reads an SGPR that a VALU instruction wrote too few wait states before, and no inner loop works from scratch
memory."""
import os
import re
import shutil

import pytest

from isa_check import HIPCC, kernel_asm, kernel_resources, valu_sgpr_vmem_hazards

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")
SOURCES = ["ssd_selective.hip", "ssd_conv1d.hip", "ssd_norm.hip"]


@pytest.mark.parametrize("src", SOURCES)
def test_valu_sgpr_write_five_wait_states_before_vmem(src):
    bad = valu_sgpr_vmem_hazards(kernel_asm(src))
    assert not bad, f"{len(bad)} vector memory reads of a VALU-written SGPR too soon, e.g. line {bad[0][0]}: {bad[0][1]}"


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_memory(src):
    """The segment scan keeps a few values of a sequence's last segment in scratch memory: written once before its loop,
    read once after it. Nothing else may use any."""
    res = kernel_resources(kernel_asm(src))
    assert res, f"no kernels found in {src}"
    for name, r in res.items():
        size = r.get("private_segment_fixed_size", 0)
        limit = 80 if "ssd_selective_scan_kernel" in name else 0
        assert size <= limit, f"{name}: {size} bytes of scratch memory"


def test_segment_scan_reads_scratch_in_no_hot_block():
    """Blocks that hold exponentials (the two passes, the gate) neither read nor write scratch memory."""
    text = kernel_asm("ssd_selective.hip")
    for body in re.findall(r"^(_ZN3ssd25ssd_selective_scan_kernel\w+):(.*?)s_endpgm", text, flags=re.S | re.M):
        for block in re.split(r"^\.LBB\w+:", body[1], flags=re.M)[1:]:
            if block.count("v_exp_f32") >= 8:
                assert "scratch_" not in block, f"{body[0]}: scratch memory beside the exponentials"
