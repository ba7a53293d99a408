"""Checks of the compiled gfx950 kernels of the decode step's operators (CPU): no vector memory instruction reads an SGPR
that a VALU instruction wrote too few wait states before, no scratch memory, and the instructions that they are built
around are there."""
import os
import re
import shutil

import pytest

from isa_check import HIPCC, _functions, kernel_asm, kernel_resources, valu_sgpr_vmem_hazards

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")
SOURCES = ["ssd_gdn_step.hip", "ssd_attention.hip", "ssd_tables.hip", "ssd_addnorm.hip"]


@pytest.mark.parametrize("src", SOURCES)
def test_valu_sgpr_write_five_wait_states_before_vmem(src):
    bad = valu_sgpr_vmem_hazards(kernel_asm(src))
    assert not bad, f"{len(bad)} vector memory reads of a VALU-written SGPR too soon, e.g. line {bad[0][0]}: {bad[0][1]}"


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_memory(src):
    res = kernel_resources(kernel_asm(src))
    assert res, f"no kernels found in {src}"
    for name, r in res.items():
        assert r.get("private_segment_fixed_size", 0) == 0, f"{name}: scratch memory"


@pytest.mark.parametrize("src", SOURCES)
def test_no_packed_float32(src):
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", kernel_asm(src))


def test_attention_runs_on_the_matrix_cores_from_streamed_lines():
    bodies = {name: [e[1] for e in body] for name, body in _functions(kernel_asm("ssd_attention.hip"))
              if "20ssd_attention_kernel" in name}
    assert len(bodies) == 12, sorted(bodies)
    for name, body in bodies.items():
        op = "v_mfma_f32_16x16x4_f32" if "kernelIf" in name else "v_mfma_f32_16x16x32_bf16"
        assert sum(e.startswith(op) for e in body) >= 16, name
        streamed = sum(e.startswith("global_load_dwordx4") and " nt" in e for e in body)
        assert (streamed > 0) == ("Lb1E" in name), name
