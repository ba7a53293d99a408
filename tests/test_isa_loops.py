"""Checks of the compiled gfx950 kernels of the selective scan, the conv1d and the group norm (CPU): no loop of a kernel,
whatever its depth, reads or writes scratch memory. Loops are the cycles of the control-flow graph, so every pass, the
gate and the joins between them count."""
import os
import shutil

import pytest

from isa_check import HIPCC, _functions, _split_blocks, kernel_asm

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")

# kernels of a source, and exponentials in the loops of each of its scans (16 states: 8 tokens x 4 of a lane's states)
KERNELS = {"ssd_selective.hip": 20 + 8 + 40, "ssd_conv1d.hip": 1, "ssd_norm.hip": 1}
EXPONENTIALS = 32


def looping_blocks(blocks, label_of):
    """Blocks from which some path leads back to them."""
    after = []
    for k, block in enumerate(blocks):
        last = block[-1][1]
        to = [label_of[last.split()[-1]]] if last.startswith(("s_branch", "s_cbranch")) else []
        if not last.startswith(("s_branch", "s_endpgm")) and k + 1 < len(blocks):
            to.append(k + 1)
        after.append(to)
    found = []
    for k in range(len(blocks)):
        seen, todo = set(), list(after[k])
        while todo:
            b = todo.pop()
            if b not in seen:
                seen.add(b)
                todo.extend(after[b])
        if k in seen:
            found.append(k)
    return found


def in_loops(body):
    """(line, instruction) of every block of a function that is part of a loop."""
    blocks, label_of = _split_blocks(body)
    return [(e[0], e[1]) for k in looping_blocks(blocks, label_of) for e in blocks[k]]


@pytest.mark.parametrize("src", KERNELS)
def test_no_loop_touches_scratch_memory(src):
    kernels = _functions(kernel_asm(src))
    assert len(kernels) >= KERNELS[src], f"{len(kernels)} kernels found in {src}"
    bad = [(name, e) for name, body in kernels for e in in_loops(body) if e[1].startswith("scratch_")]
    assert not bad, f"{len(bad)} accesses to scratch memory in loops, e.g. {bad[0][0]} line {bad[0][1][0]}: {bad[0][1][1]}"


def test_the_scans_exponentials_are_in_loops():
    """What the check above looks at holds the scans' work."""
    names = 0
    for name, body in _functions(kernel_asm("ssd_selective.hip")):
        if "ssd_selective_scan_kernel" in name or "ssd_selective_walk_kernel" in name:
            names += 1
            count = sum(t.startswith("v_exp_f32") for _, t in in_loops(body))
            assert count >= EXPONENTIALS, f"{name}: {count} exponentials in loops"
    assert names == 28


def test_the_loop_finder_on_planted_code():
    """A scratch access in an outer loop, one in its inner loop, and one behind both."""
    text = "\n".join([
        "_Zplanted:", "\ts_mov_b32 s0, 0", ".LBB0_1:", "\tscratch_store_dword off, v1, off", ".LBB0_2:",
        "\tscratch_load_dword v1, off, off", "\ts_cbranch_scc1 .LBB0_2", "\ts_nop 0", "\ts_cbranch_scc1 .LBB0_1",
        "\tscratch_load_dword v2, off, off", "\ts_endpgm", ".Lfunc_end0:"])
    (name, body), = _functions(text)
    found = [t for _, t in in_loops(body) if t.startswith("scratch_")]
    assert found == ["scratch_store_dword off, v1, off", "scratch_load_dword v1, off, off"]
