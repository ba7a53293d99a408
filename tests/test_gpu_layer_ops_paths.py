"""The conv step at the sizes of real batches: several sequences in a workgroup."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd
from test_gpu_layer_ops import BF, F32, conv_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


# Four sequences to a workgroup from 512 workgroups on (of 1024 channels each).
@pytest.mark.parametrize("s,c,w,dtype,silu", [
    (2050, 1032, 4, BF, True), (1027, 2048, 3, F32, False), (2049, 40, 2, BF, True), (2053, 8, 1, F32, True),
    (263, 8200, 4, F32, True),
])
def test_conv_step_of_four_sequences_a_workgroup(s, c, w, dtype, silu):
    """A number of sequences that four does not divide, with fresh, unsaved, in-place and refused ones in every place."""
    log(f"conv step {s, c, w, dtype, silu}")
    assert -(-s // 4) * -(-c // 1024) >= 512
    i = conv_inputs(s, c, w, dtype, seed=s)
    slots = i["states"].shape[0]
    for at in range(4):
        i["read"][4 + at * 5] = -1                  # 4, 9, 14, 19: one in each place of a workgroup
        i["write"][24 + at * 5] = -1
        i["write"][44 + at * 5] = i["read"][44 + at * 5].clone()
        i["read"][64 + at * 5] = slots + at
        i["write"][84 + at * 5] = slots
    i["write"][s - 1] = slots + 9
    refused = [64, 69, 74, 79, 84, 89, 94, 99, s - 1]
    before = i["states"].clone()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((s, c), 3.0, dtype=dtype, device="cuda")
    ssd.causal_conv1d_step(i["x"], i["weight"], i["states"], i["read"], i["write"], bias=i["bias"], silu=silu, out=out,
                           error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == ssd.DATA_BAD_SLOT
    assert (out[refused] == 3).all()
    # every sequence at once: windows oldest first, the token last
    taken = torch.tensor([k for k in range(s) if k not in refused])
    x, old, rs, ws = i["x"].cpu()[taken], before.cpu(), i["read"].cpu().long()[taken], i["write"].cpu().long()[taken]
    window = torch.where((rs >= 0)[:, None, None], old[rs.clamp(min=0)], torch.zeros_like(old[:1]))
    want, bound = ref.conv_step(x, i["weight"].cpu(), window, i["bias"].cpu(), silu)
    log(f"  worst {ref.check(out.cpu()[taken], want, bound, 'out'):.3f} of the bound")
    new = old.clone()
    new[ws[ws >= 0]] = torch.cat([window, x[:, None]], 1)[ws >= 0, 1:]
    assert torch.equal(i["states"].cpu(), new)
