"""The conv step and the group norm at the sizes of real batches: several sequences in a workgroup of the conv step, and
teams of every size and vector width of the norm that go on from row to row."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd
from test_gpu_layer_ops import BF, F32, conv_inputs, norm_inputs

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


# More (row, group) pairs than the teams of one launch (at most 1536 workgroups), so that teams go on to further rows.
MANY = [
    # rows, channels, groups, type, activation, centred, elements before each row; lanes of a team and values of an access
    (4000, 5120, 1, BF, "gate_first", False, 8),      # 1024 lanes, 8 values
    (5000, 2056, 1, F32, "silu", True, 0),            # 256 lanes, 4 values
    (9000, 337 * 7, 7, F32, "none", True, 0),         # 64 lanes, single values; 7 groups among 6144 teams
    (8000, 337 * 3, 3, BF, "gate_last", False, 1),    # the same with odd rows of bf16
    (2100, 4096, 32, BF, "gate_last", False, 8),      # 8 lanes, 8 values
    (1700, 4096, 128, F32, "gate_first", True, 4),    # 2 lanes, 4 values
    (7001, 1030, 1, BF, "silu", True, 2),             # 256 lanes, pairs
    (6500, 514 * 3, 3, BF, "gate_first", False, 2),   # 64 lanes, pairs; 3 groups
    (4300, 9000, 1, F32, "none", True, 1),            # 1024 lanes, single values, up to 9 a lane
    (6160, 1008, 2, BF, "none", True, 8),             # 32 lanes, 8 values, the last round partial
    (5200, 1537, 1, F32, "gate_last", False, 0),      # 256 lanes, single values, one lane in the last round
    (9000, 1500, 5, F32, "gate_first", True, 0),      # 32 lanes, 4 values; 5 groups among 12288 teams
    (420000, 3, 1, F32, "silu", True, 0),             # one lane
]


@pytest.mark.parametrize("k", range(len(MANY)))
def test_norm_teams_go_on_to_further_rows(k):
    rows, c, g, dtype, act, center, pad = MANY[k]
    log(f"norm {MANY[k]}")
    i = norm_inputs(rows, c, dtype, act, seed=200 + k, pad=pad)
    out = torch.full((rows, c + 8), 7.0, dtype=dtype, device="cuda")
    got = ssd.group_norm(i["x"], g, weight=i["weight"], bias=i["bias"], z=i["z"], act=act, center=center,
                         out=out[:, pad:pad + c])
    torch.cuda.synchronize()
    x, w, b = i["x"].cpu(), i["weight"].cpu(), i["bias"].cpu()
    z = None if i["z"] is None else i["z"].cpu()
    got, worst = got.cpu(), 0.0
    for r in range(0, rows, 4096):
        part = slice(r, r + 4096)
        want, bound = ref.group_norm(x[part], g, w, b, None if z is None else z[part], act, center)
        worst = max(worst, ref.check(got[part], want, bound, f"rows from {r}"))
    log(f"  worst {worst:.3f} of the bound")
    assert (out[:, :pad] == 7).all() and (out[:, pad + c:] == 7).all()
    # the rows' order does not matter: the last ones alone, which one team each takes, give the same bits
    few = slice(rows - 5, rows)
    again = ssd.group_norm(i["x"][few], g, weight=i["weight"], bias=i["bias"],
                           z=None if i["z"] is None else i["z"][few], act=act, center=center)
    torch.cuda.synchronize()
    assert torch.equal(again.cpu(), got[few])
