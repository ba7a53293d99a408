"""Log sums of rows that NaN reach: NaN, as their outputs are, and never the -infinity of rows that see nothing."""
import pytest
import torch

import test_gpu_attention as att

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32, NAN = torch.bfloat16, torch.float32, float("nan")


@pytest.mark.parametrize("lengths,counts,D,dtype", [([600, 50], [2, 3], 128, BF), ([9000, 20], [1, 2], 64, F32),
                                                     ([40, 7], [2, 1], 256, F32), ([3000, 90], [4, 4], 64, BF)])
def test_a_query_of_nan(lengths, counts, D, dtype):
    """In one part and in several, beside a sequence that sees nothing."""
    i = att.inputs(lengths + [0], counts + [1], 8, 2, D, 16, dtype, seed=51)
    clean, clean_lse = att.call(i)
    i["q"][0, 5] = NAN
    i["q"][counts[0], 2] = NAN
    out, lse = att.call(i)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 5] = hit[counts[0], 2] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert (out[-1] == 0).all() and (lse[-1] == -float("inf")).all()


@pytest.mark.parametrize("D,dtype", [(128, BF), (64, F32)])
def test_a_part_whose_keys_are_all_nan(D, dtype):
    """The other parts' sums do not hide it; other heads take no notice."""
    i = att.inputs([5000], [2], 8, 2, D, 16, dtype, seed=52)
    plan = att.plan_of(i)
    part = int(plan.part_keys.item())
    assert plan.part_start[1].item() > 2
    clean, clean_lse = att.call(i)
    i["kc"][i["table"][0, part // 16:2 * part // 16].long(), 1] = NAN
    out, lse = att.call(i)
    assert torch.isnan(out[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()
    assert torch.equal(out[:, :4], clean[:, :4]) and torch.equal(lse[:, :4], clean_lse[:, :4])


@pytest.mark.parametrize("lengths", [[150, 33], [4000, 700]])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, F32)])
def test_products_past_the_largest_number(lengths, D, dtype):
    """One finite key whose product with every query of its head is +infinity: NaN for the tokens that see it."""
    i = att.inputs(lengths, [2, 2], 8, 2, D, 16, dtype, seed=54)
    i["q"].abs_()
    clean, clean_lse = att.call(i)
    at = lengths[0] - 1   # the second token's own
    i["kc"][int(i["table"][0, at // 16]), 1, at % 16] = 3e38
    out, lse = att.call(i)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[1, 4:] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
