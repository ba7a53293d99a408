"""Step tables: batches without tokens, and tokens that were not accepted."""
import pytest
import torch

import test_gpu_step_tables as tables
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("requests", [1, 1024, 1025, 3000])
def test_no_tokens_of_any_number_of_requests(requests):
    """Nothing new: the lengths, read slots and the free list's count all the same."""
    m = tables.make([s % 50 for s in range(requests)], [0] * requests, 16, seed=requests)
    t = tables.check(m, bits=0)
    assert t.positions.shape == (0,)


def test_tokens_given_up_give_back_their_blocks():
    """Four tokens a step, some of them not accepted: the caller returns the blocks past those that are left, and every
    block stays in the list or in the table, once."""
    block, blocks = 4, 40
    table, free = tables.dev([[-1] * 12 for _ in range(3)]), tables.dev(list(range(blocks)))
    count, flag = tables.dev([blocks]), tables.dev([0])
    computed = [0, 3, 7]
    ssd.step_tables(tables.dev([0] * 3), tables.dev(computed), table, block, sum(computed), free_blocks=free, free_count=count,
                    free_count_out=count, num_blocks=blocks, error_flag=flag)
    for step in range(9):
        t = ssd.step_tables(tables.dev(computed), tables.dev([4] * 3), table, block, 12, free_blocks=free, free_count=count,
                            free_count_out=count, num_blocks=blocks, error_flag=flag)
        torch.cuda.synchronize()
        rows, at, left = table.tolist(), 0, int(count.item())
        for s in range(3):
            used = rows[s][:-(-(computed[s] + 4) // block)]
            assert t.slots.tolist()[at:at + 4] == [used[p // block] * block + p % block for p in range(computed[s], computed[s] + 4)]
            at += 4
            computed[s] += (1, 4, 2, 0, 3)[(step + 2 * s) % 5]   # accepted
            keep = -(-computed[s] // block)
            for b in range(keep, len(used)):
                free[left] = used[b]
                table[s, b] = -1
                left += 1
            rows[s] = used[:keep]
        count.fill_(left)
        held = [b for r in rows for b in r] + free.tolist()[:left]
        assert sorted(held) == list(range(blocks))
        computed = [min(c, 40) for c in computed]
    assert flag.tolist() == [0]
