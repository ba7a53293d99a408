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
