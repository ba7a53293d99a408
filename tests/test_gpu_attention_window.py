"""Windows as large as 32 bits hold, with more new tokens than keys."""
import pytest
import torch

import test_gpu_attention as att

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 31 - 60, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_windows_longer_than_any_sequence_are_none(window, dtype):
    """Tokens before position 0 see nothing; those after them see all their keys."""
    i = att.inputs([2, 5, 0, 300], [6, 9, 3, 64], 4, 2, 64, 16, dtype, seed=53)
    want, want_lse = att.call(i)
    out, lse = att.call(i, window)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    att.check(i, out, lse, f"window {window}", window, only=(0, 1, 3))
