"""Sizes at and past the ends of what the decode step's calls take, on the CPU."""
import os

import pytest
import torch

from selective_state_space_cu_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="libssd.so not built")

I32 = torch.int32


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_parts_of_any_number_of_heads():
    """Rows (tokens x heads) past 32 bits: one part fills the GPU."""
    parts = ssd.load_library().ssd_paged_attention_parts
    for tokens, heads, kv in ((64, 2 ** 30, 1), (64, 2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 30, 2 ** 29), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1),
                              (2 ** 31 - 1, 16, 1)):
        assert parts(tokens, heads, kv) == 1
    assert parts(64, 64, 1) == 8 and parts(1, 1, 1) == 2048


@pytest.mark.parametrize("total", [-1, 2 ** 31, 2 ** 32 + 3])
def test_bindings_refuse_tokens_past_32_bits(total):
    """Before anything of that size is allocated."""
    with pytest.raises(ValueError, match="total_tokens"):
        ssd.step_tables(zeros(3, dtype=I32), zeros(3, dtype=I32), zeros(3, 4, dtype=I32), 16, total)
    with pytest.raises(ValueError, match="total_tokens"):
        ssd.attention_plan(zeros(3, dtype=I32), 8, 2, cu_seqlens=zeros(4, dtype=I32), total_tokens=total)


@pytest.mark.parametrize("heads,kv", [(2 ** 31, 8), (2 ** 32 + 8, 8), (2 ** 32 + 8, 2 ** 32 + 8)])
def test_bindings_refuse_heads_past_32_bits(heads, kv):
    with pytest.raises(ValueError, match="num_heads must be"):
        ssd.attention_plan(zeros(3, dtype=I32), heads, kv)


def test_bindings_refuse_caches_without_heads_and_rows_without_channels():
    plan = ssd.AttentionPlan(3, 3, 1, 0, 20, *(zeros(24, dtype=I32) for _ in range(6)))
    with pytest.raises(ValueError, match="heads must be a multiple"):
        ssd.paged_attention_step(zeros(3, 4, 64), zeros(4, 0, 16, 64), zeros(4, 0, 64, 16), zeros(3, 4, dtype=I32), plan)
    for group in (0, 32):
        with pytest.raises(ValueError, match="GPU" if group else "group must divide"):
            ssd.add_rms_norm_e4m3(zeros(3, 0), group=group)


def test_plans_whose_tensors_are_too_short_are_refused():
    """A plan with other numbers than its tensors were made for."""
    sizes = dict(seq_lens=3, cu_seqlens=4, part_start=4, part_seq=20, part_keys=1, error_flag=1)

    def call(**other):
        plan = ssd.AttentionPlan(3, 3, 1, 0, 20, **{n: zeros(k, dtype=I32) for n, k in dict(sizes, **other).items()})
        ssd.paged_attention_step(zeros(3, 4, 64), zeros(4, 2, 16, 64), zeros(4, 2, 64, 16), zeros(3, 4, dtype=I32), plan)

    with pytest.raises(ValueError, match="on a GPU"):
        call()
    for name, size in sizes.items():
        with pytest.raises(ValueError, match="shorter"):
            call(**{name: size - 1})
