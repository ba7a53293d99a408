"""Block tables and slot maps against plain loops: whole numbers, equal everywhere."""
import random

import pytest
import torch

import step_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def dev(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def make(computed, new, block, width=None, spare=5, seed=0, permute=True):
    """Requests whose computed tokens' blocks are in the table, and a free list."""
    r = random.Random(seed)
    S = len(computed)
    total = [c + max(n, 0) for c, n in zip(computed, new)]
    width = max([-(-t // block) for t in total] + [1]) if width is None else width
    rows = r.sample(range(S + 3), S) if permute else None
    need = sum(-(-t // block) for t in total)
    ids = r.sample(range(need + spare), need + spare)
    table = [[-1] * width for _ in range(S + 3)]
    for s, c in enumerate(computed):
        for b in range(min(width, max(0, -(-c // block)))):
            table[rows[s] if permute else s][b] = ids.pop()
    return dict(computed=computed, new=new, rows=rows, table=table, block=block, free=ids, num_blocks=need + spare)


def check(m, total=None, free_count=None, allocate=True, num_blocks=None, bits=None):
    total = sum(max(n, 0) for n in m["new"]) if total is None else total
    free = m["free"] if allocate else None
    count = len(m["free"]) if free_count is None else free_count
    want, table, want_bits = ref.step_tables(m["computed"], m["new"], m["rows"], m["table"], m["block"], total, free, count,
                                             num_blocks)
    if bits is not None:
        assert want_bits == bits
    bt, fc = dev(m["table"]), dev([count])
    flag = dev([0])
    kw = dict(free_blocks=dev(m["free"]), free_count=fc, free_count_out=fc) if allocate else {}
    t = ssd.step_tables(dev(m["computed"]), dev(m["new"]), bt, m["block"], total,
                        rows=None if m["rows"] is None else dev(m["rows"]), num_blocks=num_blocks, error_flag=flag, **kw)
    torch.cuda.synchronize()
    assert int(flag.item()) == want_bits
    got = dict(cu=t.cu_seqlens, lens=t.seq_lens, read=t.read_slot, pos=t.positions, seq=t.token_seq, slots=t.slots,
               state=t.state_slot)
    for name, g in got.items():
        assert g.tolist() == want[name], name
    assert bt.tolist() == table
    if allocate:
        assert t.free_count is fc and int(fc.item()) == want["left"]
    return t


@pytest.mark.parametrize("computed,new,block", [
    ([0], [1], 16), ([16], [1], 16), ([15], [1], 16), ([0], [0], 16), ([5], [0], 1), ([0, 0, 0], [17, 64, 47], 16),
    ([31, 32, 33, 0], [1, 1, 1, 1], 32), ([3, 700, 0, 64], [5, 0, 200, 64], 64), ([100] * 70, [1] * 70, 16), ([0, 7], [3, 1], 1),
    ([10, 0, 527, 528], [600, 1, 2, 1], 528), ([0] * 1030, [1] * 1030, 16), ([9] * 2500, [2] * 2500, 4),
])
def test_against_loops(computed, new, block):
    log(f"step tables {len(computed)} requests, {sum(new)} tokens, block {block}")
    m = make(computed, new, block, seed=len(computed))
    check(m, bits=0)
    check(make(computed, new, block, permute=False), bits=0)


def test_ragged_prompts_in_two_launches():
    r = random.Random(1)
    computed = [r.choice([0, r.randint(0, 3000)]) for _ in range(200)]
    new = [r.choice([0, 1, r.randint(1, 300)]) for _ in range(200)]
    assert sum(new) > 4096
    check(make(computed, new, 16, seed=2), bits=0)


def test_padded_batch():
    m = make([3, 20], [2, 1], 16)
    t = check(m, total=8, bits=0)
    for g in (t.positions, t.token_seq, t.slots, t.state_slot):
        assert g.tolist()[3:] == [-1] * 5


def test_tables_without_a_free_list():
    m = make([30, 40], [4, 9], 16, width=4)
    for row in (0, 1):
        m["table"][m["rows"][row]] = [50 + 4 * row + j for j in range(4)]
    m["table"][m["rows"][1]][3] = -1   # a hole: no slots for its tokens
    check(m, allocate=False, bits=0)


def test_too_few_free_blocks():
    """Requests in order until the free list is short; later ones only if they need no block."""
    m = make([16, 16, 10, 32, 5], [1, 40, 3, 1, 2], 16)
    for count in range(6):
        check(m, free_count=count, bits=0 if count >= 5 else ssd.DATA_NO_BLOCK)


def test_refused_requests():
    m = make([4, 4, 4, 4], [1, 1, 1, 1], 16)
    check(dict(m, new=[1, -1, 1, 1]), total=4, bits=1)
    check(dict(m, new=[1, 9, 1, 1]), total=4, bits=1)
    check(dict(m, computed=[4, 4, -2, 4]), bits=1)
    check(dict(m, computed=[4, 4, 2 ** 31 - 1, 4]), bits=1)
    check(dict(m, rows=[m["rows"][0], 7, m["rows"][2], -1]), bits=4)
    check(dict(m, computed=[4, 16, 4, 4]), bits=8)            # a second block, in a table of one column
    check(dict(m, new=[2, 2, 2, 2]), total=5, bits=1)         # more tokens than the batch has


def test_blocks_outside_the_cache():
    m = make([20, 20, 40], [1, 13, 1], 16)
    m["table"][m["rows"][0]][1] = 9999   # holds its last computed and its new token
    m["table"][m["rows"][2]][2] = -7
    check(m, num_blocks=60, bits=8)


def test_counts_past_the_free_list_and_an_empty_batch():
    m = make([0, 3], [5, 1], 4)
    check(m, free_count=len(m["free"]))
    bt = dev([[1]])
    fc = dev([7])   # more than the list has: the list's length counts
    t = ssd.step_tables(dev([0]), dev([1]), bt, 16, 1, free_blocks=dev([3, 4]), free_count=fc)
    torch.cuda.synchronize()
    assert bt.tolist() == [[4]] and t.free_count.tolist() == [1] and fc.tolist() == [7]
    t = ssd.step_tables(dev([]), dev([]), bt, 16, 0)
    assert t.cu_seqlens.tolist() == [0]


def test_captured_steps_continue_from_each_other():
    """A decode loop's step, replayed: each takes its blocks from what the one before left."""
    S, block = 6, 4
    m = make([3, 0, 9, 4, 7, 2], [1] * S, block, width=16, spare=60)
    computed, bt, fc = dev(m["computed"]), dev(m["table"]), dev([len(m["free"])])
    new, free, rows, flag = dev([1] * S), dev(m["free"]), dev(m["rows"]), dev([0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = ssd.step_tables(computed, new, bt, block, S, rows=rows, free_blocks=free, free_count=fc, free_count_out=fc,
                            error_flag=flag)
        computed.add_(new)
    left, table, c = len(m["free"]), m["table"], list(m["computed"])
    for _ in range(9):
        graph.replay()
        torch.cuda.synchronize()
        want, table, bits = ref.step_tables(c, [1] * S, m["rows"], table, block, S, m["free"], left)
        left, c = want["left"], [x + 1 for x in c]
        assert bits == 0 and bt.tolist() == table and fc.tolist() == [left]
        assert t.slots.tolist() == want["slots"] and t.read_slot.tolist() == want["read"]
        assert t.state_slot.tolist() == want["state"] and t.seq_lens.tolist() == want["lens"]
    assert flag.tolist() == [0]
