"""Every form of the attention kernel against float64: both types, all head dims, one tile of rows and several, one part and
several joined, with and without a window; values that are not finite in later tiles; blocks that sequences share."""
import pytest
import torch

import step_ref as ref
import test_gpu_attention as att
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def parts_of(i, window=0):
    starts = att.plan_of(i, window).part_start.tolist()
    return [b - a for a, b in zip(starts, starts[1:])]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 1500])
def test_several_parts_in_one_tile(D, dtype, window):
    """Lengths around the steps of 32 and 64 keys and the waves' rounds of 128 and 256."""
    lengths, counts = [1000, 5000, 257, 2309, 4096, 1], [1, 2, 1, 4, 1, 1]
    log(f"attention {D, dtype, window}, {lengths}")
    i = att.inputs(lengths, counts, 8, 2, D, 16, dtype, seed=D + window)
    n = parts_of(i, window)
    assert n[1] > 2 and n[3] > 2 and n[4] > 2 and n[5] == 1
    log(f"  {n} parts, worst {att.check(i, *att.call(i, window), 'several parts', window):.3f} of the bound")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group,counts,window", [(8, [8, 5], 0), (5, [7, 4], 0), (7, [5, 6], 300), (32, [1, 1], 0), (17, [2, 1], 40)])
def test_several_tiles(D, dtype, group, counts, window):
    """More rows than a tile has, tokens that cross from one tile to the next; one part and several."""
    for lengths in ([200, 60], [3000, 700]):
        log(f"attention {D, dtype, group, counts, window}, {lengths}")
        i = att.inputs(lengths, counts, 2 * group, 2, D, 32, dtype, seed=D + group, pad=3)
        n = parts_of(i, window)
        assert n == [1, 1] if lengths[0] == 200 or window == 40 else n[0] > 1   # (parts have 256 keys at least)
        log(f"  {n} parts, worst {att.check(i, *att.call(i, window), 'several tiles', window):.3f} of the bound")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group,n", [(8, 8), (5, 7)])
def test_values_not_finite_that_some_tokens_of_later_tiles_see(D, dtype, group, n):
    """They reach the tokens that see them, in their own place of the head, and no other's; in one part and in several."""
    for length, bad in ((150, NAN), (2000, -INF)):
        i = att.inputs([length, 39], [n, 2], 2 * group, 2, D, 16, dtype, seed=36)
        clean, clean_lse = att.call(i)
        place, at = length - n + 5, D - 3   # tokens 5 and later of the first sequence see it
        i["vc"][int(i["table"][0, place // 16]), 1, at, place % 16] = bad
        out, lse = att.call(i)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[5:n, group:, at] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
        assert torch.isnan(out[hit]).all() if bad != bad else (out[hit] == bad).all()
        # tokens that do not see it, a window further back
        i = att.inputs([length], [n], 2 * group, 2, D, 16, dtype, seed=37)
        clean, clean_lse = att.call(i, 30)
        place = length - n - 30 + 1 + 3   # tokens 0 .. 3 see it
        i["vc"][int(i["table"][0, place // 16]), 0, at, place % 16] = bad
        out, lse = att.call(i, 30)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[:4, :group, at] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
        assert torch.isnan(out[hit]).all() if bad != bad else (out[hit] == bad).all()


@pytest.mark.parametrize("dtype,counts", [(BF, [1, 1, 1, 1]), (F32, [1, 1, 1, 1]), (BF, [4, 3, 6, 1])])
def test_sequences_that_share_the_blocks_of_a_prefix(dtype, counts):
    """Tables that name the same blocks: the same bits as with copies of them, and the float64 bound."""
    lengths, prefix = [1700, 1100, 1024 + 6, 2000], 1024
    i = att.inputs(lengths, counts, 8, 2, 128, 16, dtype, seed=38)
    for s in range(1, 4):   # copies first
        own, first = i["table"][s, :prefix // 16].long(), i["table"][0, :prefix // 16].long()
        i["kc"][own], i["vc"][own] = i["kc"][first], i["vc"][first]
    want, want_lse = att.call(i)
    for s in range(1, 4):
        i["kc"][i["table"][s, :prefix // 16].long()] = NAN
        i["table"][s, :prefix // 16] = i["table"][0, :prefix // 16]
    out, lse = att.call(i)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    att.check(i, out, lse, "shared blocks")


def test_delta_steps_that_read_one_state():
    """Sequences that go on from the same slot, as after a shared prefix: each as if it had a copy."""
    r = torch.Generator().manual_seed(39)
    n = lambda *s: torch.randn(*s, generator=r).cuda()   # noqa: E731
    S, H, G, dk, dv = 5, 4, 2, 128, 48
    q, k, v, gate, beta = n(S, G, dk), n(S, G, dk) / 11, n(S, H, dv), -n(S, H).abs(), torch.sigmoid(n(S, H))
    cache = n(2 * S + 1, H, dv, dk)
    cache[1:S] = cache[0]
    i32 = lambda *a: torch.arange(*a, dtype=torch.int32).cuda()   # noqa: E731
    copies = cache.clone()
    want = ssd.gated_delta_step(q, k, v, gate, beta, copies, i32(S), i32(S, 2 * S))
    o = ssd.gated_delta_step(q, k, v, gate, beta, cache, torch.zeros_like(i32(S)), i32(S, 2 * S))
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(cache, copies)
    exact, err, made, made_err = ref.gated_delta(q, k, v, gate, beta, copies, torch.zeros(S, dtype=torch.int64),
                                                 torch.arange(S, 2 * S))
    ref.check(o, exact, ref.rounded(exact, err, F32), "o")
    ref.check(cache, made, made_err, "states")
