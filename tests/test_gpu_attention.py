"""Attention over a paged cache, its plan and the cache's writes, against float64 at the bound that roundings give."""
import pytest
import torch

import step_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def inputs(lengths, counts, Hq, Hkv, D, block, dtype, seed=0, pad=0, extra_cols=1, spread=1.0):
    """A paged cache whose free places hold NaN."""
    r = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=r)   # noqa: E731
    need = [-(-n // block) for n in lengths]
    blocks = sum(need) + 2
    order = torch.randperm(blocks, generator=r).to(torch.int32)
    table = torch.full((len(lengths), max(need + [0]) + extra_cols), -1, dtype=torch.int32)
    kc, vc = torch.full((blocks, Hkv, block, D), NAN), torch.full((blocks, Hkv, D, block), NAN)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        for b in range(n):
            live = min(block, lengths[s] - b * block)
            kc[order[at + b], :, :live] = spread * normal(Hkv, live, D)
            vc[order[at + b], :, :, :live] = normal(Hkv, D, live)
        at += n
    T = sum(counts)
    q = normal(T, pad + Hq * D).to(dtype).cuda()[:, pad:].unflatten(1, (Hq, D))
    return dict(q=q, kc=kc.to(dtype).cuda(), vc=vc.to(dtype).cuda(), table=table.cuda(), lengths=lengths, counts=counts,
                lens=torch.tensor(lengths, dtype=torch.int32).cuda(),
                cu=torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda())


def plan_of(i, window=0, max_new=None):
    return ssd.attention_plan(i["lens"], i["q"].shape[1], i["kc"].shape[1], cu_seqlens=i["cu"],
                              total_tokens=i["q"].shape[0], max_new_tokens=max_new or max(i["counts"] + [1]), window=window)


def call(i, window=0, plan=None, **kw):
    plan = plan_of(i, window) if plan is None else plan
    lse = torch.full((i["q"].shape[0], i["q"].shape[1]), 5.0, device="cuda")
    out = ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan, lse=lse, **kw)
    torch.cuda.synchronize()
    assert int(plan.error_flag.item()) == 0
    return out, lse


def check(i, out, lse, what, window=0, scale=None, rows=None, only=None):
    worst, at = 0.0, 0
    for s, (length, n) in enumerate(zip(i["lengths"], i["counts"])):
        if n and (only is None or s in only):
            k, v = ref.gather_cache(i["kc"], i["vc"], i["table"][s if rows is None else rows[s]], length)
            want, err, log_want, log_err = ref.attention(i["q"][at:at + n].cpu(), k, v, n, window, scale,
                                                         p_step=0.0 if out.dtype == F32 else ref.HALF_STEP[BF])
            worst = max(worst, ref.check(out[at:at + n], want, ref.rounded(want, err, out.dtype), f"{what}: sequence {s}"),
                        ref.check(lse[at:at + n], log_want, log_err, f"{what}: lse of sequence {s}"))
        at += n
    return worst


CASES = [
    # lengths, new tokens, query heads, kv heads, head dim, block, type, window
    ([1], [1], 1, 1, 64, 16, F32, 0), ([1], [1], 4, 1, 128, 16, BF, 0), ([17, 64, 47], [1, 1, 1], 8, 2, 64, 16, F32, 0),
    ([31, 32, 33, 15, 16, 0], [1] * 6, 8, 2, 128, 16, BF, 0), ([255, 257, 128], [1] * 3, 5, 5, 64, 32, BF, 0),
    ([300, 5, 129], [1] * 3, 14, 2, 256, 48, BF, 0), ([77, 100], [1, 1], 16, 1, 128, 256, F32, 0),
    ([200, 3, 66, 40], [4, 3, 1, 0], 8, 2, 128, 16, BF, 0), ([65, 9], [5, 9], 16, 2, 64, 16, F32, 0),
    ([500, 64, 33], [1] * 3, 4, 2, 128, 16, BF, 50), ([130, 40], [4, 4], 8, 4, 256, 64, F32, 33),
    ([90, 70], [2, 2], 32, 2, 64, 528, BF, 1), ([2000, 1], [1, 1], 8, 1, 128, 16, BF, 0), ([40], [17], 4, 4, 64, 16, BF, 0),
    ([1500], [3], 24, 2, 256, 16, BF, 700), ([33] * 40, [1] * 40, 2, 1, 64, 16, BF, 0),
]


@pytest.mark.parametrize("c", range(len(CASES)))
def test_against_float64(c):
    lengths, counts, Hq, Hkv, D, block, dtype, window = CASES[c]
    log(f"attention {CASES[c]}")
    i = inputs(lengths, counts, Hq, Hkv, D, block, dtype, seed=c, pad=c % 3)
    out, lse = call(i, window)
    log(f"  worst {check(i, out, lse, f'case {c}', window):.3f} of the bound")


def test_long_sequences_in_many_parts_equal_float64():
    """Parts of more than one round of a workgroup's waves, joined; keys of large products."""
    i = inputs([9001, 300, 4097], [1, 1, 1], 4, 2, 128, 16, BF, seed=20, spread=4.0)
    plan = plan_of(i)
    plan = ssd.dataclasses.replace(plan, max_parts=3 + 8)   # fewer and longer parts than would fill the GPU
    ssd._enqueue("ssd_attention_plan_build", i["q"].device, ssd.ctypes.byref(plan.c_struct()))
    out, lse = call(i, plan=plan)
    starts = plan.part_start.tolist()
    assert starts[-1] <= 11 and starts[1] > 3
    check(i, out, lse, "long parts")
    check(i, *call(i), "short parts")


def test_plan_covers_every_key_once():
    for seed, (lengths, counts, window) in enumerate([([1, 0, 5000, 128, 129], [1] * 5, 0), ([70000, 3], [1, 1], 0),
                                                      ([4000, 10, 0, 300], [4, 4, 2, 0], 1000), ([0, 0], [0, 0], 0),
                                                      ([3 * s for s in range(1500)], [1] * 1500, 0), ([2 ** 30] * 1024, [1] * 1024, 0),
                                                      ([2 ** 30 - s for s in range(1025)], [2] * 1025, 0),
                                                      ([40000, 39999, 17] * 9, [3, 1, 2] * 9, 4096)]):
        lens, cu = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
        plan = ssd.attention_plan(lens, 8, 2, cu_seqlens=cu, total_tokens=sum(counts), max_new_tokens=4, window=window)
        part, starts, seqs = int(plan.part_keys.item()), plan.part_start.tolist(), plan.part_seq.tolist()
        assert part > 0 and part % 256 == 0 and starts[0] == 0 and starts[-1] <= plan.max_parts
        want = []
        for s, (n, new) in enumerate(zip(lengths, counts)):
            low = max(0, n - new - window + 1) // 32 * 32 if window else 0
            want += [s] * (max(1, -(-(n - low) // part)) if new else 0)
        assert seqs[:len(want)] == want and set(seqs[len(want):]) <= {-1} and starts[-1] == len(want)


def test_places_that_a_token_does_not_see():
    """Infinities and NaN in keys and values past a token's own, before its window and in the rest of a block."""
    for bad in (NAN, INF, -INF):
        for dtype in (BF, F32):
            i = inputs([70, 45], [4, 3], 8, 2, 64, 16, dtype, seed=21)
            clean, clean_lse = call(i)
            kc, vc = i["kc"].clone(), i["vc"].clone()
            for s, (length, n) in enumerate(zip(i["lengths"], i["counts"])):
                for p in range(length - n + 1, length):   # what the first new token does not see
                    b, at = int(i["table"][s, p // 16]), p % 16
                    i["kc"][b, :, at] = bad
                    i["vc"][b, :, :, at] = bad
            out, lse = call(i)
            first = [0, 4]
            assert torch.equal(out[first], clean[first]) and torch.equal(lse[first], clean_lse[first]), (bad, dtype)
            i.update(kc=kc, vc=vc)
            out, lse = call(i, window=20)
            for s, (length, n) in enumerate(zip(i["lengths"], i["counts"])):
                for p in range(0, length - n - 20 + 1 + n - 1):   # before the last token's window
                    b, at = int(i["table"][s, p // 16]), p % 16
                    i["kc"][b, :, at] = bad
                    i["vc"][b, :, :, at] = bad
            last = [3, 6]
            again, again_lse = call(i, window=20)
            assert torch.equal(again[last], out[last]) and torch.equal(again_lse[last], lse[last]), (bad, dtype)


@pytest.mark.parametrize("D,dtype,at", [(64, BF, 0), (64, F32, 63), (128, BF, 127), (128, F32, 5), (256, BF, 200), (256, F32, 70)])
def test_one_value_that_is_not_finite(D, dtype, at):
    """A single infinity or NaN at a place that some tokens see reaches theirs, in its own place of the head, and no other's."""
    for bad in (NAN, -INF):
        i = inputs([150, 39], [4, 2], 8, 2, D, 16, dtype, seed=36)
        clean, clean_lse = call(i)
        i["vc"][int(i["table"][0, 147 // 16]), 1, at, 147 % 16] = bad   # tokens 1, 2 and 3 see it, heads 4 .. 7
        out, lse = call(i)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[1:4, 4:, at] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
        assert torch.isnan(out[hit]).all() if bad != bad else (out[hit] == bad).all()


def test_tokens_that_see_nothing():
    """Empty sequences and tokens before position 0 get zeros and -infinity."""
    i = inputs([0, 2, 40], [1, 4, 2], 4, 2, 64, 16, BF, seed=22)
    out, lse = call(i)
    for t in (0, 1, 2):
        assert (out[t] == 0).all() and (lse[t] == -INF).all()
    assert torch.isfinite(lse[3:]).all()
    check(i, out, lse, "short", only=(2,))
    k, v = ref.gather_cache(i["kc"], i["vc"], i["table"][1], 2)
    want, err, _, _ = ref.attention(i["q"][3:5].cpu(), k, v, 2, p_step=ref.HALF_STEP[BF])
    ref.check(out[3:5], want, ref.rounded(want, err, BF), "positions 0 and 1")


def test_bad_tables_rows_and_plans():
    i = inputs([40, 50, 20, 33], [1] * 4, 4, 2, 64, 16, BF, seed=23)
    good, good_lse = call(i)
    table, flag = i["table"].clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    i["table"][1, 1] = i["kc"].shape[0]      # keys 16 .. 31 of sequence 1 are left out
    i["table"][3, 0] = -5                    # and keys 0 .. 15 of sequence 3
    out, lse = call(i, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_BLOCK
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    for s, gone in ((1, range(16, 32)), (3, range(16))):
        k, v = ref.gather_cache(i["kc"], i["vc"], table[s], i["lengths"][s])
        keep = [p for p in range(i["lengths"][s]) if p not in gone]
        want, err, lw, le = ref.attention(i["q"][s:s + 1].cpu(), k[keep], v[keep], 1, p_step=ref.HALF_STEP[BF])
        ref.check(out[s:s + 1], want, ref.rounded(want, err, BF), f"sequence {s}")
        ref.check(lse[s:s + 1], lw, le, f"lse of sequence {s}")
    # a table of two columns holds 32 keys
    i["table"] = table[:, :2].contiguous()
    flag.zero_()
    out, _ = call(i, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_BLOCK and torch.equal(out[2], good[2])
    # rows: a permutation, and one outside the table
    i["table"] = table[[2, 0, 3, 1]].contiguous()
    flag.zero_()
    rows = torch.tensor([1, 3, 0, 2], dtype=torch.int32).cuda()
    out, lse = call(i, rows=rows, error_flag=flag)
    assert int(flag.item()) == 0 and torch.equal(out, good) and torch.equal(lse, good_lse)
    rows[2] = 4
    out, lse = call(i, rows=rows, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_SLOT and (out[2] == 0).all() and (lse[2] == -INF).all()
    assert torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])


def test_sequences_outside_the_batch_or_too_long_are_left_out():
    i = inputs([40, 50, 20], [2, 3, 2], 4, 2, 64, 16, BF, seed=24)
    good, _ = call(i)
    for cu, left in (([0, 2, 5, 9], [5, 6]), ([0, 2, 7, 5], [2, 3, 4, 5, 6])):
        i["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        plan = plan_of(i, max_new=3)
        assert int(plan.error_flag.item()) == ssd.DATA_BAD_CU_SEQLENS
        out = torch.full_like(good, 3.0)
        ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan, out=out)
        torch.cuda.synchronize()
        assert (out[left] == 3).all() and torch.equal(out[:2], good[:2])


def test_sequences_left_out_do_not_hide_others():
    """The sequences around a damaged one are joined, too, when the places of their tokens do not ascend."""
    i = inputs([40, 50, 9000], [2, 2, 2], 4, 2, 64, 16, BF, seed=34)
    good, good_lse = call(i)
    plan = plan_of(i, max_new=2)
    assert plan.part_start[3].item() - plan.part_start[2].item() > 1
    for cu in ([0, 100, 4, 6], [0, -3, 4, 6], [7, 5, 4, 6]):
        i["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        plan = plan_of(i, max_new=2)
        assert int(plan.error_flag.item()) == ssd.DATA_BAD_CU_SEQLENS
        out, lse = torch.full_like(good, 3.0), torch.full_like(good_lse, 4.0)
        ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out[:4] == 3).all() and (lse[:4] == 4).all()
        check(i, out, lse, f"{cu}", only=(2,))


def test_blocks_before_the_window_may_be_gone():
    """A table whose blocks before the first token's window have been given back sets no flag; one a token sees does."""
    for dtype, length, n, window in ((BF, 100, 1, 37), (BF, 100, 3, 30), (F32, 75, 2, 11), (BF, 64, 1, 1), (F32, 100, 4, 97)):
        i = inputs([length, length], [n, n], 8, 2, 64, 16, dtype, seed=35)
        good, good_lse = call(i, window)
        first = length - n - window + 1   # the first key that a token sees
        i["table"][0, :max(first, 0) // 16] = -1
        i["table"][1, :max(first, 0) // 16] = i["kc"].shape[0]
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = call(i, window, error_flag=flag)
        assert int(flag.item()) == 0 and torch.equal(out, good) and torch.equal(lse, good_lse), (length, n, window)
        i["table"][0, max(first, 0) // 16] = -1
        call(i, window, error_flag=flag)
        assert int(flag.item()) == ssd.DATA_BAD_BLOCK, (length, n, window)


def test_lengths_past_the_limit_and_below_zero():
    """A sequence of more than 2^30 keys is left out; a negative length counts as none."""
    i = inputs([40, 50, 20], [1] * 3, 4, 2, 64, 16, BF, seed=29)
    good, _ = call(i)
    i["lens"][1] = 2 ** 30 + 1
    plan = plan_of(i)
    assert int(plan.error_flag.item()) == ssd.DATA_BAD_CU_SEQLENS
    out = torch.full_like(good, 3.0)
    ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan, out=out)
    torch.cuda.synchronize()
    assert (out[1] == 3).all() and torch.equal(out[[0, 2]], good[[0, 2]])
    i["lens"][1] = 2 ** 30   # more than the table holds: what it holds counts
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan_of(i), out=out, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == ssd.DATA_BAD_BLOCK and torch.equal(out[[0, 2]], good[[0, 2]])
    i["lens"][1] = -7
    out, lse = call(i)
    assert (out[1] == 0).all() and (lse[1] == -INF).all() and torch.equal(out[[0, 2]], good[[0, 2]])


def test_padded_batch_and_rows_of_nan():
    """Rows behind the last sequence stay as they were; a query of NaN spoils its own row alone."""
    i = inputs([600, 50], [2, 3], 8, 2, 128, 16, BF, seed=31)
    want, want_lse = call(i)
    q = torch.full((9, 8, 128), NAN, dtype=BF, device="cuda")
    q[:5] = i["q"]
    q[1, 5] = NAN
    plan = ssd.attention_plan(i["lens"], 8, 2, cu_seqlens=i["cu"], total_tokens=9, max_new_tokens=4)
    out, lse = torch.full_like(q, 3.0), torch.full((9, 8), 4.0, device="cuda")
    ssd.paged_attention_step(q, i["kc"], i["vc"], i["table"], plan, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[5:] == 3).all() and (lse[5:] == 4).all()
    assert torch.isnan(out[1, 5]).all()
    keep = torch.ones(5, 8, dtype=torch.bool)
    keep[1, 5] = False
    assert torch.equal(out[:5][keep], want[keep]) and torch.equal(lse[:5][keep], want_lse[keep])


def test_many_tokens_of_several_parts():
    """More tokens than the join has workgroups for: each takes several heads."""
    i = inputs([2600] * 130, [4] * 130, 8, 1, 64, 16, BF, seed=32)
    plan = plan_of(i)
    plan = ssd.dataclasses.replace(plan, max_parts=130 + 2000, part_seq=torch.zeros(2130, dtype=torch.int32, device="cuda"))
    ssd._enqueue("ssd_attention_plan_build", i["q"].device, ssd.ctypes.byref(plan.c_struct()))
    out, lse = call(i, plan=plan)
    assert plan.part_start[-1].item() == 130 * 3   # parts of 1024 keys
    check(i, out, lse, "several parts", only=(0, 64, 129))
    first = inputs([2600], [4], 8, 1, 64, 16, BF, seed=33)
    for s in range(0, 130, 13):
        one = dict(first, q=i["q"][4 * s:4 * s + 4], table=i["table"][s:s + 1], kc=i["kc"], vc=i["vc"])
        k, v = ref.gather_cache(i["kc"], i["vc"], i["table"][s], 2600)
        want, err, _, _ = ref.attention(one["q"][3:].cpu(), k, v, 1, p_step=ref.HALF_STEP[BF])
        ref.check(out[4 * s + 3:4 * s + 4], want, ref.rounded(want, err, BF), f"sequence {s}")


def test_scale_strides_and_a_given_workspace():
    i = inputs([400, 30], [1, 1], 6, 3, 64, 32, BF, seed=25, pad=5)
    plan = plan_of(i)
    ws = torch.full((ssd.paged_attention_workspace_size(plan, 6, 64),), 255, dtype=torch.uint8, device="cuda")
    wide = torch.full((2, 3 + 6 * 64), 7.0, dtype=BF, device="cuda")
    out = wide[:, 3:].unflatten(1, (6, 64))
    got, lse = call(i, plan=plan, scale=-0.2, workspace=ws, out=out)
    assert (wide[:, :3] == 7).all()
    check(i, got.contiguous(), lse, "scale", scale=-0.2)


def test_scores_far_apart_and_infinite_products():
    """Scores of thousands (one key takes all), and keys whose products are -infinity, which take no part."""
    i = inputs([200], [1], 4, 1, 64, 16, F32, seed=26, spread=300.0)
    check(i, *call(i), "far apart")
    i = inputs([48], [1], 4, 1, 64, 16, F32, seed=27)
    i["q"].abs_()
    for p in range(10, 20):
        i["kc"][int(i["table"][0, p // 16]), :, p % 16] = -INF
    out, lse = call(i)
    k, v = ref.gather_cache(i["kc"], i["vc"], i["table"][0], 48)
    keep = [p for p in range(48) if not 10 <= p < 20]
    want, err, _, _ = ref.attention(i["q"].cpu(), k[keep], v[keep], 1)
    ref.check(out, want, ref.rounded(want, err, F32), "minus infinity")


def test_one_new_token_each_without_cu_seqlens_and_replays():
    i = inputs([700, 3, 90], [1] * 3, 8, 2, 128, 16, BF, seed=28)
    want, _ = call(i)
    plan = ssd.attention_plan(i["lens"], 8, 2)
    ws = torch.empty(ssd.paged_attention_workspace_size(plan, 8, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd._enqueue("ssd_attention_plan_build", out.device, ssd.ctypes.byref(plan.c_struct()))
        ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], plan, out=out, workspace=ws)
    for length in (700, 650, 33):   # the lengths change between replays, as a decode loop's do
        i["lens"][0] = length
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        j = dict(i, lengths=[length, 3, 90])
        eager, lse = call(j)
        assert torch.equal(out, eager)
        check(j, eager, lse, f"length {length}")
    assert int(plan.error_flag.item()) == 0


def write_inputs(T, Hkv, D, block, dtype, seed=0, pad=0, run=False):
    r = torch.Generator().manual_seed(seed)
    blocks = -(-T // block) + 3
    wide = torch.randn(T, pad + 2 * Hkv * D, generator=r).to(dtype).cuda()[:, pad:]
    slots = torch.randperm(blocks * block, generator=r)[:T] if not run else torch.arange(T) + block // 2 + 1
    return dict(k=wide[:, :Hkv * D].unflatten(1, (Hkv, D)), v=wide[:, Hkv * D:].unflatten(1, (Hkv, D)),
                slots=slots.to(torch.int32).cuda(), kc=torch.full((blocks, Hkv, block, D), 9.0, dtype=dtype, device="cuda"),
                vc=torch.full((blocks, Hkv, D, block), 9.0, dtype=dtype, device="cuda"))


def check_write(i, flag=0):
    block = i["kc"].shape[2]
    kc, vc = torch.full_like(i["kc"], 9.0), torch.full_like(i["vc"], 9.0)
    keep = (i["slots"] >= 0) & (i["slots"] < kc.shape[0] * block)
    s = i["slots"][keep].long()
    kc[s // block, :, s % block] = i["k"][keep]
    vc[s // block, :, :, s % block] = i["v"][keep]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.kv_cache_write(i["k"], i["v"], i["kc"], i["vc"], i["slots"], error_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == flag
    assert torch.equal(i["kc"], kc) and torch.equal(i["vc"], vc)


@pytest.mark.parametrize("T,Hkv,D,block,dtype,pad,run", [
    (1, 1, 64, 16, F32, 0, False), (1, 8, 128, 16, BF, 0, False), (7, 3, 64, 48, BF, 1, False), (64, 2, 256, 16, BF, 8, True),
    (130, 2, 128, 64, F32, 3, True), (257, 1, 64, 16, BF, 0, True), (300, 4, 128, 528, BF, 2, True), (65, 8, 64, 32, F32, 0, False),
    (1000, 2, 128, 256, BF, 0, True), (33, 1, 256, 16, F32, 1, True), (1025, 8, 128, 16, BF, 0, True), (2731, 3, 64, 48, BF, 1, True),
    (8195, 1, 256, 16, F32, 3, False), (4100, 2, 64, 528, F32, 0, True), (2050, 4, 256, 32, BF, 5, False), (8200, 1, 128, 64, F32, 1, True),
])
def test_cache_write(T, Hkv, D, block, dtype, pad, run):
    log(f"cache write {T, Hkv, D, block, dtype, pad, run}")
    i = write_inputs(T, Hkv, D, block, dtype, seed=T, pad=pad, run=run)
    check_write(i)


def test_cache_write_skips_and_refuses():
    for T, run in ((90, False), (90, True), (4200, False), (4200, True)):   # (both kernels)
        i = write_inputs(T, 2, 64, 16, BF, seed=5, run=run)
        i["slots"][::7] = -1
        i["slots"][3] = i["kc"].shape[0] * 16
        i["slots"][50] = 2 ** 31 - 1
        check_write(i, ssd.DATA_BAD_SLOT)


def test_cache_past_32_bit_offsets():
    """Blocks past 2^31 elements of the caches: written, then attended to, as a small cache's are."""
    block, Hkv, D = 256, 8, 128
    blocks = 2 ** 31 // (block * Hkv * D) + 3
    i = inputs([300], [1], 8, Hkv, D, block, BF, seed=30)
    k, v = ref.gather_cache(i["kc"], i["vc"], i["table"][0], 300)
    want, lse = call(i)
    kc, vc = (torch.zeros(blocks, Hkv, *s, dtype=BF, device="cuda") for s in ((block, D), (D, block)))
    ids = [blocks - 1, blocks - 3]
    slots = torch.tensor([ids[p // block] * block + p % block for p in range(300)], dtype=torch.int32).cuda()
    ssd.kv_cache_write(k.to(BF).cuda(), v.to(BF).cuda(), kc, vc, slots)
    table = torch.tensor([ids], dtype=torch.int32).cuda()
    out = ssd.paged_attention_step(i["q"], kc, vc, table, plan_of(i))
    assert torch.equal(out, want)
