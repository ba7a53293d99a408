"""The gated delta rule's step against float64, at the bound that its roundings give."""
import pytest
import torch

import step_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def inputs(counts, H, G, dk, dv, dtype, gate_dtype=F32, raw=False, seed=0, pad=0):
    r = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=r)   # noqa: E731
    S, T = len(counts), sum(counts)
    wide = normal(T, pad + 2 * G * dk + H * dv)
    if not raw:   # unit keys
        for j in range(2 * G):
            part = wide[:, pad + j * dk:pad + (j + 1) * dk]
            part /= part.norm(dim=1, keepdim=True)
    wide = wide.to(dtype).cuda()[:, pad:]
    gates = normal(T, pad + 2 * H) if raw else torch.cat([normal(T, pad), -torch.rand(T, H, generator=r) * 0.3,
                                                          torch.rand(T, H, generator=r)], 1)
    gates = gates.to(gate_dtype).cuda()[:, pad:]
    order = torch.randperm(S + T + 1, generator=r).to(torch.int32).cuda()
    return dict(q=wide[:, :G * dk].unflatten(1, (G, dk)), k=wide[:, G * dk:2 * G * dk].unflatten(1, (G, dk)),
                v=wide[:, 2 * G * dk:].unflatten(1, (H, dv)), gate=gates[:, :H], beta=gates[:, H:],
                cache=0.5 * normal(S + T + 1, H, dv, dk).cuda(), read=order[:S].clone(), write=order[S:S + T].clone(),
                cu=torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda(),
                A=-torch.exp(torch.rand(H, generator=r) * 2.5).cuda() if raw else None,
                dt_bias=(normal(H) - 3).cuda() if raw else None, qk_eps=1e-6 if raw else None)


def call(i, single=False, **more):
    kw = dict(cu_seqlens=None if single else i["cu"], A=i["A"], dt_bias=i["dt_bias"], qk_eps=i["qk_eps"])
    kw.update(more)
    o = ssd.gated_delta_step(i["q"], i["k"], i["v"], i["gate"], i["beta"], i["cache"], i["read"], i["write"], **kw)
    torch.cuda.synchronize()
    return o


def check(i, before, o, what, skip=(), **kw):
    """o and every slot of the cache; the tokens and write slots of skipped sequences stay as they were."""
    cu = i["cu"].tolist()
    read, write, keep = i["read"].clone(), i["write"].clone(), torch.ones(o.shape[0], dtype=torch.bool)
    for s in skip:
        read[s] = -1
        write[cu[s]:cu[s + 1]] = -1
        keep[cu[s]:cu[s + 1]] = False
    want, err, cache, cache_err = ref.gated_delta(i["q"], i["k"], i["v"], i["gate"], i["beta"], before, read, write,
                                                  i["cu"], A=i["A"], dt_bias=i["dt_bias"], qk_eps=i["qk_eps"], **kw)
    a = ref.check(o.cpu()[keep], want[keep], ref.rounded(want, err, o.dtype)[keep], f"{what}: o")
    b = ref.check(i["cache"], cache, cache_err, f"{what}: states")
    return a, b


CASES = [
    # counts, value heads, key heads, dk, dv, type, gates' type, raw gates, elements before each row
    ([1], 1, 1, 64, 1, F32, F32, False, 0), ([1], 32, 16, 128, 128, BF, BF, True, 0), ([1] * 5, 6, 2, 128, 48, BF, F32, False, 3),
    ([1] * 3, 4, 4, 256, 100, F32, BF, True, 1), ([2, 0, 5, 1], 4, 2, 128, 64, BF, BF, True, 8),
    ([3, 1], 3, 1, 64, 33, F32, F32, True, 0), ([0, 0, 4], 2, 1, 256, 17, BF, F32, False, 5),
    ([70], 2, 2, 128, 40, F32, F32, False, 0), ([4] * 9, 8, 4, 64, 80, BF, BF, True, 1), ([1, 2, 3, 4], 16, 2, 128, 128, F32, F32, True, 4),
]


@pytest.mark.parametrize("c", range(len(CASES)))
def test_against_float64(c):
    counts, H, G, dk, dv, dtype, gate_dtype, raw, pad = CASES[c]
    log(f"gated delta step {CASES[c]}")
    i = inputs(counts, H, G, dk, dv, dtype, gate_dtype, raw, seed=c, pad=pad)
    before = i["cache"].clone()
    worst = check(i, before, call(i), f"case {c}")
    log(f"  worst {worst[0]:.3f} and {worst[1]:.3f} of the bounds")


def test_one_token_each_without_cu_seqlens_is_the_same_call():
    i = inputs([1] * 7, 4, 2, 128, 96, BF, BF, True, seed=1)
    before = i["cache"].clone()
    a = call(i)
    first = i["cache"].clone()
    i["cache"].copy_(before)
    assert torch.equal(call(i, single=True), a) and torch.equal(i["cache"], first)


@pytest.mark.parametrize("dk,dv,S,dtype", [(64, 20, 24, F32), (128, 20, 24, BF), (128, 9, 260, F32), (64, 130, 10, BF)])
def test_many_sequences_equal_each_alone(dk, dv, S, dtype):
    """Batches that take one or two rows a lane: the same bits as each sequence alone, at the float64 bound."""
    i = inputs([1 + s % 2 for s in range(S)], 32, 16, dk, dv, dtype, seed=41)
    before = i["cache"].clone()
    o = call(i)
    check(i, before, o, f"{S} sequences") if S < 100 else None
    cu = i["cu"].tolist()
    for s in (0, 1, S // 2, S - 1):
        t = slice(cu[s], cu[s + 1])
        one = dict(i, read=i["read"][s:s + 1], write=i["write"][t], cu=i["cu"][s:s + 2] - cu[s], cache=before.clone(),
                   **{n: i[n][t] for n in ("q", "k", "v", "gate", "beta")})
        assert torch.equal(call(one), o[t]) and torch.equal(one["cache"][one["write"].long()], i["cache"][i["write"][t].long()])


def test_slots_in_place_fresh_unsaved_and_refused():
    i = inputs([1, 2, 1, 3, 1, 2], 4, 2, 128, 70, BF, F32, False, seed=3)
    slots, cu = i["cache"].shape[0], i["cu"].tolist()
    i["write"][cu[0]] = i["read"][0]          # in place
    i["write"][cu[1]] = i["read"][1]          # the first of two tokens in place, the second elsewhere
    i["read"][2] = -1                         # fresh
    i["write"][cu[3] + 1] = -1                # the middle of three states is not kept
    i["read"][4] = slots                      # refused
    i["write"][cu[5] + 1] = slots + 7         # refused for its last token's slot
    before = i["cache"].clone()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((10, 4, 70), 3.0, dtype=BF, device="cuda")
    call(i, o=o, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_SLOT
    assert (o[cu[4]:] == 3).all()
    check(i, before, o, "slots", skip=(4, 5))


def test_sequences_outside_the_batch_are_refused():
    i = inputs([2, 3, 2], 2, 1, 64, 32, F32, seed=4)
    before = i["cache"].clone()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    i["cu"][1:3] = torch.tensor([9, 5], dtype=torch.int32)   # 0 .. 9, 9 .. 5, 5 .. 7 of 7 tokens
    o = torch.full((7, 2, 32), 3.0, device="cuda")
    call(i, o=o, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_CU_SEQLENS
    assert (o[:5] == 3).all()
    for slot in i["write"][:5].tolist():
        assert torch.equal(i["cache"][slot], before[slot])
    j = dict(i, cu=torch.tensor([0, 2], dtype=torch.int32), read=i["read"][2:], write=i["write"][5:])
    for name in ("q", "k", "v", "gate", "beta"):
        j[name] = i[name][5:]
    check(j, before, o[5:], "the last sequence")


def test_given_scale_strided_output_and_no_bias():
    i = inputs([1] * 4, 4, 2, 64, 24, BF, BF, True, seed=5)
    before, wide = i["cache"].clone(), torch.full((4, 4 * 24 + 5), 7.0, dtype=BF, device="cuda")
    o = wide[:, 5:].unflatten(1, (4, 24))
    i["dt_bias"] = None
    call(i, scale=0.3, o=o)
    assert (wide[:, :5] == 7).all()
    check(i, before, o.contiguous(), "scale", scale=0.3)


def test_no_decay_full_decay_and_strengths_of_zero_and_one():
    """e^0 and e^-inf are exact; with beta 1 and a unit key a write stores the value under the key."""
    i = inputs([1] * 4, 2, 1, 64, 16, F32, seed=6)
    i["gate"][0], i["gate"][1] = 0.0, -float("inf")
    i["beta"][2], i["beta"][3] = 0.0, 1.0
    before = i["cache"].clone()
    check(i, before, call(i), "edges")
    assert torch.isfinite(i["cache"]).all()


def test_padded_batch():
    """Tokens behind the last sequence are not computed, whatever they hold."""
    i = inputs([2, 1, 4], 4, 2, 64, 24, BF, BF, True, seed=11)
    before = i["cache"].clone()
    i["cu"] = torch.tensor([0, 2, 3], dtype=torch.int32).cuda()
    i["read"], i["v"][3:], i["write"][3:] = i["read"][:2].clone(), float("nan"), 2 ** 31 - 1
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((7, 4, 24), 3.0, dtype=BF, device="cuda")
    call(i, o=o, error_flag=flag)
    assert int(flag.item()) == 0 and (o[3:] == 3).all()
    j = dict(i, write=i["write"][:3])
    for name in ("q", "k", "v", "gate", "beta"):
        j[name] = i[name][:3]
    check(j, before, o[:3], "padded")


def test_nothing_to_do():
    i = inputs([0, 0], 2, 1, 64, 16, BF, seed=7)
    before = i["cache"].clone()
    assert call(i).shape == (0, 2, 16) and torch.equal(i["cache"], before)
    e = inputs([], 2, 1, 64, 16, BF, seed=7)
    assert call(e).shape == (0, 2, 16)


def test_equals_the_chunk_call():
    """Prompts through the chunk call and through this one: the same rule, to the chunk call's tolerance."""
    counts = [130, 64, 3]
    i = inputs(counts, 4, 2, 128, 64, BF, seed=8)
    meta = ssd.varlen_metadata(i["cu"], 64, total_tokens=sum(counts))
    read = i["read"].long()
    want, final = ssd.gated_delta_chunk_varlen(i["q"].contiguous(), i["k"].contiguous(), i["v"].contiguous(),
                                               i["gate"].contiguous(), i["beta"].contiguous(), meta,
                                               initial_states=i["cache"][read].contiguous())
    o = call(i)
    ends = i["write"][i["cu"][1:].long() - 1].long()
    torch.testing.assert_close(o.float(), want.float(), atol=2e-2, rtol=2e-2)
    torch.testing.assert_close(i["cache"][ends], final, atol=2e-2, rtol=2e-2)


def test_captured_and_replayed():
    i = inputs([1] * 6, 4, 2, 128, 64, BF, BF, True, seed=9)
    before = i["cache"].clone()
    want = call(i).clone()
    states = i["cache"].clone()
    o = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ssd.gated_delta_step(i["q"], i["k"], i["v"], i["gate"], i["beta"], i["cache"], i["read"], i["write"], o=o,
                                 A=i["A"], dt_bias=i["dt_bias"], qk_eps=i["qk_eps"])
    torch.cuda.synchronize()
    for _ in range(3):
        i["cache"].copy_(before)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(i["cache"], states)


def test_slots_past_32_bit_offsets():
    """Slots whose states begin past 2^32 bytes and past 2^31 elements."""
    H, dv, dk = 32, 128, 128
    slots = 2 ** 31 // (H * dv * dk) + 3
    i = inputs([1, 1], H, 16, dk, dv, BF, BF, True, seed=10)
    big = torch.zeros(slots, H, dv, dk, device="cuda")
    big[slots - 1].copy_(i["cache"][0])
    big[slots - 3].copy_(i["cache"][1])
    small = dict(i, cache=torch.stack([i["cache"][0], i["cache"][1], torch.zeros_like(i["cache"][0]), torch.zeros_like(i["cache"][0])]),
                 read=torch.tensor([0, 1], dtype=torch.int32).cuda(), write=torch.tensor([2, 3], dtype=torch.int32).cuda())
    want = call(small)
    i.update(cache=big, read=torch.tensor([slots - 1, slots - 3], dtype=torch.int32).cuda(),
             write=torch.tensor([slots - 2, slots - 3], dtype=torch.int32).cuda())
    assert torch.equal(call(i), want)
    assert torch.equal(big[slots - 2], small["cache"][2]) and torch.equal(big[slots - 3], small["cache"][3])
