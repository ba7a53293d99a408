"""Every form in which the selective scan and its step are launched at the sizes of real batches, against float64 with
the bound of tests/selective_bound.py: the walk and 2, 4, 8 and 16 waves of segments, several sequences of a step in one
workgroup, and products of decays that leave float32's range."""
import pytest
import torch

import selective_bound as bound
import selective_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd
from test_gpu_selective import BF, F32, call, cpu, make, starts, step, step_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def on_words(i, n):
    """Rows of B and C on 4-byte boundaries, which the walk needs."""
    wide = torch.cat([i["B"].flatten(1), i["C"].flatten(1)], 1).contiguous()
    half = i["B"].shape[1] * n
    i["B"], i["C"] = wide[:, :half].unflatten(1, (-1, n)), wide[:, half:].unflatten(1, (-1, n))


def one_sequence(c, s):
    """The float64 reference of sequence s of a batch on the CPU."""
    t0 = sum(c["lengths"][:s])
    r = slice(t0, t0 + c["lengths"][s])
    return bound.scan(c["u"][r], c["dt"][r], c["A"], c["B"][r], c["C"][r], c["dt_bias"], c["D"],
                      None if c["z"] is None else c["z"][r], starts(c, s)) + (r,)


# sequences and channels that are walked, and that go in segments
FORMS = {"walk": (256, 1040), "segments": (2, 48)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [16, 32])
def test_an_infinite_state_meets_vanishing_decays(form, n):
    """Decays of 1e-7 each leave an infinite state infinite, token by token; their product over a few tokens is below
    float32's least number. A decay that is itself 0 makes it NaN."""
    s, d = FORMS[form]
    i = make([43] * s, d, n, 1, F32, gate=False, init="none", seed=80, skip=False)
    on_words(i, n)
    i["dt"][:] = 1.0
    i["dt_bias"] = None
    delta = float(ref.softplus(torch.tensor(1.0, dtype=torch.float64)))
    i["A"][:] = -16.1 / delta     # e^-16.1 = 1.0e-7: eight of them are 1e-56
    i["A"][3] = -90.0 / delta     # below 2^-126: 0
    i["B"][2, 0, 5] = float("inf")
    fin = call(i)[1].cpu()
    other = [k for k in range(n) if k != 5]
    want = torch.where(i["u"][2].cpu() > 0, float("inf"), float("-inf"))
    want[3] = float("nan")
    assert torch.equal(torch.nan_to_num(fin[0, :, 5], nan=1.0), torch.nan_to_num(want, nan=1.0))
    assert torch.isfinite(fin[0][:, other]).all() and torch.isfinite(fin[1:]).all()


@pytest.mark.parametrize("form", FORMS)
def test_growing_states_whose_decays_overflow_together(form):
    """Rates above zero: a state of 0 stays 0 and one of 1e-30 grows to a finite one, although the product of the
    growth factors over eight tokens is more than float32 holds."""
    s, d = FORMS[form]
    lengths = [8, 40] * (s // 2)
    i = make(lengths, d, 16, 1, F32, gate=False, init="all", seed=81, skip=False)
    on_words(i, 16)
    i["dt"][:] = 0.5
    i["dt_bias"] = None
    i["A"][:] = 12.5 / float(ref.softplus(torch.tensor(0.5, dtype=torch.float64)))   # e^12.5 a token, e^100 for eight
    c0, c1 = i["init"][0::2], i["init"][1::2]
    c0.mul_(1e-30)
    c1.fill_(0.0)
    i["u"][:] = 0.0
    ends = torch.tensor(lengths).cumsum(0) - 1
    i["u"][ends[1::2].cuda()] = 1.0     # the longer sequences get their one input at the last token
    y, fin, _ = call(i)
    c = cpu(i)
    for k in (0, 1):
        ry, rh, by, bh, r = one_sequence(c, k)
        ref.check(fin[k], rh[-1], bh[-1], f"state {k}")
        ref.check(y[r], ry, by, f"y {k}")


@pytest.mark.parametrize("form", FORMS)
def test_vanishing_decays_of_large_states(form):
    """States of 1e30 through segments whose decays' product is below, near and above float32's least number."""
    s, d = FORMS[form]
    i = make([8] * s, d, 16, 1, F32, gate=False, init="all", seed=82, skip=False)
    on_words(i, 16)
    i["dt"][:] = 1.0
    i["dt_bias"] = None
    i["A"][:] = -torch.linspace(1.0, 14.0, d).cuda()[:, None]
    i["init"].mul_(1e30)
    y, fin, _ = call(i)
    c = cpu(i)
    for k in (0, 1):
        ry, rh, by, bh, r = one_sequence(c, k)
        ref.check(fin[k], rh[-1], bh[-1], f"state {k}")
        ref.check(y[r], ry, by, f"y {k}")


def check_sequences(i, y, fin, cst, chunk, sequences):
    """y, final and exported states of some sequences of a batch; returns the worst part of the bound."""
    c, worst = cpu(i), 0.0
    first = [0]
    for v in i["lengths"]:
        first.append(first[-1] + -(-v // chunk))
    for s in sequences:
        ry, rh, by, bh, r = one_sequence(c, s)
        n = i["lengths"][s]
        if n == 0:
            start = starts(c, s)
            assert torch.equal(fin[s].cpu(), torch.zeros_like(fin[s].cpu()) if start is None else start), f"empty {s}"
            continue
        worst = max(worst, ref.check(y[r], ry, by, f"y of {s}"), ref.check(fin[s], rh[-1], bh[-1], f"state of {s}"))
        for k in range(-(-n // chunk) if cst is not None else 0):
            last = min(chunk * (k + 1), n) - 1
            worst = max(worst, ref.check(cst[first[s] + k], rh[last], bh[last], f"chunk {k} of {s}"))
    return worst


SMALL = [
    # lengths, channels, states, groups, type, type of dt, gate, initial states: 16 waves of segments
    ([1], 16, 16, 1, BF, None, True, "none"), ([17, 64, 47], 64, 16, 1, F32, None, True, "even"),
    ([15, 0, 1, 33, 0], 100, 16, 2, BF, F32, True, "even"), ([129, 70], 24, 32, 3, F32, BF, True, "all"),
    ([300, 19], 72, 64, 2, BF, None, True, "all"), ([65, 31], 10, 128, 1, F32, None, False, "even"),
    ([90, 50], 18, 256, 1, BF, None, True, "all"), ([1037, 3], 31, 16, 1, F32, None, True, "even"),
]


@pytest.mark.parametrize("k", range(len(SMALL)))
def test_sixteen_waves(k):
    lengths, d, n, g, dtype, dt_dtype, gate, init = SMALL[k]
    log(f"segments {SMALL[k]}")
    i = make(lengths, d, n, g, dtype, dt_dtype, gate, init, seed=100 + k)
    meta = ssd.varlen_metadata(i["cu"], 16, total_tokens=sum(lengths))
    cst = torch.full((meta.max_chunks, d, n), float("nan"), device="cuda")
    y, fin, meta = call(i, chunk=16, chunk_states=cst)
    assert int(meta.error_flag.item()) == 0
    log(f"  worst {check_sequences(i, y, fin, cst, 16, range(len(lengths))):.3f} of the bound")


# A workgroup of segments has 2, 4 or 8 waves by the number of (sequence, 16 channels) pairs; each of its waves takes
# several segments here, and sequences end in whole and in partial ones.
WAVES = [
    # waves, sequences, tokens of the longest, channels, states, groups, type, gate, initial states
    (8, 9, 210, 520, 16, 1, BF, True, "even"), (8, 12, 150, 400, 64, 2, F32, False, "all"),
    (8, 260, 140, 12, 32, 1, BF, True, "even"), (8, 9, 140, 530, 256, 1, F32, True, "all"),
    (4, 24, 120, 520, 16, 1, F32, True, "even"), (4, 50, 90, 264, 128, 8, BF, True, "none"),
    (4, 200, 70, 90, 32, 3, F32, False, "even"), (2, 500, 70, 528, 64, 1, BF, True, "even"),
    (2, 1030, 60, 250, 64, 2, F32, False, "all"), (2, 300, 50, 1030, 16, 1, BF, True, "even"),
]


@pytest.mark.parametrize("k", range(len(WAVES)))
def test_two_to_eight_waves(k):
    waves, s, longest, d, n, g, dtype, gate, init = WAVES[k]
    log(f"segments {WAVES[k]}")
    pairs = s * g * -(-(d // g) // 16)
    assert {8: 256 < pairs < 768, 4: 768 <= pairs < 16384, 2: pairs >= 16384}[waves], pairs
    # (16 and 32 states: rows of B and C off 4-byte boundaries, or too few pairs, so that nothing is walked)
    lengths = torch.randint(0, longest + 1, (s,), generator=torch.Generator().manual_seed(k)).tolist()
    lengths[:6] = [longest, 16 * waves, 8 * waves + 3, 0, 1, 8]
    i = make(lengths, d, n, g, dtype, None, gate, init, seed=120 + k)
    meta = ssd.varlen_metadata(i["cu"], 32, total_tokens=sum(lengths))
    cst = torch.full((meta.max_chunks, d, n), float("nan"), device="cuda")
    y, fin, meta = call(i, chunk=32, chunk_states=cst)
    assert int(meta.error_flag.item()) == 0
    assert torch.isfinite(fin).all() and torch.isfinite(y).all()
    used = sum(-(-v // 32) for v in lengths)
    assert torch.isfinite(cst[:used]).all() and torch.isnan(cst[used:]).all()
    log(f"  worst {check_sequences(i, y, fin, cst, 32, [0, 1, 2, 3, 4, 5, s // 2, s - 1]):.3f} of the bound")


@pytest.mark.parametrize("n,dtype,dt_dtype,gate,g", [(16, BF, F32, True, 1), (32, F32, None, False, 2)])
def test_walk(n, dtype, dt_dtype, gate, g):
    """4096 and more pairs; a sequence more than 3 times the mean goes in segments beside the walk."""
    r = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, 45, (258,), generator=r).tolist()
    lengths[:6] = [400, 64, 33, 0, 1, 2]
    i = make(lengths, 1044, n, g, dtype, dt_dtype, gate, "even", seed=140 + n)
    on_words(i, n)
    meta = ssd.varlen_metadata(i["cu"], 32, total_tokens=sum(lengths))
    cst = torch.full((meta.max_chunks, 1044, n), float("nan"), device="cuda")
    y, fin, meta = call(i, chunk=32, chunk_states=cst)
    assert int(meta.error_flag.item()) == 0
    assert torch.isfinite(fin).all() and torch.isfinite(y).all()
    log(f"  worst {check_sequences(i, y, fin, cst, 32, [0, 1, 2, 3, 4, 5, 129, 257]):.3f} of the bound")


# A step takes two sequences to a workgroup from 2048 workgroups on (channels of a workgroup: 1024 / states).
STEPS = [
    # sequences, channels, states, groups, type, type of dt, gate
    (257, 1040, 16, 1, BF, None, True), (301, 1752, 32, 3, F32, BF, False), (121, 1100, 128, 2, BF, F32, True),
    (4097, 70, 16, 1, F32, None, True), (65, 1008, 256, 1, BF, None, True),
]


@pytest.mark.parametrize("k", range(len(STEPS)))
def test_step_of_two_sequences_a_workgroup(k):
    """An odd number of sequences, with fresh, unsaved, in-place and refused ones in both places of a pair."""
    s, d, n, g, dtype, dt_dtype, gate = STEPS[k]
    log(f"step {STEPS[k]}")
    assert -(-s // 2) * -(-d // (1024 // n)) >= 2048
    i = step_inputs(s, d, n, g, dtype, dt_dtype, gate, seed=160 + k)
    slots = i["cache"].shape[0]
    for at in (4, 7):                     # first and second of a pair, and the same again where the last one stands alone
        i["read"][at] = -1
        i["write"][at + 4] = -1
        i["write"][at + 8] = i["read"][at + 8].clone()
        i["read"][at + 12] = slots
        i["write"][at + 16] = slots + 5
    i["read"][-1] = slots + 1
    refused = [16, 19, 20, 23, s - 1]
    before = i["cache"].clone()
    y = torch.full((s, d), 3.0, dtype=dtype, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    step(i, y=y, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_SLOT
    assert (y[refused] == 3).all()
    c, old, new = cpu(i), before.cpu(), i["cache"].cpu()
    written = set()
    for q in range(s):
        rs, ws = int(c["read"][q]), int(c["write"][q])
        if q in refused:
            continue
        r = slice(q, q + 1)
        if q < 30 or q % 16 == 1 or q > s - 4:
            ry, rh, by, bh = bound.scan(c["u"][r], c["dt"][r], c["A"], c["B"][r], c["C"][r], c["dt_bias"], c["D"],
                                        None if c["z"] is None else c["z"][r], old[rs] if rs >= 0 else None)
            ref.check(y[r], ry, by, f"y of {q}")
            if ws >= 0:
                ref.check(new[ws], rh[-1], bh[-1], f"state of {q}")
        written.add(ws)
    kept = [v for v in range(slots) if v not in written]
    assert torch.equal(new[kept], old[kept]), "a slot that no sequence writes was written"
    assert torch.isfinite(new).all() and torch.isfinite(y).all()
    # alone, one sequence a workgroup: the same bits
    some = [0, 1, 4, 8, 12, s - 2]
    pick = torch.tensor(some, device="cuda")
    j = {**i, **{name: None if i[name] is None else i[name][pick] for name in ("u", "dt", "B", "C", "z")},
         "cache": before.clone(), "read": i["read"][pick], "write": i["write"][pick]}
    assert torch.equal(step(j), y[pick])
    for q in some:
        ws = int(c["write"][q])
        if ws >= 0:
            assert torch.equal(j["cache"][ws], i["cache"][ws]), f"state of {q}"


@pytest.mark.parametrize("s,d", [(5, 48), (260, 1040)], ids=["segments", "walk"])
def test_graph_of_metadata_and_scan_replays_with_other_lengths(s, d):
    """The same number of sequences and tokens, cut elsewhere before every replay (a long one among short ones, empty
    ones): what is chosen on the host holds for any cut."""
    total = 20 * s
    i = make([20] * s, d, 16, 1, BF, init="all", seed=180)
    on_words(i, 16)
    y = torch.empty_like(i["u"])
    fin = torch.empty(s, d, 16, device="cuda")
    cu = i["cu"].clone()

    def both():
        meta = ssd.varlen_metadata(cu, 16, total_tokens=total)
        ssd.selective_scan_varlen(i["u"], i["dt"], i["A"], i["B"], i["C"], meta, dt_bias=i["dt_bias"], D=i["D"], z=i["z"],
                                  initial_states=i["init"], y=y, final_states=fin)
        return meta
    with torch.cuda.stream(torch.cuda.Stream()):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    r = torch.Generator().manual_seed(181)
    for turn in range(4):
        cuts = torch.randint(0, total + 1, (s - 1,), generator=r).sort().values
        if turn == 1:
            cuts[:] = 0                      # one sequence has all the tokens
        if turn == 2:
            cuts = torch.cat([cuts[:s // 2].clamp(max=total // 2).sort().values, torch.full((s - 1 - s // 2,), total)])
        now = torch.cat([torch.tensor([0]), cuts, torch.tensor([total])]).to(torch.int32)
        cu.copy_(now)
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, fin)]
        y.fill_(-1.0)
        fin.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(fin, want[1]), f"replay {turn}"
        lengths = (now[1:] - now[:-1]).tolist()
        j = {**i, "lengths": lengths, "has": None}
        longest = max(range(s), key=lambda k: lengths[k])
        check_sequences(j, y, fin, None, 16, [longest] if lengths[longest] > 1500 else [longest, 0, s - 1])
