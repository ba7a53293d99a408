"""The selective scan and its single-token step against a float64 recurrence: types, odd widths, groups, strided
rows, lengths from none to thousands, continued and fresh sequences, exported states, refused slots, non-finite
neighbours, graph replays, two streams, and prompts continued token by token."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def make(lengths, d, n, g, dtype=BF, dt_dtype=None, gate=True, init="even", seed=0, slow=False, skip=True):
    """Random inputs on the GPU; z, B and C are slices of wider rows."""
    r = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=r)   # noqa: E731
    t, s = sum(lengths), len(lengths)
    wide = normal(t, 2 * g * n + 3).to(dtype).cuda() * n ** -0.5
    rates = torch.rand(d, n, generator=r) * (0.02 if slow else 2.7)
    return dict(
        lengths=lengths, u=normal(t, d).to(dtype).cuda(), dt=normal(t, d).to(dt_dtype or dtype).cuda(),
        A=-(torch.exp(rates) - (1.0 if slow else 0.0)).cuda(),
        B=wide[:, 3:3 + g * n].unflatten(1, (g, n)), C=wide[:, 3 + g * n:].unflatten(1, (g, n)),
        dt_bias=(-4 + 2 * torch.rand(d, generator=r)).cuda(), D=normal(d).cuda() if skip else None,
        z=normal(t, 2 * d + 1).to(dtype).cuda()[:, d + 1:] if gate else None,
        init=None if init == "none" else 0.5 * normal(s, d, n).cuda(),
        has=None if init in ("none", "all") else torch.tensor([i % 2 == 0 for i in range(s)], dtype=torch.int32).cuda(),
        cu=torch.tensor([0] + list(lengths), dtype=torch.int32).cumsum(0).to(torch.int32).cuda())


def call(i, chunk=64, **kw):
    meta = ssd.varlen_metadata(i["cu"], chunk, total_tokens=sum(i["lengths"]))
    y, fin = ssd.selective_scan_varlen(i["u"], i["dt"], i["A"], i["B"], i["C"], meta, dt_bias=i["dt_bias"], D=i["D"],
                                       z=i["z"], initial_states=i["init"], has_initial_state=i["has"], **kw)
    torch.cuda.synchronize()
    return y, fin, meta


def cpu(i):
    return {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in i.items()}


def starts(i, s):
    if i["init"] is None or (i["has"] is not None and int(i["has"][s]) == 0):
        return None
    return i["init"][s]


def expected(i):
    """Per sequence: (y, states after every token, bounds, start)."""
    c = cpu(i)
    out, t = [], 0
    for s, n in enumerate(i["lengths"]):
        r = slice(t, t + n)
        t += n
        got = ref.scan(c["u"][r], c["dt"][r], c["A"], c["B"][r], c["C"][r], c["dt_bias"], c["D"],
                       None if c["z"] is None else c["z"][r], starts(c, s))
        out.append(got + (starts(c, s),))
    return out


def check_all(i, y, fin, what):
    t, worst = 0, 0.0
    for s, (ry, rh, by, bh, start) in enumerate(expected(i)):
        n = i["lengths"][s]
        worst = max(worst, ref.check(y[t:t + n], ry, by, f"{what}: y of sequence {s}"))
        t += n
        if n == 0:
            want = torch.zeros_like(fin[s].cpu()) if start is None else start
            assert torch.equal(fin[s].cpu(), want), f"{what}: state of the empty sequence {s}"
        else:
            worst = max(worst, ref.check(fin[s], rh[-1], bh[-1], f"{what}: final state {s}"))
    return worst


SHAPES = [
    # lengths, channels, states, groups, type, type of dt, gate, initial states
    ([1], 16, 16, 1, BF, None, True, "none"),
    ([1], 1, 16, 1, F32, None, False, "all"),
    ([5], 17, 16, 1, BF, F32, True, "all"),
    ([16], 64, 16, 1, F32, BF, True, "none"),
    ([17, 64, 47], 64, 16, 1, F32, None, True, "even"),
    ([15, 0, 1, 33, 0], 100, 16, 2, BF, None, True, "even"),
    ([0, 0, 3], 40, 16, 8, BF, None, False, "all"),
    ([255, 256, 257], 48, 16, 1, BF, None, True, "even"),
    ([129, 70], 24, 32, 3, F32, None, True, "all"),
    ([77, 200, 2], 33, 32, 1, BF, None, True, "even"),
    ([130], 20, 64, 1, F32, None, False, "none"),
    ([19, 300], 72, 64, 2, BF, None, True, "all"),
    ([65, 31], 10, 128, 1, BF, None, True, "even"),
    ([40, 1], 35, 128, 5, F32, None, True, "none"),
    ([50, 90], 18, 256, 1, F32, None, True, "all"),
    ([33], 130, 256, 2, BF, F32, False, "none"),
    ([1037, 3], 31, 16, 1, BF, None, True, "even"),
]


@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_scan_against_float64(k):
    lengths, d, n, g, dtype, dt_dtype, gate, init = SHAPES[k]
    i = make(lengths, d, n, g, dtype, dt_dtype, gate, init, seed=k)
    log(f"scan {SHAPES[k]}")
    y, fin, meta = call(i)
    worst = check_all(i, y, fin, f"scan {k}")
    assert int(meta.error_flag.item()) == 0
    log(f"  worst {worst:.3f} of the bound")


def test_scan_without_bias_or_skip():
    i = make([90, 20], 50, 16, 1, F32, skip=False, seed=3)
    i["dt_bias"] = None
    i["dt"] = i["dt"] - 3
    y, fin, _ = call(i)
    check_all(i, y, fin, "no bias, no skip")


def test_scan_long_slow_decay():
    """A state that forgets over thousands of tokens: errors add up over as many."""
    i = make([9001], 20, 16, 1, BF, seed=5, slow=True)
    y, fin, _ = call(i, chunk=256)
    check_all(i, y, fin, "slow decay")


def test_scan_extreme_steps():
    """Step sizes of zero (dt of -inf: the state stays, as a padded token would leave it) and very large ones
    (the state is replaced), and steps far down softplus's tail."""
    i = make([64, 40], 32, 16, 1, F32, gate=False, init="all", seed=6)
    i["dt"][5:20] = float("-inf")
    i["dt"][30:34] = 500.0
    i["dt"][64:80] = -30.0
    y, fin, _ = call(i)
    c = cpu(i)
    c["dt"][5:20] = -1e30   # softplus of either is zero
    t = 0
    for s, n in enumerate(i["lengths"]):
        r = slice(t, t + n)
        ry, rh, by, bh = ref.scan(c["u"][r], c["dt"][r], c["A"], c["B"][r], c["C"][r], c["dt_bias"], c["D"], None,
                                  c["init"][s])
        ref.check(y[r], ry, by, f"y {s}")
        ref.check(fin[s], rh[-1], bh[-1], f"state {s}")
        t += n


def test_scan_chunk_size_changes_nothing():
    i = make([300, 17, 1, 64], 80, 16, 2, BF, seed=7)
    y0, f0, _ = call(i, chunk=16)
    for chunk in (64, 256):
        y, f, _ = call(i, chunk=chunk)
        assert torch.equal(y, y0) and torch.equal(f, f0)


def test_scan_repeats_bit_for_bit():
    i = make([700, 333, 90], 512, 16, 1, BF, seed=8)
    y0, f0, _ = call(i)
    for _ in range(3):
        y, f, _ = call(i)
        assert torch.equal(y, y0) and torch.equal(f, f0)


def test_scan_sequences_do_not_touch_each_other():
    """NaN and infinities in one sequence, and beside the rows of a slice, stay there."""
    i = make([40, 50, 60], 48, 16, 1, BF, seed=9)
    y0, f0, _ = call(i)
    j = dict(i)
    for name in ("u", "dt", "B", "C", "z"):
        wide = torch.full((150, i[name][0].numel() + 7), float("nan"), dtype=i[name].dtype, device="cuda")
        part = wide[:, 4:4 + i[name][0].numel()].unflatten(1, i[name].shape[1:])
        part.copy_(i[name])
        part[40:90] = float("nan") if name != "u" else float("inf")
        j[name] = part
    out = torch.full((150, 48 + 5), 7.0, dtype=BF, device="cuda")
    y, f, _ = call(j, y=out[:, 3:51])
    for r, s in ((slice(0, 40), 0), (slice(90, 150), 2)):
        assert torch.equal(y[r], y0[r]) and torch.equal(f[s], f0[s])
    assert torch.isnan(f[1]).any()
    assert (out[:, :3] == 7).all() and (out[:, 51:] == 7).all()


@pytest.mark.parametrize("chunk,n", [(16, 16), (64, 16), (64, 64), (256, 16)])
def test_scan_exports_every_chunk(chunk, n):
    i = make([130, 0, 16, 300, 1], 40, n, 1, BF, seed=10)
    meta = ssd.varlen_metadata(i["cu"], chunk, total_tokens=447)
    cst = torch.full((meta.max_chunks, 40, n), float("nan"), device="cuda")
    y, fin, meta = call(i, chunk=chunk, chunk_states=cst)
    check_all(i, y, fin, "export")
    c = 0
    for s, (_, rh, _, bh, _) in enumerate(expected(i)):
        for first in range(0, i["lengths"][s], chunk):
            last = min(first + chunk, i["lengths"][s]) - 1
            ref.check(cst[c], rh[last], bh[last], f"chunk {c}")
            c += 1
    assert torch.isnan(cst[c:]).all(), "slots past the last chunk were written"


def test_scan_checkpoints_through_the_plan_and_refuses_bad_slots():
    i = make([300, 70, 513], 24, 16, 1, F32, seed=11)
    chunk, block, slots = 64, 128, 12
    meta = ssd.varlen_metadata(i["cu"], chunk, total_tokens=883)
    table = torch.tensor([[4, -1, 9, -1, -1], [0, -1, -1, -1, -1], [1, 2, 3, 11, 5]], dtype=torch.int32)
    _, dst = ssd.export_chunk_states(meta, table, block, num_slots=slots)
    cache = torch.full((slots, 24, 16), 5.0, device="cuda")
    y, fin, m = call(i, chunk=chunk, chunk_states=cache, chunk_state_dst=dst)
    want = {4: (0, 128), 9: (0, 300), 0: (1, 70), 1: (2, 128), 2: (2, 256), 3: (2, 384), 11: (2, 512), 5: (2, 513)}
    e = expected(i)
    for slot in range(slots):
        if slot in want:
            s, end = want[slot]
            ref.check(cache[slot], e[s][1][end - 1], e[s][3][end - 1], f"slot {slot}")
        else:
            assert (cache[slot] == 5).all(), f"slot {slot} was written"
    bad = dst.clone()
    bad[1] = slots   # the second chunk of the first sequence
    cache2 = torch.full_like(cache, 5.0)
    y2, f2, m = call(i, chunk=chunk, chunk_states=cache2, chunk_state_dst=bad)
    assert int(m.error_flag.item()) == ssd.DATA_BAD_SLOT
    assert torch.equal(y2, y) and torch.equal(f2, fin)
    assert (cache2[4] == 5).all()
    keep = [k for k in range(slots) if k != 4]
    assert torch.equal(cache2[keep], cache[keep])


@pytest.mark.parametrize("lengths,d", [([33, 20], 24), ([3, 5] * 32, 8192)], ids=["segments", "walk"])
def test_scan_exports_no_chunk_outside_the_grid(lengths, d):
    """Chunk numbers that the grid does not have (metadata of another batch) are never used as indices."""
    i = make(lengths, d, 16, 1, BF, seed=14)
    i["B"], i["C"] = i["B"].contiguous(), i["C"].contiguous()
    meta = ssd.varlen_metadata(i["cu"], 16, total_tokens=sum(lengths))
    meta.seq_chunk_start[0] = 10 ** 9
    meta.seq_chunk_start[1] = -10 ** 6
    dst = torch.arange(meta.max_chunks, dtype=torch.int32, device="cuda")
    cst = torch.full((meta.max_chunks, d, 16), 7.0, device="cuda")
    y, fin = ssd.selective_scan_varlen(i["u"], i["dt"], i["A"], i["B"], i["C"], meta, i["dt_bias"], i["D"], i["z"],
                                       i["init"], i["has"], chunk_states=cst, chunk_state_dst=dst)
    own = [int(c) for s, c in enumerate(meta.seq_chunk_start[:-1].tolist()) if s > 1]
    rest = [c for c in range(meta.max_chunks) if c not in own]
    assert int(meta.error_flag.item()) == 0
    assert (cst[rest] == 7).all()
    want = call(i, chunk=16)
    assert torch.equal(y, want[0]) and torch.equal(fin, want[1])
    assert torch.equal(cst[own], fin[2:])


def test_scan_of_malformed_cu_seqlens_writes_nothing():
    i = make([20, 30], 16, 16, 1, F32, seed=12)
    i["cu"] = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
    y = torch.full((50, 16), 3.0, device="cuda")
    fin = torch.full((2, 16, 16), 3.0, device="cuda")
    _, _, m = call(i, y=y, final_states=fin)
    assert int(m.error_flag.item()) & ssd.DATA_BAD_CU_SEQLENS
    assert (y == 3).all() and (fin == 3).all()


def test_scan_continues_from_its_final_state():
    """A prompt in two bites equals the prompt in one (the cut moves the sums' order only)."""
    i = make([400], 64, 16, 1, F32, init="all", seed=13)
    whole = expected(i)[0]
    first = {**i, "lengths": [150], "cu": torch.tensor([0, 150], dtype=torch.int32, device="cuda"),
             **{k: i[k][:150] for k in ("u", "dt", "B", "C", "z")}}
    ya, fa, _ = call(first)
    rest = {**i, "lengths": [250], "cu": torch.tensor([0, 250], dtype=torch.int32, device="cuda"), "init": fa,
            **{k: i[k][150:] for k in ("u", "dt", "B", "C", "z")}}
    yb, fb, _ = call(rest)
    ref.check(torch.cat([ya, yb]), whole[0], whole[2], "y")
    ref.check(fb[0], whole[1][-1], whole[3][-1], "state")


def step_inputs(s, d, n, g, dtype, dt_dtype=None, gate=True, seed=0):
    i = make([s], d, n, g, dtype, dt_dtype, gate, "none", seed=seed)
    r = torch.Generator().manual_seed(seed + 99)
    order = torch.randperm(2 * s + 1, generator=r).to(torch.int32)
    i["cache"] = 0.5 * torch.randn(2 * s + 1, d, n, generator=r).cuda()
    i["read"], i["write"] = order[:s].cuda(), order[s:2 * s].cuda()
    return i


def step(i, **kw):
    y = ssd.selective_step(i["u"], i["dt"], i["A"], i["B"], i["C"], i["cache"], i["read"], i["write"],
                           dt_bias=i["dt_bias"], D=i["D"], z=i["z"], **kw)
    torch.cuda.synchronize()
    return y


def check_step(i, before, y, skip=()):
    c = cpu(i)
    untouched = set(range(before.shape[0]))
    for s in range(i["u"].shape[0]):
        if s in skip:
            continue
        rs, ws = int(i["read"][s]), int(i["write"][s])
        r = slice(s, s + 1)
        ry, rh, by, bh = ref.scan(c["u"][r], c["dt"][r], c["A"], c["B"][r], c["C"][r], c["dt_bias"], c["D"],
                                  None if c["z"] is None else c["z"][r], before[rs].cpu() if rs >= 0 else None)
        ref.check(y[r], ry, by, f"y of {s}")
        if ws >= 0:
            ref.check(i["cache"][ws], rh[-1], bh[-1], f"state of {s}")
            untouched.discard(ws)
    for k in untouched:
        assert torch.equal(i["cache"][k], before[k]), f"slot {k} was written"


@pytest.mark.parametrize("s,d,n,g,dtype,dt_dtype,gate", [
    (1, 64, 16, 1, BF, None, True), (1, 1, 16, 1, F32, None, False), (3, 37, 16, 1, BF, F32, True),
    (7, 100, 32, 4, F32, BF, True), (5, 48, 64, 2, BF, None, False), (4, 18, 128, 3, F32, None, True),
    (2, 9, 256, 1, BF, None, True), (33, 520, 16, 8, BF, None, True), (130, 16, 16, 1, F32, None, True),
])
def test_step_against_float64(s, d, n, g, dtype, dt_dtype, gate):
    log(f"step {s, d, n, g, dtype, dt_dtype, gate}")
    i = step_inputs(s, d, n, g, dtype, dt_dtype, gate, seed=s)
    before = i["cache"].clone()
    check_step(i, before, step(i))


def test_step_in_place_fresh_and_unsaved_sequences():
    i = step_inputs(5, 40, 16, 1, BF, seed=2)
    i["write"][0] = i["read"][0]     # in place
    i["read"][1] = -1                # no state yet
    i["write"][2] = -1               # state not kept
    i["read"][3], i["write"][3] = -1, -1
    before = i["cache"].clone()
    check_step(i, before, step(i))


def test_step_from_one_shared_slot():
    i = step_inputs(5, 40, 16, 1, BF, seed=5)
    i["read"][:] = i["read"][2].clone()   # branches of one sequence
    before = i["cache"].clone()
    check_step(i, before, step(i))


def test_step_refuses_slots_past_the_cache():
    i = step_inputs(4, 40, 64, 1, F32, seed=3)
    i["read"][1] = i["cache"].shape[0]
    i["write"][2] = i["cache"].shape[0] + 7
    before = i["cache"].clone()
    y = torch.full((4, 40), 3.0, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    step(i, y=y, error_flag=flag)
    assert int(flag.item()) == ssd.DATA_BAD_SLOT
    assert (y[1:3] == 3).all()
    check_step(i, before, y, skip=(1, 2))


def test_step_takes_int64_and_strided_slots():
    i = step_inputs(6, 32, 16, 1, F32, seed=4)
    before = i["cache"].clone()
    pairs = torch.stack([i["read"].long(), i["write"].long()], 1)
    i["read"], i["write"] = pairs[:, 0], pairs[:, 1]
    check_step(i, before, step(i))


def test_graph_replays_scan_and_step():
    """Captured once, replayed with new inputs in the same buffers, eager work in between."""
    i = make([100, 29], 96, 16, 1, BF, init="all", seed=14)
    k = step_inputs(3, 96, 16, 1, BF, seed=15)
    meta = ssd.varlen_metadata(i["cu"], 64, total_tokens=129)
    y, ys = torch.empty_like(i["u"]), torch.empty_like(k["u"])
    fin = torch.empty(2, 96, 16, device="cuda")

    def both():
        ssd.selective_scan_varlen(i["u"], i["dt"], i["A"], i["B"], i["C"], meta, dt_bias=i["dt_bias"], D=i["D"],
                                  z=i["z"], initial_states=i["init"], y=y, final_states=fin)
        ssd.selective_step(k["u"], k["dt"], k["A"], k["B"], k["C"], k["cache"], k["read"], k["write"],
                           dt_bias=k["dt_bias"], D=k["D"], z=k["z"], y=ys)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for turn in range(4):
        i["u"].copy_(torch.randn(129, 96, generator=torch.Generator().manual_seed(turn)))
        k["u"].copy_(torch.randn(3, 96, generator=torch.Generator().manual_seed(turn + 50)))
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, fin, ys, k["cache"])]
        for t in (y, fin, ys):
            t.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("y", "final", "step y", "cache"), (y, fin, ys, k["cache"]), want):
            assert torch.equal(a, b), f"replay {turn}: {name}"


def test_two_streams_at_once():
    i, j = make([600, 50], 256, 16, 1, BF, seed=16), make([333], 512, 16, 1, BF, seed=17)
    wi, wj = call(i)[:2], call(j)[:2]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(3):
        for st, x in zip(streams, (i, j)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                meta = ssd.varlen_metadata(x["cu"], 64, total_tokens=sum(x["lengths"]))
                got.append(ssd.selective_scan_varlen(x["u"], x["dt"], x["A"], x["B"], x["C"], meta,
                                                     dt_bias=x["dt_bias"], D=x["D"], z=x["z"],
                                                     initial_states=x["init"], has_initial_state=x["has"]) + (meta,))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        want = (wi, wj)[k % 2]
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def many(lengths, d, n, g, dtype, seed, pad=0, chunk=64, **kw):
    """Enough (sequence, channels) pairs that sequences are walked one wave each, and a few far longer ones that
    are not; every channel of a few sequences against float64, others in the batch and alone."""
    i = make(lengths, d, n, g, dtype, seed=seed, **kw)
    if pad == 0:   # rows of B and C on 4-byte boundaries
        wide = torch.cat([i["B"].reshape(-1, g * n), i["C"].reshape(-1, g * n)], 1).contiguous()
        i["B"], i["C"] = wide[:, :g * n].unflatten(1, (g, n)), wide[:, g * n:].unflatten(1, (g, n))
    meta = ssd.varlen_metadata(i["cu"], chunk, total_tokens=sum(lengths))
    cst = torch.full((meta.max_chunks, d, n), float("nan"), device="cuda")
    y, fin, meta = call(i, chunk=chunk, chunk_states=cst)
    assert int(meta.error_flag.item()) == 0
    assert torch.isfinite(fin).all()
    return i, y, fin, cst


def sequence(i, s):
    """One sequence of a batch as a batch of its own."""
    t0 = sum(i["lengths"][:s])
    r = slice(t0, t0 + i["lengths"][s])
    j = {**i, "lengths": [i["lengths"][s]], "cu": torch.tensor([0, i["lengths"][s]], dtype=torch.int32, device="cuda")}
    for k in ("u", "dt", "B", "C", "z"):
        j[k] = None if i[k] is None else i[k][r]
    j["init"] = None if i["init"] is None else i["init"][s:s + 1].contiguous()
    j["has"] = None if i["has"] is None else i["has"][s:s + 1]
    return j, r


@pytest.mark.parametrize("dtype,n,g,gate,init", [
    (BF, 16, 1, True, "even"), (BF, 32, 2, False, "all"), (F32, 16, 2, True, "none"), (F32, 32, 1, True, "even"),
])
def test_scan_of_many_sequences(dtype, n, g, gate, init):
    """512 sequences of 8 x 64 + 2 x 5 channels: 4608 or more pairs."""
    lengths = [int(v) for v in torch.randint(0, 40, (512,), generator=torch.Generator().manual_seed(n + g))]
    lengths[3], lengths[77], lengths[200], lengths[201] = 700, 333, 0, 1
    d = 522
    i, y, fin, cst = many(lengths, d, n, g, dtype, seed=30 + n, gate=gate, init=init)
    first = 0
    starts_of = []
    for v in lengths:
        starts_of.append(first)
        first += -(-v // 64)
    for s in (0, 1, 3, 77, 200, 201, 511):
        j, r = sequence(i, s)
        ry, rh, by, bh, start = expected(j)[0]
        ref.check(y[r], ry, by, f"y of {s}")
        if lengths[s] == 0:
            want = torch.zeros(d, n) if start is None else start
            assert torch.equal(fin[s].cpu(), want)
            continue
        ref.check(fin[s], rh[-1], bh[-1], f"state of {s}")
        for k in range(-(-lengths[s] // 64)):
            last = min(64 * k + 64, lengths[s]) - 1
            ref.check(cst[starts_of[s] + k], rh[last], bh[last], f"chunk {k} of {s}")
    assert torch.isnan(cst[first:]).all()
    for s in range(5, 512, 50):
        # One alone goes in segments. Sums in another order differ by float32's roundings before y's own: each result
        # is within the reference's bound (which counts those) plus one rounding of y, so each is checked against it.
        j, r = sequence(i, s)
        if lengths[s] == 0:
            continue
        y1, f1, _ = call(j)
        ry, rh, by, bh, _ = expected(j)[0]
        for name, gy, gf in (("batch", y[r], fin[s]), ("alone", y1, f1[0])):
            ref.check(gy, ry, by, f"y of {s} ({name})")
            ref.check(gf, rh[-1], bh[-1], f"state of {s} ({name})")


def test_scan_of_many_sequences_with_odd_rows():
    """Rows of B and C that do not lie on 4-byte boundaries go in segments; so does any number of sequences."""
    lengths = [7] * 300
    i, y, fin, _ = many(lengths, 1030, 16, 1, BF, seed=44, pad=1)
    j, r = sequence(i, 150)
    ry, rh, by, bh, _ = expected(j)[0]
    ref.check(y[r], ry, by, "y")
    ref.check(fin[150], rh[-1], bh[-1], "state")


@pytest.mark.parametrize("path", ["segments", "walk", "step"])
def test_extreme_rates_and_infinite_inputs(path):
    """Rates of the type's lowest value and of minus infinity (the state is replaced, but a step size of zero leaves it
    for any finite rate), and an infinite B at a sequence's ragged end, which reaches its own state and no other."""
    n, d = 16, 1040 if path == "walk" else 48
    lengths = [13] * 256 if path == "walk" else [1, 1] if path == "step" else [13, 5]
    i = make(lengths, d, n, 1, F32, gate=False, init="all", seed=51, skip=False)
    wide = torch.cat([i["B"].reshape(-1, n), i["C"].reshape(-1, n)], 1).contiguous()
    i["B"], i["C"] = wide[:, :n].unflatten(1, (1, n)), wide[:, n:].unflatten(1, (1, n))
    i["A"][1] = torch.finfo(F32).min
    i["A"][2, 3] = float("-inf")
    i["dt"][:, 1] = float("-inf")     # step sizes of zero for the channel of lowest rates
    i["dt"][:, 2] = 1.0
    last = lengths[0] - 1
    i["B"][last, 0, 5] = float("inf")
    i["u"][last, 7] = -1.5
    if path == "step":
        cache = torch.zeros(4, d, n, device="cuda")
        cache[:2] = i["init"]
        slots = torch.arange(4, dtype=torch.int32, device="cuda")
        ssd.selective_step(i["u"], i["dt"], i["A"], i["B"], i["C"], cache, slots[:2], slots[2:], dt_bias=i["dt_bias"])
        torch.cuda.synchronize()
        fin = cache[2:]
    else:
        fin = call(i, chunk=16)[1]
    c = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in cpu(i).items()}
    delta = ref.softplus(c["dt"].clamp(min=-1e30) + c["dt_bias"])
    t = 0
    for s in range(2):
        h = c["init"][s]
        for _ in range(lengths[s]):
            h = torch.exp(delta[t][:, None] * c["A"]) * h + (delta[t] * c["u"][t])[:, None] * c["B"][t]
            t += 1
        got = fin[s].cpu().double()
        # channel 1 and state 5 of zero steps: 0 x inf
        assert torch.equal(torch.isnan(got), torch.isnan(h)) and torch.equal(torch.isinf(got), torch.isinf(h))
        assert torch.equal(got[torch.isinf(h)], h[torch.isinf(h)])
        keep = torch.isfinite(h)
        # up to 13 tokens: each state is good to about 13 x 50 units of 2^-24 of the largest term, 4e-5 at most
        assert (got[keep] - h[keep]).abs().max() < 4e-5 * h[keep].abs().max()
        if s == 0:
            free = [k for k in range(n) if k != 5]
            assert torch.equal(got[1][free], c["init"][0][1][free]), "a step size of zero changed a state"
            assert got[7, 5] == float("-inf")


def test_offsets_past_32_bits():
    """Slots and rows whose element offsets pass 2^31 (and byte offsets 2^32): a cache of 6.4 GB and rows 2^26
    elements apart, the largest stride."""
    d, n, s = 48, 16, 3
    i = step_inputs(s, d, n, 1, BF, seed=60)
    slots = 2 ** 31 // (d * n) + 40
    cache = torch.empty(slots, d, n, device="cuda")
    high = torch.tensor([slots - 1, slots - 7, slots - 9], dtype=torch.int32, device="cuda")
    to = torch.tensor([slots - 2, slots - 30, 5], dtype=torch.int32, device="cuda")
    state = i["cache"][:s].clone()
    cache[high.long()] = state
    y = ssd.selective_step(i["u"], i["dt"], i["A"], i["B"], i["C"], cache, high, to, dt_bias=i["dt_bias"], D=i["D"],
                           z=i["z"])
    small = torch.cat([state, torch.zeros_like(state)])
    near = torch.arange(2 * s, dtype=torch.int32, device="cuda")
    want = ssd.selective_step(i["u"], i["dt"], i["A"], i["B"], i["C"], small, near[:s], near[s:], dt_bias=i["dt_bias"],
                              D=i["D"], z=i["z"])
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(cache[to.long()], small[s:])

    # the scan: 40 rows of u, z and y 2^26 elements apart, and a checkpoint in the last slot of the cache
    j = make([33, 7], d, n, 1, BF, seed=61)
    y0, f0, _ = call(j, chunk=16)
    far = torch.empty(40 * 2 ** 26, dtype=BF, device="cuda")
    views = [far.as_strided((40, d), (2 ** 26, 1), k * 64) for k in range(3)]
    views[0].copy_(j["u"])
    views[1].copy_(j["z"])
    k = {**j, "u": views[0], "z": views[1]}
    dst = torch.tensor([-1, slots - 3, -1, slots - 4], dtype=torch.int32, device="cuda")
    y1, f1, m = call(k, chunk=16, y=views[2], chunk_states=cache, chunk_state_dst=dst)
    assert int(m.error_flag.item()) == 0
    assert torch.equal(y1, y0) and torch.equal(f1, f0)
    assert torch.equal(cache[slots - 4], f1[1])
    del far, views, k, cache
