"""The conv step and the group norm against float64, and a layer of them with the scan: prompts continued token
by token give what the whole prompts give."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def conv_inputs(s, c, w, dtype, seed=0):
    r = torch.Generator().manual_seed(seed)
    normal = lambda *k: torch.randn(*k, generator=r)   # noqa: E731
    order = torch.randperm(2 * s + 1, generator=r).to(torch.int32)
    return dict(x=normal(s, 2 * c).to(dtype).cuda()[:, c:], weight=normal(c, w).cuda(), bias=normal(c).cuda(),
                states=normal(2 * s + 1, w - 1, c).to(dtype).cuda(), read=order[:s].cuda(), write=order[s:2 * s].cuda())


def check_conv(i, before, out, silu, bias, skip=()):
    s, w = i["x"].shape[0], i["weight"].shape[1]
    untouched = set(range(before.shape[0]))
    x, old = i["x"].cpu(), before.cpu()
    for k in range(s):
        if k in skip:
            continue
        rs, ws = int(i["read"][k]), int(i["write"][k])
        window = old[rs] if rs >= 0 else torch.zeros_like(old[0])
        want, bound = ref.conv_step(x[k:k + 1], i["weight"].cpu(), window[None], i["bias"].cpu() if bias else None,
                                    silu)
        ref.check(out[k:k + 1], want, bound, f"out of {k}")
        if ws >= 0:
            assert torch.equal(i["states"][ws].cpu(), torch.cat([window, x[k:k + 1]])[1:]), f"window of {k}"
            untouched.discard(ws)
    for k in untouched:
        assert torch.equal(i["states"][k], before[k]), f"slot {k} was written"


@pytest.mark.parametrize("s,c,w,dtype,silu,bias", [
    (1, 64, 4, BF, True, True), (1, 8, 2, F32, False, True), (3, 1032, 3, BF, True, False),
    (5, 2056, 4, F32, True, True), (17, 24, 1, BF, False, True), (9, 520, 2, BF, True, True),
])
def test_conv_step_against_float64(s, c, w, dtype, silu, bias):
    log(f"conv step {s, c, w, dtype, silu, bias}")
    i = conv_inputs(s, c, w, dtype, seed=s)
    before = i["states"].clone()
    out = ssd.causal_conv1d_step(i["x"], i["weight"], i["states"], i["read"], i["write"],
                                 bias=i["bias"] if bias else None, silu=silu)
    torch.cuda.synchronize()
    check_conv(i, before, out, silu, bias)


def test_conv_step_slots():
    """In place, no window yet, window not kept, and slots past the cache (skipped and flagged)."""
    i = conv_inputs(6, 72, 4, BF, seed=2)
    i["write"][0] = i["read"][0]
    i["read"][1] = -1
    i["write"][2] = -1
    i["read"][3] = i["states"].shape[0]
    i["write"][4] = i["states"].shape[0] + 3
    before = i["states"].clone()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((6, 80), 3.0, dtype=BF, device="cuda")
    ssd.causal_conv1d_step(i["x"], i["weight"], i["states"], i["read"], i["write"], bias=i["bias"], out=out[:, 8:],
                           error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == ssd.DATA_BAD_SLOT
    assert (out[:, :8] == 3).all() and (out[3:5] == 3).all()
    check_conv(i, before, out[:, 8:], True, True, skip=(3, 4))


def test_conv_step_equals_the_prompt_call():
    """A sequence of one token through causal_conv1d_varlen is the same call, bit for bit."""
    i = conv_inputs(7, 264, 4, BF, seed=5)
    a, b = i["states"].clone(), i["states"].clone()
    out = ssd.causal_conv1d_step(i["x"], i["weight"], a, i["read"], i["write"], bias=i["bias"])
    cu = torch.arange(8, dtype=torch.int32, device="cuda")
    meta = ssd.varlen_metadata(cu, 16, total_tokens=7)
    want = ssd.causal_conv1d_varlen(i["x"].contiguous(), i["weight"], meta, bias=i["bias"], conv_states=b,
                                    read_slot=i["read"], write_slot=i["write"])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(a, b)


def norm_inputs(rows, c, dtype, act, seed=0, pad=0, offset=0.0):
    r = torch.Generator().manual_seed(seed)
    normal = lambda *k: torch.randn(*k, generator=r)   # noqa: E731
    wide = (2 * normal(rows, c + pad) + offset).to(dtype).cuda()
    return dict(x=wide[:, pad:], z=normal(rows, c + pad).to(dtype).cuda()[:, pad:] if act.startswith("gate") else None,
                weight=1 + 0.3 * normal(c).cuda(), bias=0.5 * normal(c).cuda())


NORMS = [
    # rows, channels, groups, type, activation, centred, elements before each row
    (1, 1, 1, F32, "none", True, 0), (1, 64, 1, BF, "silu", True, 0), (5, 64, 8, BF, "gate_first", False, 0),
    (3, 5, 5, F32, "silu", False, 0), (7, 100, 4, BF, "gate_last", True, 3), (4, 129, 1, F32, "gate_first", True, 1),
    (6, 337 * 15, 15, F32, "silu", True, 0), (9, 2048, 1, BF, "gate_first", False, 8), (2, 16384, 1, F32, "none", True, 0),
    (3, 16384, 1, BF, "gate_last", False, 8), (3, 16383, 1, BF, "gate_first", True, 5), (2, 8191, 1, F32, "gate_last", True, 0),
    (300, 512, 16, BF, "gate_last", False, 8), (1000, 128, 1, BF, "gate_last", False, 0), (33, 4096, 4, F32, "gate_first", False, 4),
    (65, 1024, 128, BF, "silu", True, 0), (70, 1031, 1, BF, "none", False, 0), (11, 5120, 1, BF, "gate_first", True, 0),
    (40, 80, 8, F32, "gate_first", True, 0), (12, 6144, 2, BF, "silu", True, 2),
]


@pytest.mark.parametrize("k", range(len(NORMS)))
def test_norm_against_float64(k):
    rows, c, g, dtype, act, center, pad = NORMS[k]
    log(f"norm {NORMS[k]}")
    i = norm_inputs(rows, c, dtype, act, seed=k, pad=pad)
    for weight, bias in ((i["weight"], i["bias"]), (None, None)):
        out = ssd.group_norm(i["x"], g, weight=weight, bias=bias, z=i["z"], act=act, center=center)
        torch.cuda.synchronize()
        want, bound = ref.group_norm(i["x"].cpu(), g, None if weight is None else weight.cpu(),
                                     None if bias is None else bias.cpu(), None if i["z"] is None else i["z"].cpu(),
                                     act, center)
        worst = ref.check(out, want, bound, f"norm {k}")
    log(f"  worst {worst:.3f} of the bound")


def test_norm_far_from_zero_mean_and_constant_groups():
    """A mean of 1000 deviations (a one-pass variance loses all digits), and groups of one value (variance 0)."""
    i = norm_inputs(6, 512, F32, "none", seed=1, offset=2000.0)
    out = ssd.group_norm(i["x"], 2)
    torch.cuda.synchronize()
    ref.check(out, *ref.group_norm(i["x"].cpu(), 2), "offset")
    flat = torch.full((3, 256), 1.5, device="cuda")
    assert (ssd.group_norm(flat, 4) == 0).all()


def test_norm_in_place_and_beside_other_columns():
    i = norm_inputs(20, 96, BF, "gate_first", seed=2)
    want = ssd.group_norm(i["x"], 3, weight=i["weight"], z=i["z"], act="gate_first", center=False)
    wide = torch.full((20, 110), 7.0, dtype=BF, device="cuda")
    part = wide[:, 6:102]
    part.copy_(i["x"])
    got = ssd.group_norm(part, 3, weight=i["weight"], z=i["z"], act="gate_first", center=False, out=part)
    torch.cuda.synchronize()
    assert got.data_ptr() == part.data_ptr() and torch.equal(part, want)
    assert (wide[:, :6] == 7).all() and (wide[:, 102:] == 7).all()


def test_norm_rows_do_not_touch_each_other():
    i = norm_inputs(9, 256, BF, "gate_last", seed=3)
    want = ssd.group_norm(i["x"], 4, z=i["z"], act="gate_last")
    i["x"][4, 10] = float("nan")
    i["z"][6, 200] = float("inf")
    got = ssd.group_norm(i["x"], 4, z=i["z"], act="gate_last")
    torch.cuda.synchronize()
    assert torch.isnan(got[4, :64]).all()
    keep = [r for r in range(9) if r not in (4, 6)]
    assert torch.equal(got[keep], want[keep]) and torch.equal(got[4, 64:], want[4, 64:])


def test_norm_of_scan_rows_and_no_rows():
    """(T, H, P) is T rows of H*P channels; a batch without tokens is fine."""
    x = torch.randn(13, 6, 32, generator=torch.Generator().manual_seed(4)).cuda()
    got = ssd.group_norm(x, 6, center=False)
    assert got.shape == x.shape
    assert torch.equal(got.view(13, 192), ssd.group_norm(x.view(13, 192), 6, center=False))
    assert ssd.group_norm(x[:0], 6).shape == (0, 6, 32)


def test_norm_and_conv_step_graph_replays():
    i, k = norm_inputs(50, 512, BF, "gate_first", seed=5), conv_inputs(4, 256, 4, BF, seed=6)
    out, co = torch.empty_like(i["x"]), torch.empty(4, 256, dtype=BF, device="cuda")

    def both():
        ssd.group_norm(i["x"], 2, weight=i["weight"], z=i["z"], act="gate_first", center=False, out=out)
        ssd.causal_conv1d_step(k["x"], k["weight"], k["states"], k["read"], k["write"], bias=k["bias"], out=co)
    with torch.cuda.stream(torch.cuda.Stream()):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for turn in range(4):
        i["x"].copy_(torch.randn(50, 512, generator=torch.Generator().manual_seed(turn)))
        k["x"].copy_(torch.randn(4, 256, generator=torch.Generator().manual_seed(turn + 9)))
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (out, co, k["states"])]
        out.fill_(0)
        co.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, co, k["states"]), want)), f"replay {turn}"


def test_layer_of_prompts_then_tokens():
    """conv -> scan -> norm over prompts, then conv step -> scan step -> norm for three more tokens each, with the
    states in cache slots, against the same layer in float64 over the whole sequences."""
    r = torch.Generator().manual_seed(21)
    normal = lambda *k: torch.randn(*k, generator=r)   # noqa: E731
    lengths, more, d, n, w = [37, 5, 1], 3, 72, 16, 4
    total = [v + more for v in lengths]
    x = [normal(v, d) for v in total]
    dt, z = [normal(v, d) for v in total], [normal(v, d) for v in total]
    B, C = [normal(v, 1, n) * n ** -0.5 for v in total], [normal(v, 1, n) * n ** -0.5 for v in total]
    weight, bias, A = normal(d, w) * 0.5, normal(d) * 0.1, -torch.exp(2 * torch.rand(d, n, generator=r))
    dt_bias, skip, gain = -3 + 0.5 * normal(d), normal(d), 1 + 0.1 * normal(d)
    cuda = lambda t: t.cuda()   # noqa: E731
    prompts = lambda ts: torch.cat([t[:v] for t, v in zip(ts, lengths)]).cuda()   # noqa: E731
    cu = torch.tensor([0, 37, 42, 43], dtype=torch.int32).cuda()
    meta = ssd.varlen_metadata(cu, 16, total_tokens=43)
    convs, cache = torch.zeros(8, w - 1, d, device="cuda"), torch.zeros(8, d, n, device="cuda")
    slots = torch.tensor([6, 1, 3], dtype=torch.int32).cuda()
    u = ssd.causal_conv1d_varlen(prompts(x), cuda(weight), meta, bias=cuda(bias), conv_states=convs, write_slot=slots)
    y, fin = ssd.selective_scan_varlen(u, prompts(dt), cuda(A), prompts(B), prompts(C), meta, dt_bias=cuda(dt_bias),
                                       D=cuda(skip), z=prompts(z))
    out = [ssd.group_norm(y, 4, weight=cuda(gain), center=False)]
    cache[slots.long()] = fin
    rows = [out[0][a:a + v] for a, v in zip((0, 37, 42), lengths)]
    for k in range(more):
        at = lambda ts: torch.stack([t[v + k] for t, v in zip(ts, lengths)]).cuda()   # noqa: E731
        uk = ssd.causal_conv1d_step(at(x), cuda(weight), convs, slots, slots, bias=cuda(bias))
        yk = ssd.selective_step(uk, at(dt), cuda(A), at(B), at(C), cache, slots, slots, dt_bias=cuda(dt_bias),
                                D=cuda(skip), z=at(z))
        ok = ssd.group_norm(yk, 4, weight=cuda(gain), center=False)
        rows = [torch.cat([a, ok[s:s + 1]]) for s, a in enumerate(rows)]
    torch.cuda.synchronize()
    for s, v in enumerate(total):
        pad = torch.cat([torch.zeros(w - 1, d), x[s]]).double()
        windows = torch.stack([pad[t:t + w - 1] for t in range(v)])
        ru, _ = ref.conv_step(x[s], weight, windows, bias, True)
        ry, rh, _, _ = ref.scan(ru, dt[s], A, B[s], C[s], dt_bias, skip, z[s])
        want, _ = ref.group_norm(ry, 4, gain, None, None, "none", False)
        # float32 all through: u is off by U (w + 1 taps, silu) and its parts; the norm divides by the rows' spread.
        # 1e-5 of the largest value covers 160 U for each of the three operators' results, term by term
        off = (rows[s].cpu().double() - want).abs().max() / want.abs().max()
        assert off < 1e-5, f"sequence {s}: {off:.2e}"
        assert ((cache[int(slots[s])].cpu().double() - rh[-1]).abs().max() / rh[-1].abs().max()) < 1e-5


def test_conv_step_and_norm_offsets_past_32_bits():
    """A cache of 2^31 and more elements, and rows 2^26 elements apart."""
    i = conv_inputs(3, 64, 4, BF, seed=70)
    slots = 2 ** 31 // (3 * 64) + 20
    cache = torch.empty(slots, 3, 64, dtype=BF, device="cuda")
    high = torch.tensor([slots - 1, slots - 5, 2], dtype=torch.int32, device="cuda")
    to = torch.tensor([slots - 2, slots - 6, slots - 9], dtype=torch.int32, device="cuda")
    cache[high.long()] = i["states"][:3]
    before = i["states"].clone()
    i["read"], i["write"] = torch.arange(3, dtype=torch.int32).cuda(), torch.arange(3, 6, dtype=torch.int32).cuda()
    want = ssd.causal_conv1d_step(i["x"], i["weight"], i["states"], i["read"], i["write"], bias=i["bias"])
    out = ssd.causal_conv1d_step(i["x"], i["weight"], cache, high, to, bias=i["bias"])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache[to.long()], i["states"][3:6])
    assert torch.equal(i["states"][:3], before[:3])
    far = torch.empty(40 * 2 ** 26, dtype=BF, device="cuda")
    x, z, o = (far.as_strided((40, 96), (2 ** 26, 1), k * 128) for k in range(3))
    n = norm_inputs(40, 96, BF, "gate_last", seed=71)
    x.copy_(n["x"])
    z.copy_(n["z"])
    ssd.group_norm(x, 3, weight=n["weight"], z=z, act="gate_last", out=o)
    torch.cuda.synchronize()
    assert torch.equal(o, ssd.group_norm(n["x"], 3, weight=n["weight"], z=n["z"], act="gate_last"))


def test_norm_of_more_groups_than_teams_fill_the_card():
    """Many tiny groups, more than the teams of one launch: every (row, group) is visited once."""
    i = norm_inputs(3, 2 ** 21, F32, "silu", seed=72)
    got = ssd.group_norm(i["x"], 2 ** 20, act="silu", center=False)
    pairs = i["x"].double().view(3, -1, 2)
    v = (pairs / (pairs.square().mean(-1, keepdim=True) + 1e-5).sqrt()).view(3, -1)
    want = v * torch.sigmoid(v)
    # sums of 2 squares, 1 / sqrt, two products, silu of values below 1.5: under 24 roundings of 2^-24
    assert ((got.double() - want).abs() <= 24 * 2.0 ** -24 * want.abs() + 1e-30).all()
