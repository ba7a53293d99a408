"""The operators of a layer with a selective state space scan, as cases to measure.

A layer keeps, for every channel d of its D inner channels, N states that decay at
rates of their own (A is (D, N), the step size dt is (tokens, D)); the four operators
are the scan of packed prompts, its step for single tokens, the short causal
convolution's step for single tokens, and the norm of groups of channels with an
activation that follows the scan.

`run` computes them in elementary torch operations in float32 where `own` is false and
calls the library where it is true; `exact` computes them in float64.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# lengths of the batches that the package's workloads have
_PROMPTS_8 = "3514,1449,903,1582,1995,3430,2129,841"
_PROMPTS_64 = ("312,339,267,477,476,107,312,323,127,153,250,380,150,370,335,112,"
               "199,425,432,337,3,350,116,420,468,220,490,389,167,450,197,53,"
               "304,436,337,202,462,246,198,75,109,358,410,150,322,447,76,141,"
               "269,288,204,205,67,314,477,101,409,93,23,383,93,386,170,291")

# tokens that the plain scan takes at a time: bounds the (tokens, D, N) tensors that it holds
_PLAIN_CHUNK = 256


def listed():
    return [
        # scan: a few short float32 prompts with many states, where the call's latency counts
        dict(name="scan_short_f32", op="scan", lengths="17,64,47", channels=512, dstate=64, groups=1, dtype="f32",
             gate=False, init="even", chunk=16, block=0),
        # scan: eight prompts of one prefill step, half of them continued from a state
        dict(name="scan_prompts_8", op="scan", lengths=_PROMPTS_8, channels=5120, dstate=16, groups=1, dtype="bf16",
             gate=True, init="even", chunk=256, block=0),
        # scan: continuous batching, 64 ragged prompts that all continue, B and C in 8 groups
        dict(name="scan_mix_64", op="scan", lengths=_PROMPTS_64, channels=8192, dstate=16, groups=8, dtype="bf16",
             gate=True, init="all", chunk=256, block=0),
        # scan: prefix caching, the state of every 256-token block written to its cache slot
        dict(name="scan_prefix_cache", op="scan", lengths="8894,8894,8894,8894", channels=4096, dstate=16, groups=1,
             dtype="bf16", gate=True, init="none", chunk=64, block=256),
        # scan: one long prompt alone, few channels: little to run side by side
        dict(name="scan_long_prompt", op="scan", lengths="30001", channels=2560, dstate=16, groups=1, dtype="bf16",
             gate=True, init="none", chunk=256, block=0),
        # step: one user's next token
        dict(name="step_1", op="step", nseqs=1, channels=5120, dstate=16, groups=1, dtype="bf16", gate=True),
        # step: the next token of 256 sequences
        dict(name="step_256", op="step", nseqs=256, channels=5120, dstate=16, groups=1, dtype="bf16", gate=True),
        # conv step: one user's next token
        dict(name="conv_step_1", op="conv", nseqs=1, channels=5120, width=4, dtype="bf16", silu=True),
        # conv step: 256 sequences, x, B and C convolved together
        dict(name="conv_step_256", op="conv", nseqs=256, channels=10240, width=4, dtype="bf16", silu=True),
        # norm: one token, gated before the norm
        dict(name="norm_1", op="norm", rows=1, channels=5120, groups=1, dtype="bf16", act="gate_first", center=False),
        # norm: the tokens of the prefix-cache batch, four groups, gated before the norm
        dict(name="norm_prompts", op="norm", rows=35576, channels=4096, groups=4, dtype="bf16", act="gate_first",
             center=False),
        # norm: float32, centred, an odd group size, SiLU of the result
        dict(name="norm_odd_f32", op="norm", rows=16085, channels=5055, groups=15, dtype="f32", act="silu",
             center=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "conv", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "scan":
        groups = rng.choice([1, 1, 2, 8])
        channels = groups * _spread(rng, max(1, 64 // groups), 8192 // groups)
        dstate = rng.choice([16, 16, 16, 32, 64])
        nseqs = _spread(rng, 1, 64)
        tokens = max(nseqs, _spread(rng, 1, min(30000, 2 ** 31 // (channels * dstate))))
        cuts = sorted(rng.randint(0, tokens) for _ in range(nseqs - 1))
        lengths = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))
        chunk = rng.choice([16, 64, 256])
        return dict(op=op, lengths=lengths, channels=channels, dstate=dstate, groups=groups, dtype=dtype,
                    gate=rng.random() < 0.7, init=rng.choice(["none", "even", "all"]), chunk=chunk,
                    block=rng.choice([0, 256]))
    if op == "step":
        groups = rng.choice([1, 1, 2, 8])
        dstate = rng.choice([16, 16, 32, 64, 128])
        channels = groups * _spread(rng, max(1, 64 // groups), 8192 // groups)
        return dict(op=op, nseqs=_spread(rng, 1, 2 ** 28 // (channels * dstate * 4)) if rng.random() < 0.8 else 1,
                    channels=channels, dstate=dstate, groups=groups, dtype=dtype, gate=rng.random() < 0.7)
    if op == "conv":
        return dict(op=op, nseqs=_spread(rng, 1, 512), channels=8 * _spread(rng, 8, 2048), width=rng.randint(2, 4),
                    dtype=dtype, silu=rng.random() < 0.7)
    groups = rng.choice([1, 2, 3, 8, 16])
    channels = groups * _spread(rng, 32, 8192 // groups)
    return dict(op=op, rows=_spread(rng, 1, 2 ** 27 // channels), channels=channels, groups=groups, dtype=dtype,
                act=rng.choice(["none", "silu", "gate_first", "gate_last"]), center=rng.random() < 0.5)


def _lengths(case):
    return [int(v) for v in case["lengths"].split(",")]


def _blocks(case):
    """(sequence, tokens at the end, slot) of every checkpointed block."""
    got = []
    for s, length in enumerate(_lengths(case)):
        for end in range(case["block"], length + case["block"], case["block"]) if case["block"] else ():
            got.append((s, min(end, length), len(got)))
    return got


class _Draw:
    """Random device tensors from one seed."""

    def __init__(self, seed, dtype):
        self.gen = torch.Generator(device="cuda").manual_seed(int(seed))
        self.dtype = dtype

    def normal(self, *shape, scale=1.0, dtype=None):
        t = torch.empty(shape, device="cuda", dtype=torch.float32).normal_(generator=self.gen)
        return t.mul_(scale).to(dtype or self.dtype)

    def uniform(self, lo, hi, *shape):
        return torch.empty(shape, device="cuda", dtype=torch.float32).uniform_(lo, hi, generator=self.gen)


def _layer(r, rows, case):
    """What the projections of a layer hand to the scan: u from the convolution, z the second half of the input
    projection, B and C next to the low-rank step size in the projection of u, dt raw."""
    d, n, g = case["channels"], case["dstate"], case["groups"]
    rank = -(-d // 16)
    low = r.normal(rows, rank + 2 * g * n, scale=n ** -0.5)
    return dict(u=r.normal(rows, d), dt=r.normal(rows, d),
                B=low[:, rank:rank + g * n].unflatten(1, (g, n)), C=low[:, rank + g * n:].unflatten(1, (g, n)),
                z=r.normal(rows, 2 * d)[:, d:] if case["gate"] else None,
                A=-torch.exp(r.uniform(0.0, math.log(16.0), d, n)), dt_bias=r.uniform(-4.0, -2.0, d),
                D=r.normal(d, dtype=torch.float32))


def _slots(nseqs):
    """Each sequence reads one cache slot and writes another; the slots are scattered over the cache."""
    order = torch.randperm(2 * nseqs, generator=torch.Generator().manual_seed(nseqs)).to(torch.int32).cuda()
    return order[:nseqs].contiguous(), order[nseqs:].contiguous()


def _inputs(case, seed):
    r = _Draw(seed, _DTYPES[case["dtype"]])
    f32 = torch.float32
    i = dict(case=case)
    if case["op"] == "scan":
        lengths = _lengths(case)
        s, d, n = len(lengths), case["channels"], case["dstate"]
        i.update(_layer(r, sum(lengths), case))
        i["lengths"] = lengths
        i["cu"] = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        i["init"] = None if case["init"] == "none" else r.normal(s, d, n, scale=0.5, dtype=f32)
        i["has"] = torch.tensor([int(case["init"] == "all" or k % 2 == 0) for k in range(s)], dtype=torch.int32).cuda()
        i["blocks"] = _blocks(case)
        i["cache"] = torch.zeros(len(i["blocks"]), d, n, device="cuda") if case["block"] else None
        return i
    if case["op"] == "norm":
        rows, c = case["rows"], case["channels"]
        i.update(x=r.normal(rows, c, scale=2.0), weight=1.0 + r.normal(c, scale=0.2, dtype=f32),
                 bias=r.normal(c, scale=0.2, dtype=f32) if case["center"] else None,
                 z=r.normal(rows, 2 * c)[:, c:] if case["act"].startswith("gate") else None)
        return i
    i["read"], i["write"] = _slots(case["nseqs"])
    if case["op"] == "step":
        i.update(_layer(r, case["nseqs"], case))
        i["cache"] = r.normal(2 * case["nseqs"], case["channels"], case["dstate"], scale=0.5, dtype=f32)
    else:
        c, w = case["channels"], case["width"]
        i.update(x=r.normal(case["nseqs"], 2 * c)[:, :c], weight=r.normal(c, w, scale=w ** -0.5, dtype=f32),
                 bias=r.normal(c, scale=0.2, dtype=f32), cache=r.normal(2 * case["nseqs"], w - 1, c))
    return i


def prepare(case, seed):
    state = _inputs(case, seed)
    if own and case["op"] == "scan":
        # the chunk grid and the checkpoint plan are built once for a batch and shared by all its layers
        from selective_state_space_cu_amd import ssd
        state["meta"] = ssd.varlen_metadata(state["cu"], case["chunk"], total_tokens=sum(state["lengths"]))
        state["dst"] = None
        if case["block"]:
            most = max(1, max(-(-n // case["block"]) for n in state["lengths"]))
            table = torch.full((len(state["lengths"]), most), -1, dtype=torch.int32)
            for s, end, slot in state["blocks"]:
                table[s, -(-end // case["block"]) - 1] = slot
            state["dst"] = ssd.export_chunk_states(state["meta"], table, case["block"],
                                                   num_slots=len(state["blocks"]))[1]
    return state


def run(i):
    case = i["case"]
    if own:
        from selective_state_space_cu_amd import ssd
        if case["op"] == "scan":
            y, final = ssd.selective_scan_varlen(
                i["u"], i["dt"], i["A"], i["B"], i["C"], i["meta"], dt_bias=i["dt_bias"], D=i["D"], z=i["z"],
                initial_states=i["init"], has_initial_state=None if i["init"] is None else i["has"],
                chunk_states=i["cache"], chunk_state_dst=i["dst"])
            return {"y": y, "final": final} if i["cache"] is None else {"y": y, "final": final, "cache": i["cache"]}
        if case["op"] == "step":
            y = ssd.selective_step(i["u"], i["dt"], i["A"], i["B"], i["C"], i["cache"], i["read"], i["write"],
                                   dt_bias=i["dt_bias"], D=i["D"], z=i["z"])
            return {"y": y, "cache": i["cache"]}
        if case["op"] == "conv":
            out = ssd.causal_conv1d_step(i["x"], i["weight"], i["cache"], i["read"], i["write"], bias=i["bias"],
                                         silu=case["silu"])
            return {"out": out, "cache": i["cache"]}
        return ssd.group_norm(i["x"], case["groups"], weight=i["weight"], bias=i["bias"], z=i["z"], act=case["act"],
                              center=case["center"])
    return {"scan": _plain_scan, "step": _plain_step, "conv": _plain_conv, "norm": _plain_norm}[case["op"]](i, case)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _silu(v):
    return v / (1 + torch.exp(-v))


def _per_channel(t, channels):
    """(..., G, N) of the groups as (..., D, N) or what broadcasts to it."""
    return t if t.shape[-2] == 1 else t.repeat_interleave(channels // t.shape[-2], dim=-2)


def _recurrence(a, b):
    """h_t = a_t h_(t-1) + b_t along dimension 1, from zero: pairs of maps are composed, the half as long recurrence
    gives every second h, and one more product and sum the others."""
    n = a.shape[1]
    if n == 1:
        return b
    even = n - n % 2
    h = torch.empty_like(b)
    h[:, 1:even:2] = _recurrence(a[:, 1:even:2] * a[:, 0:even:2],
                                 torch.addcmul(b[:, 1:even:2], a[:, 1:even:2], b[:, 0:even:2]))
    h[:, 0] = b[:, 0]
    h[:, 2::2] = torch.addcmul(b[:, 2::2], a[:, 2::2], h[:, 1:n - 1:2])
    return h


def _plain_scan(i, case):
    """All sequences side by side, a chunk of tokens at a time. Tokens past a sequence's end get a step size of zero,
    which leaves its state."""
    d, lengths = case["channels"], i["lengths"]
    total, longest, f32 = sum(lengths), max(lengths), torch.float32
    starts = i["cu"][:-1].long()[:, None]
    left = i["cu"][1:].long()[:, None] - starts
    h = torch.zeros(len(lengths), d, case["dstate"], device="cuda")
    if i["init"] is not None:
        h = torch.where(i["has"][:, None, None] != 0, i["init"], h)
    y = torch.empty(total + 1, d, device="cuda", dtype=i["u"].dtype)
    for t0 in range(0, longest, _PLAIN_CHUNK):
        k = min(_PLAIN_CHUNK, longest - t0)
        at = t0 + torch.arange(k, device="cuda")[None, :]
        live = at < left
        rows = torch.where(live, starts + at, 0)
        u = i["u"][rows].to(f32)
        delta = _softplus(i["dt"][rows].to(f32) + i["dt_bias"]) * live[..., None]
        a = torch.exp(delta[..., None] * i["A"])
        b = (delta * u)[..., None] * _per_channel(i["B"][rows].to(f32), d)
        b[:, 0] += a[:, 0] * h
        states = _recurrence(a, b)
        h = states[:, -1].clone()
        out = (states * _per_channel(i["C"][rows].to(f32), d)).sum(-1) + i["D"] * u
        if i["z"] is not None:
            out = out * _silu(i["z"][rows].to(f32))
        y[torch.where(live, rows, total)] = out.to(y.dtype)
        for s, end, slot in i["blocks"]:
            if t0 < end <= t0 + k:
                i["cache"][slot] = states[s, end - 1 - t0]
    return {"y": y[:total], "final": h} if i["cache"] is None else {"y": y[:total], "final": h, "cache": i["cache"]}


def _plain_step(i, case):
    d, f32 = case["channels"], torch.float32
    u = i["u"].to(f32)
    delta = _softplus(i["dt"].to(f32) + i["dt_bias"])
    h = i["cache"][i["read"]] * torch.exp(delta[..., None] * i["A"])
    h += (delta * u)[..., None] * _per_channel(i["B"].to(f32), d)
    y = (h * _per_channel(i["C"].to(f32), d)).sum(-1) + i["D"] * u
    if i["z"] is not None:
        y = y * _silu(i["z"].to(f32))
    i["cache"][i["write"]] = h
    return {"y": y.to(i["u"].dtype), "cache": i["cache"]}


def _plain_conv(i, case):
    window = torch.cat([i["cache"][i["read"]], i["x"][:, None]], dim=1)
    out = (window.to(torch.float32) * i["weight"].t()).sum(1) + i["bias"]
    i["cache"][i["write"]] = window[:, 1:]
    return {"out": (_silu(out) if case["silu"] else out).to(i["x"].dtype), "cache": i["cache"]}


def _plain_norm(i, case):
    rows, c, g = case["rows"], case["channels"], case["groups"]
    v = i["x"].to(torch.float32)
    gate = None if i["z"] is None else _silu(i["z"].to(torch.float32))
    if case["act"] == "gate_first":
        v = v * gate
    v = v.view(rows, g, c // g)
    if case["center"]:
        v = v - v.mean(-1, keepdim=True)
    v = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-5)).view(rows, c) * i["weight"]
    if i["bias"] is not None:
        v = v + i["bias"]
    if case["act"] == "silu":
        v = _silu(v)
    if case["act"] == "gate_last":
        v = v * gate
    return v.to(i["x"].dtype)


def exact(case, seed):
    """float64, from the definitions: the scan token by token, everything else row by row at once."""
    i = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in _inputs(case, seed).items()}
    if case["op"] == "scan":
        return _exact_scan(i, case)
    if case["op"] == "step":
        cache = i["cache"]
        y, state = _exact_token(i, slice(None), cache[i["read"].long()], case)
        cache[i["write"].long()] = state
        return {"y": y, "cache": cache}
    if case["op"] == "conv":
        old, cache, w = i["cache"][i["read"].long()], i["cache"], case["width"]
        out = i["bias"] + i["weight"][:, w - 1] * i["x"]
        for k in range(w - 1):
            out = out + i["weight"][:, k] * old[:, k]
        cache[i["write"].long()] = torch.cat([old[:, 1:], i["x"].unsqueeze(1)], 1)
        return {"out": out * torch.sigmoid(out) if case["silu"] else out, "cache": cache}
    parts = []
    size = case["channels"] // case["groups"]
    gate = None if i["z"] is None else i["z"] * torch.sigmoid(i["z"])
    v = i["x"] * gate if case["act"] == "gate_first" else i["x"]
    for k in range(case["groups"]):
        p = v[:, k * size:(k + 1) * size]
        mean = p.sum(1, keepdim=True) / size if case["center"] else 0.0
        parts.append((p - mean) / torch.sqrt(((p - mean) ** 2).sum(1, keepdim=True) / size + 1e-5))
    o = torch.cat(parts, 1) * i["weight"]
    if i["bias"] is not None:
        o = o + i["bias"]
    if case["act"] == "silu":
        o = o * torch.sigmoid(o)
    return o * gate if case["act"] == "gate_last" else o


def _exact_token(i, rows, state, case):
    """One token of each sequence: (y, new state)."""
    u, raw = i["u"][rows], i["dt"][rows] + i["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    per = case["channels"] // case["groups"]
    state = state * torch.exp(delta.unsqueeze(2) * i["A"])
    shape = (state.shape[0], case["groups"], per, case["dstate"])
    state = (state.view(shape) + (delta * u).view(shape[:3]).unsqueeze(3) * i["B"][rows].unsqueeze(2)).view_as(state)
    y = (state.view(shape) * i["C"][rows].unsqueeze(2)).sum(3).view_as(u) + i["D"] * u
    if i["z"] is not None:
        y = y * (i["z"][rows] * torch.sigmoid(i["z"][rows]))
    return y, state


def _exact_scan(i, case):
    """Sequences in order of their lengths, so that the live ones stand first at every token."""
    lengths = i["lengths"]
    order = sorted(range(len(lengths)), key=lambda s: -lengths[s])
    starts = i["cu"].long()[:-1][torch.tensor(order).cuda()]
    state = torch.zeros(len(lengths), case["channels"], case["dstate"], dtype=torch.float64, device="cuda")
    if i["init"] is not None:
        state = i["init"] * (i["has"] != 0).view(-1, 1, 1)
    state = state[torch.tensor(order).cuda()]
    wanted = {}
    for s, end, slot in i["blocks"]:
        wanted.setdefault(end, []).append((order.index(s), slot))
    y = torch.empty_like(i["u"])
    for t in range(max(lengths)):
        live = sum(n > t for n in lengths)
        rows = starts[:live] + t
        y[rows], state[:live] = _exact_token(i, rows, state[:live], case)
        for place, slot in wanted.get(t + 1, ()):
            i["cache"][slot] = state[place]
    final = torch.empty_like(state)
    final[torch.tensor(order).cuda()] = state
    return {"y": y, "final": final} if i["cache"] is None else {"y": y, "final": final, "cache": i["cache"]}


def work(case):
    """Each input read once and each output written once; an exponential, a product or a sum is one operation."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["channels"]
        gate = case["act"].startswith("gate")
        return {"bytes": e * n * (3 if gate else 2) + 4 * case["channels"] * (2 if case["center"] else 1),
                "flops": n * (5 + (2 if case["center"] else 0) + (5 if case["act"] != "none" else 0))}
    if case["op"] == "conv":
        s, c, w = case["nseqs"], case["channels"], case["width"]
        return {"bytes": e * s * c * (2 + 2 * (w - 1)) + 4 * c * (w + 1) + 8 * s,
                "flops": s * c * (2 * w + (4 if case["silu"] else 0))}
    d, n, g = case["channels"], case["dstate"], case["groups"]
    rows = case["nseqs"] if case["op"] == "step" else sum(_lengths(case))
    streams = 4 if case["gate"] else 3
    moved = rows * (streams * d + 2 * g * n) * e + 4 * d * (n + 2)
    if case["op"] == "step":
        moved += rows * (8 * d * n + 8)
    else:
        s = len(_lengths(case))
        given = {"none": 0, "even": (s + 1) // 2, "all": s}[case["init"]]
        moved += 4 * d * n * (given + s + len(_blocks(case)))
    return {"bytes": moved, "flops": rows * d * (7 * n + 8 + (5 if case["gate"] else 0))}
