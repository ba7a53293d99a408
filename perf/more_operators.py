"""The operators of one decode step of a hybrid stack, as cases to measure: a few layers keep keys and values in paged
caches, the others the state of a gated delta rule.

A step begins with the tables that all its layers share (which blocks the new tokens take, where their keys and states
go); a layer adds the residual and norms, then advances its states by the new tokens, or writes their keys and values to
the cache and attends to it.

Caches of keys are (blocks, kv heads, block size, head dim), caches of values (blocks, kv heads, head dim, block size);
states are float32 (slots, value heads, dv, dk).

`run` computes the operators in elementary torch operations in float32 where `own` is false and calls the library where
it is true; `exact` computes them in float64.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_E4M3_MAX = 448.0

# lengths of a batch that the package's workloads have
_PROMPTS_64 = [312, 339, 267, 477, 476, 107, 312, 323, 127, 153, 250, 380, 150, 370, 335, 112, 199, 425, 432, 337, 3, 350,
               116, 420, 468, 220, 490, 389, 167, 450, 197, 53, 304, 436, 337, 202, 462, 246, 198, 75, 109, 358, 410, 150,
               322, 447, 76, 141, 269, 288, 204, 205, 67, 314, 477, 101, 409, 93, 23, 383, 93, 386, 170, 291]

# elements that the plain attention gathers at a time
_PLAIN_KEYS = 1 << 28


def _text(values):
    return ",".join(str(v) for v in values)


def listed():
    ones = _text([1] * 256)
    return [
        # delta rule: one user's next token
        dict(name="delta_1", op="delta", counts="1", heads=32, kheads=16, dk=128, dv=128, dtype="bf16", raw=True),
        # delta rule: the next token of 256 sequences
        dict(name="delta_256", op="delta", counts=ones, heads=32, kheads=16, dk=128, dv=128, dtype="bf16", raw=True),
        # delta rule: speculated tokens, up to four a sequence and the state kept after each; float32, gates computed before
        dict(name="delta_speculated_f32", op="delta", counts=_text([1 + n % 4 for n in _PROMPTS_64]), heads=24, kheads=8,
             dk=64, dv=80, dtype="f32", raw=False),
        # attention: short float32 prompts' next tokens, where the call's latency counts
        dict(name="attend_short_f32", op="attend", lengths="17,64,47", counts="1,1,1", heads=8, kvheads=2, dim=64, block=16,
             window=0, dtype="f32"),
        # attention: one user's next token after a long prompt
        dict(name="attend_long", op="attend", lengths="30001", counts="1", heads=32, kvheads=8, dim=128, block=16, window=0,
             dtype="bf16"),
        # attention: the next token of 64 sequences of 48 to 7872 tokens
        dict(name="attend_64", op="attend", lengths=_text([16 * n + k for k, n in enumerate(_PROMPTS_64)]),
             counts=_text([1] * 64), heads=32, kvheads=8, dim=128, block=64, window=0, dtype="bf16"),
        # cache write: the next token of 256 sequences
        dict(name="write_256", op="write", counts=ones, kvheads=8, dim=128, block=16, dtype="bf16"),
        # cache write: the prompts of a prefix-cache batch
        dict(name="write_prompts", op="write", counts="8894,8894,8894,8894", kvheads=8, dim=128, block=64, dtype="bf16"),
        # tables: the next token of 256 sequences
        dict(name="tables_256", op="tables", computed=_text([64 * n + k for k, n in enumerate(_PROMPTS_64 * 4)]),
             counts=ones, block=16),
        # tables: 64 ragged prompts beside 64 sequences' next tokens, blocks of 64
        dict(name="tables_prompts", op="tables", computed=_text([0] * 64 + [16 * n for n in _PROMPTS_64]),
             counts=_text(_PROMPTS_64 + [1] * 64), block=64),
        # norm: one token, the residual added
        dict(name="norm_1", op="norm", rows=1, channels=5120, residual=True, out="same", group=0, dtype="bf16"),
        # norm: the tokens of the prefix-cache batch, 8-bit output with a scale for every 128 channels
        dict(name="norm_prompts_e4m3", op="norm", rows=35576, channels=4096, residual=True, out="e4m3", group=128,
             dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "attend", "attend", "write", "tables", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "delta":
        kheads = _spread(rng, 1, 16)
        heads = kheads * rng.choice([1, 2, 3, 4])
        dk, dv = rng.choice([64, 128, 128, 256]), 4 * _spread(rng, 4, 64)
        most = max(1, 2 ** 27 // (heads * dk * dv))   # states that the largest listed case reads
        if rng.random() < 0.15:
            counts = [_spread(rng, 1, min(300, most))]
        else:
            per = rng.choice([1, 1, 4])
            counts = [rng.randint(0, per) if per > 1 else 1 for _ in range(_spread(rng, 1, max(1, min(300, most // per))))]
        return dict(op=op, counts=_text(counts if sum(counts) else [1]), heads=heads, kheads=kheads, dk=dk, dv=dv,
                    dtype=dtype, raw=rng.random() < 0.5)
    if op == "attend":
        kvheads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        heads = kvheads * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
        most = 2 ** (28 if dtype == "bf16" else 27) // (kvheads * dim)   # keys that the largest listed case reads
        seqs = _spread(rng, 1, 256)
        longest = _spread(rng, 1, max(1, min(100000, most // seqs)))
        lengths = [rng.randint(0, longest) for _ in range(seqs - 1)] + [longest]
        per = rng.choice([1, 1, 1, 4])
        counts = [min(n, rng.randint(0, per) if per > 1 else 1) for n in lengths[:-1]] + [1]
        return dict(op=op, lengths=_text(lengths), counts=_text(counts), heads=heads, kvheads=kvheads, dim=dim,
                    block=16 * rng.choice([1, 1, 2, 3, 4, 16, 33]), window=rng.choice([0, 0, _spread(rng, 1, 4096)]),
                    dtype=dtype)
    if op == "write":
        kvheads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        tokens = _spread(rng, 1, 2 ** 24 // (kvheads * dim))
        seqs = min(tokens, _spread(rng, 1, 256))
        cuts = sorted(rng.randint(0, tokens) for _ in range(seqs - 1))
        return dict(op=op, counts=_text(b - a for a, b in zip([0] + cuts, cuts + [tokens])), kvheads=kvheads, dim=dim,
                    block=16 * rng.choice([1, 1, 2, 3, 4, 16, 33]), dtype=dtype)
    if op == "tables":
        seqs = _spread(rng, 1, 1024)
        longest = _spread(rng, 1, max(1, 2 * 17252 // seqs))
        counts = [1] + [rng.choice([1, rng.randint(0, longest)]) for _ in range(seqs - 1)]
        return dict(op=op, computed=_text(rng.choice([0, rng.randint(0, 30000)]) for _ in range(seqs)),
                    counts=_text(counts), block=16 * rng.choice([1, 1, 2, 3, 4, 16, 33]))
    channels = 16 * _spread(rng, 4, 1024)
    rows = _spread(rng, 1, 2 ** (27 if dtype == "bf16" else 26) // channels)
    return dict(op=op, rows=rows, channels=channels, residual=rng.random() < 0.8, out=rng.choice(["same", "e4m3"]),
                group=rng.choice([0, 0, 64, 128]) if channels % 128 == 0 else 0, dtype=dtype)


def _ints(case, key):
    return [int(v) for v in case[key].split(",")]


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


def _shuffled(n, salt):
    return torch.randperm(n, generator=torch.Generator().manual_seed(n * 31 + salt)).to(torch.int32)


def _cu(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _scattered(lengths, block, spare=0):
    """A table of the blocks that hold sequences of these lengths, scattered over the cache, and the cache's blocks."""
    need = [-(-n // block) for n in lengths]
    order = _shuffled(max(1, sum(need)) + spare, len(lengths))
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, order.numel(), order[at:]


def _inputs(case, seed):
    r = _Draw(seed, _DTYPES[case.get("dtype", "f32")])
    i = dict(case=case)
    if case["op"] == "norm":
        rows, c = case["rows"], case["channels"]
        i.update(x=r.normal(rows, c), residual=r.normal(rows, c, scale=2.0) if case["residual"] else None,
                 weight=1.0 + r.normal(c, scale=0.2, dtype=torch.float32))
        return i
    counts = _ints(case, "counts")
    seqs, tokens = len(counts), sum(counts)
    i.update(counts=counts, tokens=tokens, cu=_cu(counts))
    if case["op"] == "delta":
        h, g, dk, dv = case["heads"], case["kheads"], case["dk"], case["dv"]
        # q, k and v lie side by side, as the convolution leaves them
        wide = r.normal(tokens, 2 * g * dk + h * dv)
        q, k, v = wide[:, :g * dk], wide[:, g * dk:2 * g * dk], wide[:, 2 * g * dk:]
        i.update(q=q.unflatten(1, (g, dk)), k=k.unflatten(1, (g, dk)), v=v.unflatten(1, (h, dv)))
        if case["raw"]:
            # the step size and the write strength as the projections give them, next to each other
            ab = r.normal(tokens, 2 * h)
            i.update(gate=ab[:, :h], beta=ab[:, h:], A=-torch.exp(r.uniform(0.0, math.log(16.0), h)),
                     dt_bias=r.uniform(-4.0, -2.0, h))
        else:
            for name in ("q", "k"):
                i[name] = (i[name].float() / i[name].float().square().sum(-1, keepdim=True).sqrt()).to(r.dtype)
            i.update(gate=-torch.exp(r.uniform(math.log(1e-3), math.log(0.2), tokens, h)),
                     beta=r.uniform(0.05, 0.95, tokens, h), A=None, dt_bias=None)
        # a sequence reads one slot of the cache; the state after each token goes to a slot of its own
        order = _shuffled(seqs + tokens, seqs).cuda()
        i.update(read=order[:seqs].contiguous(), write=order[seqs:].contiguous(),
                 cache=r.normal(seqs + tokens, h, dv, dk, scale=0.5, dtype=torch.float32))
        return i
    if case["op"] == "tables":
        computed, block = _ints(case, "computed"), case["block"]
        total = [a + b for a, b in zip(computed, counts)]
        need = [-(-t // block) - -(-c // block) for t, c in zip(total, computed)]
        old, blocks, free = _scattered(computed, block, spare=sum(need) + 100)
        # the table has a row for every request that may run, and columns for longer ones
        rows = _shuffled(2 * seqs, int(seed) % 1000)[:seqs]
        width = max(1, max(-(-t // block) for t in total)) + 3
        table = torch.full((2 * seqs, width), -1, dtype=torch.int32)
        table[rows.long(), :old.shape[1]] = old
        free = free[torch.randperm(free.numel(), generator=torch.Generator().manual_seed(int(seed)))]
        i.update(computed=torch.tensor(computed, dtype=torch.int32).cuda(),
                 new=torch.tensor(counts, dtype=torch.int32).cuda(), rows=rows.cuda(), table=table.cuda(),
                 free=free.cuda(), free_count=torch.tensor([free.numel()], dtype=torch.int32).cuda(),
                 free_left=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return i
    kv, d, block = case["kvheads"], case["dim"], case["block"]
    if case["op"] == "write":
        table, blocks, _ = _scattered(counts, block)
        slots = [table[s, torch.arange(n) // block] * block + torch.arange(n) % block for s, n in enumerate(counts)]
        # keys and values lie behind the queries, as the projection leaves them
        wide = r.normal(tokens, 4 * kv * d)
        i.update(k=wide[:, 2 * kv * d:3 * kv * d].unflatten(1, (kv, d)), v=wide[:, 3 * kv * d:].unflatten(1, (kv, d)),
                 slots=torch.cat(slots).to(torch.int32).cuda(),
                 kc=torch.zeros(blocks, kv, block, d, dtype=r.dtype, device="cuda"),
                 vc=torch.zeros(blocks, kv, d, block, dtype=r.dtype, device="cuda"))
        return i
    lengths = _ints(case, "lengths")
    table, blocks, _ = _scattered(lengths, block)
    wide = r.normal(tokens, (case["heads"] + 2 * kv) * d)
    i.update(q=wide[:, :case["heads"] * d].unflatten(1, (case["heads"], d)), table=table.cuda(), lengths=lengths,
             lens=torch.tensor(lengths, dtype=torch.int32).cuda(), kc=r.normal(blocks, kv, block, d),
             vc=r.normal(blocks, kv, d, block))
    return i


def prepare(case, seed):
    state = _inputs(case, seed)
    if own and case["op"] == "attend":
        # the split of the cache's length is planned once for a step and shared by all its layers
        from selective_state_space_cu_amd import ssd
        most = max(state["counts"])
        state["plan"] = ssd.attention_plan(state["lens"], case["heads"], case["kvheads"],
                                           cu_seqlens=None if min(state["counts"]) == most == 1 else state["cu"],
                                           total_tokens=state["tokens"], max_new_tokens=max(1, most),
                                           window=case["window"])
    return state


def run(i):
    case = i["case"]
    if not own:
        return {"delta": _plain_delta, "attend": _plain_attend, "write": _plain_write, "tables": _plain_tables,
                "norm": _plain_norm}[case["op"]](i, case)
    from selective_state_space_cu_amd import ssd
    if case["op"] == "delta":
        single = len(i["counts"]) == i["tokens"] and min(i["counts"]) == 1
        o = ssd.gated_delta_step(i["q"], i["k"], i["v"], i["gate"], i["beta"], i["cache"], i["read"], i["write"],
                                 cu_seqlens=None if single else i["cu"], A=i["A"], dt_bias=i["dt_bias"],
                                 qk_eps=1e-6 if case["raw"] else None)
        return {"o": o, "cache": i["cache"]}
    if case["op"] == "attend":
        return ssd.paged_attention_step(i["q"], i["kc"], i["vc"], i["table"], i["plan"])
    if case["op"] == "write":
        ssd.kv_cache_write(i["k"], i["v"], i["kc"], i["vc"], i["slots"])
        return {"k": i["kc"], "v": i["vc"]}
    if case["op"] == "tables":
        t = ssd.step_tables(i["computed"], i["new"], i["table"], case["block"], i["tokens"], rows=i["rows"],
                            free_blocks=i["free"], free_count=i["free_count"], free_count_out=i["free_left"])
        return {"table": i["table"], "cu": t.cu_seqlens, "lens": t.seq_lens, "positions": t.positions,
                "seq": t.token_seq, "slots": t.slots, "read": t.read_slot, "state": t.state_slot, "left": t.free_count}
    if case["out"] == "same":
        out, res = ssd.add_rms_norm(i["x"], weight=i["weight"], residual=i["residual"])
        return {"out": out} if res is None else {"out": out, "residual": res}
    out, scales, res = ssd.add_rms_norm_e4m3(i["x"], weight=i["weight"], residual=i["residual"], group=case["group"])
    return {"out": out, "scales": scales} if res is None else {"out": out, "scales": scales, "residual": res}


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_delta(i, case):
    """Token after token of all sequences side by side."""
    f32, counts = torch.float32, i["counts"]
    per = case["heads"] // case["kheads"]
    q, k, v = i["q"].to(f32), i["k"].to(f32), i["v"].to(f32)
    gate, beta = i["gate"].to(f32), i["beta"].to(f32)
    if case["raw"]:
        gate = i["A"] * _softplus(gate + i["dt_bias"])
        beta = 1 / (1 + torch.exp(-beta))
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q = (q * case["dk"] ** -0.5).repeat_interleave(per, 1)
    k = k.repeat_interleave(per, 1)
    o = torch.empty(i["tokens"], case["heads"], case["dv"], device="cuda", dtype=i["v"].dtype)
    starts = torch.tensor([0] + counts[:-1]).cumsum(0)
    h = i["cache"][i["read"]]
    for t in range(max(counts)):
        live = [s for s, n in enumerate(counts) if n > t]
        whole = len(live) == len(counts)
        at = (starts + t if whole else starts[live] + t).to("cuda", non_blocking=True)
        some = None if whole else torch.tensor(live).to("cuda", non_blocking=True)
        state = (h if whole else h[some]) * torch.exp(gate[at])[..., None, None]
        kt = k[at][:, :, None]
        delta = beta[at][..., None] * (v[at] - (state * kt).sum(-1))
        state = state + delta[..., None] * kt
        o[at] = (state * q[at][:, :, None]).sum(-1).to(o.dtype)
        i["cache"][i["write"][at]] = state
        if whole:
            h = state
        else:
            h[some] = state
    return {"o": o, "cache": i["cache"]}


def _plain_attend(i, case):
    """Sequences side by side, padded to the longest, as many at a time as _PLAIN_KEYS allows."""
    f32, kv, d, block = torch.float32, case["kvheads"], case["dim"], case["block"]
    g = case["heads"] // kv
    out = torch.empty_like(i["q"], memory_format=torch.contiguous_format)
    width, most = i["table"].shape[1], max(i["counts"])
    step = max(1, _PLAIN_KEYS // (width * block * kv * d))
    keys = torch.arange(width * block, device="cuda")
    starts = i["cu"].long()
    for s in range(0, len(i["counts"]), step):
        table = i["table"][s:s + step].clamp(min=0).long()
        n = table.shape[0]
        k = i["kc"][table].to(f32).permute(0, 2, 1, 3, 4).reshape(n, kv, width * block, d)
        v = i["vc"][table].to(f32).permute(0, 2, 1, 4, 3).reshape(n, kv, width * block, d)
        fresh = starts[s + 1:s + n + 1] - starts[s:s + n]
        j = torch.arange(most, device="cuda")[None]
        rows = torch.where(j < fresh[:, None], starts[s:s + n, None] + j, 0)
        last = i["lens"][s:s + n, None] - fresh[:, None] + j   # the position of each new token
        q = i["q"][rows].to(f32).view(n, most, kv, g, d).permute(0, 2, 1, 3, 4).reshape(n, kv, most * g, d)
        score = (torch.matmul(q, k.transpose(2, 3)) * d ** -0.5).view(n, kv, most, g, -1)
        seen = keys <= last[..., None]
        if case["window"]:
            seen = seen & (keys > last[..., None] - case["window"])
        seen = seen[:, None, :, None]
        top = torch.where(seen, score, -torch.inf).amax(-1, keepdim=True)
        p = torch.where(seen, torch.exp(score - top.clamp(min=-3e38)), 0.0)
        den = p.sum(-1, keepdim=True)
        r = torch.matmul(p.view(n, kv, most * g, -1), v).view(n, kv, most, g, d) / torch.where(den > 0, den, 1.0)
        r = r.permute(0, 2, 1, 3, 4).reshape(n, most, case["heads"], d).to(out.dtype)
        # rows past a sequence's tokens repeat what the batch's first rows get
        picked = torch.cat([torch.arange(c) + b * most for b, c in enumerate(i["counts"][s:s + n])])
        first = sum(i["counts"][:s])
        out[first:first + picked.numel()] = r.view(n * most, case["heads"], d)[picked.to("cuda", non_blocking=True)]
    return out


def _plain_write(i, case):
    slot = i["slots"].long()
    block, at = slot // case["block"], slot % case["block"]
    i["kc"][block, :, at] = i["k"]
    i["vc"][block, :, :, at] = i["v"]
    return {"k": i["kc"], "v": i["vc"]}


def _plain_tables(i, case):
    block, tokens, computed, new = case["block"], i["tokens"], i["computed"].long(), i["new"].long()
    seqs, total = computed.numel(), computed + new
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)])
    first = (computed + block - 1) // block
    need = (total + block - 1) // block - first
    taken = need.cumsum(0)
    at = torch.arange(i["table"].shape[1], device="cuda")[None] - first[:, None]
    fresh = i["free"].long()[(i["free_count"].long() - 1 - (taken - need)[:, None] - at).clamp(0, i["free"].numel() - 1)]
    rows = i["rows"].long()
    table = torch.where((at >= 0) & (at < need[:, None]), fresh, i["table"][rows].long())
    i["table"][rows] = table.to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), new, output_size=tokens)
    position = computed[seq] + torch.arange(tokens, device="cuda") - cu[seq]
    slot = table[seq, position // block] * block + position % block
    ends = (position + 1 == total[seq]) | ((position + 1) % block == 0)
    state = torch.where(ends, table[seq, position // block], -1)
    read = torch.where(computed > 0, table.gather(1, ((computed - 1) // block).clamp(min=0)[:, None])[:, 0], -1)
    left = i["free_count"].long() - taken[-1:]
    got = dict(cu=cu, lens=total, positions=position, seq=seq, slots=slot, read=read, state=state, left=left)
    return {"table": i["table"], **{name: t.to(torch.int32) for name, t in got.items()}}


def _plain_norm(i, case):
    v = i["x"].to(torch.float32)
    got = {}
    if i["residual"] is not None:
        v = v + i["residual"].to(torch.float32)
        got["residual"] = v.to(i["x"].dtype)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * i["weight"]
    if case["out"] == "same":
        return {"out": v.to(i["x"].dtype), **got}
    size = case["group"] or case["channels"]
    v = v.view(case["rows"], -1, size)
    top = v.abs().amax(-1)
    scales = torch.where(top > 0, top / _E4M3_MAX, 1.0)
    out = (v / scales[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(_E4M3)
    return {"out": out.view(case["rows"], -1), "scales": scales, **got}


def exact(case, seed):
    """float64 (whole numbers on the host), from the definitions, one sequence or one head after another."""
    i = _inputs(case, seed)
    if case["op"] == "tables":
        return _exact_tables(i, case)
    if case["op"] == "write":
        return _exact_write(i, case)
    i = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() and k not in ("kc", "vc") else v
         for k, v in i.items()}
    return {"delta": _exact_delta, "attend": _exact_attend, "norm": _exact_norm}[case["op"]](i, case)


def _exact_delta(i, case):
    per, dk = case["heads"] // case["kheads"], case["dk"]
    decay, strength = i["gate"].exp(), i["beta"]
    q, k = i["q"], i["k"]
    if case["raw"]:
        step = torch.logaddexp(i["gate"] + i["dt_bias"], torch.zeros_like(i["gate"]))
        decay, strength = (step * i["A"]).exp(), torch.sigmoid(i["beta"])
        q, k = (t / torch.sqrt(t.pow(2).sum(2, keepdim=True) + 1e-6) for t in (q, k))
    o, cache = torch.empty_like(i["v"]), i["cache"].clone()
    read, write, t = i["read"].tolist(), i["write"].tolist(), 0
    for s, n in enumerate(i["counts"]):
        state = i["cache"][read[s]].view(case["kheads"], per, case["dv"], dk)
        for t in range(t, t + n):
            a, b = (x[t].view(case["kheads"], per, 1) for x in (decay, strength))
            state = state * a.unsqueeze(3)
            miss = i["v"][t].view(case["kheads"], per, -1) - torch.matmul(state, k[t].view(-1, 1, dk, 1)).squeeze(3)
            state = state + (b * miss).unsqueeze(3) * k[t].view(-1, 1, 1, dk)
            o[t] = (torch.matmul(state, q[t].view(-1, 1, dk, 1)) / math.sqrt(dk)).reshape(case["heads"], -1)
            cache[write[t]] = state.reshape(case["heads"], -1, dk)
        t = t + 1 if n else t
    return {"o": o, "cache": cache}


def _exact_attend(i, case):
    kv, d, block = case["kvheads"], case["dim"], case["block"]
    g, t, out = case["heads"] // kv, 0, torch.zeros_like(i["q"])
    for s, (length, n) in enumerate(zip(i["lengths"], i["counts"])):
        if not n:
            continue
        blocks = i["table"][s, :-(-length // block)].long()
        for h in range(kv):
            k = i["kc"][blocks, h].double().reshape(-1, d)[:length]
            v = i["vc"][blocks, h].double().transpose(1, 2).reshape(-1, d)[:length]
            for j in range(n):
                end = length - n + j + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= begin:
                    continue
                score = i["q"][t + j, h * g:(h + 1) * g] @ k[begin:end].t() / math.sqrt(d)
                out[t + j, h * g:(h + 1) * g] = torch.softmax(score, 1) @ v[begin:end]
        t += n
    return out


def _exact_write(i, case):
    kc, vc = i["kc"].clone(), i["vc"].clone()
    flat = kc.transpose(1, 2).reshape(-1, case["kvheads"], case["dim"])
    flat[i["slots"].long()] = i["k"]
    shape = (kc.shape[0], case["block"], case["kvheads"], case["dim"])
    turned = vc.permute(0, 3, 1, 2).reshape(flat.shape)
    turned[i["slots"].long()] = i["v"]
    return {"k": flat.view(shape).permute(0, 2, 1, 3).double(), "v": turned.view(shape).permute(0, 2, 3, 1).double()}


def _exact_tables(i, case):
    block, table, rows, free = case["block"], i["table"].tolist(), i["rows"].tolist(), i["free"].tolist()
    free = free[:int(i["free_count"])]
    got = dict(cu=[0], lens=[], positions=[], seq=[], slots=[], read=[], state=[])
    for s, (computed, n) in enumerate(zip(i["computed"].tolist(), i["counts"])):
        row = table[rows[s]]
        got["read"].append(row[(computed - 1) // block] if computed else -1)
        for p in range(computed, computed + n):
            if p % block == 0:
                row[p // block] = free.pop()
            got["positions"].append(p)
            got["seq"].append(s)
            got["slots"].append(row[p // block] * block + p % block)
            got["state"].append(row[p // block] if p == computed + n - 1 or p % block == block - 1 else -1)
        got["cu"].append(got["cu"][-1] + n)
        got["lens"].append(computed + n)
    got["left"] = [len(free)]
    return {"table": torch.tensor(table, dtype=torch.int32).cuda(),
            **{name: torch.tensor(v, dtype=torch.int32).cuda() for name, v in got.items()}}


def _exact_norm(i, case):
    got = {}
    v = i["x"]
    if i["residual"] is not None:
        v = got["residual"] = v + i["residual"]
    v = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / case["channels"] + 1e-6) * i["weight"]
    if case["out"] == "same":
        return {"out": v, **got}
    parts = v.split(case["group"] or case["channels"], 1)
    scales = torch.stack([p.abs().max(1).values for p in parts], 1) / _E4M3_MAX
    # 8-bit values have no value between their steps to be near to
    return {"out": None, "scales": torch.where(scales > 0, scales, torch.ones_like(scales)), **got}


def work(case):
    """Each input read once and each output written once; an exponential, a product or a sum is one operation."""
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["channels"]
        out = n * e if case["out"] == "same" else n + 4 * n // (case["group"] or case["channels"])
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + 4 * case["channels"],
                "flops": n * (5 if case["residual"] else 4) + (2 * n if case["out"] == "e4m3" else 0)}
    counts = _ints(case, "counts")
    seqs, tokens = len(counts), sum(counts)
    if case["op"] == "delta":
        h, g, dk, dv = case["heads"], case["kheads"], case["dk"], case["dv"]
        started = sum(1 for n in counts if n)
        gates = 2 * tokens * h * (e if case["raw"] else 4)
        states = 4 * h * dk * dv * (started + tokens)
        return {"bytes": states + tokens * (2 * g * dk + 2 * h * dv) * e + gates + 4 * (seqs + tokens),
                "flops": tokens * h * (7 * dk * dv + 3 * dv + 20)}
    if case["op"] == "tables":
        block = case["block"]
        fresh = sum(-(-(c + n) // block) - -(-c // block) for c, n in zip(_ints(case, "computed"), counts))
        return {"bytes": 4 * (7 * seqs + 4 * tokens + 3 * fresh), "flops": 6 * (seqs + tokens)}
    kv, d = case["kvheads"], case["dim"]
    if case["op"] == "write":
        return {"bytes": tokens * (4 * kv * d * e + 4), "flops": 2 * tokens * kv * d}
    keys = pairs = 0
    for length, n in zip(_ints(case, "lengths"), counts):
        ends = range(length - n + 1, length + 1)
        seen = [min(end, case["window"] or end) for end in ends]
        pairs += sum(seen)
        keys += min(length, seen[0] + n - 1) if n else 0
    return {"bytes": 2 * keys * kv * d * e + 2 * tokens * case["heads"] * d * e,
            "flops": pairs * case["heads"] * (4 * d + 5)}
