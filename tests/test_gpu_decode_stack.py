"""The decode step's operators together, as a server of a hybrid stack runs them: a delta-rule layer and an attention layer
with their caches, token after token through block tables, against the whole sequences in float64."""
import pytest
import torch

import step_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F32 = torch.float32
C, H, G, DK, DV, WIDTH = 64, 4, 2, 64, 32, 4     # residual channels; value and key heads of the delta rule; conv taps
HQ, HKV, D = 4, 2, 64                            # heads of the attention
CONV = 2 * G * DK + H * DV
KV_BLOCK, STATE_BLOCK = 16, 8


def weights(seed=0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)   # noqa: E731
    return dict(n1=1 + 0.1 * n(C), n2=1 + 0.1 * n(C), n3=1 + 0.1 * n(C), w1=n(C, CONV + 2 * H + H * DV) / 8, conv=n(CONV, WIDTH) / 2,
                A=-torch.exp(n(H) * 0.5), bias=n(H) - 2, out1=n(H * DV, C) / 12, w2=n(C, (HQ + 2 * HKV) * D) / 8,
                out2=n(HQ * D, C) / 16)


def norm(v, w, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * w


def whole(x, w):
    """One sequence in float64: (the residual stream after both layers, the last norm)."""
    w = {k: v.double() for k, v in w.items()}
    L = x.shape[0]
    res = x.double()
    p = norm(res, w["n1"], 1e-6) @ w["w1"]
    u, a, b, z = p.split([CONV, H, H, H * DV], 1)
    padded = torch.cat([torch.zeros(WIDTH - 1, CONV, dtype=torch.float64), u])
    u = sum(padded[k:k + L] * w["conv"][:, k] for k in range(WIDTH))
    u = u * torch.sigmoid(u)
    q, k, v = u.split([G * DK, G * DK, H * DV], 1)
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()   # noqa: E731
    q, k = (unit(t.view(L, G, DK)).repeat_interleave(H // G, 1) for t in (q, k))
    v, state, o = v.view(L, H, DV), torch.zeros(H, DV, DK, dtype=torch.float64), []
    decay = torch.exp(w["A"] * torch.nn.functional.softplus(a + w["bias"]))
    for t in range(L):
        state = state * decay[t][:, None, None]
        miss = torch.sigmoid(b[t])[:, None] * (v[t] - (state * k[t][:, None]).sum(-1))
        state = state + miss[:, :, None] * k[t][:, None]
        o.append((state * q[t][:, None]).sum(-1) * DK ** -0.5)
    o = torch.stack(o) * (z * torch.sigmoid(z)).view(L, H, DV)
    o = (o / (o.square().mean(-1, keepdim=True) + 1e-5).sqrt()).reshape(L, -1)
    res = res + o @ w["out1"]
    p = norm(res, w["n2"], 1e-6) @ w["w2"]
    q, k, v = p.split([HQ * D, HKV * D, HKV * D], 1)
    q, k, v = q.view(L, HQ, D), k.view(L, HKV, D), v.view(L, HKV, D)
    out = torch.zeros(L, HQ, D, dtype=torch.float64)
    for h in range(HQ):
        s = (q[:, h] @ k[:, h * HKV // HQ].t()) * D ** -0.5
        s = s.masked_fill(torch.ones(L, L, dtype=torch.bool).triu(1), -float("inf"))
        out[:, h] = torch.softmax(s, 1) @ v[:, h * HKV // HQ]
    res = res + out.reshape(L, -1) @ w["out2"]
    return res, norm(res, w["n3"], 1e-6)


class Server:
    """The caches, tables and free lists of a few requests."""

    def __init__(self, w, requests, longest):
        dev = dict(device="cuda")
        i32 = dict(dtype=torch.int32, **dev)
        self.w = {k: v.cuda() for k, v in w.items()}
        kv_blocks, state_blocks = requests * (-(-longest // KV_BLOCK)) + 2, requests * (-(-longest // STATE_BLOCK)) + 2
        self.kc = torch.full((kv_blocks, HKV, KV_BLOCK, D), float("nan"), **dev)
        self.vc = torch.full((kv_blocks, HKV, D, KV_BLOCK), float("nan"), **dev)
        self.states = torch.full((state_blocks, H, DV, DK), float("nan"), **dev)
        self.conv = torch.full((state_blocks, WIDTH - 1, CONV), float("nan"), **dev)
        self.kv_table = torch.full((requests, -(-longest // KV_BLOCK)), -1, **i32)
        self.state_table = torch.full((requests, -(-longest // STATE_BLOCK)), -1, **i32)
        r = torch.Generator().manual_seed(1)
        self.kv_free, self.state_free = (torch.randperm(n, generator=r).to(**i32) for n in (kv_blocks, state_blocks))
        self.kv_left, self.state_left = torch.tensor([kv_blocks], **i32), torch.tensor([state_blocks], **i32)
        self.flag = torch.zeros(1, **i32)

    def step(self, x, computed, rows):
        """One new token x (S, C) of each request in `rows`, which have `computed` tokens."""
        w, s, flag = self.w, x.shape[0], self.flag
        new = torch.ones_like(computed)
        kv = ssd.step_tables(computed, new, self.kv_table, KV_BLOCK, s, rows=rows, free_blocks=self.kv_free,
                             free_count=self.kv_left, free_count_out=self.kv_left, num_blocks=self.kc.shape[0], error_flag=flag)
        st = ssd.step_tables(computed, new, self.state_table, STATE_BLOCK, s, rows=rows, free_blocks=self.state_free,
                             free_count=self.state_left, free_count_out=self.state_left, num_blocks=self.states.shape[0],
                             error_flag=flag)
        plan = ssd.attention_plan(kv.seq_lens, HQ, HKV)
        n, _ = ssd.add_rms_norm(x, weight=w["n1"])
        u, a, b, z = (n @ w["w1"]).split([CONV, H, H, H * DV], 1)
        u = ssd.causal_conv1d_step(u, w["conv"], self.conv, st.read_slot, st.state_slot, error_flag=flag)
        q, k, v = u.split([G * DK, G * DK, H * DV], 1)
        o = ssd.gated_delta_step(q.unflatten(1, (G, DK)), k.unflatten(1, (G, DK)), v.unflatten(1, (H, DV)), a, b, self.states,
                                 st.read_slot, st.state_slot, A=w["A"], dt_bias=w["bias"], qk_eps=1e-6, error_flag=flag)
        o = ssd.group_norm(o.flatten(1), H, z=z.contiguous(), act="gate_first", center=False)
        n, res = ssd.add_rms_norm(o @ w["out1"], weight=w["n2"], residual=x)
        q, k, v = (n @ w["w2"]).split([HQ * D, HKV * D, HKV * D], 1)
        ssd.kv_cache_write(k.unflatten(1, (HKV, D)), v.unflatten(1, (HKV, D)), self.kc, self.vc, kv.slots, error_flag=flag)
        out = ssd.paged_attention_step(q.unflatten(1, (HQ, D)), self.kc, self.vc, self.kv_table, plan, rows=rows, error_flag=flag)
        n, res = ssd.add_rms_norm(out.flatten(1) @ w["out2"], weight=w["n3"], residual=res)
        code, scales, _ = ssd.add_rms_norm_e4m3(res, weight=w["n3"], group=32)
        return n, res, code, scales


def prompts(lengths, seed=2):
    r = torch.Generator().manual_seed(seed)
    return [torch.randn(n, C, generator=r) for n in lengths]


def test_stack_token_by_token_equals_the_whole_sequences():
    """Requests that start at different steps and rows; every token of each against its float64 forward."""
    lengths, starts, rows = [41, 17, 30, 5], [0, 3, 11, 40], [2, 0, 3, 1]
    w, xs = weights(), prompts(lengths)
    server, want = Server(w, 4, 41), [whole(x, w) for x in xs]
    worst = 0.0
    for step in range(max(s + n for s, n in zip(starts, lengths))):
        live = [k for k in range(4) if starts[k] <= step < starts[k] + lengths[k]]
        at = [step - starts[k] for k in live]
        x = torch.stack([xs[k][p] for k, p in zip(live, at)]).cuda()
        n, res, code, scales = server.step(x, torch.tensor(at, dtype=torch.int32).cuda(),
                                           torch.tensor([rows[k] for k in live], dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        # twelve float32 operations of at most 128 terms each, every one within 300 x 2^-24 = 2e-5 of values of order 1,
        # through maps of gains up to 4: 12 x 4 x 2e-5
        tol = 1e-3
        for j, (k, p) in enumerate(zip(live, at)):
            for name, got, exact in (("norm", n[j], want[k][1][p]), ("residual", res[j], want[k][0][p])):
                err = (got.double().cpu() - exact).abs()
                assert (err <= tol * (1 + exact.abs())).all(), f"{name} of request {k}, token {p}: {err.max().item():.2e}"
                worst = max(worst, err.max().item())
            exact = want[k][1][p]
            back = code[j].double().cpu() * scales[j].double().cpu().repeat_interleave(32)
            half = torch.maximum(exact.abs() * 2.0 ** -4, scales[j].double().cpu().repeat_interleave(32) * 2.0 ** -10)
            assert ((back - exact).abs() <= half * 1.01 + tol * (1 + exact.abs())).all(), f"codes of request {k}, token {p}"
    assert int(server.flag.item()) == 0
    log(f"  worst error {worst:.2e}")


def test_stack_captured_and_replayed():
    """The whole step in one graph, replayed as a decode loop does: inputs and lengths change, blocks are taken."""
    lengths = [38, 38, 38]
    w, xs = weights(1), prompts(lengths, 3)
    eager, graphed = Server(w, 3, 38), Server(w, 3, 38)
    rows = torch.tensor([1, 2, 0], dtype=torch.int32).cuda()
    x, computed = torch.zeros(3, C, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    warm = Server(w, 3, 38)
    warm.step(x, computed, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = graphed.step(x, computed, rows)
        computed.add_(1)
    computed.zero_()
    for p in range(38):
        x.copy_(torch.stack([s[p] for s in xs]))
        graph.replay()
        torch.cuda.synchronize()
        want = eager.step(torch.stack([s[p] for s in xs]).cuda(), torch.full((3,), p, dtype=torch.int32, device="cuda"), rows)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.float(), b.float()), f"token {p}"
    assert int(graphed.flag.item()) == 0 and torch.equal(graphed.kv_table, eager.kv_table)


def test_speculated_tokens_continue_from_the_accepted_one():
    """Four tokens at once with a slot for the state after each, two of them accepted: the next step reads the second's
    slot, and everything is bit for bit what one token at a time gives."""
    r = torch.Generator().manual_seed(4)
    T, heads, kheads, dk, dv = 4, 4, 2, 128, 40
    one = lambda *s: torch.randn(*s, generator=r).cuda()   # noqa: E731
    q, k, v, ab = one(T, kheads, dk), one(T, kheads, dk), one(T, heads, dv), one(T, 2 * heads)
    A, cache = -torch.exp(one(heads)), one(12, heads, dv, dk)
    slot = lambda *s: torch.tensor(s, dtype=torch.int32).cuda()   # noqa: E731
    kw = dict(A=A, qk_eps=1e-6)
    serial = cache.clone()
    outs = [ssd.gated_delta_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], ab[t:t + 1, :heads], ab[t:t + 1, heads:], serial,
                                 slot(0 if t == 0 else 4 + t), slot(5 + t), **kw) for t in range(T)]
    o = ssd.gated_delta_step(q, k, v, ab[:, :heads], ab[:, heads:], cache, slot(0), slot(5, 6, 7, 8), cu_seqlens=slot(0, T), **kw)
    assert torch.equal(o, torch.cat(outs)) and torch.equal(cache, serial)
    # the third and fourth were rejected: other tokens follow the second
    again = ssd.gated_delta_step(q[:2], k[:2], v[2:], ab[:2, :heads], ab[:2, heads:], cache, slot(6), slot(7, 8),
                                 cu_seqlens=slot(0, 2), **kw)
    first = ssd.gated_delta_step(q[:1], k[:1], v[2:3], ab[:1, :heads], ab[:1, heads:], serial, slot(6), slot(9), **kw)
    second = ssd.gated_delta_step(q[1:2], k[1:2], v[3:], ab[1:2, :heads], ab[1:2, heads:], serial, slot(9), slot(10), **kw)
    assert torch.equal(again, torch.cat([first, second])) and torch.equal(cache[8], serial[10])


def test_calls_on_two_streams_with_their_own_workspaces():
    """Two attention calls that overlap, each with its workspace, give what each gives alone."""
    r = torch.Generator().manual_seed(5)
    q = torch.randn(2, 3, 8, 128, generator=r).cuda().to(torch.bfloat16)
    kc, vc = (torch.randn(200, 2, *s, generator=r).cuda().to(torch.bfloat16) for s in ((16, 128), (128, 16)))
    table = torch.randperm(200, generator=r)[:186].to(torch.int32).view(3, 62).cuda()
    plan = ssd.attention_plan(torch.tensor([990, 500, 77], dtype=torch.int32).cuda(), 8, 2)
    want = [ssd.paged_attention_step(q[i], kc, vc, table, plan) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append((i, ssd.paged_attention_step(q[i], kc, vc, table, plan)))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i])


def test_large_norms_stream_and_equal_the_small_calls():
    """Rows past what the last-level cache holds take the same values."""
    x = torch.empty(30000, 2048, device="cuda", dtype=torch.bfloat16).normal_()
    res = torch.empty_like(x).normal_()
    out, new = ssd.add_rms_norm(x, residual=res)
    code, scales, _ = ssd.add_rms_norm_e4m3(x, residual=res, group=128)
    for at in (0, 12345, 29000):
        a, b = ssd.add_rms_norm(x[at:at + 1000], residual=res[at:at + 1000])
        c, d, _ = ssd.add_rms_norm_e4m3(x[at:at + 1000], residual=res[at:at + 1000], group=128)
        assert torch.equal(a, out[at:at + 1000]) and torch.equal(b, new[at:at + 1000])
        assert torch.equal(c.float(), code[at:at + 1000].float()) and torch.equal(d, scales[at:at + 1000])
