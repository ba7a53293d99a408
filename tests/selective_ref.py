"""float64 references of the selective scan, its step, the conv step and the group norm, each with a bound on
what a float32 evaluation may be off (torch on the CPU, from the definitions).

Bounds count roundings in units of U = 2^-24 (half a step of float32 relative to the value). The hardware's
exp2, log2 and reciprocal are good to one step, 2 U.
"""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # torch.finfo(t).eps / 2


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def silu(v):
    return v * torch.sigmoid(v)


def _silu_units(v):
    """Relative error of v / (1 + e^-v) in units: the exponent's product (3 |v|), exp2, 1 + e, reciprocal, product."""
    return 3 * v.abs() + 8


def scan(u, dt, A, B, C, dt_bias=None, D=None, z=None, state=None):
    """One sequence: u, dt, z (L, D), B, C (L, G, N), state (D, N) or None.
    Returns y, every state (L, D, N), and the bounds of both."""
    u, dt, A, B, C = (t.double() for t in (u, dt, A, B, C))
    L, d = u.shape
    g, n = B.shape[1:]
    per = d // g
    raw = dt + (0 if dt_bias is None else dt_bias.double())
    delta = softplus(raw)
    # delta: sum dt + bias and the exponent's product carry |raw|, the series or the logarithm the rest
    units_d = 16 + 4 * raw.abs().clamp(max=100)
    h = torch.zeros(d, n, dtype=torch.float64) if state is None else state.double().clone()
    err = torch.zeros_like(h)
    y, yerr = torch.zeros(L, d, dtype=torch.float64), torch.zeros(L, d, dtype=torch.float64)
    hs, herr = [], []
    for t in range(L):
        e = delta[t][:, None] * A
        a = torch.exp(e)
        b = (delta[t] * u[t])[:, None] * B[t].repeat_interleave(per, 0)
        # a h: exp2 (2), product and sum (2), a sum over a run of tokens joined in another order (4); the exponent
        # itself is off by the units of delta, of A log2 e and of sums of up to 16 tokens' delta
        err = a * err + U * ((8 + (24 + units_d[t][:, None]) * e.abs()) * a * h.abs()
                             + (8 + units_d[t][:, None]) * b.abs())
        h = a * h + b
        hs.append(h)
        herr.append(err.clone())
        c = C[t].repeat_interleave(per, 0)
        skip = 0 if D is None else D.double() * u[t]
        y[t] = (h * c).sum(1) + skip
        yerr[t] = (err * c.abs()).sum(1) + U * (n + 4) * ((h * c).abs().sum(1) + (skip.abs() if D is not None else 0))
        if z is not None:
            zz = z[t].double()
            s = silu(zz)
            yerr[t] = yerr[t] * s.abs() + U * _silu_units(zz) * (y[t] * s).abs()
            y[t] = y[t] * s
    stack = (lambda v: torch.stack(v) if v else torch.zeros(0, d, n, dtype=torch.float64))
    return y, stack(hs), yerr, stack(herr)


def conv_step(x, weight, window, bias=None, act=True):
    """x (S, C), window (S, W-1, C). Returns out and its bound."""
    taps = torch.cat([window.double(), x.double()[:, None]], 1) * weight.double().t()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if bias is None else bias.double()
    v = taps.sum(1) + b
    err = U * (weight.shape[1] + 1) * (taps.abs().sum(1) + b.abs())
    if act:
        # silu's slope is below 1.1
        return silu(v), 1.1 * err + U * _silu_units(v) * silu(v).abs()
    return v, err


def group_norm(x, ngroups, weight=None, bias=None, z=None, act="none", center=True, eps=1e-5):
    """x, z (rows, C). Returns out and its bound."""
    rows, c = x.shape
    v = x.double()
    verr = torch.zeros_like(v)
    gate = gate_units = None
    if z is not None:
        gate, gate_units = silu(z.double()), _silu_units(z.double()) + 1
    if act == "gate_first":
        v = v * gate
        verr = U * gate_units * v.abs()
    v, verr = v.view(rows, ngroups, -1), verr.view(rows, ngroups, -1)
    k = v.shape[-1]
    # sums of k values: a tree over lanes and at most 64 values one after the other, so 80 roundings at most
    depth = min(k, 80) + 4
    if center:
        mu = v.mean(-1, keepdim=True)
        verr = verr + verr.mean(-1, keepdim=True) + U * (depth * v.abs().mean(-1, keepdim=True) + (v - mu).abs())
        v = v - mu
    var = (v * v).mean(-1, keepdim=True)
    varerr = (2 * v.abs() * verr + verr ** 2).mean(-1, keepdim=True) + U * depth * var
    scale = (var + eps) ** -0.5
    # 1 / sqrt: half the argument's relative error, and the function's own roundings
    rel = 0.5 * varerr / (var + eps) + 6 * U
    o = v * scale
    oerr = verr * scale + o.abs() * (rel * 1.1 + 2 * U)
    o, oerr = o.view(rows, c), oerr.view(rows, c)
    if weight is not None:
        o, oerr = o * weight.double(), oerr * weight.double().abs() + U * (o * weight.double()).abs()
    if bias is not None:
        o = o + bias.double()
        oerr = oerr + U * o.abs()
    if act == "silu":
        oerr = 1.1 * oerr + U * _silu_units(o) * silu(o).abs()
        o = silu(o)
    if act == "gate_last":
        oerr = oerr * gate.abs() + U * gate_units * (o * gate).abs()
        o = o * gate
    return o, oerr


def check(got, want, bound, what):
    """|got - want| within the bound, one rounding to got's type and nothing else (float32 minimum normal for
    results that the hardware may flush to zero)."""
    half = HALF[got.dtype]
    g = got.detach().cpu().double()
    assert g.shape == want.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(want.shape)}"
    assert torch.isfinite(g).all(), f"{what}: not finite"
    allowed = bound + half * (want.abs() + bound) + 2.0 ** -125
    worst = ((g - want).abs() / allowed).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.3f} of the bound"
    return worst
