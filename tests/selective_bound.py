"""A float64 reference of the selective scan with a rigorous bound on what its float32 kernels may be off.

Units of U = 2^-24 (half a step of float32 relative to the value); the hardware's exp2 and reciprocal are good to one
step, 2 U. With `size` the sum of the absolute terms of a state (no cancellation, whatever order they are added in):
  delta: raw = dt + bias rounds (1 |raw|), the exponent raw log2 e its product and its constant (2 |raw|), exp2 2,
    polynomial 3.2, last sum 1                                                               -> 3 |raw| + 7
  decay a = exp2((delta log2 e) A): delta's, one constant, two products, times |delta A|; exp2 2; in segments one
    more product in the factor that joins them                                               -> (delta + 3) |delta A| + 3
  input b = (delta u) B: delta's and two products                                            -> delta + 2
  state a h + b: its rounding, and one more where segments are joined                        -> 2
  y: n / 2 + 4 sums one after the other at most; the gate: exponent 2 |z|, exp2 2, sum 1, reciprocal 2, products 2
A decay below 2^-126 counts as 0, and the product of the decays of up to eight tokens is off by up to 2^-149 more.
The sum of first-order terms is taken 1.01 times: |delta A| is below 104 where a is not 0, so a relative error is below
(3 x 10 + 10) x 104 x 2^-24 = 2.5e-4, and its square below a thousandth of it.
"""
import torch

from selective_ref import U, silu, softplus


def scan(u, dt, A, B, C, dt_bias=None, D=None, z=None, state=None):
    """One sequence: u, dt, z (L, D), B, C (L, G, N), state (D, N) or None.
    Returns y, every state (L, D, N), and the bounds of both."""
    u, dt, A, B, C = (t.double() for t in (u, dt, A, B, C))
    L, d = u.shape
    n = B.shape[2]
    per = d // B.shape[1]
    raw = dt + (0 if dt_bias is None else dt_bias.double())
    delta = softplus(raw)
    units = 3 * raw.abs().clamp(max=120) + 7
    h = torch.zeros(d, n, dtype=torch.float64) if state is None else state.double().clone()
    size, err = h.abs(), torch.zeros_like(h)
    y, yerr = torch.zeros(L, d, dtype=torch.float64), torch.zeros(L, d, dtype=torch.float64)
    hs, herr, sizes = [], [], [size]
    for t in range(L):
        e = delta[t][:, None] * A
        a = torch.exp(e)
        b = (delta[t] * u[t])[:, None] * B[t].repeat_interleave(per, 0)
        k = units[t][:, None]
        bound = 1.01 * U * (((k + 3) * e.abs() + 3) * a * size + (k + 2) * b.abs()) + 2.0 ** -126 * size
        err = a * err + bound
        size = a * size + b.abs()
        sizes = sizes[-8:] + [size]
        err = err + 1.01 * U * 2 * size + 2.0 ** -149 * torch.stack(sizes).amax(0)
        h = a * h + b
        hs.append(h)
        herr.append(err.clone())
        c = C[t].repeat_interleave(per, 0)
        skip = torch.zeros(d, dtype=torch.float64) if D is None else D.double() * u[t]
        y[t] = (h * c).sum(1) + skip
        yerr[t] = (err * c.abs()).sum(1) + 1.01 * U * (n / 2 + 4) * ((size * c.abs()).sum(1) + skip.abs())
        if z is not None:
            g = silu(z[t].double())
            yerr[t] = yerr[t] * g.abs() + 1.01 * U * (2 * z[t].double().abs() + 7) * ((y[t] * g).abs() + yerr[t] * g.abs())
            y[t] = y[t] * g
    stack = (lambda v: torch.stack(v) if v else torch.zeros(0, d, n, dtype=torch.float64))
    return y, stack(hs), yerr, stack(herr)
