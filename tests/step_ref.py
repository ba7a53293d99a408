"""Float64 forms of the decode-step operators, each with a bound on what float32 arithmetic and the roundings of its
outputs may add. EPS is half a step of float32 relative to the value; every bound counts roundings to first order and
adds one per cent for the rest."""
import torch

EPS = 2.0 ** -24
HALF_STEP = {torch.float32: EPS, torch.bfloat16: 2.0 ** -8}   # torch.finfo(t).eps / 2
MORE = 1.01


def check(got, want, bound, what):
    """Every value within its bound; infinities and NaN in the same places. Returns the worst share of the bound."""
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), f"{what}: infinities in other places"
    share = ((got - want).abs() / bound.clamp(min=1e-300))[fine & (got != want)]
    worst = share.max().item() if share.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound, max abs err {(got - want)[fine].abs().max().item():.3e}"
    return worst


def gated_delta(q, k, v, gate, beta, cache, read, write, cu=None, scale=None, A=None, dt_bias=None, qk_eps=None):
    """Token by token. Returns (o, its bound, the cache, its bound, sequences' skipped flags are the caller's)."""
    q, k, v, gate, beta, cache = (t.double().cpu() for t in (q, k, v, gate, beta, cache))
    T, H, dv = v.shape
    G, dk = k.shape[1:]
    cu = list(range(T + 1)) if cu is None else cu.tolist()
    read, write = read.tolist(), write.tolist()
    scale = dk ** -0.5 if scale is None else scale
    per = H // G
    sums = (dk / 8 + 4) * EPS           # a sum of dk products: 8 lanes' chains and their joins
    gate_err = 2 * EPS * gate.abs()
    beta_err = torch.zeros_like(beta)
    if A is not None:
        A = A.double().cpu()
        bias = torch.zeros_like(A) if dt_bias is None else dt_bias.double().cpu()
        x = gate + bias
        sp = torch.logaddexp(x, torch.zeros_like(x))
        gate = A * sp
        gate_err = A.abs() * (EPS * x.abs() + 3.2 * EPS * sp + EPS * sp) + 3 * EPS * gate.abs()
        beta_err = torch.sigmoid(beta) * (6 * EPS + 2 * EPS * beta.abs())
        beta = torch.sigmoid(beta)
    kn_err = qn_err = 0.0
    if qk_eps is not None:
        q = q / (q.square().sum(-1, keepdim=True) + qk_eps).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + qk_eps).sqrt()
        kn_err = qn_err = sums / 2 + 4 * EPS
    alpha = gate.exp()
    alpha_err = (alpha * (4 * EPS + gate_err)).nan_to_num(0.0)   # (e^-inf is exact)
    out, out_err = torch.zeros(T, H, dv, dtype=torch.float64), torch.zeros(T, H, dv, dtype=torch.float64)
    made, made_err = cache.clone(), torch.zeros_like(cache)
    for s in range(len(cu) - 1):
        st = cache[read[s]].clone() if read[s] >= 0 else torch.zeros_like(cache[0])
        err = torch.zeros_like(st)
        for t in range(cu[s], cu[s + 1]):
            kt, qt = (x[t].repeat_interleave(per, 0)[:, None, :] for x in (k, q))
            a, ea, b, eb = (x[t][:, None] for x in (alpha, alpha_err, beta, beta_err))
            dot = lambda m, n: (m * n).sum(-1)   # noqa: E731
            r, w, kq = dot(st, kt), dot(st, qt), dot(kt, qt)
            r_err = dot(err, kt.abs()) + dot(st.abs(), kt.abs()) * (sums + kn_err)
            w_err = dot(err, qt.abs()) + dot(st.abs(), qt.abs()) * (sums + qn_err)
            kq_err = dot(kt.abs(), qt.abs()) * (sums + kn_err + qn_err)
            d = b * (v[t] - a * r)
            # (an error of the strength multiplies the difference, whose own roundings are relative to its terms)
            d_err = b * (a * r_err + ea * r.abs() + 4 * EPS * (v[t].abs() + a * r.abs())) + (eb / b.clamp(min=1e-300) + 3 * EPS) * d.abs()
            out[t] = scale * (a * w + d * kq)
            out_err[t] = abs(scale) * (a * w_err + ea * w.abs() + d_err * kq.abs() + d.abs() * kq_err
                                       + 5 * EPS * (a * w.abs() + d.abs() * kq.abs()))
            new = a[..., None] * st + d[..., None] * kt
            err = (a[..., None] * err + ea[..., None] * st.abs() + d_err[..., None] * kt.abs()
                   + (d.abs()[..., None] * kt.abs()) * (kn_err + 3 * EPS) + 2 * EPS * (a[..., None] * st.abs()))
            st = new
            if write[t] >= 0:
                made[write[t]], made_err[write[t]] = st, err
    return out, out_err * MORE, made, made_err * MORE


def rounded(value, err, dtype):
    """The bound of a value whose error before its rounding to `dtype` is at most err."""
    return err + HALF_STEP[dtype] * (value.abs() + err) * MORE


def attention(q, keys, values, n, window=0, scale=None, p_step=0.0):
    """One sequence: q (n, Hq, D), keys and values (L, Hkv, D), the n last positions' rows. p_step: half a step of what
    probabilities are rounded to. Returns (out, bound before rounding, lse, its bound)."""
    q, keys, values = q.double(), keys.double(), values.double()
    L, hkv, D = keys.shape
    hq = q.shape[1]
    g = hq // hkv
    scale = D ** -0.5 if scale is None else scale
    out, bound = torch.zeros(n, hq, D, dtype=torch.float64), torch.zeros(n, hq, D, dtype=torch.float64)
    lse = torch.full((n, hq), -float("inf"), dtype=torch.float64)
    lse_bound = torch.zeros(n, hq, dtype=torch.float64)
    for j in range(n):
        hi = L - n + j + 1
        lo = max(0, hi - window) if window else 0
        if hi <= lo:
            continue
        for h in range(hq):
            k, v = keys[lo:hi, h // g], values[lo:hi, h // g]
            s = scale * (k @ q[j, h])
            s_err = abs(scale) * (k.abs() @ q[j, h].abs()) * (D + 2) * EPS
            top = s.max()
            e = (s - top).exp()
            # scaling to powers of two, the maximum's subtraction (of an equally scaled maximum), the exponential
            rel = s_err + 3 * EPS * s.abs() + 2 * EPS * top.abs() + 4 * EPS + (hi - lo + 40) * EPS
            den = e.sum()
            out[j, h] = (e @ v) / den
            bound[j, h] = ((e * (rel + p_step)) @ v.abs()) / den + out[j, h].abs() * ((e * rel).sum() / den + 6 * EPS)
            lse[j, h] = top + den.log()
            lse_bound[j, h] = (e * rel).sum() / den + 4 * EPS * (top.abs() + den.log().abs() + 1)
    return out, bound * MORE, lse, lse_bound * MORE


def gather_cache(k_cache, v_cache, table_row, length):
    """Keys and values (length, Hkv, D) of a sequence from the paged caches."""
    block = k_cache.shape[2]
    ids = table_row[:-(-length // block)].long().cpu() if length else torch.empty(0, dtype=torch.long)
    k = k_cache.cpu()[ids].permute(0, 2, 1, 3).reshape(-1, k_cache.shape[1], k_cache.shape[3])[:length]
    v = v_cache.cpu()[ids].permute(0, 3, 1, 2).reshape(-1, k_cache.shape[1], k_cache.shape[3])[:length]
    return k, v


def add_rms_norm(x, residual, weight, eps):
    """(r, norm, relative bound of the norm before its rounding)."""
    r = x.double().cpu() + (0 if residual is None else residual.double().cpu())
    c = r.shape[1]
    n = r / (r.square().mean(1, keepdim=True) + eps).sqrt()
    if weight is not None:
        n = n * weight.double().cpu()
    # the sum's rounding (and its square's), chains of at most 16 and their joins, root, reciprocal, products
    return r, n, ((16 + 24) / 2 + 10) * EPS * MORE


def step_tables(computed, new, rows, table, block, total, free, free_count, num_blocks=None):
    """What ssd_step_tables gives, in plain loops. Returns a dict of lists, the table and the error bits."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    num_blocks = (2 ** 31 - 1) // block if num_blocks is None else num_blocks
    got = dict(cu=[0], lens=[], read=[], pos=[-1] * total, seq=[-1] * total, slots=[-1] * total, state=[-1] * total)
    wanted, bits, left, at = 0, 0, free_count, 0
    for s, (c, n) in enumerate(zip(computed, new)):
        row, refused = rows[s] if rows is not None else s, 0
        if n < 0 or n > total:
            refused, n = 1, 0
        if c < 0 or c + n > 2 ** 31 - 1:
            refused = refused or 1
        elif not refused and not 0 <= row < len(table):
            refused = 4
        elif not refused and -(-(c + n) // block) > width:
            refused = 8
        need = 0
        if not refused and free is not None:
            first = -(-c // block)
            need = -(-(c + n) // block) - first
            wanted += need
            if need and wanted > free_count:
                refused = 16
            elif need:
                for j in range(need):
                    table[row][first + j] = free[free_count - 1 - (wanted - need + j)]
                left = free_count - wanted
        bits |= refused
        ok = lambda b: 0 <= b < num_blocks   # noqa: E731
        read = table[row][(c - 1) // block] if not refused and c > 0 else -1
        if read >= num_blocks:
            bits |= 8
        got["read"].append(read if ok(read) else -1)
        got["lens"].append(0 if refused else c + n)
        for j in range(n):
            if at + j >= total:
                bits |= 1
                break
            got["seq"][at + j] = s
            if refused:
                continue
            p = c + j
            b = table[row][p // block]
            got["pos"][at + j] = p
            if b >= num_blocks:
                bits |= 8
            if ok(b):
                got["slots"][at + j] = b * block + p % block
                if j == n - 1 or p % block == block - 1:
                    got["state"][at + j] = b
        at += n
        got["cu"].append(at)
    got["left"] = left
    return got, table, bits
