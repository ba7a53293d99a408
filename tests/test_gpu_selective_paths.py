"""Every form in which the selective scan and its step are launched at the sizes of real batches, against float64 with
the bound of tests/selective_bound.py: the walk and 2, 4, 8 and 16 waves of segments, several sequences of a step in one
workgroup, and products of decays that leave float32's range."""
import pytest
import torch

import selective_bound as bound
import selective_ref as ref
from selective_state_space_cu_amd import ssd
from test_gpu_selective import BF, F32, call, cpu, make, starts

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
