"""The 8-bit output's codes where a rounding border decides: e4m3(n / scale) of the float32 quotient, scales max |n| / 448.

Rows of +-1 have a mean square of 1, so with eps 0 the norm is the weights themselves, and every expected scale and code is
exact."""
import pytest
import torch

from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


def signs(rows, c, dtype, seed):
    r = torch.Generator().manual_seed(seed)
    return (2.0 * torch.randint(0, 2, (rows, c), generator=r) - 1).to(dtype)


def codes(quotient):
    """What the codes of float32 quotients stand for (NaN stays NaN)."""
    return quotient.clamp(-448, 448).to(E4M3).float()


def call(x, w, **kw):
    out, scales, _ = ssd.add_rms_norm_e4m3(x.cuda(), weight=w.cuda(), eps=0.0, **kw)
    torch.cuda.synchronize()
    return out.float().cpu(), scales.cpu()


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=1e9), torch.nan_to_num(b, nan=1e9))


@pytest.mark.parametrize("dtype,c,group", [(BF, 256, 64), (F32, 256, 64), (F32, 1024, 512), (BF, 1024, 0), (F32, 31, 0)])
def test_groups_too_small_for_their_quotient_by_448(dtype, c, group):
    """Non-zero values below 448 x 2^-150, whose scale would round to 0: it is the smallest there is, and zeros stay zeros."""
    size = group or c
    w = torch.arange(c) % 25 * 2.0 ** -149   # 0 .. 24 steps
    x = signs(3, c, dtype, 65)
    out, scales = call(x, w, group=group)
    assert (scales == 2.0 ** -149).all() and scales.shape == (3, c // size)
    assert same(out, codes((torch.arange(c) % 25).float()) * x.float())


@pytest.mark.parametrize("scale", [-0.25, -3.0, -2.0 ** 33, 2.0 ** 33, -2.0 ** -110, 2.0 ** -130, 2.0 ** 126, 0.0, INF, NAN])
def test_given_scales_of_any_sign_and_size(scale):
    w = torch.tensor([0.0, 1.0, 25.0, 2.0 ** 40, 3 * 2.0 ** 39, 2.0 ** 127, 7 * 2.0 ** -149, 2.0 ** -105, INF, NAN, 0.3, 2.0 ** 31,
                      2.0 ** 128 - 2.0 ** 104, 2.0 ** -140, 1e-30, 1e30])
    x = signs(2, 16, F32, 64)
    given = torch.tensor([scale])
    out, _ = call(x, w, scale=given.cuda())
    assert same(out, codes(w / given * x))


def ties():
    """Values half way between two codes: 2^e (2 k + 1) / 16 for k = 8 .. 15, and those below the smallest normal code."""
    normal = [2.0 ** e * (2 * k + 1) / 16 for e in range(-6, 9) for k in range(8, 16)]
    return torch.tensor([v for v in normal if v < 448] + [(2 * k + 1) * 2.0 ** -10 for k in range(8)])


@pytest.mark.parametrize("dtype,odd", [(BF, False), (F32, False), (BF, True), (F32, True)])
def test_exact_ties_under_a_given_scale(dtype, odd):
    """n = tie x scale without a rounding, so n / scale is the tie itself, which goes to the even code."""
    r = torch.Generator().manual_seed(61)
    t = ties()
    t = t[:len(t) // 8 * 8 - (3 if odd else 0)]
    x = signs(3, t.numel(), dtype, 62)
    for k in range(60):
        scale = torch.randint(1 << 15, 1 << 16, (1,), generator=r).float() * 2.0 ** (k % 40 - 35)   # 16 bits, t has 5
        w = t * scale
        assert torch.equal(w.double(), t.double() * scale.double())
        out, _ = call(x, w, scale=scale.cuda())
        assert same(out, codes(t) * x.float()), float(scale)


CASES = [(2, 4096, 0, BF), (3, 4096, 128, BF), (3, 1024, 512, F32), (2, 512, 64, F32), (5, 320, 32, BF), (2, 1031, 0, BF), (4, 96, 32, F32),
         (2, 16384, 256, BF), (2, 9728, 256, F32)]


@pytest.mark.parametrize("rows,c,group,dtype", CASES)
def test_scales_and_codes_are_those_of_the_float32_quotients(rows, c, group, dtype):
    w = torch.randn(c, generator=torch.Generator().manual_seed(c)).abs() * 3
    x = signs(rows, c, dtype, 63)
    size = group or c
    want = w.view(-1, size).amax(1) / 448
    out, scales = call(x, w, group=group)
    assert torch.equal(scales, want.expand(rows, -1))
    assert same(out, codes(w / want.repeat_interleave(size)) * x.float())
    given = torch.tensor([0.0171])
    out, _ = call(x, w, scale=given.cuda())
    assert same(out, codes(w / given) * x.float())
