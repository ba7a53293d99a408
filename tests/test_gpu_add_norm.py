"""The norm with the residual's addition and its 8-bit output against float64."""
import pytest
import torch

import step_ref as ref
from gpu_util import log
from selective_state_space_cu_amd import ssd

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


def inputs(rows, c, dtype, residual=True, pad=0, seed=0):
    r = torch.Generator().manual_seed(seed)
    wide = [torch.randn(rows, c + pad, generator=r).to(dtype).cuda()[:, pad:] for _ in range(2)]
    return dict(x=wide[0], residual=2 * wide[1] if residual else None, weight=1 + 0.3 * torch.randn(c, generator=r).cuda())


def check_codes(out, scales, norm, rel, group, what):
    """The values that the 8 bits stand for: within half a step of norm / scale, and the float32 error before it."""
    rows, c = norm.shape
    size = group or c
    wide = scales.double().cpu().reshape(rows if scales.dim() == 2 else 1, -1).expand(rows, -1)
    wide = wide.repeat_interleave(c // wide.shape[1], 1)
    if scales.dim() == 2:
        top = norm.view(rows, -1, size).abs().amax(-1)
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        ref.check(scales, want, want * (rel + 3 * ref.EPS), f"{what}: scales")
    y = norm / wide
    err = y.abs() * (rel + 3 * ref.EPS)
    half = torch.maximum((y.abs() + err) * 2.0 ** -4, torch.full_like(y, 2.0 ** -10))   # smallest step 2^-9
    ref.check(out.float(), y.clamp(-448, 448), half + err, f"{what}: codes")


CASES = [
    # rows, channels, type, residual, elements before each row
    (1, 1, F32, True, 0), (1, 64, BF, True, 0), (3, 5, F32, False, 0), (5, 100, BF, True, 3), (2, 4096, BF, True, 0),
    (3, 4100, F32, True, 0), (4, 5120, BF, False, 8), (1, 16384, BF, True, 0), (2, 16383, F32, True, 1), (300, 512, BF, True, 0),
    (7, 2056, BF, True, 4), (33, 96, F32, False, 4), (1000, 128, BF, True, 0), (6, 8192, F32, True, 0), (70, 1031, BF, True, 0),
    (9, 2048, BF, True, 2), (3, 6144, BF, True, 8), (5, 256, F32, True, 0), (131, 64, F32, True, 4), (9, 128, F32, True, 0),
    (77, 160, BF, False, 8), (5, 1040, BF, True, 0), (3, 2064, F32, True, 4), (4, 512, BF, True, 3), (67, 32, BF, True, 0),
    (35, 320, F32, True, 0), (6, 768, F32, True, 1), (2, 12288, BF, True, 0), (3, 9728, F32, False, 0),
]


@pytest.mark.parametrize("c", range(len(CASES)))
def test_against_float64(c):
    rows, ch, dtype, residual, pad = CASES[c]
    log(f"add norm {CASES[c]}")
    i = inputs(rows, ch, dtype, residual, pad, seed=c)
    for weight in (i["weight"], None):
        out, res = ssd.add_rms_norm(i["x"], weight=weight, residual=i["residual"], eps=1e-5)
        torch.cuda.synchronize()
        r, norm, rel = ref.add_rms_norm(i["x"], i["residual"], weight, 1e-5)
        ref.check(out, norm, ref.rounded(norm, norm.abs() * rel, dtype), "out")
        if residual:
            ref.check(res, r, ref.rounded(r, r.abs() * ref.EPS, dtype), "residual")
        else:
            assert res is None


@pytest.mark.parametrize("c", range(len(CASES)))
def test_8_bit_output_against_float64(c):
    rows, ch, dtype, residual, pad = CASES[c]
    log(f"add norm e4m3 {CASES[c]}")
    i = inputs(rows, ch, dtype, residual, pad, seed=100 + c)
    r, norm, rel = ref.add_rms_norm(i["x"], i["residual"], i["weight"], 1e-6)
    for group in [0] + [g for g in (32, 64, 128, 256, 512) if ch % g == 0]:
        out, scales, res = ssd.add_rms_norm_e4m3(i["x"], weight=i["weight"], residual=i["residual"], group=group)
        torch.cuda.synchronize()
        assert out.dtype == E4M3 and scales.shape == (rows, ch // (group or ch))
        check_codes(out, scales, norm, rel, group, f"group {group}")
        if residual:
            ref.check(res, r, ref.rounded(r, r.abs() * ref.EPS, dtype), "residual")
    given = torch.tensor([0.01], device="cuda")   # clamps the largest
    out, scales, _ = ssd.add_rms_norm_e4m3(i["x"], weight=i["weight"], residual=i["residual"], scale=given)
    torch.cuda.synchronize()
    assert scales is given
    check_codes(out, given, norm, rel, 0, "given scale")


def test_zero_rows_infinities_and_nan():
    x = torch.randn(5, 256, generator=torch.Generator().manual_seed(3)).cuda()
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = float("inf")
    x[3, 200] = NAN
    out, _ = ssd.add_rms_norm(x)
    code, scales, _ = ssd.add_rms_norm_e4m3(x, group=128)
    torch.cuda.synchronize()
    r, norm, rel = ref.add_rms_norm(x, None, None, 1e-6)
    ref.check(out, norm, ref.rounded(norm, norm.abs() * rel, F32), "out")
    assert (code[0].float() == 0).all() and (scales[0] == 1).all()
    assert (code[1, :128].float() == 0).all() and scales[1, 0] == 1
    assert torch.isnan(code[3].float()).all() and torch.isnan(scales[3]).all()   # the row's mean is none
    # an infinity makes its own place NaN, and with it its group's scale; the others are 0
    assert torch.isnan(code[2, :128].float()).all() and torch.isnan(scales[2, 0])
    assert (code[2, 128:].float() == 0).all() and scales[2, 1] == 1
    check_codes(code[4:], scales[4:], norm[4:], rel, 128, "a plain row")


def test_values_far_from_one():
    """Sums of squares near float32's ends would be lost; these are not, and eps holds small rows."""
    for scale in (1e-12, 1e12):
        i = inputs(4, 777, F32, seed=4)
        x, res = i["x"] * scale, i["residual"] * scale
        out, _ = ssd.add_rms_norm(x, weight=i["weight"], residual=res, eps=1e-6)
        torch.cuda.synchronize()
        _, norm, rel = ref.add_rms_norm(x, res, i["weight"], 1e-6)
        ref.check(out, norm, ref.rounded(norm, norm.abs() * rel + 1e-45, F32), f"scale {scale}")


def test_8_bit_output_of_values_near_the_smallest():
    """Scales whose reciprocals are past float32's largest."""
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(6)).cuda()
    x[:, 5] = 0
    w = torch.full((256,), 1e-37, device="cuda")
    code, scales, _ = ssd.add_rms_norm_e4m3(x, weight=w, group=64)
    torch.cuda.synchronize()
    _, norm, rel = ref.add_rms_norm(x, None, w, 1e-6)
    assert (scales < 2.0 ** -126).all() and (code[:, 5].float() == 0).all()
    wide = scales.double().cpu().repeat_interleave(64, 1)
    y = norm / wide
    # scales and norms of this size are off by up to 2^-149, the smallest step; codes by that, and by half a step
    top = norm.view(3, -1, 64).abs().amax(-1)
    ref.check(scales, top / 448, torch.full_like(top, 2.0 ** -149) + top / 448 * (rel + 3 * ref.EPS), "scales")
    err = y.abs() * (rel + 3 * ref.EPS) + 2.0 ** -149 / wide
    ref.check(code.float(), y.clamp(-448, 448), torch.maximum((y.abs() + err) * 2.0 ** -4, torch.full_like(y, 2.0 ** -10)) + err, "codes")


def test_in_place_and_beside_other_columns():
    i = inputs(20, 96, BF, seed=5)
    want, want_res = ssd.add_rms_norm(i["x"], weight=i["weight"], residual=i["residual"])
    x, res = i["x"].clone(), i["residual"].clone()
    out, got = ssd.add_rms_norm(x, weight=i["weight"], residual=res, residual_out=res, out=x)
    assert out is x and got is res and torch.equal(x, want) and torch.equal(res, want_res)
    wide, wide8 = torch.full((20, 110), 7.0, dtype=BF, device="cuda"), torch.full((20, 110), 7.0, device="cuda").to(E4M3)
    ssd.add_rms_norm(i["x"], weight=i["weight"], residual=i["residual"], out=wide[:, 6:102])
    assert torch.equal(wide[:, 6:102], want) and (wide[:, :6] == 7).all() and (wide[:, 102:] == 7).all()
    code, scales, _ = ssd.add_rms_norm_e4m3(i["x"], weight=i["weight"], residual=i["residual"], group=32)
    for first in (4, 5):   # whole words of codes, and odd bytes
        wide8.copy_(torch.full((20, 110), 7.0, device="cuda").to(E4M3))
        part = wide8[:, first:first + 96]
        ssd.add_rms_norm_e4m3(i["x"], weight=i["weight"], residual=i["residual"], group=32, out=part)
        torch.cuda.synchronize()
        assert torch.equal(part.float(), code.float())
        assert (wide8[:, :first].float() == 7).all() and (wide8[:, first + 96:].float() == 7).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    assert ssd.add_rms_norm(x, residual=x)[0].shape == (0, 64)
    code, scales, _ = ssd.add_rms_norm_e4m3(x, group=32)
    assert code.shape == (0, 64) and scales.shape == (0, 2)
