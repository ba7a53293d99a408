"""The decode step's operators (gated delta step, tables, cache write, paged attention and its plan, norms with a residual)
on the CPU: argument errors of the C ABI (nothing is launched) and the bindings' refusals."""
import ctypes
import os

import pytest
import torch

from selective_state_space_cu_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="libssd.so not built")

FAKE = 0x1000   # a non-NULL, 16-byte aligned address that is never dereferenced
NULL, SHAPE, BLOCK, CAPACITY, DTYPE, UNSUPPORTED = 1, 3, 4, 5, 6, 8
NAN = float("nan")


def call(fn, defaults, kw):
    assert not set(kw) - set(defaults), kw
    a = dict(defaults)
    a.update(kw)
    return getattr(ssd.load_library(), fn)(*a.values(), None)


DELTA = dict(q=FAKE, qs=256, k=FAKE, ks=256, v=FAKE, vs=384, gate=FAKE, gs=4, beta=FAKE, bs=4, A=FAKE, bias=FAKE, eps=1e-6,
             scale=0.1, dtype=1, gdtype=0, S=3, T=3, cu=None, H=4, G=2, dk=128, dv=96, cache=FAKE, slots=8, rs=FAKE, ws=FAKE,
             o=FAKE, os=384, flag=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(gdtype=-1), DTYPE), (dict(S=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=4), SHAPE), (dict(T=2 ** 30 + 1, cu=FAKE), SHAPE),
    (dict(H=0), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE), (dict(dv=0), SHAPE), (dict(dk=0), SHAPE), (dict(slots=-1), SHAPE),
    (dict(eps=NAN), SHAPE), (dict(scale=NAN), SHAPE), (dict(dk=32), UNSUPPORTED), (dict(dk=96), UNSUPPORTED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(gate=None), NULL), (dict(beta=None), NULL),
    (dict(cache=None), NULL), (dict(rs=None), NULL), (dict(ws=None), NULL), (dict(o=None), NULL), (dict(qs=255), SHAPE),
    (dict(ks=0), SHAPE), (dict(vs=-384), SHAPE), (dict(gs=3), SHAPE), (dict(bs=3), SHAPE), (dict(os=383), SHAPE),
    (dict(vs=2 ** 26 + 1), SHAPE), (dict(q=FAKE + 1), SHAPE), (dict(dtype=0, v=FAKE + 2), SHAPE), (dict(gate=FAKE + 2), SHAPE),
    (dict(A=FAKE + 2), SHAPE), (dict(cache=FAKE + 8), SHAPE),
])
def test_delta_step_rejects_bad_arguments(kw, code):
    assert call("ssd_gated_delta_step", DELTA, kw) == code


def test_delta_step_of_nothing_launches_nothing():
    none = dict(q=None, k=None, v=None, gate=None, beta=None, cache=None, rs=None, ws=None, o=None)
    assert call("ssd_gated_delta_step", DELTA, dict(S=0, T=0, **none)) == 0
    assert call("ssd_gated_delta_step", DELTA, dict(S=2, T=0, cu=FAKE, **none)) == 0


TABLES = dict(S=3, T=5, nc=FAKE, nn=FAKE, rows=None, table=FAKE, trows=4, width=8, block=16, blocks=100, free=FAKE, nfree=10,
              count=FAKE, left=FAKE, cu=FAKE, lens=FAKE, pos=FAKE, seq=FAKE, slots=FAKE, read=FAKE, state=FAKE, flag=None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), SHAPE), (dict(S=2 ** 20 + 1), SHAPE), (dict(T=-1), SHAPE), (dict(T=2 ** 20 + 1), SHAPE), (dict(trows=-1), SHAPE),
    (dict(width=-1), SHAPE), (dict(width=2 ** 20 + 1), SHAPE), (dict(blocks=-1), SHAPE), (dict(nfree=-1), SHAPE),
    (dict(nfree=2 ** 29 + 1), SHAPE), (dict(block=0), BLOCK), (dict(block=-16), BLOCK), (dict(blocks=2 ** 27), SHAPE),
    (dict(nc=None), NULL), (dict(nn=None), NULL), (dict(table=None), NULL), (dict(count=None), NULL), (dict(left=None), NULL),
    (dict(cu=None), NULL), (dict(lens=None), NULL), (dict(pos=None), NULL), (dict(seq=None), NULL), (dict(slots=None), NULL),
    (dict(read=None), NULL), (dict(state=None), NULL), (dict(nc=FAKE + 2), SHAPE), (dict(state=FAKE + 1), SHAPE),
])
def test_tables_reject_bad_arguments(kw, code):
    assert call("ssd_step_tables", TABLES, kw) == code


WRITE = dict(k=FAKE, ks=256, v=FAKE, vs=256, dtype=1, T=3, H=2, D=128, kc=FAKE, vc=FAKE, blocks=9, block=16, slots=FAKE, flag=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), DTYPE), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(D=0), SHAPE), (dict(D=80), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED), (dict(blocks=-1), SHAPE), (dict(block=0), BLOCK), (dict(block=8), BLOCK), (dict(block=24), BLOCK),
    (dict(blocks=2 ** 27), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(slots=None), NULL), (dict(ks=255), SHAPE), (dict(vs=2 ** 26 + 1), SHAPE), (dict(k=FAKE + 1), SHAPE),
    (dict(kc=FAKE + 8), SHAPE), (dict(vc=FAKE + 2), SHAPE), (dict(slots=FAKE + 2), SHAPE),
])
def test_cache_write_rejects_bad_arguments(kw, code):
    assert call("ssd_kv_cache_write", WRITE, kw) == code


def test_cache_write_of_nothing_launches_nothing():
    assert call("ssd_kv_cache_write", WRITE, dict(T=0, k=None, v=None, kc=None, vc=None, slots=None)) == 0


def plan(S=3, T=3, most=1, window=0, parts=20, null=(), **at):
    p = ssd._Plan(S, T, most, window, parts, *([FAKE] * 6))
    p.cu_seqlens = None
    for name in null:
        setattr(p, name, None)
    for name, v in at.items():
        setattr(p, name, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=4), SHAPE), (dict(most=0), SHAPE), (dict(most=65), SHAPE),
    (dict(window=-1), SHAPE), (dict(parts=3), CAPACITY), (dict(parts=-4), CAPACITY), (dict(parts=2 ** 26 + 1), SHAPE),
    (dict(null=["seq_lens"]), NULL), (dict(null=["part_start"]), NULL), (dict(null=["part_seq"]), NULL),
    (dict(null=["part_keys"]), NULL), (dict(null=["error_flag"]), NULL), (dict(seq_lens=FAKE + 2), SHAPE),
    (dict(T=9, cu_seqlens=FAKE + 1), SHAPE),
])
def test_plans_are_checked(kw, code):
    lib, p = ssd.load_library(), plan(**kw)
    assert lib.ssd_attention_plan_build(ctypes.byref(p), None) == code
    assert attend(p=p) == code
    assert lib.ssd_attention_plan_build(None, None) == NULL


ATTEND = dict(q=FAKE, qs=1024, kc=FAKE, vc=FAKE, dtype=1, scale=0.1, plan=None, Hq=8, Hkv=2, D=128, table=FAKE, trows=3, width=7,
              rows=None, blocks=30, block=16, out=FAKE, os=1024, lse=None, ws=FAKE, wsb=2 ** 40, flag=None)


def attend(p=None, **kw):
    p = plan() if p is None else p
    return call("ssd_paged_attention_step", dict(ATTEND, plan=ctypes.byref(p)), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=3), SHAPE), (dict(trows=-1), SHAPE),
    (dict(width=-1), SHAPE), (dict(scale=NAN), SHAPE), (dict(D=96), UNSUPPORTED), (dict(block=8), BLOCK), (dict(block=0), BLOCK),
    (dict(block=2 ** 20 + 16, blocks=1), BLOCK), (dict(blocks=2 ** 27), SHAPE), (dict(blocks=-1), SHAPE), (dict(q=None), NULL),
    (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL), (dict(qs=1023), SHAPE),
    (dict(os=2 ** 26 + 1), SHAPE), (dict(q=FAKE + 1), SHAPE), (dict(out=FAKE + 1), SHAPE), (dict(kc=FAKE + 8), SHAPE),
    (dict(ws=FAKE + 8), SHAPE), (dict(lse=FAKE + 2), SHAPE), (dict(table=FAKE + 2), SHAPE), (dict(ws=None), CAPACITY),
    (dict(wsb=20 * 8 * 130 * 4 - 1), CAPACITY),
])
def test_attention_rejects_bad_arguments(kw, code):
    assert attend(**kw) == code


def test_attention_of_nothing_launches_nothing():
    none = dict(q=None, kc=None, vc=None, table=None, out=None, ws=None, wsb=0)
    assert attend(plan(S=0, T=0), **none) == 0
    assert attend(plan(S=2, T=0, cu_seqlens=FAKE), **none) == 0


def test_parts_and_workspace():
    lib = ssd.load_library()
    assert lib.ssd_paged_attention_workspace_size(20, 1, 8, 128) == 20 * 8 * 130 * 4
    assert lib.ssd_paged_attention_workspace_size(0, 1, 8, 128) == lib.ssd_paged_attention_workspace_size(5, 0, 8, 128) == 0
    assert lib.ssd_paged_attention_parts(1, 32, 8) * 8 >= 256
    assert lib.ssd_paged_attention_parts(4, 32, 2) == -(-lib.ssd_paged_attention_parts(1, 32, 2) // 4)
    assert lib.ssd_paged_attention_parts(1, 7, 2) == lib.ssd_paged_attention_parts(0, 8, 2) == 0


NORM = dict(x=FAKE, xs=64, res=FAKE, rs=64, w=FAKE, dtype=1, rows=3, ch=64, eps=1e-6, ro=FAKE, ros=64, out=FAKE, os=64)
NORM8 = dict(x=FAKE, xs=64, res=FAKE, rs=64, w=FAKE, dtype=1, rows=3, ch=64, group=64, eps=1e-6, scale=None, scales=FAKE,
             ro=FAKE, ros=64, out=FAKE, os=64)
BOTH = [
    (dict(dtype=5), DTYPE), (dict(rows=-1), SHAPE), (dict(ch=0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(xs=63), SHAPE), (dict(rs=1), SHAPE), (dict(ros=0), SHAPE), (dict(os=2 ** 26 + 1), SHAPE), (dict(x=None), NULL),
    (dict(out=None), NULL), (dict(x=FAKE + 1), SHAPE), (dict(res=FAKE + 1), SHAPE), (dict(ro=FAKE + 1), SHAPE),
    (dict(w=FAKE + 2), SHAPE),
]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(out=FAKE + 1), SHAPE), (dict(ch=16385, xs=2 ** 15, rs=2 ** 15, ros=2 ** 15,
                                                                              os=2 ** 15), UNSUPPORTED)])
def test_norm_rejects_bad_arguments(kw, code):
    assert call("ssd_add_rms_norm", NORM, kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(group=0), UNSUPPORTED), (dict(group=48), UNSUPPORTED), (dict(group=128), UNSUPPORTED), (dict(group=16), UNSUPPORTED),
    (dict(ch=80, xs=80, rs=80, ros=80, os=80, group=32), UNSUPPORTED), (dict(scales=None), NULL), (dict(scales=FAKE + 2), SHAPE),
    (dict(scale=FAKE + 1), SHAPE),
])
def test_8_bit_norm_rejects_bad_arguments(kw, code):
    assert call("ssd_add_rms_norm_e4m3", NORM8, kw) == code


def test_norms_of_no_rows_launch_nothing():
    assert call("ssd_add_rms_norm", NORM, dict(rows=0, x=None, out=None)) == 0
    assert call("ssd_add_rms_norm_e4m3", NORM8, dict(rows=0, x=None, out=None, scales=None)) == 0


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_bindings_refuse_what_does_not_fit():
    i32 = torch.int32
    d = dict(q=zeros(3, 2, 64), k=zeros(3, 2, 64), v=zeros(3, 4, 8), gate=zeros(3, 4), beta=zeros(3, 4),
             state_cache=zeros(5, 4, 8, 64), read_slot=zeros(3, dtype=i32), write_slot=zeros(3, dtype=i32))
    for bad in (dict(q=zeros(2, 2, 64)), dict(k=zeros(3, 2, 32)), dict(v=zeros(3, 4, 8, dtype=torch.float16)),
                dict(gate=zeros(3, 5)), dict(beta=zeros(3, 4, dtype=torch.bfloat16)), dict(state_cache=zeros(5, 4, 64, 8)),
                dict(write_slot=zeros(2, dtype=i32)), dict(read_slot=zeros(2, dtype=i32)), dict(dt_bias=zeros(4)),
                dict(qk_eps=-1e-6), dict(A=zeros(3)), dict(cu_seqlens=zeros(3, dtype=i32)), dict(o=zeros(3, 4, 9)),
                dict(error_flag=zeros(1)), dict()):   # and the last: no GPU
        with pytest.raises(ValueError):
            ssd.gated_delta_step(**dict(d, **bad))
    t = dict(num_computed=zeros(3, dtype=i32), num_new=zeros(3, dtype=i32), block_table=zeros(3, 4, dtype=i32), block_size=16,
             total_tokens=3)
    for bad in (dict(num_new=zeros(2, dtype=i32)), dict(block_table=zeros(3, dtype=i32)), dict(block_size=0),
                dict(total_tokens=-1), dict(rows=zeros(4, dtype=i32)), dict(free_blocks=zeros(9, dtype=i32)),
                dict(free_count=zeros(1, dtype=i32)), dict(block_table=zeros(3, 4)),
                dict(free_blocks=zeros(9, dtype=i32), free_count=zeros(2, dtype=i32)), dict()):
        with pytest.raises(ValueError):
            ssd.step_tables(**dict(t, **bad))
    w = dict(k=zeros(3, 2, 64), v=zeros(3, 2, 64), k_cache=zeros(4, 2, 16, 64), v_cache=zeros(4, 2, 64, 16),
             slots=zeros(3, dtype=i32))
    for bad in (dict(v_cache=zeros(4, 2, 16, 64)), dict(k=zeros(3, 4, 64)), dict(v=zeros(3, 2, 32)), dict(slots=zeros(4, dtype=i32)),
                dict(k_cache=zeros(4, 16, 64)), dict(k_cache=zeros(4, 2, 16, 64, dtype=torch.bfloat16)), dict()):
        with pytest.raises(ValueError):
            ssd.kv_cache_write(**dict(w, **bad))
    for bad in (dict(num_heads=7), dict(num_kv_heads=0), dict(total_tokens=4), dict(cu_seqlens=zeros(4, dtype=i32)), dict()):
        with pytest.raises(ValueError):
            ssd.attention_plan(**dict(dict(seq_lens=zeros(3, dtype=i32), num_heads=8, num_kv_heads=2), **bad))
    p = ssd.AttentionPlan(3, 3, 1, 0, 20, *(zeros(4, dtype=i32) for _ in range(6)))
    a = dict(q=zeros(3, 4, 64), k_cache=zeros(4, 2, 16, 64), v_cache=zeros(4, 2, 64, 16), block_table=zeros(3, 4, dtype=i32),
             plan=p)
    for bad in (dict(q=zeros(2, 4, 64)), dict(q=zeros(3, 4, 128)), dict(q=zeros(3, 5, 64)), dict(block_table=zeros(2, 4, dtype=i32)),
                dict(block_table=zeros(12, dtype=i32)), dict(rows=zeros(2, dtype=i32)), dict(lse=zeros(3, 5)),
                dict(out=zeros(3, 4, 65)), dict(workspace=zeros(9)), dict()):
        with pytest.raises(ValueError):
            ssd.paged_attention_step(**dict(a, **bad))
    for bad in (dict(x=zeros(4)), dict(weight=zeros(63)), dict(residual=zeros(3, 63)), dict(residual_out=zeros(3, 64)),
                dict(residual=zeros(3, 64), residual_out=zeros(4, 64)), dict(out=zeros(3, 64, dtype=torch.bfloat16)), dict()):
        with pytest.raises(ValueError):
            ssd.add_rms_norm(**dict(dict(x=zeros(3, 64)), **bad))
    for bad in (dict(group=48), dict(group=-32), dict(scale=zeros(2)), dict(scale=zeros(1), scales=zeros(3, 1)),
                dict(scales=zeros(3, 2)), dict(out=zeros(3, 64)), dict()):
        with pytest.raises(ValueError):
            ssd.add_rms_norm_e4m3(**dict(dict(x=zeros(3, 64)), **bad))


def test_bindings_refuse_numbers_that_do_not_fit_32_bits():
    i32 = torch.int32
    for bad in (dict(max_new_tokens=0), dict(max_new_tokens=65), dict(max_new_tokens=2 ** 32 + 1), dict(window=-1),
                dict(window=2 ** 32 + 5)):
        with pytest.raises(ValueError, match="max_new_tokens must be"):
            ssd.attention_plan(zeros(3, dtype=i32), 8, 2, **bad)
    for bad in (-1, 2 ** 27, 2 ** 32 + 4):
        with pytest.raises(ValueError, match="num_blocks"):
            ssd.step_tables(zeros(3, dtype=i32), zeros(3, dtype=i32), zeros(3, 4, dtype=i32), 16, 3, num_blocks=bad)
    with pytest.raises(ValueError, match="block_size"):
        ssd.step_tables(zeros(3, dtype=i32), zeros(3, dtype=i32), zeros(3, 4, dtype=i32), 2 ** 32 + 16, 3)
