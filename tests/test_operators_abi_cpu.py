"""The selective scan, its step, the conv step and the group norm on the CPU: argument errors of the C ABI (nothing
is launched) and the bindings' refusals."""
import ctypes
import os

import pytest
import torch

from selective_state_space_cu_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="libssd.so not built")

FAKE = 0x1000   # a non-NULL, 16-byte aligned address that is never dereferenced
NULL, CHUNK, SHAPE, CAPACITY, DTYPE, UNSUPPORTED = 1, 2, 3, 5, 6, 8


def _meta(S=2, T=100, cs=64, max_chunks=None, null_field=None):
    m = ssd._Meta(S, T, cs, T // cs + S if max_chunks is None else max_chunks, *([FAKE] * 7))
    if null_field:
        setattr(m, null_field, None)
    return m


def _scan(m=None, **kw):
    a = dict(u=FAKE, us=64, dt=FAKE, ds=64, bias=None, A=FAKE, B=FAKE, Bs=32, C=FAKE, Cs=32, D=None, z=FAKE, zs=64,
             dtype=1, dtd=1, ch=64, N=16, G=2, init=None, has=None, y=FAKE, ys=64, fin=FAKE, cst=None, dst=None, cap=0)
    assert not set(kw) - set(a)
    a.update(kw)
    m = _meta() if m is None else m
    return ssd.load_library().ssd_selective_scan_varlen(
        a["u"], a["us"], a["dt"], a["ds"], a["bias"], a["A"], a["B"], a["Bs"], a["C"], a["Cs"], a["D"], a["z"], a["zs"],
        a["dtype"], a["dtd"], ctypes.byref(m), a["ch"], a["N"], a["G"], a["init"], a["has"], a["y"], a["ys"], a["fin"],
        a["cst"], a["dst"], a["cap"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(dtd=-1), DTYPE), (dict(ch=0), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE),
    (dict(N=8), UNSUPPORTED), (dict(N=48), UNSUPPORTED), (dict(N=512), UNSUPPORTED), (dict(u=None), NULL),
    (dict(dt=None), NULL), (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(y=None), NULL),
    (dict(fin=None), NULL), (dict(us=63), SHAPE), (dict(ds=0), SHAPE), (dict(ys=-64), SHAPE), (dict(Bs=31), SHAPE),
    (dict(Cs=16), SHAPE), (dict(zs=1), SHAPE), (dict(us=2 ** 26 + 1), SHAPE), (dict(u=FAKE + 1), SHAPE),
    (dict(dtype=0, u=FAKE + 2), SHAPE), (dict(dtd=0, dt=FAKE + 2), SHAPE), (dict(A=FAKE + 4), SHAPE),
    (dict(init=FAKE + 8), SHAPE), (dict(fin=FAKE + 8), SHAPE), (dict(D=FAKE + 2), SHAPE), (dict(bias=FAKE + 1), SHAPE),
    (dict(cst=FAKE, cap=0), CAPACITY), (dict(cst=FAKE, cap=2), CAPACITY), (dict(cst=FAKE + 4, cap=9), SHAPE),
])
def test_scan_rejects_bad_arguments(kw, code):
    assert _scan(**kw) == code


def test_scan_rejects_bad_meta_and_takes_an_empty_batch():
    assert _scan(m=_meta(null_field="seq_order")) == NULL
    assert _scan(m=_meta(cs=48)) == CHUNK
    assert _scan(m=_meta(max_chunks=1)) == CAPACITY
    assert _scan(m=_meta(T=2 ** 30 + 1, max_chunks=2 ** 30)) == SHAPE
    none = dict(u=None, dt=None, B=None, C=None, y=None, z=None, fin=None)
    assert _scan(m=_meta(S=0, T=0, max_chunks=0), **none) == 0


def _step(**kw):
    a = dict(u=FAKE, us=64, dt=FAKE, ds=64, bias=None, A=FAKE, B=FAKE, Bs=32, C=FAKE, Cs=32, D=None, z=None, zs=0,
             dtype=1, dtd=0, S=3, ch=64, N=16, G=2, cache=FAKE, slots=8, rs=FAKE, ws=FAKE, y=FAKE, ys=64)
    assert not set(kw) - set(a)
    a.update(kw)
    return ssd.load_library().ssd_selective_step(
        a["u"], a["us"], a["dt"], a["ds"], a["bias"], a["A"], a["B"], a["Bs"], a["C"], a["Cs"], a["D"], a["z"], a["zs"],
        a["dtype"], a["dtd"], a["S"], a["ch"], a["N"], a["G"], a["cache"], a["slots"], a["rs"], a["ws"], a["y"], a["ys"],
        None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), DTYPE), (dict(S=-1), SHAPE), (dict(slots=-1), SHAPE), (dict(N=24), UNSUPPORTED), (dict(G=5), SHAPE),
    (dict(cache=None), NULL), (dict(rs=None), NULL), (dict(ws=None), NULL), (dict(u=None), NULL), (dict(A=None), NULL),
    (dict(cache=FAKE + 4), SHAPE), (dict(us=10), SHAPE), (dict(z=FAKE, zs=3), SHAPE), (dict(dt=FAKE + 2), SHAPE),
])
def test_step_rejects_bad_arguments(kw, code):
    assert _step(**kw) == code


def test_step_of_no_sequences_launches_nothing():
    assert _step(S=0, u=None, dt=None, B=None, C=None, y=None, cache=None, rs=None, ws=None) == 0


def _conv(**kw):
    a = dict(x=FAKE, xs=64, w=FAKE, bias=None, dtype=1, S=3, C=64, W=4, act=1, states=FAKE, slots=8, rs=FAKE, ws=FAKE,
             out=FAKE, os=64)
    assert not set(kw) - set(a)
    a.update(kw)
    return ssd.load_library().ssd_causal_conv1d_step(
        a["x"], a["xs"], a["w"], a["bias"], a["dtype"], a["S"], a["C"], a["W"], a["act"], a["states"], a["slots"],
        a["rs"], a["ws"], a["out"], a["os"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=4), DTYPE), (dict(S=-2), SHAPE), (dict(C=0), SHAPE), (dict(C=12), UNSUPPORTED), (dict(W=0), UNSUPPORTED),
    (dict(W=5), UNSUPPORTED), (dict(act=3), UNSUPPORTED), (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(states=None), NULL), (dict(xs=56), SHAPE), (dict(xs=68), SHAPE), (dict(os=65), SHAPE), (dict(x=FAKE + 8), SHAPE),
    (dict(out=FAKE + 2), SHAPE), (dict(states=FAKE + 4), SHAPE), (dict(w=FAKE + 2), SHAPE), (dict(slots=-1), SHAPE),
])
def test_conv_step_rejects_bad_arguments(kw, code):
    assert _conv(**kw) == code


def test_conv_step_of_no_sequences_launches_nothing():
    assert _conv(S=0, x=None, out=None, states=None, rs=None, ws=None) == 0


def _norm(**kw):
    a = dict(x=FAKE, xs=96, z=FAKE, zs=96, w=FAKE, b=None, dtype=1, rows=5, C=96, G=3, eps=1e-5, center=1, act=2, out=FAKE,
             os=96)
    assert not set(kw) - set(a)
    a.update(kw)
    return ssd.load_library().ssd_group_norm(a["x"], a["xs"], a["z"], a["zs"], a["w"], a["b"], a["dtype"], a["rows"], a["C"],
                                             a["G"], a["eps"], a["center"], a["act"], a["out"], a["os"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(rows=-1), SHAPE), (dict(C=0), SHAPE), (dict(G=5), SHAPE), (dict(G=0), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(act=4), UNSUPPORTED), (dict(act=-1), UNSUPPORTED),
    (dict(x=None), NULL), (dict(z=None), NULL), (dict(act=3, z=None), NULL), (dict(out=None), NULL), (dict(xs=95), SHAPE),
    (dict(zs=90), SHAPE), (dict(os=0), SHAPE), (dict(x=FAKE + 1), SHAPE), (dict(w=FAKE + 2), SHAPE),
    (dict(C=16385, G=1, xs=16385, zs=16385, os=16385), UNSUPPORTED),
])
def test_norm_rejects_bad_arguments(kw, code):
    assert _norm(**kw) == code


def test_norm_of_no_rows_launches_nothing():
    assert _norm(rows=0, x=None, z=None, out=None) == 0


def test_bindings_refuse():
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)   # noqa: E731
    i32 = torch.int32
    meta = ssd.VarlenMeta(2, 10, 16, 3, *([z(1, dt=i32)] * 7))
    good = dict(u=z(10, 32), dt=z(10, 32), A=z(32, 16), B=z(10, 2, 16), C=z(10, 2, 16))

    def scan(meta=meta, kw=None, **over):
        a = {**good, **over}
        return ssd.selective_scan_varlen(a["u"], a["dt"], a["A"], a["B"], a["C"], meta, **(kw or {}))
    for match, over, kw in [
            ("dt must have", dict(dt=z(10, 31)), {}), ("dt must be", dict(dt=z(10, 32, dt=torch.float16)), {}),
            ("A must", dict(A=z(32, 8)), {}), ("A must", dict(A=z(32, 16, dt=torch.bfloat16)), {}),
            ("C must", dict(C=z(10, 2, 8)), {}), ("B must", dict(B=z(9, 2, 16), C=z(9, 2, 16)), {}),
            ("B must", dict(B=z(10, 2, 16, dt=torch.bfloat16)), {}), ("contiguous rows", dict(u=z(32, 10).t()), {}),
            ("contiguous rows", dict(C=z(10, 16, 2).transpose(1, 2)), {}), ("z must", {}, dict(z=z(10, 33))),
            ("dt_bias must", {}, dict(dt_bias=z(31))), ("initial_states must", {}, dict(initial_states=z(1, 32, 16))),
            ("has_initial_state must", {}, dict(has_initial_state=z(3, dt=i32))),
            ("chunk_states must", {}, dict(chunk_states=z(4, 32, 8))),
            ("chunk_state_dst needs", {}, dict(chunk_states=z(4, 32, 16), chunk_state_dst=z(2, dt=i32))),
            ("y must", {}, dict(y=z(10, 32, dt=torch.bfloat16))), ("final_states must", {}, dict(final_states=z(2, 32, 8))),
            ("on a GPU", {}, {})]:
        with pytest.raises(ValueError, match=match):
            scan(kw=kw, **over)
    with pytest.raises(ValueError, match="tokens"):
        scan(meta=ssd.VarlenMeta(2, 11, 16, 3, *([z(1, dt=i32)] * 7)))
    away = torch.zeros(1, dtype=i32, device="meta")
    with pytest.raises(ValueError, match="metadata must be on"):
        scan(meta=ssd.VarlenMeta(2, 10, 16, 3, *([away] * 7)))
    step = (z(3, 32), z(3, 32), z(32, 16), z(3, 1, 16), z(3, 1, 16))
    slots = z(3, dt=i32)
    with pytest.raises(ValueError, match="state_cache must"):
        ssd.selective_step(*step, z(6, 32, 8), slots, slots)
    with pytest.raises(ValueError, match="state_cache must"):
        ssd.selective_step(*step, z(6, 32, 16, dt=torch.bfloat16), slots, slots)
    with pytest.raises(ValueError, match="write_slot must"):
        ssd.selective_step(*step, z(6, 32, 16), slots, z(2, dt=i32))
    with pytest.raises(ValueError, match="conv_states must"):
        ssd.causal_conv1d_step(z(3, 32), z(32, 4), z(6, 4, 32), slots, slots)
    with pytest.raises(ValueError, match="weight must"):
        ssd.causal_conv1d_step(z(3, 32), z(24, 4), z(6, 3, 32), slots, slots)
    with pytest.raises(ValueError, match="read_slot must"):
        ssd.causal_conv1d_step(z(3, 32), z(32, 4), z(6, 3, 32), z(4, dt=i32), slots)
    with pytest.raises(ValueError, match="weight must"):
        ssd.group_norm(z(3, 32), 2, weight=z(31))
    with pytest.raises(ValueError, match="act must"):
        ssd.group_norm(z(3, 32), 2, act="gelu")
    with pytest.raises(ValueError, match="gated forms"):
        ssd.group_norm(z(3, 32), 2, z=z(3, 32))
    with pytest.raises(ValueError, match="gated forms"):
        ssd.group_norm(z(3, 32), 2, act="gate_last")
    with pytest.raises(ValueError, match="out must"):
        ssd.group_norm(z(3, 32), 2, out=z(3, 31))
    for groups in (0, -1, 33, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="ngroups must"):
            ssd.group_norm(z(3, 32), groups)
    with pytest.raises(ValueError, match="more than"):
        ssd.group_norm(torch.empty(2 ** 31, 1, dtype=torch.bfloat16, device="meta"), 1)
