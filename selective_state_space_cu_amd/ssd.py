"""Thin ctypes binding of libssd.so (declared in include/ssd.h).

Argument marshalling only: torch tensors provide device memory and the current
HIP stream; every step of the scan runs in the library's HIP kernels. There is
no fallback: if libssd.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
NORM_ACTS = {"none": 0, "silu": 1, "gate_first": 2, "gate_last": 3}   # ssd_norm_act
DATA_BAD_CU_SEQLENS, DATA_TOO_MANY_CHUNKS, DATA_BAD_SLOT, DATA_BAD_BLOCK, DATA_NO_BLOCK = 1, 2, 4, 8, 16

# names exported by libssd.so (checked by the CPU tests against include/ssd.h)
EXPORTS = ("ssd_varlen_metadata", "ssd_chunk_scan_varlen", "ssd_export_chunk_states",
           "ssd_decode_step", "ssd_causal_conv1d_varlen", "ssd_gated_delta_chunk_varlen", "ssd_gated_delta_workspace_size",
           "ssd_gated_delta_chunk_varlen_noalloc",
           "ssd_prefill_bites",
           "ssd_selective_scan_varlen", "ssd_selective_step", "ssd_causal_conv1d_step", "ssd_group_norm",
           "ssd_gated_delta_step", "ssd_step_tables", "ssd_kv_cache_write", "ssd_attention_plan_build",
           "ssd_paged_attention_step", "ssd_paged_attention_parts", "ssd_paged_attention_workspace_size",
           "ssd_add_rms_norm", "ssd_add_rms_norm_e4m3",
           "ssd_status_string")


class SSDError(RuntimeError):
    """A libssd call returned a non-zero ssd_status."""

    def __init__(self, fn, status, text):
        super().__init__(f"{fn} failed: status {status} ({text})")
        self.status = status


class _Meta(ctypes.Structure):
    _fields_ = [("nseqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("chunk_size", ctypes.c_int32), ("max_chunks", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("chunk_offsets", ctypes.c_void_p),
                ("chunk_seq_idx", ctypes.c_void_p), ("seq_chunk_start", ctypes.c_void_p),
                ("nchunks", ctypes.c_void_p), ("seq_order", ctypes.c_void_p),
                ("error_flag", ctypes.c_void_p)]


class _Plan(ctypes.Structure):
    _fields_ = [("nseqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32), ("max_new_tokens", ctypes.c_int32),
                ("window", ctypes.c_int32), ("max_parts", ctypes.c_int32), ("seq_lens", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("part_start", ctypes.c_void_p), ("part_seq", ctypes.c_void_p),
                ("part_keys", ctypes.c_void_p), ("error_flag", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libssd.so (once). Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libssd.so not found at {path}: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [st]
    lib.ssd_varlen_metadata.restype = st
    lib.ssd_varlen_metadata.argtypes = [ctypes.POINTER(_Meta), vp]
    lib.ssd_chunk_scan_varlen.restype = st
    lib.ssd_chunk_scan_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, st, ctypes.POINTER(_Meta),
                                          i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp]
    lib.ssd_export_chunk_states.restype = st
    lib.ssd_export_chunk_states.argtypes = [ctypes.POINTER(_Meta), vp, vp, i32, i32, vp, vp, vp,
                                            i32, vp, i32, vp]
    lib.ssd_decode_step.restype = st
    lib.ssd_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, st, i32, i32, i32, i32, i32, vp, i32,
                                    vp, vp, vp, vp, vp]
    lib.ssd_causal_conv1d_varlen.restype = st
    lib.ssd_causal_conv1d_varlen.argtypes = [vp, vp, vp, st, ctypes.POINTER(_Meta), i32, i32, i32, vp, i32,
                                             vp, vp, vp, vp]
    lib.ssd_gated_delta_chunk_varlen.restype = st
    lib.ssd_gated_delta_chunk_varlen.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, st, ctypes.POINTER(_Meta),
                                                 i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp,
                                                 ctypes.c_size_t, vp]
    lib.ssd_gated_delta_chunk_varlen_noalloc.restype = st
    lib.ssd_gated_delta_chunk_varlen_noalloc.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, st,
                                                         ctypes.POINTER(_Meta), i32, i32, i32, i32, vp, vp, vp, vp,
                                                         vp, vp, i32, vp]
    lib.ssd_gated_delta_workspace_size.restype = ctypes.c_size_t
    lib.ssd_gated_delta_workspace_size.argtypes = [i32, i32]
    i64 = ctypes.c_int64
    lib.ssd_selective_scan_varlen.restype = st
    lib.ssd_selective_scan_varlen.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64, st, st,
                                              ctypes.POINTER(_Meta), i32, i32, i32, vp, vp, vp, i64, vp, vp, vp,
                                              i32, vp]
    lib.ssd_selective_step.restype = st
    lib.ssd_selective_step.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64, st, st, i32, i32,
                                       i32, i32, vp, i32, vp, vp, vp, i64, vp, vp]
    lib.ssd_causal_conv1d_step.restype = st
    lib.ssd_causal_conv1d_step.argtypes = [vp, i64, vp, vp, st, i32, i32, i32, i32, vp, i32, vp, vp, vp, i64, vp, vp]
    lib.ssd_group_norm.restype = st
    lib.ssd_group_norm.argtypes = [vp, i64, vp, i64, vp, vp, st, i32, i32, i32, ctypes.c_float, i32, st, vp, i64, vp]
    f32, size = ctypes.c_float, ctypes.c_size_t
    lib.ssd_gated_delta_step.restype = st
    lib.ssd_gated_delta_step.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32, f32, st, st, i32, i32,
                                         vp, i32, i32, i32, i32, vp, i32, vp, vp, vp, i64, vp, vp]
    lib.ssd_step_tables.restype = st
    lib.ssd_step_tables.argtypes = [i32, i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                    vp, vp, vp]
    lib.ssd_kv_cache_write.restype = st
    lib.ssd_kv_cache_write.argtypes = [vp, i64, vp, i64, st, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp]
    lib.ssd_attention_plan_build.restype = st
    lib.ssd_attention_plan_build.argtypes = [ctypes.POINTER(_Plan), vp]
    lib.ssd_paged_attention_step.restype = st
    lib.ssd_paged_attention_step.argtypes = [vp, i64, vp, vp, st, f32, ctypes.POINTER(_Plan), i32, i32, i32, vp, i32,
                                             i32, vp, i32, i32, vp, i64, vp, vp, size, vp, vp]
    lib.ssd_paged_attention_parts.restype = i32
    lib.ssd_paged_attention_parts.argtypes = [i32, i32, i32]
    lib.ssd_paged_attention_workspace_size.restype = size
    lib.ssd_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.ssd_add_rms_norm.restype = st
    lib.ssd_add_rms_norm.argtypes = [vp, i64, vp, i64, vp, st, i32, i32, f32, vp, i64, vp, i64, vp]
    lib.ssd_add_rms_norm_e4m3.restype = st
    lib.ssd_add_rms_norm_e4m3.argtypes = [vp, i64, vp, i64, vp, st, i32, i32, i32, f32, vp, vp, vp, i64, vp, i64, vp]
    lib.ssd_prefill_bites.restype = st
    lib.ssd_prefill_bites.argtypes = [i32, vp, vp, vp, i32, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().ssd_status_string(status).decode()


def _check(fn, status):
    if status != 0:
        raise SSDError(fn, status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _data(t: torch.Tensor, name: str, device, dtype=None):
    """Data tensors must already be contiguous and on the device (no hidden copies)."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _shape(t: Optional[torch.Tensor], name: str, *shape):
    """The kernels index every buffer from the sizes passed beside it: a tensor of
    another shape would be read or written out of its bounds, so refuse it here."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dst_len(dst: Optional[torch.Tensor], meta):
    """The kernels read one checkpoint slot per chunk of the batch's chunk grid."""
    if dst is not None and dst.numel() < meta.max_chunks:
        raise ValueError(f"chunk_state_dst needs {meta.max_chunks} entries (one per chunk), got {dst.numel()}")


def _index(t: torch.Tensor, device):
    """Index arrays are normalised to contiguous int32 on the device."""
    t = t.to(device=device, dtype=torch.int32)
    return t if t.stride(-1) == 1 and t.is_contiguous() else t.contiguous()


@dataclasses.dataclass
class VarlenMeta:
    """Device-resident chunk metadata of one packed batch (see ssd_varlen_meta)."""
    nseqs: int
    total_tokens: int
    chunk_size: int
    max_chunks: int
    cu_seqlens: torch.Tensor
    chunk_offsets: torch.Tensor
    chunk_seq_idx: torch.Tensor
    seq_chunk_start: torch.Tensor
    nchunks: torch.Tensor
    seq_order: torch.Tensor
    error_flag: torch.Tensor

    def c_struct(self) -> _Meta:
        return _Meta(self.nseqs, self.total_tokens, self.chunk_size, self.max_chunks,
                     *(t.data_ptr() for t in (self.cu_seqlens, self.chunk_offsets,
                                              self.chunk_seq_idx, self.seq_chunk_start,
                                              self.nchunks, self.seq_order, self.error_flag)))


def varlen_metadata(cu_seqlens: torch.Tensor, chunk_size: int, total_tokens: Optional[int] = None,
                    max_chunks: Optional[int] = None, device=None) -> VarlenMeta:
    """ssd_varlen_metadata: build the chunk grid on the device (no host sync).

    `total_tokens` defaults to cu_seqlens[-1] (read on the host if cu_seqlens is a
    CPU tensor; pass it explicitly for device-resident cu_seqlens)."""
    lib = load_library()
    device = torch.device(device) if device is not None else (
        cu_seqlens.device if cu_seqlens.is_cuda else torch.device("cuda", torch.cuda.current_device()))
    S = cu_seqlens.numel() - 1
    if total_tokens is None:
        if cu_seqlens.is_cuda:
            raise ValueError("pass total_tokens when cu_seqlens lives on the device")
        total_tokens = int(cu_seqlens[-1])
    if max_chunks is None:
        max_chunks = total_tokens // chunk_size + S
    cu = _index(cu_seqlens, device)
    i32 = dict(dtype=torch.int32, device=device)
    meta = VarlenMeta(S, int(total_tokens), int(chunk_size), int(max_chunks), cu,
                      torch.empty(max_chunks + 1, **i32), torch.empty(max(max_chunks, 1), **i32),
                      torch.empty(S + 1, **i32), torch.empty(1, **i32),
                      torch.empty(max(S, 1), **i32), torch.zeros(1, **i32))
    c = meta.c_struct()
    _check("ssd_varlen_metadata", lib.ssd_varlen_metadata(ctypes.byref(c), _stream(device)))
    return meta


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise ValueError(f"x/B/C must be float32 or bfloat16, got {t.dtype}")


def chunk_scan_varlen(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                      C: torch.Tensor, meta: VarlenMeta, dt_bias: Optional[torch.Tensor] = None,
                      D: Optional[torch.Tensor] = None,
                      initial_states: Optional[torch.Tensor] = None,
                      has_initial_state: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None,
                      final_states: Optional[torch.Tensor] = None,
                      chunk_states: Optional[torch.Tensor] = None,
                      chunk_state_dst: Optional[torch.Tensor] = None):
    """ssd_chunk_scan_varlen. x (T,H,P), dt (T,H), A (H,), B/C (T,G,N).

    Returns (y, final_states). `chunk_states` (float32 [slots,H,P,N]) receives the
    state after each chunk, at index c or at chunk_state_dst[c] when given."""
    lib = load_library()
    device = x.device
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    S = meta.nseqs
    _data(x, "x", device)
    if T != meta.total_tokens:
        raise ValueError(f"x has {T} tokens, the metadata {meta.total_tokens}")
    for name, t, shp in (("B", B, (T, G, N)), ("C", C, (T, G, N)), ("dt", dt, (T, H)), ("A", A, (H,)),
                         ("dt_bias", dt_bias, (H,)), ("D", D, (H,)),
                         ("initial_states", initial_states, (S, H, P, N)), ("y", y, (T, H, P)),
                         ("final_states", final_states, (S, H, P, N))):
        _shape(t, name, *shp)
    if has_initial_state is not None:
        _shape(has_initial_state, "has_initial_state", S)
    if chunk_states is not None:
        _shape(chunk_states, "chunk_states", chunk_states.shape[0], H, P, N)
    _dst_len(chunk_state_dst, meta)
    dtype = x.dtype
    for name, t in (("B", B), ("C", C)):
        _data(t, name, device, dtype)
    _data(dt, "dt", device, torch.float32)
    _data(A, "A", device, torch.float32)
    for name, t in (("dt_bias", dt_bias), ("D", D), ("initial_states", initial_states)):
        if t is not None:
            _data(t, name, device, torch.float32)
    if y is None:
        y = torch.empty_like(x)
    _data(y, "y", device, dtype)
    if final_states is None:
        final_states = torch.empty((S, H, P, N), dtype=torch.float32, device=device)
    _data(final_states, "final_states", device, torch.float32)
    has = _index(has_initial_state, device) if has_initial_state is not None else None
    dst = _index(chunk_state_dst, device) if chunk_state_dst is not None else None
    cap = 0
    if chunk_states is not None:
        _data(chunk_states, "chunk_states", device, torch.float32)
        cap = chunk_states.shape[0]
    m = meta.c_struct()
    _check("ssd_chunk_scan_varlen", lib.ssd_chunk_scan_varlen(
        _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _dtype_code(x),
        ctypes.byref(m), H, P, N, G, _ptr(initial_states), _ptr(has), _ptr(y),
        _ptr(final_states), _ptr(chunk_states), _ptr(dst), cap, _stream(device)))
    return y, final_states


def export_chunk_states(meta: VarlenMeta, block_table: torch.Tensor, block_size: int,
                        num_computed_tokens: Optional[torch.Tensor] = None,
                        chunk_states: Optional[torch.Tensor] = None,
                        state_cache: Optional[torch.Tensor] = None,
                        num_slots: Optional[int] = None):
    """ssd_export_chunk_states: block-checkpoint plan (and scatter when chunk_states
    is given). Returns (ckpt_src [S, max_blocks], chunk_state_dst [max_chunks])."""
    lib = load_library()
    device = meta.cu_seqlens.device
    bt = _index(block_table, device)
    S, maxb = bt.shape if bt.dim() == 2 else (meta.nseqs, 0)
    ncomp = _index(num_computed_tokens, device) if num_computed_tokens is not None else None
    ckpt_src = torch.empty((S, maxb), dtype=torch.int32, device=device)
    dst = torch.empty(max(meta.max_chunks, 1), dtype=torch.int32, device=device)
    state_elems = 0
    if state_cache is not None:
        _data(state_cache, "state_cache", device, torch.float32)
        state_elems = state_cache[0].numel() if state_cache.shape[0] else 0
        if num_slots is None:
            num_slots = state_cache.shape[0]
    if chunk_states is not None:
        _data(chunk_states, "chunk_states", device, torch.float32)
    m = meta.c_struct()
    _check("ssd_export_chunk_states", lib.ssd_export_chunk_states(
        ctypes.byref(m), _ptr(ncomp), _ptr(bt), maxb, int(block_size), _ptr(ckpt_src), _ptr(dst),
        _ptr(chunk_states), state_elems, _ptr(state_cache), int(num_slots or 0), _stream(device)))
    return ckpt_src, dst[: meta.max_chunks]


def gated_delta_chunk_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor,
                             beta: torch.Tensor, meta: VarlenMeta, scale: Optional[float] = None,
                             initial_states: Optional[torch.Tensor] = None,
                             has_initial_state: Optional[torch.Tensor] = None,
                             o: Optional[torch.Tensor] = None, final_states: Optional[torch.Tensor] = None,
                             chunk_states: Optional[torch.Tensor] = None,
                             chunk_state_dst: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, no_alloc: bool = False):
    """ssd_gated_delta_chunk_varlen: q, k (T,G,dk), v (T,H,dv) bf16; gate, beta (T,H) float32;
    states (S,H,dv,dk) float32. `workspace` (uint8 on the device, at least
    gated_delta_workspace_size(meta, H) bytes) is allocated per call when not
    given. no_alloc=True calls ssd_gated_delta_chunk_varlen_noalloc instead (the
    library's static workspace; pass o and final_states too for a call that
    allocates nothing).
    Returns (o, final_states)."""
    lib = load_library()
    device = v.device
    T, H, DV = v.shape
    G, DK = k.shape[1], k.shape[2]
    S = meta.nseqs
    for name, t, shp in (("q", q, (T, G, DK)), ("k", k, (T, G, DK)), ("gate", gate, (T, H)), ("beta", beta, (T, H)),
                         ("o", o, (T, H, DV)), ("initial_states", initial_states, (S, H, DV, DK)),
                         ("final_states", final_states, (S, H, DV, DK)), ("has_initial_state", has_initial_state, (S,))):
        _shape(t, name, *shp)
    if chunk_states is not None:
        _shape(chunk_states, "chunk_states", chunk_states.shape[0], H, DV, DK)
    _dst_len(chunk_state_dst, meta)
    if T != meta.total_tokens:
        raise ValueError(f"v has {T} tokens, the metadata {meta.total_tokens}")
    dtype = v.dtype
    _data(v, "v", device)
    for name, t in (("q", q), ("k", k)):
        _data(t, name, device, dtype)
    for name, t in (("gate", gate), ("beta", beta)):
        _data(t, name, device, torch.float32)
    if o is None:
        o = torch.empty_like(v)
    _data(o, "o", device, dtype)
    if final_states is None:
        final_states = torch.empty((S, H, DV, DK), dtype=torch.float32, device=device)
    _data(final_states, "final_states", device, torch.float32)
    if initial_states is not None:
        _data(initial_states, "initial_states", device, torch.float32)
    has = _index(has_initial_state, device) if has_initial_state is not None else None
    cap = 0
    if chunk_states is not None:
        _data(chunk_states, "chunk_states", device, torch.float32)
        cap = chunk_states.shape[0]
    dst = _index(chunk_state_dst, device) if chunk_state_dst is not None else None
    if no_alloc:
        m = meta.c_struct()
        _check("ssd_gated_delta_chunk_varlen_noalloc", lib.ssd_gated_delta_chunk_varlen_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), float(scale if scale is not None else DK ** -0.5),
            _dtype_code(v), ctypes.byref(m), H, G, DK, DV, _ptr(initial_states), _ptr(has), _ptr(o),
            _ptr(final_states), _ptr(chunk_states), _ptr(dst), cap, _stream(device)))
        return o, final_states
    ws_bytes = gated_delta_workspace_size(meta, H)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=device)
    _data(workspace, "workspace", device, torch.uint8)
    m = meta.c_struct()
    _check("ssd_gated_delta_chunk_varlen", lib.ssd_gated_delta_chunk_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), float(scale if scale is not None else DK ** -0.5),
        _dtype_code(v), ctypes.byref(m), H, G, DK, DV, _ptr(initial_states), _ptr(has), _ptr(o), _ptr(final_states),
        _ptr(chunk_states), _ptr(dst), cap, _ptr(workspace), workspace.numel(), _stream(device)))
    return o, final_states


def gated_delta_workspace_size(meta: VarlenMeta, nheads: int) -> int:
    """Bytes of device workspace ssd_gated_delta_chunk_varlen needs for this batch."""
    return int(load_library().ssd_gated_delta_workspace_size(meta.max_chunks, int(nheads)))


def prefill_bites(num_computed_tokens, prompt_len, budget, align: int):
    """ssd_prefill_bites (host): tokens each prefilling sequence gets this step.
    Arguments are host sequences, arrays or CPU tensors of nseqs entries (budget may
    be a single int); returns a host int32 tensor of nseqs entries."""
    lib = load_library()
    nc = torch.as_tensor(num_computed_tokens, dtype=torch.int32).reshape(-1).contiguous()
    pl = torch.as_tensor(prompt_len, dtype=torch.int32).reshape(-1).contiguous()
    bu = torch.as_tensor(budget, dtype=torch.int32).reshape(-1).expand(nc.numel()).contiguous()
    if pl.numel() != nc.numel():
        raise ValueError("prompt_len and num_computed_tokens differ in length")
    out = torch.empty_like(nc)
    _check("ssd_prefill_bites", lib.ssd_prefill_bites(nc.numel(), nc.data_ptr(), pl.data_ptr(), bu.data_ptr(),
                                                     int(align), out.data_ptr()))
    return out


def decode_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                C: torch.Tensor, state_cache: torch.Tensor, read_slot: torch.Tensor,
                write_slot: torch.Tensor, dt_bias: Optional[torch.Tensor] = None,
                D: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                error_flag: Optional[torch.Tensor] = None):
    """ssd_decode_step: one token per sequence, state read from
    state_cache[read_slot[s]] (zero if < 0) and written to
    state_cache[write_slot[s]] (skipped if < 0). x (S,H,P), dt (S,H), A (H,),
    B/C (S,G,N), state_cache float32 (slots,H,P,N). Returns y (S,H,P)."""
    lib = load_library()
    device = x.device
    S, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    _data(x, "x", device)
    for name, t, shp in (("B", B, (S, G, N)), ("C", C, (S, G, N)), ("dt", dt, (S, H)), ("A", A, (H,)),
                         ("dt_bias", dt_bias, (H,)), ("D", D, (H,)), ("y", y, (S, H, P)),
                         ("state_cache", state_cache, (state_cache.shape[0], H, P, N)),
                         ("read_slot", read_slot, (S,)), ("write_slot", write_slot, (S,))):
        _shape(t, name, *shp)
    dtype = x.dtype
    for name, t in (("B", B), ("C", C)):
        _data(t, name, device, dtype)
    _data(dt, "dt", device, torch.float32)
    _data(A, "A", device, torch.float32)
    _data(state_cache, "state_cache", device, torch.float32)
    for name, t in (("dt_bias", dt_bias), ("D", D)):
        if t is not None:
            _data(t, name, device, torch.float32)
    if y is None:
        y = torch.empty_like(x)
    _data(y, "y", device, dtype)
    rs, ws = _index(read_slot, device), _index(write_slot, device)
    if error_flag is not None:
        _data(error_flag, "error_flag", device, torch.int32)
    _check("ssd_decode_step", lib.ssd_decode_step(
        _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _dtype_code(x),
        S, H, P, N, G, _ptr(state_cache), state_cache.shape[0], _ptr(rs), _ptr(ws), _ptr(y),
        _ptr(error_flag), _stream(device)))
    return y


def causal_conv1d_varlen(x: torch.Tensor, weight: torch.Tensor, meta: VarlenMeta,
                         bias: Optional[torch.Tensor] = None, silu: bool = True,
                         conv_states: Optional[torch.Tensor] = None,
                         read_slot: Optional[torch.Tensor] = None,
                         write_slot: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None):
    """ssd_causal_conv1d_varlen: depthwise causal conv1d of x (T, C) with
    weight (C, W) float32 over the chunk grid of `meta`; the W-1 inputs before
    each sequence come from conv_states[read_slot[s]] (zero if < 0) and its last
    W-1 inputs go to conv_states[write_slot[s]] (skipped if < 0); conv_states
    (slots, W-1, C) has x's dtype. Returns out (T, C)."""
    lib = load_library()
    device = x.device
    _data(x, "x", device)
    T, C = x.shape
    W = weight.shape[1]
    if T != meta.total_tokens:
        raise ValueError(f"x has {T} tokens, the metadata {meta.total_tokens}")
    S = meta.nseqs
    for name, t, shp in (("weight", weight, (C, W)), ("bias", bias, (C,)), ("out", out, (T, C)),
                         ("read_slot", read_slot, (S,)), ("write_slot", write_slot, (S,))):
        _shape(t, name, *shp)
    if conv_states is not None:
        _shape(conv_states, "conv_states", conv_states.shape[0], W - 1, C)
    _data(weight, "weight", device, torch.float32)
    if bias is not None:
        _data(bias, "bias", device, torch.float32)
    if conv_states is not None:
        _data(conv_states, "conv_states", device, x.dtype)
    if out is None:
        out = torch.empty_like(x)
    _data(out, "out", device, x.dtype)
    rs = _index(read_slot, device) if read_slot is not None else None
    ws = _index(write_slot, device) if write_slot is not None else None
    m = meta.c_struct()
    _check("ssd_causal_conv1d_varlen", lib.ssd_causal_conv1d_varlen(
        _ptr(x), _ptr(weight), _ptr(bias), _dtype_code(x), ctypes.byref(m), C, W, int(bool(silu)),
        _ptr(conv_states), 0 if conv_states is None else conv_states.shape[0], _ptr(rs), _ptr(ws),
        _ptr(out), _stream(device)))
    return out


def _enqueue(fn, device, *args):
    """Call the library's `fn` on the current stream of `device`, with that device current."""
    if device.type != "cuda":
        raise ValueError(f"{fn} needs tensors on a GPU, got {device}")
    f = getattr(_lib or load_library(), fn)
    if device.index == torch.cuda.current_device():
        status = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            status = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status != 0:
        raise SSDError(fn, status, status_string(status))


def _refuse(t: torch.Tensor, name: str, device, dtype, shape):
    """Says what is wrong with a tensor that is not as it has to be."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous, or where rows may lie apart have contiguous rows; got strides "
                     f"{t.stride()}")


def _whole(t: Optional[torch.Tensor], name: str, device, dtype, shape):
    """Checks a contiguous tensor; returns its address (None for None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        _refuse(t, name, device, dtype, shape)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, device, dtype, shape, row: int) -> int:
    """Checks a tensor of `shape` (rows first, `row` elements each) whose rows are contiguous but may lie any distance
    apart, as a slice of a wider projection has them. Returns the elements from one row to the next."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(t, name, device, dtype, shape)
    if shape[0] > 0x7fffffff:
        raise ValueError(f"{name} has {shape[0]} rows, more than 2^31 - 1")
    if t.is_contiguous():
        return row
    stride = t.stride()
    if stride[-1] == 1 and shape[0] > 1 and (len(shape) == 2 or len(shape) == 3 and stride[1] == shape[2]):
        return stride[0]
    step = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != step:
            _refuse(t, name, device, dtype, shape)
        step *= size
    return t.stride(0) if shape[0] > 1 else row


def _out_rows(out: Optional[torch.Tensor], name: str, like: torch.Tensor, row: int):
    """The output and the elements between its rows: `out` if given, else a new contiguous one."""
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format), row
    return out, _rows(out, name, like.device, like.dtype, like.shape, row)


def _selective_inputs(u, dt, A, B, C, dt_bias, D, z):
    """Checks what the selective scan and its step share; returns the library's leading arguments and sizes."""
    if u.dim() != 2 or B.dim() != 3:
        raise ValueError(f"u must be (rows, channels) and B (rows, groups, states), got {tuple(u.shape)} and "
                         f"{tuple(B.shape)}")
    device, dtype, shape, bshape = u.device, u.dtype, u.shape, B.shape
    rows, channels = shape
    brows, groups, n = bshape
    code = _dtype_code(u)
    if dt.dtype != dtype and dt.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dt must be float32 or bfloat16, got {dt.dtype}")
    if brows != rows:
        raise ValueError(f"B must have {rows} rows, got {brows}")
    return (u.data_ptr(), _rows(u, "u", device, dtype, shape, channels),
            dt.data_ptr(), _rows(dt, "dt", device, dt.dtype, shape, channels),
            _whole(dt_bias, "dt_bias", device, torch.float32, (channels,)),
            _whole(A, "A", device, torch.float32, (channels, n)),
            B.data_ptr(), _rows(B, "B", device, dtype, bshape, groups * n),
            C.data_ptr(), _rows(C, "C", device, dtype, bshape, groups * n),
            _whole(D, "D", device, torch.float32, (channels,)),
            None if z is None else z.data_ptr(), 0 if z is None else _rows(z, "z", device, dtype, shape, channels),
            code, code if dt.dtype == dtype else _dtype_code(dt)), channels, n, groups


def _slots(t: torch.Tensor, name: str, device, nseqs: int):
    """A slot array as contiguous int32 on the device."""
    if t.shape != (nseqs,):
        raise ValueError(f"{name} must have shape {(nseqs,)}, got {tuple(t.shape)}")
    if t.dtype == torch.int32 and t.device == device and t.is_contiguous():
        return t
    return _index(t, device)


def selective_scan_varlen(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                          meta: VarlenMeta, dt_bias: Optional[torch.Tensor] = None,
                          D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                          initial_states: Optional[torch.Tensor] = None,
                          has_initial_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                          final_states: Optional[torch.Tensor] = None, chunk_states: Optional[torch.Tensor] = None,
                          chunk_state_dst: Optional[torch.Tensor] = None):
    """ssd_selective_scan_varlen: the scan with a decay per channel and state. u, dt, z (T, D) and B, C (T, G, N)
    may be slices with rows further apart; A (D, N), dt_bias, D (D,) and the states (S, D, N) are float32.
    `chunk_states` (float32 [slots, D, N]) receives the state after each chunk, at index c or at
    chunk_state_dst[c] when given. Float32 roundings of a sequence's results may differ with the batch around it.
    Returns (y, final_states)."""
    head, channels, n, groups = _selective_inputs(u, dt, A, B, C, dt_bias, D, z)
    device, f32 = u.device, torch.float32
    if u.shape[0] != meta.total_tokens:
        raise ValueError(f"u has {u.shape[0]} tokens, the metadata {meta.total_tokens}")
    if meta.cu_seqlens.device != device:
        raise ValueError(f"the metadata must be on {device}, got {meta.cu_seqlens.device}")
    states = (meta.nseqs, channels, n)
    cap = 0 if chunk_states is None else chunk_states.shape[0]
    init = _whole(initial_states, "initial_states", device, f32, states)
    cst = _whole(chunk_states, "chunk_states", device, f32, (cap, channels, n))
    has = None if has_initial_state is None else _slots(has_initial_state, "has_initial_state", device, meta.nseqs)
    _dst_len(chunk_state_dst, meta)
    dst = None if chunk_state_dst is None else _slots(chunk_state_dst, "chunk_state_dst", device,
                                                      chunk_state_dst.numel())
    y, y_stride = _out_rows(y, "y", u, channels)
    if final_states is None:
        final_states = torch.empty(states, dtype=f32, device=device)
    m = meta.c_struct()
    _enqueue("ssd_selective_scan_varlen", device, *head, ctypes.byref(m), channels, n, groups, init,
             None if has is None else has.data_ptr(), y.data_ptr(), y_stride,
             _whole(final_states, "final_states", device, f32, states), cst,
             None if dst is None else dst.data_ptr(), cap)
    return y, final_states


def selective_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   state_cache: torch.Tensor, read_slot: torch.Tensor, write_slot: torch.Tensor,
                   dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   error_flag: Optional[torch.Tensor] = None):
    """ssd_selective_step: one token per sequence, the state read from state_cache[read_slot[s]] (zero if < 0) and
    written to state_cache[write_slot[s]] (skipped if < 0). u, dt, z (S, D), B, C (S, G, N), state_cache float32
    (slots, D, N). Returns y (S, D)."""
    head, channels, n, groups = _selective_inputs(u, dt, A, B, C, dt_bias, D, z)
    device, nseqs, slots = u.device, u.shape[0], state_cache.shape[0]
    cache = _whole(state_cache, "state_cache", device, torch.float32, (slots, channels, n))
    rs = _slots(read_slot, "read_slot", device, nseqs)
    ws = _slots(write_slot, "write_slot", device, nseqs)
    flag = _whole(error_flag, "error_flag", device, torch.int32, (1,))
    y, y_stride = _out_rows(y, "y", u, channels)
    _enqueue("ssd_selective_step", device, *head, nseqs, channels, n, groups, cache, slots, rs.data_ptr(),
             ws.data_ptr(), y.data_ptr(), y_stride, flag)
    return y


def causal_conv1d_step(x: torch.Tensor, weight: torch.Tensor, conv_states: Optional[torch.Tensor] = None,
                       read_slot: Optional[torch.Tensor] = None, write_slot: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, silu: bool = True, out: Optional[torch.Tensor] = None,
                       error_flag: Optional[torch.Tensor] = None):
    """ssd_causal_conv1d_step: causal_conv1d_varlen for one token per sequence. x (S, C) may be a slice with rows
    further apart; the window of W-1 inputs comes from conv_states[read_slot[s]] (zero if < 0) and goes, shifted by
    x, to conv_states[write_slot[s]] (skipped if < 0). Returns out (S, C)."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"x must be (sequences, channels) and weight (channels, width), got {tuple(x.shape)} and "
                         f"{tuple(weight.shape)}")
    device, dtype, f32 = x.device, x.dtype, torch.float32
    nseqs, channels = x.shape
    width = weight.shape[1]
    slots = 0 if conv_states is None else conv_states.shape[0]
    x_stride = _rows(x, "x", device, dtype, x.shape, channels)
    w = _whole(weight, "weight", device, f32, (channels, width))
    b = _whole(bias, "bias", device, f32, (channels,))
    states = _whole(conv_states, "conv_states", device, dtype, (slots, width - 1, channels))
    rs = None if read_slot is None else _slots(read_slot, "read_slot", device, nseqs)
    ws = None if write_slot is None else _slots(write_slot, "write_slot", device, nseqs)
    flag = _whole(error_flag, "error_flag", device, torch.int32, (1,))
    out, out_stride = _out_rows(out, "out", x, channels)
    _enqueue("ssd_causal_conv1d_step", device, x.data_ptr(), x_stride, w, b, _dtype_code(x), nseqs, channels, width,
             1 if silu else 0, states, slots, None if rs is None else rs.data_ptr(),
             None if ws is None else ws.data_ptr(), out.data_ptr(), out_stride, flag)
    return out


def group_norm(x: torch.Tensor, ngroups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, act: str = "none",
               center: bool = True, eps: float = 1e-5, out: Optional[torch.Tensor] = None):
    """ssd_group_norm: every row of x (rows, C), or of a scan's output (T, H, P) read as T rows of H*P channels, is
    normed in `ngroups` groups of channels (mean and variance, or the mean square alone when `center` is false),
    scaled by weight and bias (C,), with act "none", "silu" (of the result), "gate_first" (norm of x silu(z)) or
    "gate_last" (norm of x, times silu(z)). Rows of x and z may lie further apart. Returns out, shaped like x."""
    if x.dim() < 2:
        raise ValueError(f"x must have rows and channels, got {tuple(x.shape)}")
    if act not in NORM_ACTS:
        raise ValueError(f"act must be one of {sorted(NORM_ACTS)}, got {act!r}")
    if (z is not None) != act.startswith("gate"):
        raise ValueError("z is given exactly with the gated forms")
    device, dtype, shape, f32 = x.device, x.dtype, x.shape, torch.float32
    channels = shape[1] if len(shape) == 2 else shape[1:].numel()
    if not 0 < ngroups <= channels:
        raise ValueError(f"ngroups must be between 1 and the {channels} channels, got {ngroups}")
    x_stride = _rows(x, "x", device, dtype, shape, channels)
    z_stride = 0 if z is None else _rows(z, "z", device, dtype, shape, channels)
    w = _whole(weight, "weight", device, f32, (channels,))
    b = _whole(bias, "bias", device, f32, (channels,))
    out, out_stride = _out_rows(out, "out", x, channels)
    _enqueue("ssd_group_norm", device, x.data_ptr(), x_stride, None if z is None else z.data_ptr(), z_stride, w, b,
             _dtype_code(x), shape[0], channels, int(ngroups), float(eps), 1 if center else 0, NORM_ACTS[act],
             out.data_ptr(), out_stride)
    return out


def gated_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor, beta: torch.Tensor,
                     state_cache: torch.Tensor, read_slot: torch.Tensor, write_slot: torch.Tensor,
                     cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     A: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                     qk_eps: Optional[float] = None, o: Optional[torch.Tensor] = None,
                     error_flag: Optional[torch.Tensor] = None):
    """ssd_gated_delta_step: the gated delta rule for the new tokens of every sequence (one each, or cu_seqlens). The
    state is read from state_cache[read_slot[s]] (zero if < 0); after token t it is written to
    state_cache[write_slot[t]] (skipped if < 0). q, k (T, G, dk), v (T, H, dv), gate, beta (T, H) (float32 or bf16) may be
    slices with rows further apart; state_cache float32 (slots, H, dv, dk), read_slot (S,), write_slot (T,). With A (H,),
    gate and beta are raw: the log-decay is A softplus(gate + dt_bias) and the strength sigmoid(beta). With qk_eps, q and
    k are divided by sqrt(|.|^2 + qk_eps). scale: dk ** -0.5 unless given. Returns o (T, H, dv)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q must be (tokens, key heads, dk) and v (tokens, heads, dv), got {tuple(q.shape)} and "
                         f"{tuple(v.shape)}")
    device, dtype, vshape, qshape = v.device, v.dtype, v.shape, q.shape
    tokens, heads, dv = vshape
    qtokens, kheads, dk = qshape
    if qtokens != tokens:
        raise ValueError(f"q must have {tokens} tokens, got {qtokens}")
    code = _dtype_code(v)
    if gate.dtype != dtype and gate.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"gate must be float32 or bfloat16, got {gate.dtype}")
    if A is None and dt_bias is not None:
        raise ValueError("dt_bias is given only with A")
    if qk_eps is not None and not qk_eps >= 0:
        raise ValueError(f"qk_eps must not be negative, got {qk_eps}")
    f32, slots, nseqs = torch.float32, state_cache.shape[0], read_slot.shape[0]
    if cu_seqlens is None and nseqs != tokens:
        raise ValueError(f"{tokens} tokens of {nseqs} sequences need cu_seqlens")
    cache = _whole(state_cache, "state_cache", device, f32, (slots, heads, dv, dk))
    rs = _slots(read_slot, "read_slot", device, nseqs)
    ws = _slots(write_slot, "write_slot", device, tokens)
    cu = None if cu_seqlens is None else _slots(cu_seqlens, "cu_seqlens", device, nseqs + 1)
    flag = _whole(error_flag, "error_flag", device, torch.int32, (1,))
    row, keys, gshape, gtype = heads * dv, kheads * dk, (tokens, heads), gate.dtype
    args = (q.data_ptr(), _rows(q, "q", device, dtype, qshape, keys),
            k.data_ptr(), _rows(k, "k", device, dtype, qshape, keys), v.data_ptr(),
            _rows(v, "v", device, dtype, vshape, row), gate.data_ptr(),
            _rows(gate, "gate", device, gtype, gshape, heads), beta.data_ptr(),
            _rows(beta, "beta", device, gtype, gshape, heads),
            _whole(A, "A", device, f32, (heads,)), _whole(dt_bias, "dt_bias", device, f32, (heads,)),
            -1.0 if qk_eps is None else float(qk_eps), dk ** -0.5 if scale is None else float(scale))
    o, o_stride = _out_rows(o, "o", v, row)
    _enqueue("ssd_gated_delta_step", device, *args, code, code if gate.dtype == dtype else _dtype_code(gate), nseqs, tokens,
             None if cu is None else cu.data_ptr(), heads, kheads, dk, dv, cache, slots, rs.data_ptr(), ws.data_ptr(),
             o.data_ptr(), o_stride, flag)
    return o


@dataclasses.dataclass
class StepTables:
    """Device-resident maps of one step (see ssd_step_tables)."""
    cu_seqlens: torch.Tensor    # (S+1,)
    seq_lens: torch.Tensor      # (S,)
    positions: torch.Tensor     # (T,)
    token_seq: torch.Tensor     # (T,)
    slots: torch.Tensor         # (T,)
    read_slot: torch.Tensor     # (S,)
    state_slot: torch.Tensor    # (T,)
    free_count: Optional[torch.Tensor]   # (1,) blocks left


def step_tables(num_computed: torch.Tensor, num_new: torch.Tensor, block_table: torch.Tensor, block_size: int,
                total_tokens: int, rows: Optional[torch.Tensor] = None, free_blocks: Optional[torch.Tensor] = None,
                free_count: Optional[torch.Tensor] = None, free_count_out: Optional[torch.Tensor] = None,
                num_blocks: Optional[int] = None, error_flag: Optional[torch.Tensor] = None) -> StepTables:
    """ssd_step_tables: block tables and slot maps of one step. num_computed, num_new (S,): tokens of each request in
    the caches and new in this step; total_tokens: their sum, or the padded batch's tokens. block_table int32 (table rows,
    blocks) holds request s in row rows[s] (s without rows) and gets the new blocks, taken from the end of
    free_blocks[:free_count]; what is left is written to free_count_out (a new tensor unless given; free_count itself
    updates it in place). num_blocks bounds the table's entries (2^31 - 1 slots unless given). Tokens that are given up
    after a step: their blocks, from column ceil(num_computed / block_size) on, go back to the free list before the next
    call, which overwrites those entries; states after such tokens need slots of the caller's own (see ssd_step_tables)."""
    device, i32 = block_table.device, torch.int32
    if block_table.dim() != 2:
        raise ValueError(f"block_table must be (rows, blocks), got {tuple(block_table.shape)}")
    if not 1 <= block_size <= 0x7fffffff:
        raise ValueError(f"block_size must be 1 .. 2^31 - 1, got {block_size}")
    nseqs, total_tokens = num_computed.shape[0], int(total_tokens)
    if not 0 <= total_tokens <= 0x7fffffff:
        raise ValueError(f"total_tokens must be 0 .. 2^31 - 1, got {total_tokens}")
    table_rows, width = block_table.shape
    nc = _slots(num_computed, "num_computed", device, nseqs)
    nn = _slots(num_new, "num_new", device, nseqs)
    rw = None if rows is None else _slots(rows, "rows", device, nseqs)
    table = _whole(block_table, "block_table", device, i32, (table_rows, width))
    if free_blocks is None:
        if free_count is not None or free_count_out is not None:
            raise ValueError("free_count and free_count_out are given only with free_blocks")
        free, nfree = None, 0
    else:
        if free_count is None:
            raise ValueError("free_blocks needs free_count")
        nfree = free_blocks.shape[0]
        free = _whole(free_blocks, "free_blocks", device, i32, (nfree,))
        if free_count_out is None:
            free_count_out = torch.empty(1, dtype=i32, device=device)
    count = _whole(free_count, "free_count", device, i32, (1,))
    left = _whole(free_count_out, "free_count_out", device, i32, (1,))
    flag = _whole(error_flag, "error_flag", device, i32, (1,))
    # one allocation for the maps
    maps = torch.empty(3 * nseqs + 1 + 4 * total_tokens, dtype=i32, device=device)
    parts = maps.split_with_sizes((nseqs + 1, nseqs, nseqs, total_tokens, total_tokens, total_tokens, total_tokens))
    cu = maps.data_ptr()
    lens = cu + 4 * (nseqs + 1)
    read = lens + 4 * nseqs
    pos = read + 4 * nseqs
    one = 4 * total_tokens
    most = 0x7fffffff // block_size
    if num_blocks is None:
        num_blocks = most
    elif not 0 <= num_blocks <= most:
        raise ValueError(f"num_blocks of {block_size} tokens must be 0 .. {most}, got {num_blocks}")
    _enqueue("ssd_step_tables", device, nseqs, total_tokens, nc.data_ptr(), nn.data_ptr(),
             None if rw is None else rw.data_ptr(), table, table_rows, width, int(block_size), int(num_blocks), free, nfree,
             count, left, cu, lens, pos, pos + one, pos + 2 * one, read, pos + 3 * one, flag)
    cu, lens, read, pos, seq, slots, state = parts
    return StepTables(cu, lens, pos, seq, slots, read, state, free_count_out)


def _paged(k_cache, v_cache, device, dtype):
    """Checks a paged cache; returns (blocks, kv heads, block size, head dim)."""
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be (blocks, kv heads, block size, head dim), got {tuple(k_cache.shape)}")
    blocks, heads, size, dim = k_cache.shape
    _whole(k_cache, "k_cache", device, dtype, k_cache.shape)
    _whole(v_cache, "v_cache", device, dtype, (blocks, heads, dim, size))
    return blocks, heads, size, dim


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slots: torch.Tensor, error_flag: Optional[torch.Tensor] = None):
    """ssd_kv_cache_write: the keys and values of token t, k, v (T, kv heads, head dim) (rows may lie further apart), go to
    slot slots[t] = block * block size + place of k_cache (blocks, kv heads, block size, head dim) and v_cache (blocks, kv
    heads, head dim, block size); negative slots are skipped."""
    device, dtype, shape = k.device, k.dtype, k.shape
    blocks, heads, size, dim = _paged(k_cache, v_cache, device, dtype)
    if len(shape) != 3 or shape[1:] != (heads, dim):
        raise ValueError(f"k must be (tokens, {heads}, {dim}), got {tuple(shape)}")
    to = _slots(slots, "slots", device, shape[0])
    flag = _whole(error_flag, "error_flag", device, torch.int32, (1,))
    row = heads * dim
    _enqueue("ssd_kv_cache_write", device, k.data_ptr(), _rows(k, "k", device, dtype, shape, row), v.data_ptr(),
             _rows(v, "v", device, dtype, shape, row), _dtype_code(k), shape[0], heads, dim, k_cache.data_ptr(),
             v_cache.data_ptr(), blocks, size, to.data_ptr(), flag)


@dataclasses.dataclass(frozen=True)
class AttentionPlan:
    """How one step's attention is split (see ssd_attention_plan)."""
    nseqs: int
    total_tokens: int
    max_new_tokens: int
    window: int
    max_parts: int
    seq_lens: torch.Tensor
    cu_seqlens: Optional[torch.Tensor]
    part_start: torch.Tensor
    part_seq: torch.Tensor
    part_keys: torch.Tensor
    error_flag: torch.Tensor

    def __post_init__(self):
        # what every layer's call passes is made once
        c = _Plan(self.nseqs, self.total_tokens, self.max_new_tokens, self.window, self.max_parts,
                  self.seq_lens.data_ptr(), None if self.cu_seqlens is None else self.cu_seqlens.data_ptr(),
                  self.part_start.data_ptr(), self.part_seq.data_ptr(), self.part_keys.data_ptr(),
                  self.error_flag.data_ptr())
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_device", self.part_start.device)
        sizes = ((self.seq_lens, self.nseqs), (self.cu_seqlens, self.nseqs + 1), (self.part_start, self.nseqs + 1),
                 (self.part_seq, self.max_parts), (self.part_keys, 1), (self.error_flag, 1))
        object.__setattr__(self, "_fits", all(t is None or t.numel() >= n for t, n in sizes))

    def c_struct(self) -> _Plan:
        return self._c


def attention_plan(seq_lens: torch.Tensor, num_heads: int, num_kv_heads: int, cu_seqlens: Optional[torch.Tensor] = None,
                   total_tokens: Optional[int] = None, max_new_tokens: int = 1, window: int = 0) -> AttentionPlan:
    """ssd_attention_plan_build: the split of one step's attention, for all layers with these heads and this window.
    seq_lens (S,): keys of each sequence, its new tokens' among them. Without cu_seqlens every sequence has one new token;
    with cu_seqlens (S+1,) pass total_tokens and max_new_tokens (the most of a sequence, up to 64)."""
    device, i32 = seq_lens.device, torch.int32
    if not 0 < num_heads <= 0x7fffffff or num_kv_heads <= 0 or num_heads % num_kv_heads:
        raise ValueError(f"num_heads must be a multiple of num_kv_heads and at most 2^31 - 1, got {num_heads} and {num_kv_heads}")
    if not 1 <= max_new_tokens <= 64 or not 0 <= window <= 0x7fffffff:
        raise ValueError(f"max_new_tokens must be 1 .. 64 and window 0 .. 2^31 - 1, got {max_new_tokens} and {window}")
    nseqs = seq_lens.shape[0]
    if cu_seqlens is None:
        if total_tokens not in (None, nseqs):
            raise ValueError(f"{total_tokens} tokens of {nseqs} sequences need cu_seqlens")
        total_tokens = nseqs
    elif total_tokens is None or not 0 <= total_tokens <= 0x7fffffff:
        raise ValueError(f"pass total_tokens, 0 .. 2^31 - 1, with cu_seqlens, got {total_tokens}")
    lens = _slots(seq_lens, "seq_lens", device, nseqs)
    cu = None if cu_seqlens is None else _slots(cu_seqlens, "cu_seqlens", device, nseqs + 1)
    parts = nseqs + int((_lib or load_library()).ssd_paged_attention_parts(int(max_new_tokens), num_heads, num_kv_heads))
    made = torch.zeros(nseqs + 3 + parts, dtype=i32, device=device)
    plan = AttentionPlan(nseqs, int(total_tokens), int(max_new_tokens), int(window), parts, lens, cu, made[:nseqs + 1],
                         made[nseqs + 3:], made[nseqs + 1:nseqs + 2], made[nseqs + 2:nseqs + 3])
    _enqueue("ssd_attention_plan_build", device, ctypes.byref(plan.c_struct()))
    return plan


def paged_attention_step(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                         plan: AttentionPlan, rows: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, error_flag: Optional[torch.Tensor] = None):
    """ssd_paged_attention_step: attention of the plan's new tokens, q (T, heads, head dim) (rows may lie further apart),
    over the keys and values of their sequences in a paged cache (see kv_cache_write). block_table int32 (table rows,
    blocks) holds sequence s in row rows[s] (s without rows). scale: head dim ** -0.5 unless given. lse (T, heads)
    float32 receives the logarithms of the sums of exponentials. workspace (uint8, at least
    paged_attention_workspace_size bytes) is allocated per call when not given. Returns out (T, heads, head dim)."""
    device, dtype, shape = q.device, q.dtype, q.shape
    blocks, kv_heads, size, dim = _paged(k_cache, v_cache, device, dtype)
    if len(shape) != 3 or shape[0] != plan.total_tokens or shape[2] != dim:
        raise ValueError(f"q must be ({plan.total_tokens}, heads, {dim}), got {tuple(shape)}")
    if plan._device != device:
        raise ValueError(f"the plan must be on {device}, got {plan._device}")
    if not plan._fits:
        raise ValueError("the plan's tensors are shorter than its numbers of sequences and parts")
    heads = shape[1]
    if kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"q's heads must be a multiple of the cache's {kv_heads}, got {heads}")
    if block_table.dim() != 2:
        raise ValueError(f"block_table must be (rows, blocks), got {tuple(block_table.shape)}")
    table_rows, width = block_table.shape
    table = _whole(block_table, "block_table", device, torch.int32, (table_rows, width))
    if rows is None and table_rows < plan.nseqs:
        raise ValueError(f"block_table must have {plan.nseqs} rows, got {table_rows}")
    rw = None if rows is None else _slots(rows, "rows", device, plan.nseqs)
    flag = _whole(error_flag, "error_flag", device, torch.int32, (1,))
    q_stride = _rows(q, "q", device, dtype, shape, heads * dim)
    log = _whole(lse, "lse", device, torch.float32, (shape[0], heads))
    need = paged_attention_workspace_size(plan, heads, dim)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    ws = _whole(workspace, "workspace", device, torch.uint8, (workspace.numel(),))
    out, out_stride = _out_rows(out, "out", q, heads * dim)
    _enqueue("ssd_paged_attention_step", device, q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(),
             _dtype_code(q), dim ** -0.5 if scale is None else float(scale), ctypes.byref(plan.c_struct()), heads, kv_heads,
             dim, table, table_rows, width, None if rw is None else rw.data_ptr(), blocks, size, out.data_ptr(), out_stride,
             log, ws, workspace.numel(), flag)
    return out


def paged_attention_workspace_size(plan: AttentionPlan, num_heads: int, head_dim: int) -> int:
    """Bytes of device workspace that paged_attention_step needs for this plan."""
    return int((_lib or load_library()).ssd_paged_attention_workspace_size(plan.max_parts, plan.max_new_tokens,
                                                                            int(num_heads), int(head_dim)))


def _add_norm_inputs(x, weight, residual, residual_out):
    """Checks what the two norms with a residual share; returns the library's leading arguments, the residual's output
    and the rest of the arguments that describe it."""
    if x.dim() != 2:
        raise ValueError(f"x must be (rows, channels), got {tuple(x.shape)}")
    device, dtype, shape = x.device, x.dtype, x.shape
    channels = shape[1]
    if residual is None and residual_out is not None:
        raise ValueError("residual_out is given only with residual")
    head = (x.data_ptr(), _rows(x, "x", device, dtype, shape, channels),
            None if residual is None else residual.data_ptr(),
            0 if residual is None else _rows(residual, "residual", device, dtype, shape, channels),
            _whole(weight, "weight", device, torch.float32, (channels,)), _dtype_code(x), shape[0], channels)
    if residual is None:
        return head, None, (None, 0)
    residual_out, stride = _out_rows(residual_out, "residual_out", x, channels)
    return head, residual_out, (residual_out.data_ptr(), stride)


def add_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """ssd_add_rms_norm: r = x + residual, out = r / sqrt(mean(r^2) + eps) * weight, over the rows of x (rows, channels)
    (which may lie further apart). residual_out receives r (a new tensor unless given; residual itself updates it in
    place). Returns (out, residual_out), the latter None without residual."""
    head, residual_out, res = _add_norm_inputs(x, weight, residual, residual_out)
    out, out_stride = _out_rows(out, "out", x, x.shape[1])
    _enqueue("ssd_add_rms_norm", x.device, *head, float(eps), *res, out.data_ptr(), out_stride)
    return out, residual_out


def add_rms_norm_e4m3(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, group: int = 0, scale: Optional[torch.Tensor] = None,
                      residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None):
    """ssd_add_rms_norm_e4m3: add_rms_norm with its result in 8 bits, out = e4m3(norm / scale) as float8_e4m3fn. `scale`
    (1,) is used as given; without it every `group` channels (0: a whole row) get the scale max |norm| / 448 (1 where all
    are zero). Returns (out, scales (rows, channels / group) or the given scale, residual_out or None)."""
    head, residual_out, res = _add_norm_inputs(x, weight, residual, residual_out)
    device, (rows, channels), f32 = x.device, x.shape, torch.float32
    group = int(group) or channels
    if group <= 0 or channels % group:
        raise ValueError(f"group must divide the {channels} channels, got {group}")
    if scale is not None and scales is not None:
        raise ValueError("scales is written only without a given scale")
    given = _whole(scale, "scale", device, f32, (1,))
    if scale is None and scales is None:
        scales = torch.empty(rows, channels // group, dtype=f32, device=device)
    made = None if scales is None else _whole(scales, "scales", device, f32, (rows, channels // group))
    if out is None:
        out = torch.empty(rows, channels, dtype=torch.float8_e4m3fn, device=device)
    out_stride = _rows(out, "out", device, torch.float8_e4m3fn, x.shape, channels)
    _enqueue("ssd_add_rms_norm_e4m3", device, *head, group, float(eps), given, made, *res, out.data_ptr(), out_stride)
    return out, scales if scale is None else scale, residual_out
