// C ABI of libssd.so: argument validation and launches (declarations and
// contracts in include/ssd.h). Every argument error is reported before
// anything is enqueued; the library never synchronises the host.
#include <stdint.h>

#include "ssd_internal.h"

namespace {

bool pow2_chunk(int32_t cs) { return cs >= 16 && cs <= 256 && (cs & (cs - 1)) == 0; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ssd_status check_meta(const ssd_varlen_meta *m) {
    if (m == nullptr || m->cu_seqlens == nullptr || m->chunk_offsets == nullptr ||
        m->chunk_seq_idx == nullptr || m->seq_chunk_start == nullptr || m->nchunks == nullptr ||
        m->seq_order == nullptr || m->error_flag == nullptr)
        return SSD_ERR_NULL_ARG;
    if (m->nseqs < 0 || m->total_tokens < 0 || m->max_chunks < 0) return SSD_ERR_SHAPE;
    if (!pow2_chunk(m->chunk_size)) return SSD_ERR_CHUNK_SIZE;
    // every sequence adds at most one partial chunk to T / chunk_size full ones
    if ((int64_t)m->max_chunks < (int64_t)m->total_tokens / m->chunk_size + m->nseqs) return SSD_ERR_CAPACITY;
    return SSD_OK;
}

bool aligned_to(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool known_dtype(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }

uintptr_t elem_bytes(ssd_dtype t) { return t == SSD_BF16 ? 2 : 4; }

// Rows of `row` contiguous elements, `stride` elements apart. The bound keeps
// every byte offset inside 16 rows below 2^32.
bool row_stride(int64_t stride, int64_t row) { return stride >= row && stride <= (int64_t(1) << 26); }

// What the selective scan and its step ask of their shared arguments.
ssd_status check_selective(const ssd::SelectiveArgs &a, ssd_dtype in_dtype, ssd_dtype dt_dtype, bool rows) {
    if (!known_dtype(in_dtype) || !known_dtype(dt_dtype)) return SSD_ERR_DTYPE;
    if (a.C_total <= 0 || a.N <= 0 || a.G <= 0 || a.C_total % a.G != 0) return SSD_ERR_SHAPE;
    if (!(a.N == 16 || a.N == 32 || a.N == 64 || a.N == 128 || a.N == 256)) return SSD_ERR_UNSUPPORTED;
    if (a.A == nullptr) return SSD_ERR_NULL_ARG;
    if (rows && (a.u == nullptr || a.dt == nullptr || a.B == nullptr || a.C == nullptr || a.y == nullptr))
        return SSD_ERR_NULL_ARG;
    const int64_t C = a.C_total, GN = (int64_t)a.G * a.N;
    if (GN > (int64_t(1) << 26) || C > (int64_t(1) << 26)) return SSD_ERR_SHAPE;
    if (rows && (!row_stride(a.u_stride, C) || !row_stride(a.dt_stride, C) || !row_stride(a.y_stride, C) ||
                 !row_stride(a.B_stride, GN) || !row_stride(a.C_stride, GN) ||
                 (a.z != nullptr && !row_stride(a.z_stride, C))))
        return SSD_ERR_SHAPE;
    const uintptr_t e = elem_bytes(in_dtype);
    for (const void *p : {a.u, a.B, a.C, a.z, (const void *)a.y})
        if (!aligned_to(p, e)) return SSD_ERR_SHAPE;
    if (!aligned_to(a.dt, elem_bytes(dt_dtype))) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)a.A, (const void *)a.init, (const void *)a.final_states,
                          (const void *)a.chunk_states, (const void *)a.cache})
        if (!aligned16(p)) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)a.dt_bias, (const void *)a.D})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// What the calls on a paged cache ask of its sizes (`heads`: of q, or of the cache).
ssd_status check_paged(int32_t heads, int32_t head_dim, int32_t num_blocks, int32_t block_size) {
    if (heads <= 0 || head_dim <= 0 || num_blocks < 0) return SSD_ERR_SHAPE;
    if (block_size < 16 || block_size % 16 != 0) return SSD_ERR_BLOCK_SIZE;
    if (!(head_dim == 64 || head_dim == 128 || head_dim == 256)) return SSD_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * block_size > INT32_MAX) return SSD_ERR_SHAPE;
    return SSD_OK;
}

ssd_status check_plan(const ssd_attention_plan *p) {
    if (p == nullptr || p->part_start == nullptr || p->part_seq == nullptr || p->part_keys == nullptr ||
        p->error_flag == nullptr)
        return SSD_ERR_NULL_ARG;
    if (p->nseqs < 0 || p->total_tokens < 0 || p->max_new_tokens < 1 || p->max_new_tokens > 64 || p->window < 0 ||
        p->max_parts > (1 << 26))
        return SSD_ERR_SHAPE;
    if (p->max_parts <= p->nseqs) return SSD_ERR_CAPACITY;
    if (p->nseqs > 0 && p->seq_lens == nullptr) return SSD_ERR_NULL_ARG;
    if (p->cu_seqlens == nullptr && p->total_tokens != p->nseqs) return SSD_ERR_SHAPE;
    for (const void *q : {(const void *)p->seq_lens, (const void *)p->cu_seqlens, (const void *)p->part_start,
                          (const void *)p->part_seq, (const void *)p->part_keys, (const void *)p->error_flag})
        if (!aligned_to(q, 4)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// A window of 2^30 keys is none (sequences have no more), so the kernels' positions less a window stay in 32 bits.
int32_t attention_window(const ssd_attention_plan *p) { return p->window >= (1 << 30) ? 0 : p->window; }

// Tiles of 16 rows (tokens x query heads of a kv head).
int64_t attention_tiles(int32_t max_new_tokens, int32_t group) { return ((int64_t)max_new_tokens * group + 15) / 16; }

// What the two norms with a residual ask of their shared arguments.
ssd_status check_add_norm(const ssd::AddNormArgs &a, ssd_dtype in_dtype) {
    if (!known_dtype(in_dtype)) return SSD_ERR_DTYPE;
    if (a.rows < 0 || a.channels <= 0 || !(a.eps >= 0.0f)) return SSD_ERR_SHAPE;
    if (a.channels > ssd::kNormMaxGroup) return SSD_ERR_UNSUPPORTED;
    if (a.rows == 0) return SSD_OK;
    if (a.x == nullptr || a.out == nullptr) return SSD_ERR_NULL_ARG;
    if (!row_stride(a.x_stride, a.channels) || !row_stride(a.out_stride, a.channels) ||
        (a.residual != nullptr && !row_stride(a.residual_stride, a.channels)) ||
        (a.residual_out != nullptr && !row_stride(a.residual_out_stride, a.channels)))
        return SSD_ERR_SHAPE;
    for (const void *p : {a.x, a.residual, (const void *)a.residual_out})
        if (!aligned_to(p, elem_bytes(in_dtype))) return SSD_ERR_SHAPE;
    return aligned_to(a.weight, 4) ? SSD_OK : SSD_ERR_SHAPE;
}

}  // namespace

extern "C" {

const char *ssd_status_string(ssd_status status) {
    switch (status) {
    case SSD_OK: return "ok";
    case SSD_ERR_NULL_ARG: return "a required pointer is NULL";
    case SSD_ERR_CHUNK_SIZE: return "chunk_size must be a power of two in [16, 256]";
    case SSD_ERR_SHAPE: return "invalid sizes, nheads % ngroups != 0, or a pointer not 16-byte aligned";
    case SSD_ERR_BLOCK_SIZE: return "block_size must be a positive multiple of chunk_size (of 16 in a cache of keys and values)";
    case SSD_ERR_CAPACITY: return "capacity below the required bound (max_chunks, chunk_states, max_parts or workspace)";
    case SSD_ERR_DTYPE: return "unknown dtype";
    case SSD_ERR_HIP: return "a HIP call failed";
    case SSD_ERR_UNSUPPORTED: return "unsupported dtype/shape combination (headdim, dstate, dk, dv, chunk size, channels or group)";
    }
    return "unknown status";
}

ssd_status ssd_varlen_metadata(const ssd_varlen_meta *meta, void *stream) {
    const ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    ssd::MetaArgs a{meta->cu_seqlens, meta->chunk_offsets, meta->chunk_seq_idx, meta->seq_chunk_start,
                    meta->nchunks, meta->seq_order, meta->error_flag, meta->nseqs, meta->total_tokens,
                    meta->chunk_size, meta->max_chunks};
    return ssd::launch_metadata(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_chunk_scan_varlen(const void *x, const float *dt, const float *dt_bias, const float *A,
                                 const void *B, const void *C, const float *D, ssd_dtype in_dtype,
                                 const ssd_varlen_meta *meta, int32_t nheads, int32_t headdim,
                                 int32_t dstate, int32_t ngroups, const float *initial_states,
                                 const int32_t *has_initial_state, void *y, float *final_states,
                                 float *chunk_states, const int32_t *chunk_state_dst,
                                 int32_t chunk_states_capacity, void *stream) {
    ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_DTYPE;
    const bool empty = meta->total_tokens == 0;
    if ((!empty && (x == nullptr || dt == nullptr || B == nullptr || C == nullptr || y == nullptr)) ||
        A == nullptr || (meta->nseqs > 0 && final_states == nullptr))
        return SSD_ERR_NULL_ARG;
    if (nheads <= 0 || headdim <= 0 || dstate <= 0 || ngroups <= 0 || nheads % ngroups != 0)
        return SSD_ERR_SHAPE;
    if (headdim % 16 != 0) return SSD_ERR_UNSUPPORTED;
    const bool n_ok = dstate == 16 || dstate == 32 || dstate == 64 || dstate == 128 ||
                      (dstate == 256 && in_dtype == SSD_BF16);
    if (!n_ok) return SSD_ERR_UNSUPPORTED;
    if (chunk_states != nullptr) {
        if (chunk_states_capacity <= 0) return SSD_ERR_CAPACITY;
        if (chunk_state_dst == nullptr && chunk_states_capacity < meta->max_chunks) return SSD_ERR_CAPACITY;
    }
    for (const void *p : {x, B, C, (const void *)y, (const void *)final_states, (const void *)initial_states,
                          (const void *)chunk_states})
        if (p != nullptr && !aligned16(p)) return SSD_ERR_SHAPE;

    ssd::ScanArgs a{};
    a.x = x; a.dt = dt; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.D = D;
    a.init = initial_states; a.has_init = has_initial_state;
    a.y = y; a.final_states = final_states; a.chunk_states = chunk_states;
    a.chunk_state_dst = chunk_state_dst;
    a.cu_seqlens = meta->cu_seqlens; a.seq_chunk_start = meta->seq_chunk_start;
    a.seq_order = meta->seq_order; a.error_flag = meta->error_flag;
    a.T = meta->total_tokens; a.S = meta->nseqs; a.H = nheads; a.P = headdim; a.G = ngroups;
    a.cs = meta->chunk_size; a.max_chunks = meta->max_chunks;
    a.capacity = chunk_states ? chunk_states_capacity : 0;
    // headdim tile per workgroup: 64 columns when it divides headdim (4 waves,
    // or 8 with the state split between wave pairs for bf16 with dstate 128),
    // else 32 (2 waves) or 16 (1 wave)
    const int waves = headdim % 64 == 0 ? 4 : (headdim % 32 == 0 ? 2 : 1);
    const bool split = in_dtype == SSD_BF16 && dstate == 128 && headdim % 64 == 0;
    a.nptiles = headdim / (16 * waves);
    a.xcd_mode = ssd::xcd_mode_for(meta->nseqs, nheads, ngroups, a.nptiles);
    // the warp-specialised kernel walks 64-token tiles (chunk_size >= 64), of
    // one head or of a.items heads per workgroup
    const bool ws = split && meta->chunk_size >= 64;
    const int64_t wgs = (int64_t)meta->nseqs * nheads * a.nptiles;
    a.items = ws ? ssd::ws_items_for(a.xcd_mode, wgs, nheads / ngroups)
                 : split ? ssd::split_items_for(a.xcd_mode, wgs, nheads / ngroups) : 1;
    if (meta->nseqs == 0) return SSD_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = ws ? ssd::launch_scan_ws_bf16(a, dstate, s)
                         : split ? ssd::launch_scan_split_bf16(a, dstate, s)
                         : in_dtype == SSD_BF16 ? ssd::launch_scan_bf16(a, waves, dstate, s)
                                                : ssd::launch_scan_f32(a, waves, dstate, s);
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_export_chunk_states(const ssd_varlen_meta *meta, const int32_t *num_computed_tokens,
                                   const int32_t *block_table, int32_t max_blocks_per_seq,
                                   int32_t block_size, int32_t *ckpt_src, int32_t *chunk_state_dst,
                                   const float *chunk_states, int32_t state_elems, float *state_cache,
                                   int32_t num_slots, void *stream) {
    ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    if (max_blocks_per_seq < 0 || num_slots < 0) return SSD_ERR_SHAPE;
    if ((meta->nseqs > 0 && max_blocks_per_seq > 0 && (block_table == nullptr || ckpt_src == nullptr)) ||
        (meta->max_chunks > 0 && chunk_state_dst == nullptr))
        return SSD_ERR_NULL_ARG;
    if (block_size <= 0 || block_size % meta->chunk_size != 0) return SSD_ERR_BLOCK_SIZE;
    if (chunk_states != nullptr) {
        if (state_cache == nullptr) return SSD_ERR_NULL_ARG;
        if (state_elems <= 0 || state_elems % 4 != 0) return SSD_ERR_SHAPE;
        if (!aligned16(chunk_states) || !aligned16(state_cache)) return SSD_ERR_SHAPE;
    }
    ssd::PlanArgs a{};
    a.cu_seqlens = meta->cu_seqlens; a.seq_chunk_start = meta->seq_chunk_start;
    a.chunk_seq_idx = meta->chunk_seq_idx; a.nchunks = meta->nchunks;
    a.num_computed_tokens = num_computed_tokens; a.block_table = block_table;
    a.ckpt_src = ckpt_src; a.chunk_state_dst = chunk_state_dst; a.error_flag = meta->error_flag;
    a.chunk_states = chunk_states; a.state_cache = state_cache;
    a.S = meta->nseqs; a.cs = meta->chunk_size; a.max_chunks = meta->max_chunks;
    a.max_blocks = max_blocks_per_seq; a.block_size = block_size; a.state_elems = state_elems;
    a.num_slots = num_slots;
    return ssd::launch_plan(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_decode_step(const void *x, const float *dt, const float *dt_bias, const float *A,
                           const void *B, const void *C, const float *D, ssd_dtype in_dtype,
                           int32_t nseqs, int32_t nheads, int32_t headdim, int32_t dstate,
                           int32_t ngroups, float *state_cache, int32_t num_slots,
                           const int32_t *read_slot, const int32_t *write_slot, void *y,
                           int32_t *error_flag, void *stream) {
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (nseqs < 0 || nheads <= 0 || headdim <= 0 || dstate <= 0 || ngroups <= 0 ||
        nheads % ngroups != 0 || num_slots < 0)
        return SSD_ERR_SHAPE;
    if (!(dstate == 16 || dstate == 32 || dstate == 64 || dstate == 128 || dstate == 256))
        return SSD_ERR_UNSUPPORTED;
    if (A == nullptr) return SSD_ERR_NULL_ARG;
    if (nseqs > 0 && (x == nullptr || dt == nullptr || B == nullptr || C == nullptr || y == nullptr ||
                      state_cache == nullptr || read_slot == nullptr || write_slot == nullptr))
        return SSD_ERR_NULL_ARG;
    if (state_cache != nullptr && !aligned16(state_cache)) return SSD_ERR_SHAPE;
    ssd::DecodeArgs a{};
    a.x = x; a.dt = dt; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.D = D;
    a.cache = state_cache; a.read_slot = read_slot; a.write_slot = write_slot; a.y = y;
    a.error_flag = error_flag;
    a.S = nseqs; a.H = nheads; a.P = headdim; a.G = ngroups; a.num_slots = num_slots;
    a.pchunks = ssd::decode_pchunks(headdim, dstate);
    return ssd::launch_decode(a, in_dtype == SSD_BF16, dstate, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_causal_conv1d_varlen(const void *x, const float *weight, const float *bias,
                                    ssd_dtype in_dtype, const ssd_varlen_meta *meta, int32_t channels,
                                    int32_t width, int32_t activation, void *conv_states,
                                    int32_t num_slots, const int32_t *read_slot,
                                    const int32_t *write_slot, void *out, void *stream) {
    ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (channels <= 0 || num_slots < 0) return SSD_ERR_SHAPE;
    if (channels % 8 != 0 || width < 1 || width > 4 || (activation != 0 && activation != 1))
        return SSD_ERR_UNSUPPORTED;
    if (weight == nullptr || (meta->total_tokens > 0 && (x == nullptr || out == nullptr)))
        return SSD_ERR_NULL_ARG;
    if (width > 1 && num_slots > 0 && (read_slot != nullptr || write_slot != nullptr) && conv_states == nullptr)
        return SSD_ERR_NULL_ARG;
    for (const void *p : {x, (const void *)out, (const void *)conv_states})
        if (p != nullptr && !aligned16(p)) return SSD_ERR_SHAPE;
    ssd::Conv1dArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.out = out; a.states = conv_states;
    a.read_slot = read_slot; a.write_slot = write_slot;
    a.chunk_offsets = meta->chunk_offsets; a.chunk_seq_idx = meta->chunk_seq_idx;
    a.seq_chunk_start = meta->seq_chunk_start; a.error_flag = meta->error_flag;
    a.S = meta->nseqs; a.C = channels; a.W = width; a.num_slots = (conv_states != nullptr || width == 1) ? num_slots : 0;   // (width 1 keeps no rows)
    a.max_chunks = meta->max_chunks; a.channel_blocks = ssd::conv1d_channel_blocks(channels);
    a.silu = activation;
    return ssd::launch_conv1d(a, in_dtype == SSD_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

size_t ssd_gated_delta_workspace_size(int32_t max_chunks, int32_t nheads) {
    if (max_chunks <= 0 || nheads <= 0) return 0;
    return (size_t)max_chunks * (size_t)nheads * ssd::kGdnWsBytes;
}

ssd_status ssd_gated_delta_chunk_varlen(const void *q, const void *k, const void *v, const float *gate,
                                        const float *beta, float scale, ssd_dtype in_dtype,
                                        const ssd_varlen_meta *meta, int32_t nheads, int32_t nkheads, int32_t dk,
                                        int32_t dv, const float *initial_states, const int32_t *has_initial_state,
                                        void *o, float *final_states, float *chunk_states,
                                        const int32_t *chunk_state_dst, int32_t chunk_states_capacity,
                                        void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_DTYPE;
    const bool empty = meta->total_tokens == 0;
    if ((!empty && (q == nullptr || k == nullptr || v == nullptr || gate == nullptr || beta == nullptr ||
                    o == nullptr)) ||
        (meta->nseqs > 0 && final_states == nullptr))
        return SSD_ERR_NULL_ARG;
    if (nheads <= 0 || nkheads <= 0 || dk <= 0 || dv <= 0 || nheads % nkheads != 0) return SSD_ERR_SHAPE;
    if (in_dtype != SSD_BF16 || dk != 128 || dv % 64 != 0 || meta->chunk_size != 64) return SSD_ERR_UNSUPPORTED;
    if (chunk_states != nullptr) {
        if (chunk_states_capacity <= 0) return SSD_ERR_CAPACITY;
        if (chunk_state_dst == nullptr && chunk_states_capacity < meta->max_chunks) return SSD_ERR_CAPACITY;
    }
    if (!empty && (workspace == nullptr || workspace_bytes < ssd_gated_delta_workspace_size(meta->max_chunks, nheads)))
        return SSD_ERR_CAPACITY;
    for (const void *p : {q, k, v, (const void *)o, (const void *)final_states, (const void *)initial_states,
                          (const void *)chunk_states, (const void *)workspace})
        if (p != nullptr && !aligned16(p)) return SSD_ERR_SHAPE;
    ssd::GdnArgs a{};
    a.q = static_cast<const uint16_t *>(q); a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v); a.gate = gate; a.beta = beta;
    a.init = initial_states; a.has_init = has_initial_state;
    a.o = static_cast<uint16_t *>(o); a.final_states = final_states;
    a.chunk_states = chunk_states; a.chunk_state_dst = chunk_state_dst;
    a.workspace = static_cast<uint16_t *>(workspace);
    a.cu_seqlens = meta->cu_seqlens; a.seq_chunk_start = meta->seq_chunk_start; a.seq_order = meta->seq_order;
    a.chunk_offsets = meta->chunk_offsets; a.chunk_seq_idx = meta->chunk_seq_idx;
    a.error_flag = meta->error_flag; a.scale = scale;
    a.T = meta->total_tokens; a.S = meta->nseqs; a.H = nheads; a.G = nkheads; a.dv = dv;
    a.max_chunks = meta->max_chunks; a.capacity = chunk_states ? chunk_states_capacity : 0;
    a.nptiles = dv / 64;
    if (meta->nseqs == 0) return SSD_OK;
    return ssd::launch_gdn(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_gated_delta_chunk_varlen_noalloc(const void *q, const void *k, const void *v, const float *gate,
                                                const float *beta, float scale, ssd_dtype in_dtype,
                                                const ssd_varlen_meta *meta, int32_t nheads, int32_t nkheads,
                                                int32_t dk, int32_t dv, const float *initial_states,
                                                const int32_t *has_initial_state, void *o, float *final_states,
                                                float *chunk_states, const int32_t *chunk_state_dst,
                                                int32_t chunk_states_capacity, void *stream) {
    const ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    const size_t need = meta->total_tokens > 0 ? ssd_gated_delta_workspace_size(meta->max_chunks, nheads) : 0;
    if (need > ssd::kGdnScratchBytes) return SSD_ERR_CAPACITY;
    void *ws = nullptr;
    if (need > 0 && ssd::gdn_scratch(&ws) != hipSuccess) return SSD_ERR_HIP;
    return ssd_gated_delta_chunk_varlen(q, k, v, gate, beta, scale, in_dtype, meta, nheads, nkheads, dk, dv,
                                        initial_states, has_initial_state, o, final_states, chunk_states,
                                        chunk_state_dst, chunk_states_capacity, ws, ws ? ssd::kGdnScratchBytes : 0,
                                        stream);
}

ssd_status ssd_prefill_bites(int32_t nseqs, const int32_t *num_computed_tokens, const int32_t *prompt_len,
                             const int32_t *budget, int32_t align, int32_t *num_scheduled) {
    if (nseqs < 0 || align <= 0) return SSD_ERR_SHAPE;
    if (nseqs > 0 && (num_computed_tokens == nullptr || prompt_len == nullptr || budget == nullptr ||
                      num_scheduled == nullptr))
        return SSD_ERR_NULL_ARG;
    for (int32_t s = 0; s < nseqs; ++s)
        if (num_computed_tokens[s] < 0 || num_computed_tokens[s] > prompt_len[s] || budget[s] < align)
            return SSD_ERR_SHAPE;
    for (int32_t s = 0; s < nseqs; ++s) {
        const int64_t pos = num_computed_tokens[s], total = prompt_len[s];
        const int64_t grid_end = total - total % align;            // last block boundary of the prompt
        const int64_t boundary = pos - pos % align + align;        // first boundary after pos
        const int64_t want = pos + budget[s];
        int64_t stop = want < total ? want : total;
        if (pos % align != 0) {
            if (boundary <= grid_end && boundary < stop) stop = boundary;   // back onto the grid
        } else if (stop < grid_end) {
            stop -= stop % align;                                           // end on the grid
        }
        num_scheduled[s] = (int32_t)(stop - pos);
    }
    return SSD_OK;
}

ssd_status ssd_selective_scan_varlen(const void *u, int64_t u_stride, const void *dt, int64_t dt_stride,
                                     const float *dt_bias, const float *A, const void *B, int64_t B_stride,
                                     const void *C, int64_t C_stride, const float *D, const void *z,
                                     int64_t z_stride, ssd_dtype in_dtype, ssd_dtype dt_dtype,
                                     const ssd_varlen_meta *meta, int32_t channels, int32_t dstate, int32_t ngroups,
                                     const float *initial_states, const int32_t *has_initial_state, void *y,
                                     int64_t y_stride, float *final_states, float *chunk_states,
                                     const int32_t *chunk_state_dst, int32_t chunk_states_capacity, void *stream) {
    ssd_status st = check_meta(meta);
    if (st != SSD_OK) return st;
    if (meta->total_tokens > (1 << 30)) return SSD_ERR_SHAPE;   // token counts stay in 32 bits past a segment's end
    ssd::SelectiveArgs a{};
    a.u = u; a.dt = dt; a.B = B; a.C = C; a.z = z; a.dt_bias = dt_bias; a.A = A; a.D = D; a.y = y;
    a.u_stride = u_stride; a.dt_stride = dt_stride; a.B_stride = B_stride; a.C_stride = C_stride;
    a.z_stride = z_stride; a.y_stride = y_stride;
    a.S = meta->nseqs; a.T = meta->total_tokens; a.C_total = channels; a.N = dstate; a.G = ngroups;
    a.error_flag = meta->error_flag;
    a.init = initial_states; a.has_init = has_initial_state; a.final_states = final_states;
    a.chunk_states = chunk_states; a.chunk_state_dst = chunk_state_dst;
    a.cu_seqlens = meta->cu_seqlens; a.seq_chunk_start = meta->seq_chunk_start; a.seq_order = meta->seq_order;
    a.cs = meta->chunk_size; a.max_chunks = meta->max_chunks;
    a.capacity = chunk_states != nullptr ? chunk_states_capacity : 0;
    st = check_selective(a, in_dtype, dt_dtype, meta->total_tokens > 0);
    if (st != SSD_OK) return st;
    if (meta->nseqs > 0 && final_states == nullptr) return SSD_ERR_NULL_ARG;
    if (chunk_states != nullptr) {
        if (chunk_states_capacity <= 0) return SSD_ERR_CAPACITY;
        if (chunk_state_dst == nullptr && chunk_states_capacity < meta->max_chunks) return SSD_ERR_CAPACITY;
    }
    if (meta->nseqs == 0) return SSD_OK;
    return ssd::launch_selective_scan(a, in_dtype == SSD_BF16, dt_dtype == SSD_BF16,
                                      static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_selective_step(const void *u, int64_t u_stride, const void *dt, int64_t dt_stride,
                              const float *dt_bias, const float *A, const void *B, int64_t B_stride, const void *C,
                              int64_t C_stride, const float *D, const void *z, int64_t z_stride, ssd_dtype in_dtype,
                              ssd_dtype dt_dtype, int32_t nseqs, int32_t channels, int32_t dstate, int32_t ngroups,
                              float *state_cache, int32_t num_slots, const int32_t *read_slot,
                              const int32_t *write_slot, void *y, int64_t y_stride, int32_t *error_flag,
                              void *stream) {
    if (nseqs < 0 || num_slots < 0) return SSD_ERR_SHAPE;
    ssd::SelectiveArgs a{};
    a.u = u; a.dt = dt; a.B = B; a.C = C; a.z = z; a.dt_bias = dt_bias; a.A = A; a.D = D; a.y = y;
    a.u_stride = u_stride; a.dt_stride = dt_stride; a.B_stride = B_stride; a.C_stride = C_stride;
    a.z_stride = z_stride; a.y_stride = y_stride;
    a.S = nseqs; a.T = nseqs; a.C_total = channels; a.N = dstate; a.G = ngroups;
    a.error_flag = error_flag;
    a.cache = state_cache; a.num_slots = num_slots; a.read_slot = read_slot; a.write_slot = write_slot;
    const ssd_status st = check_selective(a, in_dtype, dt_dtype, nseqs > 0);
    if (st != SSD_OK) return st;
    if (nseqs == 0) return SSD_OK;
    if (state_cache == nullptr || read_slot == nullptr || write_slot == nullptr) return SSD_ERR_NULL_ARG;
    return ssd::launch_selective_step(a, in_dtype == SSD_BF16, dt_dtype == SSD_BF16,
                                      static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_causal_conv1d_step(const void *x, int64_t x_stride, const float *weight, const float *bias,
                                  ssd_dtype in_dtype, int32_t nseqs, int32_t channels, int32_t width,
                                  int32_t activation, void *conv_states, int32_t num_slots,
                                  const int32_t *read_slot, const int32_t *write_slot, void *out,
                                  int64_t out_stride, int32_t *error_flag, void *stream) {
    if (!known_dtype(in_dtype)) return SSD_ERR_DTYPE;
    if (nseqs < 0 || channels <= 0 || num_slots < 0) return SSD_ERR_SHAPE;
    if (channels % 8 != 0 || width < 1 || width > 4 || (activation != 0 && activation != 1))
        return SSD_ERR_UNSUPPORTED;
    if (weight == nullptr || (nseqs > 0 && (x == nullptr || out == nullptr))) return SSD_ERR_NULL_ARG;
    if (width > 1 && num_slots > 0 && (read_slot != nullptr || write_slot != nullptr) && conv_states == nullptr)
        return SSD_ERR_NULL_ARG;
    if (nseqs > 0 && (!row_stride(x_stride, channels) || !row_stride(out_stride, channels) || x_stride % 8 != 0 ||
                      out_stride % 8 != 0))
        return SSD_ERR_SHAPE;
    for (const void *p : {x, (const void *)out, (const void *)conv_states})
        if (!aligned16(p)) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)weight, (const void *)bias})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    if (nseqs == 0) return SSD_OK;
    ssd::Conv1dStepArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.out = out; a.states = conv_states;
    a.read_slot = read_slot; a.write_slot = write_slot; a.error_flag = error_flag;
    a.x_stride = x_stride; a.out_stride = out_stride;
    a.S = nseqs; a.C = channels; a.W = width; a.silu = activation;
    a.num_slots = (conv_states != nullptr || width == 1) ? num_slots : 0;   // (width 1 keeps no rows)
    return ssd::launch_conv1d_step(a, in_dtype == SSD_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_group_norm(const void *x, int64_t x_stride, const void *z, int64_t z_stride, const float *weight,
                          const float *bias, ssd_dtype in_dtype, int32_t rows, int32_t channels, int32_t ngroups,
                          float eps, int32_t center, ssd_norm_act act, void *out, int64_t out_stride,
                          void *stream) {
    if (!known_dtype(in_dtype)) return SSD_ERR_DTYPE;
    if (rows < 0 || channels <= 0 || ngroups <= 0 || channels % ngroups != 0 || !(eps >= 0.0f))
        return SSD_ERR_SHAPE;
    if (act < SSD_NORM_NONE || act > SSD_NORM_GATE_LAST || channels / ngroups > ssd::kNormMaxGroup)
        return SSD_ERR_UNSUPPORTED;
    const bool gated = act == SSD_NORM_GATE_FIRST || act == SSD_NORM_GATE_LAST;
    if (rows > 0 && (x == nullptr || out == nullptr || (gated && z == nullptr))) return SSD_ERR_NULL_ARG;
    if (rows > 0 && (!row_stride(x_stride, channels) || !row_stride(out_stride, channels) ||
                     (gated && !row_stride(z_stride, channels))))
        return SSD_ERR_SHAPE;
    for (const void *p : {x, gated ? z : nullptr, (const void *)out})
        if (!aligned_to(p, elem_bytes(in_dtype))) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)weight, (const void *)bias})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    if (rows == 0) return SSD_OK;
    ssd::NormArgs a{};
    a.x = x; a.z = gated ? z : nullptr; a.weight = weight; a.bias = bias; a.out = out;
    a.x_stride = x_stride; a.z_stride = z_stride; a.out_stride = out_stride;
    a.rows = rows; a.groups = ngroups; a.size = channels / ngroups;
    a.eps = eps; a.center = center != 0; a.act = act;
    return ssd::launch_group_norm(a, in_dtype == SSD_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_gated_delta_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                int64_t v_stride, const void *gate, int64_t gate_stride, const void *beta,
                                int64_t beta_stride, const float *A, const float *dt_bias, float qk_eps, float scale,
                                ssd_dtype in_dtype, ssd_dtype gate_dtype, int32_t nseqs, int32_t total_tokens,
                                const int32_t *cu_seqlens, int32_t nheads, int32_t nkheads, int32_t dk, int32_t dv,
                                float *state_cache, int32_t num_slots, const int32_t *read_slot,
                                const int32_t *write_slot, void *o, int64_t o_stride, int32_t *error_flag,
                                void *stream) {
    if (!known_dtype(in_dtype) || !known_dtype(gate_dtype)) return SSD_ERR_DTYPE;
    if (nseqs < 0 || total_tokens < 0 || total_tokens > (1 << 30) || num_slots < 0 || nheads <= 0 || nkheads <= 0 ||
        dk <= 0 || dv <= 0 || nheads % nkheads != 0 || qk_eps != qk_eps || scale != scale)
        return SSD_ERR_SHAPE;
    if (cu_seqlens == nullptr && total_tokens != nseqs) return SSD_ERR_SHAPE;
    if (!(dk == 64 || dk == 128 || dk == 256)) return SSD_ERR_UNSUPPORTED;
    if (nseqs == 0 || total_tokens == 0) return SSD_OK;
    if (q == nullptr || k == nullptr || v == nullptr || gate == nullptr || beta == nullptr || o == nullptr ||
        state_cache == nullptr || read_slot == nullptr || write_slot == nullptr)
        return SSD_ERR_NULL_ARG;
    const int64_t keys = (int64_t)nkheads * dk, values = (int64_t)nheads * dv;
    if (!row_stride(q_stride, keys) || !row_stride(k_stride, keys) || !row_stride(v_stride, values) ||
        !row_stride(o_stride, values) || !row_stride(gate_stride, nheads) || !row_stride(beta_stride, nheads))
        return SSD_ERR_SHAPE;
    for (const void *p : {q, k, v, (const void *)o})
        if (!aligned_to(p, elem_bytes(in_dtype))) return SSD_ERR_SHAPE;
    for (const void *p : {gate, beta})
        if (!aligned_to(p, elem_bytes(gate_dtype))) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)A, (const void *)dt_bias})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    if (!aligned16(state_cache)) return SSD_ERR_SHAPE;
    ssd::GdnStepArgs a{};
    a.q = q; a.k = k; a.v = v; a.gate = gate; a.beta = beta; a.A = A; a.dt_bias = dt_bias;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.gate_stride = gate_stride;
    a.beta_stride = beta_stride; a.o_stride = o_stride;
    a.qk_eps = qk_eps; a.scale = scale; a.cu_seqlens = cu_seqlens; a.cache = state_cache;
    a.read_slot = read_slot; a.write_slot = write_slot; a.o = o; a.error_flag = error_flag;
    a.S = nseqs; a.T = total_tokens; a.H = nheads; a.G = nkheads; a.dv = dv; a.num_slots = num_slots;
    return ssd::launch_gdn_step(a, in_dtype == SSD_BF16, gate_dtype == SSD_BF16, dk,
                                static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_step_tables(int32_t nseqs, int32_t total_tokens, const int32_t *num_computed, const int32_t *num_new,
                           const int32_t *rows, int32_t *block_table, int32_t table_rows, int32_t max_blocks,
                           int32_t block_size, int32_t num_blocks, const int32_t *free_blocks, int32_t num_free,
                           const int32_t *free_count, int32_t *free_count_out, int32_t *cu_seqlens,
                           int32_t *seq_lens, int32_t *positions, int32_t *token_seq, int32_t *slots,
                           int32_t *read_slot, int32_t *state_slot, int32_t *error_flag, void *stream) {
    constexpr int32_t most = 1 << 20;
    if (nseqs < 0 || nseqs > most || total_tokens < 0 || total_tokens > most || table_rows < 0 || max_blocks < 0 ||
        max_blocks > most || num_blocks < 0 || num_free < 0 || num_free > (1 << 29))
        return SSD_ERR_SHAPE;
    if (block_size < 1) return SSD_ERR_BLOCK_SIZE;
    if ((int64_t)num_blocks * block_size > INT32_MAX) return SSD_ERR_SHAPE;
    if (cu_seqlens == nullptr || (free_blocks != nullptr && (free_count == nullptr || free_count_out == nullptr)))
        return SSD_ERR_NULL_ARG;
    if (nseqs > 0 && (num_computed == nullptr || num_new == nullptr || seq_lens == nullptr || read_slot == nullptr ||
                      (block_table == nullptr && table_rows > 0 && max_blocks > 0)))
        return SSD_ERR_NULL_ARG;
    if (total_tokens > 0 && (positions == nullptr || token_seq == nullptr || slots == nullptr || state_slot == nullptr))
        return SSD_ERR_NULL_ARG;
    for (const void *p : {(const void *)num_computed, (const void *)num_new, (const void *)rows,
                          (const void *)block_table, (const void *)free_blocks, (const void *)free_count,
                          (const void *)free_count_out, (const void *)cu_seqlens, (const void *)seq_lens,
                          (const void *)positions, (const void *)token_seq, (const void *)slots,
                          (const void *)read_slot, (const void *)state_slot, (const void *)error_flag})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    ssd::TablesArgs a{};
    a.num_computed = num_computed; a.num_new = num_new; a.rows = rows; a.block_table = block_table;
    a.free_blocks = free_blocks; a.free_count = free_count; a.free_count_out = free_blocks ? free_count_out : nullptr;
    a.cu_seqlens = cu_seqlens; a.seq_lens = seq_lens; a.positions = positions; a.token_seq = token_seq;
    a.slots = slots; a.read_slot = read_slot; a.state_slot = state_slot; a.error_flag = error_flag;
    a.S = nseqs; a.T = total_tokens; a.table_rows = table_rows; a.max_blocks = max_blocks; a.block = block_size;
    a.num_blocks = num_blocks; a.num_free = num_free;
    return ssd::launch_step_tables(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_kv_cache_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, ssd_dtype dtype,
                              int32_t total_tokens, int32_t nkvheads, int32_t head_dim, void *k_cache, void *v_cache,
                              int32_t num_blocks, int32_t block_size, const int32_t *slots, int32_t *error_flag,
                              void *stream) {
    if (!known_dtype(dtype)) return SSD_ERR_DTYPE;
    if (total_tokens < 0) return SSD_ERR_SHAPE;
    const ssd_status st = check_paged(nkvheads, head_dim, num_blocks, block_size);
    if (st != SSD_OK) return st;
    if (total_tokens == 0) return SSD_OK;
    if (k == nullptr || v == nullptr || slots == nullptr || (num_blocks > 0 && (k_cache == nullptr || v_cache == nullptr)))
        return SSD_ERR_NULL_ARG;
    const int64_t row = (int64_t)nkvheads * head_dim;
    if (!row_stride(k_stride, row) || !row_stride(v_stride, row)) return SSD_ERR_SHAPE;
    for (const void *p : {k, v})
        if (!aligned_to(p, elem_bytes(dtype))) return SSD_ERR_SHAPE;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned_to(slots, 4)) return SSD_ERR_SHAPE;
    ssd::KvWriteArgs a{};
    a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride; a.k_cache = k_cache; a.v_cache = v_cache;
    a.slots = slots; a.error_flag = error_flag;
    a.T = total_tokens; a.Hkv = nkvheads; a.D = head_dim; a.block = block_size; a.num_slots = num_blocks * block_size;
    return ssd::launch_kv_write(a, dtype == SSD_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK
                                                                                                     : SSD_ERR_HIP;
}

ssd_status ssd_attention_plan_build(const ssd_attention_plan *plan, void *stream) {
    const ssd_status st = check_plan(plan);
    if (st != SSD_OK) return st;
    ssd::AttnPlanArgs a{};
    a.seq_lens = plan->seq_lens; a.cu_seqlens = plan->cu_seqlens; a.part_start = plan->part_start;
    a.part_seq = plan->part_seq; a.part_keys = plan->part_keys; a.error_flag = plan->error_flag;
    a.S = plan->nseqs; a.T = plan->total_tokens; a.max_new = plan->max_new_tokens; a.window = attention_window(plan);
    a.max_parts = plan->max_parts;
    return ssd::launch_attention_plan(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

int32_t ssd_paged_attention_parts(int32_t max_new_tokens, int32_t nheads, int32_t nkvheads) {
    if (max_new_tokens <= 0 || nheads <= 0 || nkvheads <= 0 || nheads % nkvheads != 0) return 0;
    const int64_t per_part = nkvheads * attention_tiles(max_new_tokens, nheads / nkvheads);
    return (int32_t)((ssd::kAttnWorkgroups + per_part - 1) / per_part);
}

size_t ssd_paged_attention_workspace_size(int32_t max_parts, int32_t max_new_tokens, int32_t nheads, int32_t head_dim) {
    if (max_parts <= 0 || max_new_tokens <= 0 || nheads <= 0 || head_dim <= 0) return 0;
    return (size_t)max_parts * (size_t)max_new_tokens * (size_t)nheads * ((size_t)head_dim + 2) * sizeof(float);
}

ssd_status ssd_paged_attention_step(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                                    ssd_dtype dtype, float scale, const ssd_attention_plan *plan, int32_t nheads,
                                    int32_t nkvheads, int32_t head_dim, const int32_t *block_table,
                                    int32_t table_rows, int32_t max_blocks, const int32_t *rows, int32_t num_blocks,
                                    int32_t block_size, void *out, int64_t out_stride, float *lse, void *workspace,
                                    size_t workspace_bytes, int32_t *error_flag, void *stream) {
    ssd_status st = check_plan(plan);
    if (st != SSD_OK) return st;
    if (!known_dtype(dtype)) return SSD_ERR_DTYPE;
    if (nheads <= 0 || nkvheads <= 0 || nheads % nkvheads != 0 || table_rows < 0 || max_blocks < 0 || scale != scale)
        return SSD_ERR_SHAPE;
    st = check_paged(nheads, head_dim, num_blocks, block_size);
    if (st != SSD_OK) return st;
    if (block_size > (1 << 20)) return SSD_ERR_BLOCK_SIZE;
    if (plan->nseqs == 0 || plan->total_tokens == 0) return SSD_OK;
    if (q == nullptr || out == nullptr || (num_blocks > 0 && (k_cache == nullptr || v_cache == nullptr)) ||
        (table_rows > 0 && max_blocks > 0 && block_table == nullptr))
        return SSD_ERR_NULL_ARG;
    const int64_t row = (int64_t)nheads * head_dim;
    if (!row_stride(q_stride, row) || !row_stride(out_stride, row)) return SSD_ERR_SHAPE;
    for (const void *p : {q, (const void *)out})
        if (!aligned_to(p, elem_bytes(dtype))) return SSD_ERR_SHAPE;
    for (const void *p : {k_cache, v_cache, (const void *)workspace})
        if (!aligned16(p)) return SSD_ERR_SHAPE;
    for (const void *p : {(const void *)block_table, (const void *)rows, (const void *)lse})
        if (!aligned_to(p, 4)) return SSD_ERR_SHAPE;
    const size_t parts = (size_t)plan->max_parts * plan->max_new_tokens * nheads;
    if (workspace == nullptr ||
        workspace_bytes < ssd_paged_attention_workspace_size(plan->max_parts, plan->max_new_tokens, nheads, head_dim))
        return SSD_ERR_CAPACITY;
    ssd::AttnArgs a{};
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.q_stride = q_stride; a.out_stride = out_stride;
    a.seq_lens = plan->seq_lens; a.cu_seqlens = plan->cu_seqlens; a.part_start = plan->part_start;
    a.part_seq = plan->part_seq; a.part_keys = plan->part_keys; a.block_table = block_table; a.rows = rows;
    a.out = out; a.lse = lse;
    a.part_o = static_cast<float *>(workspace); a.part_ml = a.part_o + parts * head_dim;
    a.error_flag = error_flag; a.scale_log2 = scale * 1.4426950408889634f;
    a.S = plan->nseqs; a.T = plan->total_tokens; a.max_new = plan->max_new_tokens; a.window = attention_window(plan);
    a.max_parts = plan->max_parts; a.Hq = nheads; a.Hkv = nkvheads; a.group = nheads / nkvheads;
    a.tiles = (int32_t)attention_tiles(plan->max_new_tokens, a.group);   // (64 tokens of 2^26 / 64 heads at most)
    // no cache, no table: no keys
    a.table_rows = num_blocks > 0 && max_blocks > 0 ? table_rows : 0;
    a.max_blocks = max_blocks; a.num_blocks = num_blocks; a.block = block_size;
    // exact division of 31-bit keys: 2^(31+L) / block rounded up has 32 bits, L = ceil(log2(block))
    uint32_t L = 1;
    while ((INT64_C(1) << L) < block_size) ++L;
    a.block_magic = (uint32_t)(((UINT64_C(1) << (31 + L)) + block_size - 1) / block_size);
    a.block_shift = L - 1;
    return ssd::launch_attention(a, dtype == SSD_BF16, head_dim, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_add_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                            const float *weight, ssd_dtype in_dtype, int32_t rows, int32_t channels, float eps,
                            void *residual_out, int64_t residual_out_stride, void *out, int64_t out_stride,
                            void *stream) {
    ssd::AddNormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out; a.out = out;
    a.x_stride = x_stride; a.residual_stride = residual_stride; a.residual_out_stride = residual_out_stride;
    a.out_stride = out_stride; a.rows = rows; a.channels = channels; a.group = channels; a.eps = eps;
    const ssd_status st = check_add_norm(a, in_dtype);
    if (st != SSD_OK || rows == 0) return st;
    if (!aligned_to(out, elem_bytes(in_dtype))) return SSD_ERR_SHAPE;
    return ssd::launch_add_rms_norm(a, in_dtype == SSD_BF16, false, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

ssd_status ssd_add_rms_norm_e4m3(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                                 const float *weight, ssd_dtype in_dtype, int32_t rows, int32_t channels,
                                 int32_t group, float eps, const float *scale, float *scales, void *residual_out,
                                 int64_t residual_out_stride, void *out, int64_t out_stride, void *stream) {
    ssd::AddNormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out; a.out = out;
    a.scale = scale; a.scales = scales;
    a.x_stride = x_stride; a.residual_stride = residual_stride; a.residual_out_stride = residual_out_stride;
    a.out_stride = out_stride; a.rows = rows; a.channels = channels; a.group = group; a.eps = eps;
    const ssd_status st = check_add_norm(a, in_dtype);
    if (st != SSD_OK) return st;
    if (group != channels && !((group == 32 || group == 64 || group == 128 || group == 256 || group == 512) &&
                               channels % group == 0))
        return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    if (scale == nullptr && scales == nullptr) return SSD_ERR_NULL_ARG;
    if (!aligned_to(scale, 4) || !aligned_to(scales, 4)) return SSD_ERR_SHAPE;
    return ssd::launch_add_rms_norm(a, in_dtype == SSD_BF16, true, static_cast<hipStream_t>(stream)) == hipSuccess
               ? SSD_OK : SSD_ERR_HIP;
}

}  // extern "C"
