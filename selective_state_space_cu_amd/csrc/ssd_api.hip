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

}  // namespace

extern "C" {

const char *ssd_status_string(ssd_status status) {
    switch (status) {
    case SSD_OK: return "ok";
    case SSD_ERR_NULL_ARG: return "a required pointer is NULL";
    case SSD_ERR_CHUNK_SIZE: return "chunk_size must be a power of two in [16, 256]";
    case SSD_ERR_SHAPE: return "invalid sizes, nheads % ngroups != 0, or a pointer not 16-byte aligned";
    case SSD_ERR_BLOCK_SIZE: return "block_size must be a positive multiple of chunk_size";
    case SSD_ERR_CAPACITY: return "capacity below the required bound (max_chunks or chunk_states)";
    case SSD_ERR_DTYPE: return "unknown dtype";
    case SSD_ERR_HIP: return "a HIP call failed";
    case SSD_ERR_UNSUPPORTED: return "unsupported dtype/shape combination (headdim, dstate, dk, dv or chunk size)";
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

}  // extern "C"
