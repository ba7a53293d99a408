// Selective scan with a decay per channel and state, and its single-token step.
//   delta  = softplus(dt[t,d] + dt_bias[d])
//   h[d,n] = 2^(delta A[d,n] log2 e) h[d,n] + delta u[t,d] B[t,g,n]
//   y[t,d] = (sum_n h[d,n] C[t,g,n] + D[d] u[t,d]) silu(z[t,d])
//
// The decay differs per (token, channel, state), so a chunk has no form as a
// matrix product (a per-head decay has one): what there is to compute is one
// exponential and a few products and sums per (token, channel, state).
//
// Lanes: a wave owns 16 channels; lane = 16 q + c holds the states
// n = q N/4 .. (q + 1) N/4 - 1 of channel c.
#include "ssd_scan.hpp"

namespace ssd {

// log(1 + e^v) in float32. For small e^v the logarithm's own argument 1 + e^v
// has lost the digits that count, so its series is summed instead
// (z <= 1/8: the first term left out is below z^7/8 = 6e-8 of the result).
__device__ __forceinline__ float softplus_full(float v) {
    const float z = fast_exp2(-fabsf(v) * kLog2e);
    const float big = __builtin_amdgcn_logf(1.0f + z) * 0.6931471805599453f;
    float p = fmaf(z, 1.0f / 7.0f, -1.0f / 6.0f);
    p = fmaf(z, p, 1.0f / 5.0f);
    p = fmaf(z, p, -1.0f / 4.0f);
    p = fmaf(z, p, 1.0f / 3.0f);
    p = fmaf(z, p, -1.0f / 2.0f);
    p = fmaf(z, p, 1.0f);
    return fmaxf(v, 0.0f) + (z <= 0.125f ? z * p : big);
}

__device__ __forceinline__ float silu_full(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

template <typename T> __device__ __forceinline__ float load_f(const void *p, int64_t i) {
    return (float)reinterpret_cast<const T *>(p)[i];
}

template <typename T, typename DT, int N>
__global__ __launch_bounds__(64) void ssd_selective_scan_kernel(SelectiveArgs a) {
    constexpr int NB = N / 4;   // states of a lane
    if (__builtin_nontemporal_load(a.error_flag) & SSD_DATA_BAD_CU_SEQLENS) return;
    const int cblocks = (a.C_total + 15) / 16;
    const int rank = blockIdx.x / cblocks, cb = blockIdx.x - rank * cblocks;
    const int s = a.seq_order[rank];
    if (s < 0 || s >= a.S) return;
    int64_t tb = a.cu_seqlens[s], te = a.cu_seqlens[s + 1];
    tb = tb < 0 ? 0 : (tb > a.T ? a.T : tb);
    te = te < tb ? tb : (te > a.T ? a.T : te);
    const int L = (int)(te - tb), c0 = a.seq_chunk_start[s];
    const int lane = threadIdx.x, q = lane >> 4, ch = cb * 16 + (lane & 15);
    const bool live = ch < a.C_total;
    const int d = live ? ch : a.C_total - 1;
    const int g = d / (a.C_total / a.G);
    const int64_t row = ((int64_t)s * a.C_total + d) * N + q * NB;

    float h[NB], a2[NB];
    const bool start = a.init != nullptr && (a.has_init == nullptr || a.has_init[s] != 0);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        a2[i] = a.A[(int64_t)d * N + q * NB + i] * kLog2e;
        h[i] = start ? a.init[row + i] : 0.0f;
    }
    const float bias = a.dt_bias != nullptr ? a.dt_bias[d] : 0.0f, skip = a.D != nullptr ? a.D[d] : 0.0f;
    for (int t = 0; t < L; ++t) {
        const int64_t tok = tb + t;
        const float u = load_f<T>(a.u, tok * a.u_stride + d);
        const float delta = softplus_full(load_f<DT>(a.dt, tok * a.dt_stride + d) + bias);
        const float du = delta * u;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int n = g * N + q * NB + i;
            h[i] = fmaf(fast_exp2(delta * a2[i]), h[i], du * load_f<T>(a.B, tok * a.B_stride + n));
            y = fmaf(h[i], load_f<T>(a.C, tok * a.C_stride + n), y);
        }
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        y = fmaf(skip, u, y);
        if (a.z != nullptr) y *= silu_full(load_f<T>(a.z, tok * a.z_stride + d));
        if (live && q == 0) reinterpret_cast<T *>(a.y)[tok * a.y_stride + d] = (T)y;
        if (a.chunk_states != nullptr && ((t + 1) % a.cs == 0 || t + 1 == L)) {
            const int chunk = c0 + t / a.cs;
            const int slot = a.chunk_state_dst != nullptr ? a.chunk_state_dst[chunk] : chunk;
            if (slot >= a.capacity) {
                if (lane == 0 && cb == 0) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
            } else if (slot >= 0 && live) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    a.chunk_states[((int64_t)slot * a.C_total + d) * N + q * NB + i] = h[i];
            }
        }
    }
    if (live)
#pragma unroll
        for (int i = 0; i < NB; ++i) a.final_states[row + i] = h[i];
}

// Step: lanes own 4 consecutive states of one channel (N / 4 lanes a channel).
constexpr int kSelStepThreads = 256;

template <typename T, typename DT, int N>
__global__ __launch_bounds__(kSelStepThreads) void ssd_selective_step_kernel(SelectiveArgs a, int64_t items) {
    constexpr int LPC = N / 4;   // lanes of a channel
    for (int64_t id = (int64_t)blockIdx.x * kSelStepThreads + threadIdx.x; id < items;
         id += (int64_t)gridDim.x * kSelStepThreads) {
        const int64_t sc = id / LPC;
        const int nq = (int)(id - sc * LPC);
        const int s = (int)(sc / a.C_total), d = (int)(sc - (int64_t)s * a.C_total);
        const int rs = a.read_slot[s], ws = a.write_slot[s];
        if (rs >= a.num_slots || ws >= a.num_slots) {   // refused: nothing read or written
            if (d == 0 && nq == 0 && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
            continue;   // whole channels, so whole shuffle groups, leave together
        }
        const int g = d / (a.C_total / a.G);
        const int64_t slot = (int64_t)a.C_total * N, at = (int64_t)d * N + 4 * nq;
        f32x4 h = rs >= 0 ? *reinterpret_cast<const f32x4 *>(a.cache + rs * slot + at) : f32x4{0, 0, 0, 0};
        const f32x4 rate = *reinterpret_cast<const f32x4 *>(a.A + at);
        const float u = load_f<T>(a.u, s * a.u_stride + d);
        const float delta = softplus_full(load_f<DT>(a.dt, s * a.dt_stride + d) + (a.dt_bias ? a.dt_bias[d] : 0.0f));
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = g * N + 4 * nq + i;
            h[i] = fmaf(fast_exp2(delta * (rate[i] * kLog2e)), h[i],
                        delta * u * load_f<T>(a.B, s * a.B_stride + n));
            y = fmaf(h[i], load_f<T>(a.C, s * a.C_stride + n), y);
        }
        if (ws >= 0) *reinterpret_cast<f32x4 *>(a.cache + ws * slot + at) = h;
#pragma unroll
        for (int m = LPC / 2; m >= 1; m >>= 1) y += __shfl_xor(y, m, LPC);
        if (nq == 0) {
            y = fmaf(a.D != nullptr ? a.D[d] : 0.0f, u, y);
            if (a.z != nullptr) y *= silu_full(load_f<T>(a.z, s * a.z_stride + d));
            reinterpret_cast<T *>(a.y)[s * a.y_stride + d] = (T)y;
        }
    }
}

template <typename T, typename DT, int N> struct SelectiveLaunch {
    static hipError_t scan(const SelectiveArgs &a, hipStream_t stream) {
        const int64_t blocks = (int64_t)a.S * ((a.C_total + 15) / 16);
        hipLaunchKernelGGL((ssd_selective_scan_kernel<T, DT, N>), dim3((unsigned)blocks), dim3(64), 0, stream, a);
        return hipGetLastError();
    }
    static hipError_t step(const SelectiveArgs &a, hipStream_t stream) {
        const int64_t items = (int64_t)a.S * a.C_total * (N / 4);
        const int64_t want = (items + kSelStepThreads - 1) / kSelStepThreads;
        const unsigned blocks = (unsigned)(want < (1 << 20) ? want : (1 << 20));
        hipLaunchKernelGGL((ssd_selective_step_kernel<T, DT, N>), dim3(blocks), dim3(kSelStepThreads), 0, stream, a,
                           items);
        return hipGetLastError();
    }
};

template <typename T, typename DT, typename F> static hipError_t selective_for(int N, F &&f) {
    switch (N) {
        case 16: return f(SelectiveLaunch<T, DT, 16>{});
        case 32: return f(SelectiveLaunch<T, DT, 32>{});
        case 64: return f(SelectiveLaunch<T, DT, 64>{});
        case 128: return f(SelectiveLaunch<T, DT, 128>{});
        case 256: return f(SelectiveLaunch<T, DT, 256>{});
        default: return hipErrorInvalidValue;
    }
}

template <typename F> static hipError_t selective_typed(int N, bool bf16, bool dt_bf16, F &&f) {
    if (bf16) return dt_bf16 ? selective_for<__bf16, __bf16>(N, f) : selective_for<__bf16, float>(N, f);
    return dt_bf16 ? selective_for<float, __bf16>(N, f) : selective_for<float, float>(N, f);
}

hipError_t launch_selective_scan(const SelectiveArgs &a, bool bf16, bool dt_bf16, hipStream_t stream) {
    return selective_typed(a.N, bf16, dt_bf16, [&](auto l) { return decltype(l)::scan(a, stream); });
}

hipError_t launch_selective_step(const SelectiveArgs &a, bool bf16, bool dt_bf16, hipStream_t stream) {
    return selective_typed(a.N, bf16, dt_bf16, [&](auto l) { return decltype(l)::step(a, stream); });
}

}  // namespace ssd
