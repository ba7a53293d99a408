// RMS norm of rows with the residual's addition before it, and an output in the
// inputs' type or in 8 bits (e4m3) with scales:
//   r = x + residual;  n = r / sqrt(mean(r^2) + eps) w;
//   out = n,  or  out = e4m3(n / s) with s = max |n| / 448 over the row or over
//   groups of channels (1 where all are zero), or with a given s.
// The norm takes r before its rounding to residual_out.
//
// Memory-bound: x, the residual and the outputs pass once; a row stays in the
// registers of one workgroup (lane l holds vectors l, l + THREADS, ..) between
// the loads, the sum of squares, the maxima and the stores.
#include "ssd_norm.hpp"

namespace ssd {

constexpr float kE4m3Max = 448.0f;

// e4m3 of four values, clamped to the largest (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    auto clamp = [](float v) { return v != v ? v : fminf(fmaxf(v, -kE4m3Max), kE4m3Max); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(a), clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(c), clamp(d), w, true);
}

template <typename T, int THREADS, int V, int R, bool Q>
__global__ __launch_bounds__(THREADS) void ssd_add_rms_norm_kernel(AddNormArgs a) {
    using IO = NormIO<T, V>;
    using Raw = typename IO::Raw;
    constexpr int SPAN = THREADS * V;
    __shared__ float part[THREADS / 64];
    __shared__ uint32_t top[Q ? kNormMaxGroup / 32 : 1];   // bits of the groups' largest absolute values
    const int tid = threadIdx.x, C = a.channels;
    const int64_t row = blockIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride;
    const T *res = a.residual ? reinterpret_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
    T *res_out = a.residual_out ? reinterpret_cast<T *>(a.residual_out) + row * a.residual_out_stride : nullptr;
    auto at = [&](int r) { return r * SPAN + tid * V; };
    Raw rx[R], rr[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (at(r) < C) {
            rx[r] = *reinterpret_cast<const Raw *>(x + at(r));
            if (res) rr[r] = *reinterpret_cast<const Raw *>(res + at(r));
        }
    if constexpr (Q)
        if (a.scale == nullptr)
            for (int i = tid; i < C / a.group; i += THREADS) top[i] = 0;
    float v[R * V], sq = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[r * V + i] = 0.0f;
        if (at(r) >= C) continue;
        IO::unpack(rx[r], v + r * V);
        if (res) {
            float y[V];
            IO::unpack(rr[r], y);
#pragma unroll
            for (int i = 0; i < V; ++i) v[r * V + i] += y[i];
        }
        if (res_out) *reinterpret_cast<Raw *>(res_out + at(r)) = IO::pack(v + r * V);
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(v[r * V + i], v[r * V + i], sq);
    }
    const float inv = 1.0f / sqrtf(team_sum<THREADS>(sq, part) / (float)C + a.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (at(r) >= C) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) v[r * V + i] *= inv * (a.weight ? a.weight[at(r) + i] : 1.0f);
        if constexpr (!Q) *reinterpret_cast<Raw *>(reinterpret_cast<T *>(a.out) + row * a.out_stride + at(r)) = IO::pack(v + r * V);
    }
    if constexpr (Q) {
        uint8_t *out = reinterpret_cast<uint8_t *>(a.out) + row * a.out_stride;
        if (a.scale == nullptr) {
            // (absolute values compare as their bits do, a NaN above all)
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (at(r) >= C) continue;
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[r * V + i]) & 0x7fffffffu);
                atomicMax(&top[at(r) / a.group], m);
            }
            __syncthreads();
            for (int i = tid; i < C / a.group; i += THREADS) {
                const float t = __uint_as_float(top[i]);
                a.scales[row * (C / a.group) + i] = t == 0.0f ? 1.0f : t / kE4m3Max;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (at(r) >= C) continue;
            float s;
            if (a.scale != nullptr) {
                s = *a.scale;
            } else {
                const float t = __uint_as_float(top[at(r) / a.group]);
                s = t == 0.0f ? 1.0f : t / kE4m3Max;
            }
            if constexpr (V >= 4) {
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    *reinterpret_cast<uint32_t *>(out + at(r) + i) =
                        pack_e4m3(v[r * V + i] / s, v[r * V + i + 1] / s, v[r * V + i + 2] / s, v[r * V + i + 3] / s);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) out[at(r) + i] = (uint8_t)pack_e4m3(v[r * V + i] / s, 0.0f, 0.0f, 0.0f);
            }
        }
    }
}

template <typename T, int THREADS, int V, bool Q> static hipError_t launch_addnorm_threads(const AddNormArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((ssd_add_rms_norm_kernel<T, THREADS, V, 16 / V, Q>), dim3((unsigned)a.rows), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int V, bool Q> static hipError_t launch_addnorm_v(const AddNormArgs &a, hipStream_t stream) {
    if (a.channels <= 256 * 16) return launch_addnorm_threads<T, 256, V, Q>(a, stream);
    return launch_addnorm_threads<T, 1024, V, Q>(a, stream);
}

template <typename T, bool Q> static hipError_t launch_addnorm_t(const AddNormArgs &a, hipStream_t stream) {
    const uint64_t rows = (uint64_t)(a.x_stride | (a.residual ? a.residual_stride : 0) |
                                     (a.residual_out ? a.residual_out_stride : 0) | (Q ? 0 : a.out_stride) | a.channels);
    const uint64_t starts = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                            reinterpret_cast<uintptr_t>(a.residual_out) | (Q ? 0 : reinterpret_cast<uintptr_t>(a.out)) |
                            rows * sizeof(T);
    const uint64_t codes = Q ? reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.out_stride : 0;   // whole words of 8-bit values
    if (starts % 16 == 0 && codes % 4 == 0) return launch_addnorm_v<T, 16 / sizeof(T), Q>(a, stream);
    return launch_addnorm_v<T, 1, Q>(a, stream);
}

hipError_t launch_add_rms_norm(const AddNormArgs &a, bool bf16, bool e4m3, hipStream_t stream) {
    if (bf16) return e4m3 ? launch_addnorm_t<__bf16, true>(a, stream) : launch_addnorm_t<__bf16, false>(a, stream);
    return e4m3 ? launch_addnorm_t<float, true>(a, stream) : launch_addnorm_t<float, false>(a, stream);
}

}  // namespace ssd
