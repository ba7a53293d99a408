// Norm of groups of channels with an activation, channels last:
//   v = x (or x silu(z));  mu = mean(v) or 0;  out = (v - mu) / sqrt(mean((v - mu)^2) + eps) w + b,
// then SiLU or a gate silu(z). One token's group at a time.
#include "ssd_scan.hpp"

namespace ssd {

constexpr int kNormThreads = 256;

template <typename T> __device__ __forceinline__ float norm_load(const void *p, int64_t i) {
    return (float)reinterpret_cast<const T *>(p)[i];
}

__device__ __forceinline__ float norm_silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

// Sum over the workgroup (every thread gets it).
__device__ __forceinline__ float block_sum(float v, float *part) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 64; ++w) sum += part[w];
    return sum;
}

template <typename T>
__global__ __launch_bounds__(kNormThreads) void ssd_group_norm_kernel(NormArgs a) {
    __shared__ float part[kNormThreads / 64];
    const int64_t row = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x - row * a.groups) * a.size;
    const int64_t xo = row * a.x_stride + c0, zo = row * a.z_stride + c0, oo = row * a.out_stride + c0;
    auto value = [&](int i) {
        const float v = norm_load<T>(a.x, xo + i);
        return a.act == SSD_NORM_GATE_FIRST ? v * norm_silu(norm_load<T>(a.z, zo + i)) : v;
    };
    float sum = 0.0f, sq = 0.0f, mu = 0.0f;
    if (a.center) {
        for (int i = threadIdx.x; i < a.size; i += kNormThreads) sum += value(i);
        mu = block_sum(sum, part) / (float)a.size;
    }
    for (int i = threadIdx.x; i < a.size; i += kNormThreads) {
        const float v = value(i) - mu;
        sq = fmaf(v, v, sq);
    }
    const float scale = 1.0f / sqrtf(block_sum(sq, part) / (float)a.size + a.eps);
    for (int i = threadIdx.x; i < a.size; i += kNormThreads) {
        float v = (value(i) - mu) * scale;
        if (a.weight != nullptr) v *= a.weight[c0 + i];
        if (a.bias != nullptr) v += a.bias[c0 + i];
        if (a.act == SSD_NORM_SILU) v = norm_silu(v);
        if (a.act == SSD_NORM_GATE_LAST) v *= norm_silu(norm_load<T>(a.z, zo + i));
        reinterpret_cast<T *>(a.out)[oo + i] = (T)v;
    }
}

hipError_t launch_group_norm(const NormArgs &a, bool bf16, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.rows * a.groups)), block(kNormThreads);
    if (bf16) hipLaunchKernelGGL(ssd_group_norm_kernel<__bf16>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(ssd_group_norm_kernel<float>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace ssd
