// What the norms share: vectors of values in memory, and sums over a team of lanes.
#pragma once

#include "ssd_scan.hpp"

namespace ssd {

// V consecutive values of type T in memory.
template <typename T, int V> struct NormIO;
template <> struct NormIO<__bf16, 8> {
    struct __attribute__((aligned(16))) Raw { uint32_t w[4]; };
    __device__ static void unpack(const Raw &r, float *v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(r.w[i]);
            v[2 * i + 1] = bf16_hi(r.w[i]);
        }
    }
    __device__ static Raw pack(const float *v) {
        Raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        return r;
    }
};
template <> struct NormIO<float, 4> {
    struct __attribute__((aligned(16))) Raw { float w[4]; };
    __device__ static void unpack(const Raw &r, float *v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r.w[i];
    }
    __device__ static Raw pack(const float *v) { return Raw{{v[0], v[1], v[2], v[3]}}; }
};
template <> struct NormIO<__bf16, 2> {
    struct Raw { uint32_t w; };
    __device__ static void unpack(const Raw &r, float *v) {
        v[0] = bf16_lo(r.w);
        v[1] = bf16_hi(r.w);
    }
    __device__ static Raw pack(const float *v) { return Raw{pack_bf16(v[0], v[1])}; }
};
template <typename T> struct NormIO<T, 1> {
    using Raw = T;
    __device__ static void unpack(const Raw &r, float *v) { *v = (float)r; }
    __device__ static Raw pack(const float *v) { return (T)*v; }
};

// Sum over a team; every lane gets it. A team of several waves is a workgroup.
template <int TEAM> __device__ __forceinline__ float team_sum(float v, float *part) {
#pragma unroll
    for (int m = (TEAM < 64 ? TEAM : 64) / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (TEAM > 64) {
        __syncthreads();   // the sums before have been read
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TEAM / 64; ++w) v += part[w];
    }
    return v;
}

}  // namespace ssd
