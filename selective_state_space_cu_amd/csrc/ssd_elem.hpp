// Elements of the layers around the scans: values as they lie in memory, softplus and SiLU.
#pragma once

#include "ssd_scan.hpp"

namespace ssd {

// log(1 + e^v) = max(v, 0) + log1p(z), z = e^-|v| in (0, 1]. log1p(z) / z is a
// polynomial of degree 8 fitted over all of (0, 1] for the least relative error
// (with the roundings of its evaluation at most 3.2 * 2^-24): the hardware's
// logarithm of 1 + z has lost the digits of a small z, and costs as much as three sums.
__device__ __forceinline__ float softplus_full(float v) {
    const float z = fast_exp2(-fabsf(v) * kLog2e);
    float p = fmaf(z, 0.0052319662645459175f, -0.029502321034669876f);
    p = fmaf(z, p, 0.07822119444608688f);
    p = fmaf(z, p, -0.1366284191608429f);
    p = fmaf(z, p, 0.1910581737756729f);
    p = fmaf(z, p, -0.2484293431043625f);
    p = fmaf(z, p, 0.33319091796875f);
    p = fmaf(z, p, -0.4999949336051941f);
    p = fmaf(z, p, 1.0f);
    return fmaf(z, p, fmaxf(v, 0.0f));
}

__device__ __forceinline__ float silu_full(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

template <typename T> __device__ __forceinline__ float load_f(const void *p, int64_t i) {
    return (float)reinterpret_cast<const T *>(p)[i];
}

template <typename T> struct RawOf;
template <> struct RawOf<__bf16> {
    using One = uint16_t;
    struct __attribute__((packed, aligned(2))) Four { uint32_t w[2]; };
    __device__ static float f(One v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static f32x4 f4(const Four &v) {
        return f32x4{bf16_lo(v.w[0]), bf16_hi(v.w[0]), bf16_lo(v.w[1]), bf16_hi(v.w[1])};
    }
};
template <> struct RawOf<float> {
    using One = float;
    struct __attribute__((packed, aligned(4))) Four { float w[4]; };
    __device__ static float f(One v) { return v; }
    __device__ static f32x4 f4(const Four &v) { return f32x4{v.w[0], v.w[1], v.w[2], v.w[3]}; }
};

}  // namespace ssd
