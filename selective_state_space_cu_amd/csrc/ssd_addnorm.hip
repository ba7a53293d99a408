// RMS norm of rows with the residual's addition before it, and an output in the
// inputs' type or in 8 bits (e4m3) with scales:
//   r = x + residual;  n = r / sqrt(mean(r^2) + eps) w;
//   out = n,  or  out = e4m3(n / s) with s = max |n| / 448 over the row or over
//   groups of channels (1 where all are zero), or with a given s.
// The norm takes r before its rounding to residual_out.
//
// Memory-bound: x, the residual and the outputs pass once; a row stays in the
// registers of its team of lanes (lane l holds vectors l, l + TEAM, ..) between
// the loads, the sum of squares, the maxima and the stores. 35576 x 4096 bf16 to
// e4m3 in groups of 128 takes 168 to 184 us, 5.6 to 6.1 TB/s (a large copy reaches 5.1).
#include <algorithm>

#include "ssd_norm.hpp"

namespace ssd {

constexpr float kE4m3Max = 448.0f;

// e4m3 of four values, clamped to the largest (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    auto clamp = [](float v) { return v != v ? v : __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(a), clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(c), clamp(d), w, true);
}

// f / scale in float32 for V values, of which those past 512 only stay past it: the product with the reciprocal, whose two
// roundings would move quotients half way between two codes off it, and one step by what it leaves of f. (Divisions would
// be a third more instructions; this and the scales' own division are a seventh: 35576 x 4096 bf16 takes as long as
// without, 35576 x 5120 2 % longer, one row 0.1 us.)
template <int V> __device__ __forceinline__ void divide_all(float *f, float scale) {
    const float per = 1.0f / scale, by = fabsf(scale) == INFINITY ? 0.0f : scale;   // (0 x infinity is no 0)
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float y = __builtin_amdgcn_fmed3f(f[i] * per, -512.0f, 512.0f);   // (what is left of f stays finite)
        f[i] = fmaf(-fmaf(y, by, -f[i]), per, y);
    }
}

// Largest of `lanes` neighbouring lanes (a power of two up to 64, uniform); every lane gets it.
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lanes) {
    auto dpp = [&](auto ctrl) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, true));
    };
    if (lanes > 1) dpp(std::integral_constant<int, 0xB1>{});    // lane ^ 1
    if (lanes > 2) dpp(std::integral_constant<int, 0x4E>{});    // lane ^ 2
    if (lanes > 4) dpp(std::integral_constant<int, 0x141>{});   // 7 - lane of 8
    if (lanes > 8) dpp(std::integral_constant<int, 0x140>{});   // 15 - lane of 16
    if (lanes > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(r[0], r[1]);
    }
    if (lanes > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(r[0], r[1]);
    }
    return v;
}

// Loads and stores of 16 bytes with the streaming policy (narrower ones share their lines and go without).
template <typename Raw> __device__ __forceinline__ Raw load_streamed(const void *p) {
    if constexpr (sizeof(Raw) == 16) return __builtin_bit_cast(Raw, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)));
    else return *reinterpret_cast<const Raw *>(p);
}
template <typename Raw> __device__ __forceinline__ void store_streamed(void *p, const Raw &v) {
    if constexpr (sizeof(Raw) == 16) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4 *>(p));
    else *reinterpret_cast<Raw *>(p) = v;
}

// Where a row's scales come from: none (no 8 bits), a given one, the whole row, groups inside a round of a team's lanes of a
// wave, larger groups.
enum Scales { kNoScale, kGiven, kRowScale, kLaneGroups, kWideGroups };

template <typename T, int TEAM, int V, int R, Scales Q>
__global__ __launch_bounds__(TEAM > 64 ? TEAM : 256) void ssd_add_rms_norm_kernel(AddNormArgs a) {
    using IO = NormIO<T, V>;
    using Raw = typename IO::Raw;
    struct __attribute__((packed, aligned(4))) Weights { float w[V]; };
    constexpr int THREADS = TEAM > 64 ? TEAM : 256, SPAN = TEAM * V, LANES = TEAM < 64 ? TEAM : 64;   // LANES: of a team in a wave
    __shared__ float part[TEAM > 64 ? TEAM / 64 : 1];
    constexpr int TOPS = Q == kWideGroups ? TEAM * 16 / 32 : Q == kRowScale && TEAM > 64 ? TEAM / 64 : 1;   // (groups have 32 channels at least)
    __shared__ uint32_t tops[THREADS / TEAM * TOPS];
    const int lane = threadIdx.x % TEAM, C = a.channels;
    uint32_t *top = tops + threadIdx.x / TEAM * TOPS;
    auto team_sync = [] {   // a wave's LDS operations are in order by themselves
        if constexpr (TEAM > 64) __syncthreads();
        else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    const int64_t row = (int64_t)blockIdx.x * (THREADS / TEAM) + threadIdx.x / TEAM;
    if (row >= a.rows) return;   // (whole teams; a team of more than a wave is a workgroup)
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride + lane * V;
    const T *res = reinterpret_cast<const T *>(a.residual) + row * a.residual_stride + lane * V;
    T *res_out = reinterpret_cast<T *>(a.residual_out) + row * a.residual_out_stride + lane * V;
    auto live = [&](int r) { return r * SPAN + lane * V < C; };
    Raw rx[R], rr[R];
    Weights w[R];
    auto load = [&](auto from) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (live(r)) {
                rx[r] = from(x + r * SPAN);
                if (a.residual) rr[r] = from(res + r * SPAN);
            }
    };
    if (a.stream) load([](const T *at) { return load_streamed<Raw>(at); });
    else load([](const T *at) { return *reinterpret_cast<const Raw *>(at); });
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (live(r)) {
            if (a.weight) w[r] = *reinterpret_cast<const Weights *>(a.weight + r * SPAN + lane * V);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) w[r].w[i] = 1.0f;
        }
    if constexpr (Q == kWideGroups) {
        for (int i = lane; i < C / a.group; i += TEAM) top[i] = 0;
        team_sync();
    }
    float v[R * V], sq = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[r * V + i] = 0.0f;
        if (!live(r)) continue;
        IO::unpack(rx[r], v + r * V);
        if (a.residual) {
            float y[V];
            IO::unpack(rr[r], y);
#pragma unroll
            for (int i = 0; i < V; ++i) v[r * V + i] += y[i];
        }
        if (a.residual_out) {
            if (a.stream) store_streamed(res_out + r * SPAN, IO::pack(v + r * V));
            else *reinterpret_cast<Raw *>(res_out + r * SPAN) = IO::pack(v + r * V);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(v[r * V + i], v[r * V + i], sq);
    }
    const float inv = 1.0f / sqrtf(team_sum<TEAM>(sq, part) / (float)C + a.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (!live(r)) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) v[r * V + i] *= inv * w[r].w[i];
        if constexpr (Q == kNoScale)
            *reinterpret_cast<Raw *>(reinterpret_cast<T *>(a.out) + row * a.out_stride + r * SPAN + lane * V) = IO::pack(v + r * V);
    }
    if constexpr (Q != kNoScale) {
        // (absolute values compare as their bits do, a NaN above all)
        uint32_t m[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) m[r] = max(m[r], __float_as_uint(v[r * V + i]) & 0x7fffffffu);
        }
        // (a scale that would round to 0, whose reciprocal makes NaN of zeros, is the smallest value above it)
        auto scale_of = [](uint32_t bits) {
            return bits == 0 ? 1.0f : __uint_as_float(max(__float_as_uint(__uint_as_float(bits) / kE4m3Max), 1u));
        };
        float scale[R];
        if constexpr (Q == kGiven) {
#pragma unroll
            for (int r = 0; r < R; ++r) scale[r] = *a.scale;
        } else if constexpr (Q == kRowScale) {
            uint32_t all = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) all = max(all, m[r]);
            all = lanes_max(all, LANES);
            if constexpr (TEAM > 64) {
                if ((lane & 63) == 0) top[lane >> 6] = all;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < TEAM / 64; ++k) all = max(all, top[k]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) scale[r] = scale_of(all);
            if (lane == 0) a.scales[row] = scale[0];
        } else if constexpr (Q == kLaneGroups) {
            const int lanes = a.group / V;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                scale[r] = scale_of(lanes_max(m[r], lanes));
                if (live(r) && (lane & (lanes - 1)) == 0)
                    a.scales[row * (C / a.group) + (r * SPAN + lane * V) / a.group] = scale[r];
            }
        } else {   // a group spans several waves, or several rounds of a team
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t most = lanes_max(m[r], LANES);
                if (live(r) && (lane & (LANES - 1)) == 0) atomicMax(&top[(r * SPAN + lane * V) / a.group], most);
            }
            team_sync();
            for (int i = lane; i < C / a.group; i += TEAM) a.scales[row * (C / a.group) + i] = scale_of(top[i]);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (live(r)) scale[r] = scale_of(top[(r * SPAN + lane * V) / a.group]);
        }
        // RUN vectors divided at a time: all of a lane's where values are moved one by one, so that they take the reciprocal
        // of their one scale once (20000 x 4097 bf16 172 us, 195 with 16 reciprocals); one where they are wide, two at a
        // time need half as many registers again (35576 x 5120 bf16, a scale a row, 230 us for 220).
        constexpr int RUN = V == 1 && (Q == kGiven || Q == kRowScale) ? R : 1;
        uint8_t *out = reinterpret_cast<uint8_t *>(a.out) + row * a.out_stride + lane * V;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!live(r)) continue;
            float *f = v + r * V;
            if (r % RUN == 0) {
                if (fabsf(scale[r]) < 0x1p-100f) {   // whose reciprocal may be infinite
                    scale[r] *= 0x1p100f;
#pragma unroll
                    for (int i = 0; i < RUN * V; ++i) f[i] *= 0x1p100f;
                }
                divide_all<RUN * V>(f, scale[r]);
            }
            if constexpr (V == 8) {
                *reinterpret_cast<u32x2 *>(out + r * SPAN) = u32x2{pack_e4m3(f[0], f[1], f[2], f[3]), pack_e4m3(f[4], f[5], f[6], f[7])};
            } else if constexpr (V == 4) {
                *reinterpret_cast<uint32_t *>(out + r * SPAN) = pack_e4m3(f[0], f[1], f[2], f[3]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) out[r * SPAN + i] = (uint8_t)pack_e4m3(f[i], 0.0f, 0.0f, 0.0f);
            }
        }
    }
}

template <typename T, int TEAM, int V, Scales Q> static hipError_t launch_addnorm_scales(const AddNormArgs &a, hipStream_t stream) {
    constexpr int THREADS = TEAM > 64 ? TEAM : 256, ROWS = THREADS / TEAM;
    const int64_t blocks = ((int64_t)a.rows + ROWS - 1) / ROWS;
    if (!fits_grid(blocks, THREADS)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssd_add_rms_norm_kernel<T, TEAM, V, 16 / V, Q>), dim3((unsigned)blocks), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int TEAM, int V> static hipError_t launch_addnorm_team(const AddNormArgs &a, bool e4m3, hipStream_t stream) {
    constexpr int LANES = TEAM < 64 ? TEAM : 64;
    if (!e4m3) return launch_addnorm_scales<T, TEAM, V, kNoScale>(a, stream);
    if (a.scale != nullptr) return launch_addnorm_scales<T, TEAM, V, kGiven>(a, stream);
    if (a.group == a.channels) return launch_addnorm_scales<T, TEAM, V, kRowScale>(a, stream);
    if constexpr (V < 8)   // (a group is half a row at most, which 8 values of each lane hold, and 512 channels)
        if (a.group > LANES * V) return launch_addnorm_scales<T, TEAM, V, kWideGroups>(a, stream);
    return launch_addnorm_scales<T, TEAM, V, kLaneGroups>(a, stream);
}

// The smallest team that holds a row with 16 values a lane, of 8 lanes at least, or of a wave where values are moved one
// by one, whose lanes are filled by 64 of them already (2^20 rows of 64 channels bf16: 316 us with a wave each, 85
// with 8 lanes).
template <typename T, int V, int TEAM = (V == 1 ? 64 : 8)> static hipError_t launch_addnorm_size(const AddNormArgs &a, bool e4m3, hipStream_t stream) {
    if constexpr (TEAM < 1024) {
        if (a.channels <= TEAM * 16) return launch_addnorm_team<T, TEAM, V>(a, e4m3, stream);
        return launch_addnorm_size<T, V, 2 * TEAM>(a, e4m3, stream);
    } else {
        static_assert(1024 * 16 >= kNormMaxGroup, "the largest team holds the largest row");
        return launch_addnorm_team<T, 1024, V>(a, e4m3, stream);
    }
}

// Vectors of 16 bytes where all rows start on such, single values elsewhere.
template <typename T> static hipError_t launch_addnorm_t(const AddNormArgs &a, bool e4m3, hipStream_t stream) {
    const uint64_t rows = (uint64_t)(a.x_stride | (a.residual ? a.residual_stride : 0) |
                                     (a.residual_out ? a.residual_out_stride : 0) | (e4m3 ? 0 : a.out_stride) | a.channels);
    const uint64_t starts = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                            reinterpret_cast<uintptr_t>(a.residual_out) | (e4m3 ? 0 : reinterpret_cast<uintptr_t>(a.out)) |
                            rows * sizeof(T);
    constexpr int V = 16 / sizeof(T);
    const uint64_t codes = e4m3 ? reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.out_stride : 0;   // V 8-bit values at a time
    if (starts % 16 == 0 && codes % V == 0) return launch_addnorm_size<T, V>(a, e4m3, stream);
    return launch_addnorm_size<T, 1>(a, e4m3, stream);
}

// Inputs and the residual that the last-level cache (256 MB) cannot hold are streamed past it (35576 x 4096 bf16 to e4m3 in
// groups of 128 184 -> 168 us, to bf16 203 -> 195, 16000 x 8192 float32 378 -> 377; 4096 x 4096 bf16, which it holds, would
// go from 24.8 to 25.6).
constexpr int64_t kStreamBytes = int64_t(256) << 20;

hipError_t launch_add_rms_norm(AddNormArgs a, bool bf16, bool e4m3, hipStream_t stream) {
    a.stream = (int64_t)a.rows * a.channels * (bf16 ? 2 : 4) * (1 + (a.residual != nullptr) + (a.residual_out != nullptr)) > kStreamBytes;
    return bf16 ? launch_addnorm_t<__bf16>(a, e4m3, stream) : launch_addnorm_t<float>(a, e4m3, stream);
}

}  // namespace ssd
