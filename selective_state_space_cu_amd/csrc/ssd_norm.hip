// Norm of groups of channels with an activation, channels last:
//   v = x (or x silu(z));  mu = mean(v) or 0;  out = (v - mu) / sqrt(mean((v - mu)^2) + eps) w + b,
// then SiLU or a gate silu(z). One token's group at a time.
//
// Memory-bound: x (and z) are read once and out is written once, so a group
// stays in registers between the loads, the two sums and the store. A team of
// TEAM lanes (a power of two: part of a wave, a wave, or a workgroup) owns one
// group of one row and each of its lanes R vectors of V values, TEAM vectors
// apart; a team goes on to the same group of other rows, so its weights are
// loaded once. V is the widest of 16 bytes, 4 bytes and one value that the
// group's size and all row starts are multiples of (16-byte accesses at odd
// 4-byte places took twice the time of single values). 16085 x 5055 float32 in
// groups of 337 take 138 us, 4.7 TB/s, and 35576 x 4096 bf16 with a gate in groups
// of 1024 170 us, 5.1 TB/s, a large copy's rate.
#include <algorithm>

#include "ssd_norm.hpp"

namespace ssd {

__device__ __forceinline__ float norm_silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

template <typename T, int TEAM, int V, int R>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void ssd_group_norm_kernel(NormArgs a) {
    using IO = NormIO<T, V>;
    using Raw = typename IO::Raw;
    constexpr int THREADS = TEAM > 256 ? TEAM : 256, TEAMS = THREADS / TEAM, SPAN = TEAM * V;
    __shared__ float part[TEAM > 64 ? TEAM / 64 : 1];
    const int lane = threadIdx.x % TEAM;
    const int64_t team = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM, teams = (int64_t)gridDim.x * TEAMS;
    // teams t, t + groups, ... own group t mod groups, in as many rows at a time as there are whole sets of teams
    const int64_t row0 = team / a.groups, rows_step = teams / a.groups;
    if (row0 >= rows_step) return;
    const int c0 = (int)(team - row0 * a.groups) * a.size, size = a.size;
    // Round r holds values r SPAN + lane V ..: `whole` rounds are full, one more may be partial, whose lanes past the
    // group's end hold zeros and store nothing.
    const int whole = size / SPAN;
    const bool tail = lane * V < size - whole * SPAN;
    auto present = [&](int r) { return r * SPAN < size; };   // uniform
    auto live = [&](int r) { return r < whole || tail; };    // of a round that is present
    float w[R * V], bias[R * V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = c0 + r * SPAN + lane * V + i;
            w[r * V + i] = a.weight != nullptr && present(r) && live(r) ? a.weight[at] : 1.0f;
            bias[r * V + i] = a.bias != nullptr && present(r) && live(r) ? a.bias[at] : 0.0f;
        }
    const float inv = 1.0f / (float)size;
    for (int64_t row = row0; row < a.rows; row += rows_step) {
        // (loading the next row here while this one is computed took 1.4 times as long for groups of 337 float32: the
        // registers cost waves)
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride + c0 + lane * V;
        const T *z = reinterpret_cast<const T *>(a.z) + row * a.z_stride + c0 + lane * V;
        T *out = reinterpret_cast<T *>(a.out) + row * a.out_stride + c0 + lane * V;
        Raw rx[R], rz[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rx[r] = Raw{};
            if (present(r) && live(r)) {
                rx[r] = *reinterpret_cast<const Raw *>(x + r * SPAN);
                if (a.z != nullptr) rz[r] = *reinterpret_cast<const Raw *>(z + r * SPAN);
            }
        }
        float v[R * V], sum = 0.0f, sq = 0.0f, mu = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!present(r)) continue;
            IO::unpack(rx[r], v + r * V);
            if (a.act == SSD_NORM_GATE_FIRST) {
                float g[V];
                IO::unpack(rz[r], g);
#pragma unroll
                for (int i = 0; i < V; ++i) v[r * V + i] = live(r) ? v[r * V + i] * norm_silu(g[i]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[r * V + i];
        }
        if (a.center) {
            mu = team_sum<TEAM>(sum, part) * inv;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!present(r)) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) v[r * V + i] = live(r) ? v[r * V + i] - mu : 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!present(r)) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) sq = fmaf(v[r * V + i], v[r * V + i], sq);
        }
        const float scale = 1.0f / sqrtf(team_sum<TEAM>(sq, part) * inv + a.eps);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!present(r)) continue;
            float o[V], g[V];
            if (a.act == SSD_NORM_GATE_LAST) IO::unpack(rz[r], g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = fmaf(v[r * V + i] * scale, w[r * V + i], bias[r * V + i]);
                if (a.act == SSD_NORM_SILU) o[i] = norm_silu(o[i]);
                if (a.act == SSD_NORM_GATE_LAST) o[i] *= norm_silu(g[i]);
            }
            if (live(r)) *reinterpret_cast<Raw *>(out + r * SPAN) = IO::pack(o);
        }
    }
}

// Workgroups of a launch: one round of what the CUs hold at once (a second, partial round costs as much as a full one: 8 a CU
// instead took 154 us for 138 with groups of 337 float32, 388 for 294 in bf16), and of those only as many as have 48 KB of
// inputs on their way in each CU (32 / 48 / 64 KB: 183 / 170 / 178 us for 35576 x 4096 bf16 with a gate in groups of 1024,
// 141 / 136 / 135 for 20011 x 5120 in groups of 640). The runtime says 7 for kernels of few registers, but 7 a CU take
// 168 us where 6 take 138.
constexpr int64_t kNormCus = 256, kNormBytesAhead = 48 * 1024;
constexpr int kNormMost = 6;

template <typename T, int TEAM, int V, int R> static hipError_t launch_norm_team(const NormArgs &a, hipStream_t stream) {
    constexpr int THREADS = TEAM > 256 ? TEAM : 256, TEAMS = THREADS / TEAM;
    static const int resident = [] {
        int n = 0;
        const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, ssd_group_norm_kernel<T, TEAM, V, R>, THREADS, 0);
        return e == hipSuccess && n > 0 ? std::min(n, kNormMost) : 1;
    }();
    const int64_t bytes = (int64_t)TEAMS * a.size * sizeof(T) * (a.z != nullptr ? 2 : 1);   // of a workgroup's inputs at a time
    const int64_t most = kNormCus * std::min<int64_t>(resident, (kNormBytesAhead + bytes - 1) / bytes);
    const int64_t need = ((int64_t)a.rows * a.groups + TEAMS - 1) / TEAMS;   // one team for every (row, group)
    int64_t blocks = need < most ? need : most;
    if (blocks * TEAMS < a.groups) blocks = (a.groups + TEAMS - 1) / TEAMS;
    hipLaunchKernelGGL((ssd_group_norm_kernel<T, TEAM, V, R>), dim3((unsigned)blocks), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

// The smallest team that holds a group with 16 values a lane (8 where they are moved one by one, which leaves more
// waves: 14 % less time for groups of 337 float32; 16 in the largest team).
template <typename T, int V, int TEAM = 1> static hipError_t launch_norm_size(const NormArgs &a, hipStream_t stream) {
    if constexpr (TEAM < 1024) {
        constexpr int R = V == 1 ? 8 : 16 / V;
        if (a.size <= TEAM * V * R) return launch_norm_team<T, TEAM, V, R>(a, stream);
        return launch_norm_size<T, V, TEAM == 64 ? 256 : TEAM == 256 ? 1024 : 2 * TEAM>(a, stream);
    } else {
        static_assert(1024 * 16 >= kNormMaxGroup, "the largest team holds the largest group");
        return launch_norm_team<T, 1024, V, 16 / V>(a, stream);
    }
}

template <typename T> static hipError_t launch_norm_t(const NormArgs &a, hipStream_t stream) {
    const uint64_t starts = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.z) |
                            reinterpret_cast<uintptr_t>(a.out) |
                            (uint64_t)(a.x_stride | (a.z ? a.z_stride : 0) | a.out_stride | a.size) * sizeof(T);
    if (starts % 16 == 0) return launch_norm_size<T, 16 / sizeof(T)>(a, stream);
    if (sizeof(T) == 2 && starts % 4 == 0) return launch_norm_size<T, 4 / sizeof(T)>(a, stream);
    return launch_norm_size<T, 1>(a, stream);
}

hipError_t launch_group_norm(const NormArgs &a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_norm_t<__bf16>(a, stream) : launch_norm_t<float>(a, stream);
}

}  // namespace ssd
