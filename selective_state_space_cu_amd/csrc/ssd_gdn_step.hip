// Gated delta rule token by token, with dual state anchors: the new tokens of
// every sequence (one, or a few speculated ones) advance the state read from one
// cache slot, and the state after each token that has a write slot goes there.
// Per value head h (key head g = h / (H/G)), with the state S (dv x dk):
//   S'  = alpha S + beta (v - alpha S k) k^T,   o = scale S' q
// Both products need only the entering state, so one pass over S gives them:
//   r = S k, w = S q;  d = beta (v - alpha r);  S' = alpha S + d k^T;
//   o = scale (alpha w + d (k . q))
// q and k may still have to be normed: k = kn k_raw, kn = 1 / sqrt(|k_raw|^2 + eps).
//
// Memory-bound: the states are the traffic (4 dk dv bytes read and written per
// (sequence, head)). Eight lanes own a state row, in float4 pieces 8 lanes apart,
// so that eight rows of a wave's access are whole 128-byte lines, and the two
// sums over a row take three lane exchanges each. 256 sequences x 32 heads of
// 128 x 128 take 186 us, 5.8 TB/s (a large copy reaches 5.1). A sequence's tokens
// follow one another at 1.0 us, all of a token's loads on their way at once;
// loading the next tokens' inputs ahead, and working out what the state is not
// needed for beside the state's update, saved no more of that and cost up to 25 %
// with 8 tokens, by the registers that it takes.
#include "ssd_elem.hpp"

namespace ssd {

constexpr int kGdnStepThreads = 64;
// State rows of a lane, from the waves that one row makes. Few waves (two a SIMD): one row, a shorter chain. More: two
// rows halve the waves to be started and to fetch q, k and the gates, until there are so many (16 a SIMD) that one row's 64
// bytes of states a lane keep memory busy by themselves; 32 bytes, of dk 64, never do, the 128 of dk 256 always.
// One / two / four rows, 32 heads x 128 rows, us: dk 128 with 4 sequences 5.7 / 6.2 / 7.2, 8 9.0 / 8.0 / 8.6, 16 16.2 / 14.7 /
// 13.2, 24 22.0 / 21.8, 32 27.0 / 27.9 / 29.0, 128 95 / 98 / 106; dk 64 with 4 4.8 / 5.1 / 6.4, 8 6.9 / 5.9, 16 11.0 / 8.5 /
// 8.2, 128 55.8 / 52.4 / 55.3; dk 256 (16 heads x 256 rows) with 4 8.3 / 8.3 / 9.0, 64 90 / 93 / 95. A wave is a workgroup;
// two or four take 0 to 2 % longer. (Four rows gain in a narrow band alone, 16 sequences here, 4 to 10 %, and lose on both
// sides of it; they are not built.)
static int gdn_step_rows(int dk, int64_t waves) { return dk <= 128 && waves > 2048 && (dk == 64 || waves < 16384) ? 2 : 1; }

// Sum over the 8 lanes of a row; every lane gets it.
__device__ __forceinline__ float sum8(float v) {
    auto add = [&](auto ctrl) {
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    add(std::integral_constant<int, 0xB1>{});    // lane ^ 1
    add(std::integral_constant<int, 0x4E>{});    // lane ^ 2
    add(std::integral_constant<int, 0x141>{});   // 7 - lane
    return v;
}

template <typename T, typename GT, int DK, int R>
__global__ __launch_bounds__(kGdnStepThreads) void ssd_gdn_step_kernel(GdnStepArgs a) {
    constexpr int PIECES = DK / 32, GROUPS = kGdnStepThreads / 8;
    using E = RawOf<T>;
    const int lr = threadIdx.x % 8, rg = threadIdx.x / 8;
    int64_t b = blockIdx.x;
    const int rb = (int)(b % a.row_blocks);
    b /= a.row_blocks;
    const int h = (int)(b % a.H), s = (int)(b / a.H);
    const bool first = rb == 0 && h == 0 && threadIdx.x == 0;   // speaks for the sequence
    int t0 = s, t1 = s + 1;
    if (a.cu_seqlens != nullptr) {
        t0 = a.cu_seqlens[s];
        t1 = a.cu_seqlens[s + 1];
        if (t0 < 0 || t1 < t0 || t1 > a.T) {
            if (first && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_CU_SEQLENS);
            return;
        }
    }
    if (t0 == t1) return;
    const int rs = a.read_slot[s];
    bool bad = rs >= a.num_slots;
    for (int t = t0 + (int)threadIdx.x; t < t1; t += kGdnStepThreads) bad |= a.write_slot[t] >= a.num_slots;
    if (__syncthreads_or(bad)) {   // refused: nothing read or written
        if (first && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
        return;
    }
    const int g = h / (a.H / a.G);
    const int p0 = rb * GROUPS * R + rg;   // rows p0, p0 + GROUPS, ..
    const int64_t slot = (int64_t)a.H * a.dv * DK, head = (int64_t)h * a.dv * DK + 4 * lr;
    f32x4 st[R][PIECES];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = p0 + r * GROUPS;
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
            st[r][j] = rs >= 0 && p < a.dv
                           ? __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(a.cache + rs * slot + head + (int64_t)p * DK + 32 * j))
                           : f32x4{0, 0, 0, 0};
    }
    const T *kp = reinterpret_cast<const T *>(a.k) + (int64_t)g * DK + 4 * lr, *qp = reinterpret_cast<const T *>(a.q) + (int64_t)g * DK + 4 * lr;
    const float rate = a.A != nullptr ? a.A[h] : 0.0f, bias = a.A != nullptr && a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;
    for (int t = t0; t < t1; ++t) {
        using Four = typename E::Four;
        Four rk[PIECES], rq[PIECES];
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            rk[j] = *reinterpret_cast<const Four *>(kp + t * a.k_stride + 32 * j);
            rq[j] = *reinterpret_cast<const Four *>(qp + t * a.q_stride + 32 * j);
        }
        float gate = load_f<GT>(a.gate, t * a.gate_stride + h), beta = load_f<GT>(a.beta, t * a.beta_stride + h), v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = load_f<T>(a.v, t * a.v_stride + (int64_t)h * a.dv + min(p0 + r * GROUPS, a.dv - 1));
        const int ws = a.write_slot[t];
        f32x4 k[PIECES], q[PIECES];
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            k[j] = E::f4(rk[j]);
            q[j] = E::f4(rq[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kk = fmaf(k[j][i], k[j][i], kk);
                qq = fmaf(q[j][i], q[j][i], qq);
                kq = fmaf(k[j][i], q[j][i], kq);
            }
        }
        if (a.A != nullptr) {
            gate = rate * softplus_full(gate + bias);
            beta = 1.0f / (1.0f + fast_exp2(-beta * kLog2e));
        }
        const float alpha = fast_exp2(gate * kLog2e);
        kq = sum8(kq);
        float kn = 1.0f, qn = a.scale;
        if (a.qk_eps >= 0.0f) {
            kn = 1.0f / sqrtf(sum8(kk) + a.qk_eps);
            qn *= 1.0f / sqrtf(sum8(qq) + a.qk_eps);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int p = p0 + r * GROUPS;
            float sk = 0.0f, sq = 0.0f;
#pragma unroll
            for (int j = 0; j < PIECES; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sk = fmaf(st[r][j][i], k[j][i], sk);
                    sq = fmaf(st[r][j][i], q[j][i], sq);
                }
            sk = sum8(sk);
            sq = sum8(sq);
            if (p >= a.dv) continue;
            const float d = beta * fmaf(-(alpha * kn), sk, v[r]) * kn;
            if (lr == 0)
                reinterpret_cast<T *>(a.o)[t * a.o_stride + (int64_t)h * a.dv + p] = (T)(qn * fmaf(alpha, sq, d * kq));
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) st[r][j][i] = fmaf(alpha, st[r][j][i], d * k[j][i]);
                if (ws >= 0)
                    __builtin_nontemporal_store(st[r][j], reinterpret_cast<f32x4 *>(a.cache + ws * slot + head + (int64_t)p * DK + 32 * j));
            }
        }
    }
}

template <typename T, typename GT, int DK, int R> static hipError_t launch_gdn_step_rows(GdnStepArgs a, hipStream_t stream) {
    constexpr int ROWS = kGdnStepThreads / 8 * R;
    a.row_blocks = (a.dv + ROWS - 1) / ROWS;
    const int64_t blocks = (int64_t)a.S * a.H * a.row_blocks;
    if (!fits_grid(blocks, kGdnStepThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssd_gdn_step_kernel<T, GT, DK, R>), dim3((unsigned)blocks), dim3(kGdnStepThreads), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename T, typename GT> static hipError_t launch_gdn_step_t(const GdnStepArgs &a, int dk, hipStream_t stream) {
    const int64_t waves = (int64_t)a.S * a.H * ((a.dv + kGdnStepThreads / 8 - 1) / (kGdnStepThreads / 8));
    const bool two = gdn_step_rows(dk, waves) == 2;
    switch (dk) {
        case 64: return two ? launch_gdn_step_rows<T, GT, 64, 2>(a, stream) : launch_gdn_step_rows<T, GT, 64, 1>(a, stream);
        case 128: return two ? launch_gdn_step_rows<T, GT, 128, 2>(a, stream) : launch_gdn_step_rows<T, GT, 128, 1>(a, stream);
        case 256: return launch_gdn_step_rows<T, GT, 256, 1>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gdn_step(const GdnStepArgs &a, bool bf16, bool gate_bf16, int dk, hipStream_t stream) {
    if (bf16) return gate_bf16 ? launch_gdn_step_t<__bf16, __bf16>(a, dk, stream) : launch_gdn_step_t<__bf16, float>(a, dk, stream);
    return gate_bf16 ? launch_gdn_step_t<float, __bf16>(a, dk, stream) : launch_gdn_step_t<float, float>(a, dk, stream);
}

}  // namespace ssd
