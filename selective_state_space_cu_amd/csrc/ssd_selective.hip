// Selective scan with a decay per channel and state, and its single-token step.
//   delta  = softplus(dt[t,d] + dt_bias[d])
//   h[d,n] = 2^(delta A[d,n] log2 e) h[d,n] + delta u[t,d] B[t,g,n]
//   y[t,d] = (sum_n h[d,n] C[t,g,n] + D[d] u[t,d]) silu(z[t,d])
//
// The decay differs per (token, channel, state), so a chunk has no form as a
// matrix product (a per-head decay has one): what there is to compute is one
// exponential and a few products and sums per (token, channel, state).
// (delta is scaled by log2 e, not A: delta = 0 leaves the state for any finite A.)
#include <type_traits>

#include "ssd_scan.hpp"

namespace ssd {

typedef float f32x2 __attribute__((ext_vector_type(2)));

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

// ---------------------------------------------------------------------------
// Scan, in segments. A workgroup owns 16 channels of one sequence; its waves take
// segments of kSeg tokens in turn (wave w of W: segments w, w + W, ...). A segment
// is an affine map of the state, h -> P h + e, and only that map's use is serial:
//   pass 1 (any time): the decays a_t = 2^(delta_t A log2 e) and the inputs
//     b_t = delta_t u_t B_t, kept in registers; e, the state after the segment
//     from a zero state; P, the product of the a_t;
//   chain (in order): wait for the state h_in that enters the segment, publish
//     P h_in + e for the next segment's wave;
//   pass 2: h_t = a_t h_(t-1) + b_t again from h_in, and y_t = h_t . C_t.
// The exponentials, which cost most, are computed once; the price of running W
// segments side by side is one product and one sum more. The chain runs through
// LDS: one state buffer, which each segment's wave reads and then overwrites, and
// a counter of finished segments. Every wave of the workgroup is resident and
// takes its segments in order, so the wave that the others wait for never waits
// for them: every wait ends.
//
// Lanes: lane = 16 q + c holds the states n = 16 nb + 4 q + i (i < 4) of channel
// c, for one block nb of 16 states at a time. What is per (token, channel) only -
// softplus, gate, loads, stores - is done by lane (q, c) for the tokens 4 j + q,
// so nothing is computed four times; delta and delta u reach the other lanes
// through LDS, as B_t and C_t do, and the four partial sums of y_t come back by
// three half swaps per four tokens.
//
// What bounds it: instruction issue. Per token and 16 channels x 16 states a wave
// issues 4 exponentials (3.4 ns of a SIMD each), 20 products and sums (about 1 ns
// with vector operands and an even number of waves) and its share of the rest, 56
// ns in all; 75 are measured (4 x 8894 tokens, 4096 channels: 672 us, 1.8 TB/s).
// Counters of that call: 314 vector instructions a segment and wave (64 scalar, 32
// LDS, 9 memory ones), 0.24 a cycle and SIMD with one exponential in eight; loops of
// nothing else reach 0.26 (one in five) and 0.40 (none) with as many waves. Of 3.4
// waves a SIMD 0.7 waits for LDS, memory or the chain. LDS is taken 38 % of the
// time, without bank conflicts.
// Tried and slower: b_t as an outer product on v_mfma_f32_4x4x1 (it holds the
// vector unit for 5 ns and saves 4 products), 64 channels to a wave with B and C as
// scalar operands (each such product takes twice as long), 16 tokens to a segment
// or 5 waves a SIMD (the decays no longer fit the registers), token after token with
// 8 lanes to a channel and two states a lane (15 % fewer instructions, but 4 x 8894
// tokens give it two waves a SIMD, too few to hide what each waits for: 929 us).
constexpr int kSeg = 8;    // tokens of a segment
constexpr int kCh = 16;    // channels of a workgroup

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

// One element at a uniform address plus a lane offset. The address is kept in scalar registers (the compiler would
// add both per lane, in 64 bits) and the access stays a global one.
template <typename V> using Global = __attribute__((address_space(1))) V;
template <typename V> __device__ __forceinline__ V load_at(const char *base, uint32_t off) {
    Global<const char> *p = (Global<const char> *)base;
    asm("" : "+s"(p));
    return *(Global<const V> *)(p + off);
}
template <typename V> __device__ __forceinline__ void store_at(char *base, uint32_t off, V v) {
    Global<char> *p = (Global<char> *)base;
    asm("" : "+s"(p));
    *(Global<V> *)(p + off) = v;
}

// Sums of y_j (j < 4) over the four lanes 16 apart: lane (q, c) gets that of y_q.
__device__ __forceinline__ float sum_scatter4(const float (&y)[4]) {
    auto swap32 = [](float a, float b) {   // [a.lo | b.lo] + [a.hi | b.hi]
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    };
    const float r0 = swap32(y[0], y[2]), r1 = swap32(y[1], y[3]);
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(r0), __float_as_uint(r1), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Whether some lane of the wave has a rate above 0.
__device__ __forceinline__ bool any_above_zero(const f32x4 &r) {
    return __any(fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3])) > 0.0f);
}

// The slot that receives the state after a chunk (-1: none, also for a chunk that is not in the grid).
__device__ __forceinline__ int chunk_slot(const SelectiveArgs &a, int chunk, bool report) {
    if (chunk < 0 || chunk >= a.max_chunks) return -1;
    const int slot = a.chunk_state_dst != nullptr ? a.chunk_state_dst[chunk] : chunk;
    if (slot < a.capacity) return slot;
    if (report) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
    return -1;
}

template <typename T, typename DT, int N>
__global__ __launch_bounds__(1024) void ssd_selective_scan_kernel(SelectiveArgs a) {
    constexpr int NBLK = N / 16, SEG = kSeg, J = SEG / 4;
    using R = RawOf<T>;
    using RD = RawOf<DT>;
    using One = typename R::One;
    using OneD = typename RD::One;
    using Four = typename R::Four;
    typedef __attribute__((address_space(3))) volatile int lds_counter;   // (a generic pointer's access waits for all loads)
    extern __shared__ __attribute__((aligned(16))) float lds[];
    if (__builtin_nontemporal_load(a.error_flag) & SSD_DATA_BAD_CU_SEQLENS) return;
    const int per = a.C_total / a.G, bpg = (per + kCh - 1) / kCh, cblocks = a.G * bpg;   // blocks stay inside a group
    // four neighbouring channel blocks (one 128-byte line of bf16) on one XCD: blocks go to the 8 XCDs in turn
    int b = blockIdx.x;
    if ((b | 31) < (int)gridDim.x) b = (b & ~31) | ((b & 7) << 2) | ((b >> 3) & 3);
    const int rank = b / cblocks, cb = b - rank * cblocks;
    const int s = a.seq_order[rank];
    if (s < 0 || s >= a.S) return;
    int64_t tb = a.cu_seqlens[s], te = a.cu_seqlens[s + 1];
    tb = tb < 0 ? 0 : (tb > a.T ? a.T : tb);
    te = te < tb ? tb : (te > a.T ? a.T : te);
    const int L = (int)(te - tb), c0 = a.seq_chunk_start[s];
    if (L <= a.walk_to) return;   // the walk's
    const int nseg = (L + SEG - 1) / SEG, nw = (int)blockDim.x >> 6;
    // Waves of the workgroups of a CU are served oldest first, so one workgroup ran ahead of the others and the last was
    // left alone on its CU. Priorities by what is left to do, in thirds of the longest sequence, keep them together (4 x
    // 8894 tokens, 4096 channels, 4 workgroups of 4 waves on every CU: 737 us without, 672 with).
    const int longest = a.seq_order[0];
    const int third = longest < 0 || longest >= a.S ? nseg : (a.cu_seqlens[longest + 1] - a.cu_seqlens[longest]) / (3 * SEG);
    const int chunk_segs = a.cs / SEG, chunk_shift = __builtin_ctz(chunk_segs);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15, g = cb / bpg, ch = (cb - g * bpg) * kCh + c;
    // Lanes past the group's channels are copies of its last channel: they compute and store the same values to the
    // same places. (Stores without a branch keep the waits for the loads ahead of them exact.)
    const int d = g * per + min(ch, per - 1);

    float *carry = lds;                                           // [NBLK][64][4]
    lds_counter *done = (lds_counter *)(__attribute__((address_space(3))) int *)(lds + NBLK * 256);   // [NBLK] segments finished
    lds_counter *rising = done + NBLK;                                    // [NBLK] whether some rate is above 0
    float *mine = lds + NBLK * 256 + ((2 * NBLK + 3) & ~3) + wave * (SEG * 64);
    float *ldsD = mine;                 // [SEG tokens][16 channels] (delta log2 e, delta u)
    float *ldsB = mine + SEG * 32;      // [SEG tokens][16 states]
    float *ldsC = mine + SEG * 48;

    const int64_t state_row = (int64_t)s * a.C_total * N;
    float *final = a.final_states + state_row;
    // What is needed once a segment or less often is worked out anew from the lane's number, which the compiler is kept
    // from knowing: kept over the segments, it pushes other values out to scratch memory inside the loops. state_col is the
    // lane's place in a state. (One block of states leaves room for d; without it nothing goes to scratch memory at all, but
    // 30001 bf16 tokens of 2560 channels take 568 us for 549, 4 float32 prompts of 4096 channels 161 for 151.)
    auto anew = [&] {
        int here = lane;
        asm volatile("" : "+v"(here));
        return here;
    };
    auto channel = [&](int lane) { return g * per + min((cb - g * bpg) * kCh + (lane & 15), per - 1); };
    auto state_col = [&]() -> int64_t {
        if constexpr (NBLK == 1) {
            uint32_t channel = d;
            asm volatile("" : "+v"(channel));
            return channel * N + (__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)) >> 2 & 12);
        }
        const int here = anew();
        return (int64_t)channel(here) * N + 4 * (here >> 4);
    };
    const bool start = a.init != nullptr && (a.has_init == nullptr || a.has_init[s] != 0);
    for (int nb = wave; nb < NBLK; nb += nw) {
        const f32x4 h = start ? *reinterpret_cast<const f32x4 *>(a.init + state_row + nb * 16 + state_col()) : f32x4{0, 0, 0, 0};
        *reinterpret_cast<f32x4 *>(carry + (nb * 64 + lane) * 4) = h;
        if (nseg == 0) *reinterpret_cast<f32x4 *>(final + nb * 16 + state_col()) = h;
        const bool up = any_above_zero(*reinterpret_cast<const f32x4 *>(a.A + nb * 16 + state_col()));
        if (lane == 0) {
            done[nb] = 0;
            rising[nb] = up;
        }
    }
    __syncthreads();
    if (wave >= nseg) return;
    const bool growing = __any(lane < NBLK && rising[lane < NBLK ? lane : 0] != 0);

    const float bias = a.dt_bias != nullptr ? a.dt_bias[d] : 0.0f, skip = a.D != nullptr ? a.D[d] : 0.0f;
    f32x4 rate = *reinterpret_cast<const f32x4 *>(a.A + (int64_t)d * N + 4 * q);

    // Addresses: uniform pointers to the first row of a segment, advanced from segment to segment, plus 32-bit lane
    // offsets (the API's bound on strides keeps 16 rows below 2^32 bytes).
    constexpr int ES = sizeof(One), ED = sizeof(OneD);
    const int64_t first = tb + wave * SEG;
    const int64_t su = a.u_stride * ES, sd = a.dt_stride * ED, sz = (a.z ? a.z_stride : a.u_stride) * ES, sy = a.y_stride * ES,
                  sB = a.B_stride * ES, sC = a.C_stride * ES;
    const char *pu = reinterpret_cast<const char *>(a.u) + first * su, *pd = reinterpret_cast<const char *>(a.dt) + first * sd;
    const char *pz = reinterpret_cast<const char *>(a.z ? a.z : a.u) + first * sz;   // (no gate: loaded again, unused)
    char *py = reinterpret_cast<char *>(a.y) + first * sy;
    const uint32_t offU = q * (uint32_t)su + d * ES, offD = q * (uint32_t)sd + d * ED, offZ = q * (uint32_t)sz + d * ES,
                   offY = q * (uint32_t)sy + d * ES;
    // B and C: every lane four states of one token, lanes 0 .. 31 of B and the others of C, through a pointer of its own
    const int tokBC = lane >> 2 & (SEG - 1);
    const int64_t sBC = lane < 32 ? sB : sC;
    const char *pBC = reinterpret_cast<const char *>(lane < 32 ? a.B : a.C) + (first + tokBC) * sBC +
                      (g * N + 4 * (lane & 3)) * ES;

    // bytes from a wave's segment to its next
    const int64_t ahead = (int64_t)nw * SEG, nextU = ahead * su, nextD = ahead * sd, nextZ = ahead * sz, nextY = ahead * sy,
                  nextB = ahead * sB, nextC = ahead * sC, nextBC = ahead * sBC;

    // raw inputs of a segment, fetched one segment ahead
    One ru[J], rz[J];
    OneD rd[J];
    Four rBC;
    auto fetch_bc = [&](int rows, int nb) {   // rows past the end: the last one
        const int64_t back = max(tokBC - (rows - 1), 0);
        rBC = *reinterpret_cast<const Four *>(pBC + nb * 16 * ES - (rows >= SEG ? 0 : back * sBC));
    };
    auto fetch = [&] {   // a segment of SEG tokens
#pragma unroll
        for (int j = 0; j < J; ++j) {
            ru[j] = load_at<One>(pu + 4 * j * su, offU);
            rd[j] = load_at<OneD>(pd + 4 * j * sd, offD);
            rz[j] = load_at<One>(pz + 4 * j * sz, offZ);
        }
        fetch_bc(SEG, 0);
    };
    auto fetch_rest = [&](int rows, int q, int d) {   // a segment of fewer: past the end, the last token again
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t r = min(4 * j + q, rows - 1);
            ru[j] = *reinterpret_cast<const One *>(pu + (r * (uint32_t)su + d * ES));
            rd[j] = *reinterpret_cast<const OneD *>(pd + (r * (uint32_t)sd + d * ED));
            rz[j] = *reinterpret_cast<const One *>(pz + (r * (uint32_t)sz + d * ES));
        }
        fetch_bc(rows, 0);
    };
    if ((wave + 1) * SEG <= L) fetch();

    auto segment = [&](int seg, auto whole) {
        constexpr bool FULL = decltype(whole)::value;   // all SEG tokens exist
        // (the sequence's last segment works its places out anew: kept, they would not fit beside the loop's)
        const int here = FULL ? lane : anew();
        const int q = here >> 4, c = here & 15, d = channel(here), lane = here;
        const int left = L - seg * SEG;                 // tokens from the segment's first on
        if constexpr (!FULL) fetch_rest(left, q, d);    // once a sequence: not ahead
        // the slot that receives the state after this segment, if a chunk ends here
        int slot = -1;
        if (a.chunk_states != nullptr && (!FULL || left == SEG || ((seg + 1) & (chunk_segs - 1)) == 0)) {
            slot = __builtin_amdgcn_readfirstlane(chunk_slot(a, c0 + (seg >> chunk_shift), cb == 0 && lane == 0));
        }
        float u[J];
        One z[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            u[j] = R::f(ru[j]);
            z[j] = rz[j];
            const float delta = softplus_full(RD::f(rd[j]) + bias);
            *reinterpret_cast<f32x2 *>(ldsD + ((4 * j + q) * 16 + c) * 2) = f32x2{delta * kLog2e, delta * u[j]};
        }

        auto emit = [&](int j, const float (&part)[4]) {   // tokens 4 j .. 4 j + 3
            float v = fmaf(skip, u[j], sum_scatter4(part));
            if (a.z != nullptr) v *= silu_full(R::f(z[j]));
            uint32_t to = offY;
            if constexpr (NBLK > 1) {
                const int here = anew();
                to = (here >> 4) * (uint32_t)sy + channel(here) * ES;
            }
            if (FULL || 4 * j + q < left) store_at<T>(py + 4 * j * sy, to, (T)v);
        };
        float y[NBLK > 1 ? SEG : 4];
        if constexpr (NBLK > 1) {
#pragma unroll
            for (int t = 0; t < SEG; ++t) y[t] = 0.0f;
        }

#pragma unroll 1
        for (int nb = 0; nb < NBLK; ++nb) {
            *reinterpret_cast<f32x4 *>(ldsB + lane * 4) = R::f4(rBC);   // C follows B
            if (NBLK > 1) rate = *reinterpret_cast<const f32x4 *>(a.A + nb * 16 + state_col());
            if (nb + 1 < NBLK) {
                fetch_bc(FULL ? SEG : left, nb + 1);
            } else if (FULL) {
                pu += nextU;
                pd += nextD;
                pz += nextZ;
                pBC += NBLK == 1 ? nextBC : anew() < 32 ? nextB : nextC;
                if (left >= (nw + 1) * SEG) fetch();
            }
            __builtin_amdgcn_wave_barrier();

            // LDS values of the next token are on their way while one is computed (the compiler, left alone, either waits
            // for each read or reads everything ahead and spills)
            constexpr int G2 = 2;   // tokens of a read group in the second pass
            f32x4 dec[SEG], inp[SEG], h, p;
            f32x2 dd[2];
            f32x4 bv[2];
            auto read1 = [&](int t) {
                dd[t & 1] = *reinterpret_cast<const f32x2 *>(ldsD + (t * 16 + c) * 2);
                bv[t & 1] = *reinterpret_cast<const f32x4 *>(ldsB + t * 16 + 4 * q);
            };
            read1(0);
#pragma unroll
            for (int t = 0; t < SEG; ++t) {
                if (t + 1 < SEG) read1(t + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dec[t][i] = fast_exp2(dd[t & 1][0] * rate[i]);
                    inp[t][i] = dd[t & 1][1] * bv[t & 1][i];
                    if (!FULL && t >= left) {   // past the end (uniform): the state stays
                        dec[t][i] = 1.0f;
                        inp[t][i] = 0.0f;
                    }
                    h[i] = t == 0 ? inp[t][i] : fmaf(dec[t][i], h[i], inp[t][i]);
                    p[i] = t == 0 ? dec[t][i] : p[i] * dec[t][i];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x4 cv[2][G2];
            auto read2 = [&](int grp) {
#pragma unroll
                for (int k = 0; k < G2; ++k)
                    cv[grp & 1][k] = *reinterpret_cast<const f32x4 *>(ldsC + (grp * G2 + k) * 16 + 4 * q);
            };
            read2(0);
#pragma unroll
            for (int t = 0; t < SEG; ++t) asm volatile("" : "+v"(dec[t]), "+v"(inp[t]));   // before the wait, not after it
            asm volatile("" : "+v"(p), "+v"(h));
            // Whether a lane's decays may have a product outside float32's range.
            const bool doubtful = growing || __any(fminf(fminf(p[0], p[1]), fminf(p[2], p[3])) == 0.0f);
            __builtin_amdgcn_s_setprio(3);     // the other waves wait for what follows

            // the chain: segment seg's wave is the only one that touches the buffer between done = seg and seg + 1.
            // LDS operations of a wave take effect in order: a state read after a counter that says so is that state
            f32x4 *state = reinterpret_cast<f32x4 *>(carry + (nb * 64 + lane) * 4);
            f32x4 in;
            for (;;) {
                const int n = done[nb];
                asm volatile("" ::: "memory");
                in = *state;
                const int ahead = seg - __builtin_amdgcn_readfirstlane(n);   // segments before this one's turn
                if (ahead <= 0) break;
                if (ahead > 1) __builtin_amdgcn_s_sleep(1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fmaf(p[i], in[i], h[i]);
            // Such a product times the state is not the decays one by one: 0 times an infinite state is NaN where each decay
            // leaves it infinite, infinity times a small one is not finite. So states that are not go token by token.
            if (doubtful) {
                const float sum = (h[0] + h[1]) + (h[2] + h[3]);
                if (__builtin_expect(__any(!(fabsf(sum) < __builtin_inff())), 0)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = in[i];
#pragma unroll
                        for (int t = 0; t < SEG; ++t) v = fmaf(dec[t][i], v, inp[t][i]);
                        if (!(fabsf(h[i]) < __builtin_inff())) h[i] = v;
                    }
                }
            }
            *state = h;
            asm volatile("" ::: "memory");
            if (lane == 0) done[nb] = seg + 1;
            if (nseg - seg > 2 * third) __builtin_amdgcn_s_setprio(2);
            else if (nseg - seg > third) __builtin_amdgcn_s_setprio(1);
            else __builtin_amdgcn_s_setprio(0);
            asm volatile("" ::: "memory");
            if (slot >= 0) {
                float *to = a.chunk_states + (int64_t)slot * a.C_total * N + nb * 16;   // uniform
                *reinterpret_cast<f32x4 *>(to + state_col()) = h;
            }

#pragma unroll
            for (int grp = 0; grp < SEG / G2; ++grp) {
                if (grp + 1 < SEG / G2) read2(grp + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < G2; ++k) {
                    const int t = grp * G2 + k;
                    const f32x4 ct = cv[grp & 1][k];
#pragma unroll
                    for (int i = 0; i < 4; ++i) in[i] = fmaf(dec[t][i], in[i], inp[t][i]);
                    float v = NBLK > 1 ? fmaf(in[0], ct[0], y[NBLK > 1 ? t : 0]) : in[0] * ct[0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) v = fmaf(in[i], ct[i], v);
                    y[NBLK > 1 ? t : t & 3] = v;
                }
                if constexpr (NBLK == 1) {
                    if ((grp + 1) * G2 % 4 == 0) emit((grp + 1) * G2 / 4 - 1, {y[0], y[1], y[2], y[3]});
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_wave_barrier();
        }
        if constexpr (NBLK > 1) {
#pragma unroll
            for (int j = 0; j < J; ++j) emit(j, {y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]});
        }
        py += nextY;
    };
    int seg = wave;
    for (; (seg + 1) * SEG <= L; seg += nw) segment(seg, std::true_type{});
    if (seg < nseg) segment(seg, std::false_type{});
    if ((nseg - 1) % nw == wave) {   // this wave's segment was the last: what it left in the buffer is the final state
#pragma unroll 1
        for (int nb = 0; nb < NBLK; ++nb)
            *reinterpret_cast<f32x4 *>(final + nb * 16 + state_col()) = *reinterpret_cast<f32x4 *>(carry + (nb * 64 + lane) * 4);
    }
}

// ---------------------------------------------------------------------------
// Scan, walked once: where there are sequences and channels enough to fill the
// card, nothing runs side by side along a sequence, and the second pass and the
// chain go. A wave owns 64 channels, lane = channel with all N states, and takes
// token after token. B_t and C_t are the same for all lanes: they come through the
// scalar cache into scalar registers, which the products take as operands (their
// rows have to lie on 4-byte boundaries). Inputs are fetched K tokens ahead (2 and
// 4 tokens: 461 and 473 us).
// Bound by instruction issue: 16 exponentials (3.4 ns of a SIMD), 32 products with a
// scalar operand (1.9 ns) and about 60 others (1 ns) a token, 172 ns in all; 220 are
// measured (64 prompts of 8192 channels, 470 us, 2.6 TB/s). B and C as vector operands
// from LDS took as long: twice the registers, half the waves.
template <typename T, typename DT, int N, int K>
__global__ __launch_bounds__(64) void ssd_selective_walk_kernel(SelectiveArgs a) {
    using R = RawOf<T>;
    using RD = RawOf<DT>;
    using One = typename R::One;
    using OneD = typename RD::One;
    constexpr int ES = sizeof(One), ED = sizeof(OneD), W = N * ES / 4;   // W: dwords of a row of B or C
    typedef const __attribute__((address_space(4))) uint32_t scalar_words;
    if (__builtin_nontemporal_load(a.error_flag) & SSD_DATA_BAD_CU_SEQLENS) return;
    const int per = a.C_total / a.G, bpg = (per + 63) / 64, cblocks = a.G * bpg;
    const int rank = blockIdx.x / cblocks, cb = blockIdx.x - rank * cblocks;
    const int s = a.seq_order[rank];
    if (s < 0 || s >= a.S) return;
    int64_t tb = a.cu_seqlens[s], te = a.cu_seqlens[s + 1];
    tb = tb < 0 ? 0 : (tb > a.T ? a.T : tb);
    te = te < tb ? tb : (te > a.T ? a.T : te);
    const int L = (int)(te - tb);
    if (L > a.walk_to) return;   // the chain's
    const int g = cb / bpg, lane = threadIdx.x;
    const int d = g * per + min((cb - g * bpg) * 64 + lane, per - 1);   // (lanes past the end: copies of the last channel)
    const int64_t state_row = (int64_t)s * a.C_total * N, state_col = (int64_t)d * N;
    float h[N], rate[N];
    const bool start = a.init != nullptr && (a.has_init == nullptr || a.has_init[s] != 0);
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const f32x4 r = *reinterpret_cast<const f32x4 *>(a.A + state_col + n);
        const f32x4 v = start ? *reinterpret_cast<const f32x4 *>(a.init + state_row + state_col + n) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rate[n + i] = r[i];
            h[n + i] = v[i];
        }
    }
    auto save = [&](float *to) {
#pragma unroll
        for (int n = 0; n < N; n += 4)
            *reinterpret_cast<f32x4 *>(to + state_col + n) = f32x4{h[n], h[n + 1], h[n + 2], h[n + 3]};
    };
    const float bias = a.dt_bias != nullptr ? a.dt_bias[d] : 0.0f, skip = a.D != nullptr ? a.D[d] : 0.0f;
    // uniform row pointers, advanced token by token (strides are below 2^28 bytes), plus 32-bit lane offsets
    const uint32_t su = (uint32_t)a.u_stride * ES, sd = (uint32_t)a.dt_stride * ED, sy = (uint32_t)a.y_stride * ES,
                   sz = (uint32_t)(a.z ? a.z_stride : a.u_stride) * ES, sB = (uint32_t)a.B_stride * ES,
                   sC = (uint32_t)a.C_stride * ES;
    const char *pu = reinterpret_cast<const char *>(a.u) + tb * su, *pd = reinterpret_cast<const char *>(a.dt) + tb * sd;
    const char *pz = reinterpret_cast<const char *>(a.z ? a.z : a.u) + tb * sz;   // (no gate: u again, unused)
    char *py = reinterpret_cast<char *>(a.y) + tb * sy;
    const char *pB = reinterpret_cast<const char *>(a.B) + tb * sB + g * N * ES;
    const char *pC = reinterpret_cast<const char *>(a.C) + tb * sC + g * N * ES;
    const uint32_t offT = d * ES, offD = d * ED;

    One ru[K], rz[K];
    OneD rd[K];
    int ahead = 0;   // the token that the next fetch reads (past the end: the last one again)
    auto fetch = [&](int k) {
        ru[k] = load_at<One>(pu, offT);
        rd[k] = load_at<OneD>(pd, offD);
        rz[k] = load_at<One>(pz, offT);
        const bool more = ++ahead < L;
        pu += more ? su : 0;
        pd += more ? sd : 0;
        pz += more ? sz : 0;
    };
    auto value = [](const uint32_t (&w)[W], int n) -> float {
        if constexpr (ES == 4) return __uint_as_float(w[n]);
        else return __uint_as_float(n & 1 ? w[n / 2] & 0xffff0000u : w[n / 2] << 16);
    };
    auto token = [&](int k) {
        uint32_t wB[W], wC[W];
#pragma unroll
        for (int i = 0; i < W; ++i) wB[i] = ((scalar_words *)pB)[i];
#pragma unroll
        for (int i = 0; i < W; ++i) wC[i] = ((scalar_words *)pC)[i];
        const float u = R::f(ru[k]), delta = softplus_full(RD::f(rd[k]) + bias), du = delta * u,
                    delta2 = delta * kLog2e;
        const One z = rz[k];
        fetch(k);
        float y[2] = {skip * u, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            h[n] = fmaf(fast_exp2(delta2 * rate[n]), h[n], du * value(wB, n));
            y[n & 1] = fmaf(h[n], value(wC, n), y[n & 1]);
        }
        float v = y[0] + y[1];
        if (a.z != nullptr) v *= silu_full(R::f(z));
        store_at<T>(py, offT, (T)v);
        pB += sB;
        pC += sC;
        py += sy;
    };
    if (L > 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) fetch(k);
    }
    // chunks of the batch's grid, in runs of K tokens (K divides the chunk size)
    const int step = a.chunk_states != nullptr ? a.cs : L;
    int chunk = a.seq_chunk_start[s];
    for (int t0 = 0; t0 < L; t0 += step, ++chunk) {
        const int end = min(t0 + step, L);
        int t = t0;
        for (; t + K <= end; t += K) {
#pragma unroll
            for (int k = 0; k < K; ++k) token(k);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)   // the sequence's last tokens
            if (t + k < end) token(k);
        if (a.chunk_states != nullptr) {
            const int slot = chunk_slot(a, chunk, cb == 0 && lane == 0);
            if (slot >= 0) save(a.chunk_states + (int64_t)slot * a.C_total * N);
        }
    }
    save(a.final_states + state_row);
}

// ---------------------------------------------------------------------------
// Step. Memory-bound: the state slots are the traffic (8 N bytes a sequence and
// channel). Lanes own 4 consecutive states of one channel (N / 4 lanes a
// channel), so a workgroup moves whole contiguous runs; it takes SEQS sequences
// at once, whose slots and states are then on their way together and share the
// rates A.
constexpr int kSelStepThreads = 256;

template <typename T, typename DT, int N, int SEQS>
__global__ __launch_bounds__(kSelStepThreads) void ssd_selective_step_kernel(SelectiveArgs a) {
    constexpr int LPC = N / 4, CH = kSelStepThreads / LPC;   // lanes of a channel, channels of a workgroup
    using R = RawOf<T>;
    const int cblocks = (a.C_total + CH - 1) / CH;
    const int sg = blockIdx.x / cblocks, cb = blockIdx.x - sg * cblocks;
    const int nq = threadIdx.x % LPC, d = cb * CH + (int)threadIdx.x / LPC;
    if (d >= a.C_total) return;   // whole channels, so whole shuffle groups, leave together
    const int n0 = d / (a.C_total / a.G) * N + 4 * nq;
    const int64_t slot = (int64_t)a.C_total * N, at = (int64_t)d * N + 4 * nq;
    int ws[SEQS];
    bool taken[SEQS];
    f32x4 h[SEQS];
    // states first (the traffic), then the small operands
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const int s = sg * SEQS + k;
        h[k] = f32x4{0, 0, 0, 0};
        taken[k] = s < a.S;
        if (!taken[k]) continue;
        const int rs = a.read_slot[s];
        ws[k] = a.write_slot[s];
        if (rs >= a.num_slots || ws[k] >= a.num_slots) {   // refused: nothing read or written
            if (d == 0 && nq == 0 && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
            taken[k] = false;
            continue;
        }
        if (rs >= 0) h[k] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(a.cache + rs * slot + at));
    }
    const f32x4 rate = *reinterpret_cast<const f32x4 *>(a.A + at);
    const float bias = a.dt_bias != nullptr ? a.dt_bias[d] : 0.0f, skip = a.D != nullptr ? a.D[d] : 0.0f;
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        if (!taken[k]) continue;
        const int64_t s = sg * SEQS + k;
        const float u = load_f<T>(a.u, s * a.u_stride + d);
        const float delta = softplus_full(load_f<DT>(a.dt, s * a.dt_stride + d) + bias), du = delta * u,
                    delta2 = delta * kLog2e;
        const f32x4 bv = R::f4(*reinterpret_cast<const typename R::Four *>(reinterpret_cast<const T *>(a.B) + s * a.B_stride + n0));
        const f32x4 cv = R::f4(*reinterpret_cast<const typename R::Four *>(reinterpret_cast<const T *>(a.C) + s * a.C_stride + n0));
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[k][i] = fmaf(fast_exp2(delta2 * rate[i]), h[k][i], du * bv[i]);
            y = fmaf(h[k][i], cv[i], y);
        }
        if (ws[k] >= 0) __builtin_nontemporal_store(h[k], reinterpret_cast<f32x4 *>(a.cache + ws[k] * slot + at));
#pragma unroll
        for (int m = LPC / 2; m >= 1; m >>= 1) y += __shfl_xor(y, m, LPC);
        if (nq == 0) {
            y = fmaf(skip, u, y);
            if (a.z != nullptr) y *= silu_full(load_f<T>(a.z, s * a.z_stride + d));
            reinterpret_cast<T *>(a.y)[s * a.y_stride + d] = (T)y;
        }
    }
}

// Waves of a workgroup that splits sequences into segments: the fewer (sequence,
// 16 channels) pairs there are, the more. Microseconds with 2 / 4 / 8 / 16 waves:
// 16384 pairs (64 x 300 tokens) 390 / 395; 8192 (32 x 500) 324 / 320; 2560 (8 ragged
// prompts) 405 / 369 / 392 / 435; 1024 (4 x 4000) 362 / 300 / 320 / 346; 800 (5 x
// 4000) 355 / 272 / 278 / 309; 512 (2 x 8000) 670 / 359 / 320 / 350; 320 (1 x 8000)
// 670 / 335 / 269 / 295; 256 (1 x 8000) 564 / 273 / 197 / 184.
static int segment_waves(int64_t pairs) { return pairs >= 16384 ? 2 : pairs >= 768 ? 4 : pairs > 256 ? 8 : 16; }

// From this many (sequence, 64 channels) pairs on, 4 for every SIMD, sequences
// are walked (64 prompts of 3 to 490 tokens, 8192 channels, 8192 pairs: 665 us in
// segments, 470 walked; 4096 channels: 64 x 300 tokens, 4096 pairs, 375 and 354;
// 32 x 500 tokens 319 and 399; 16 x 1000 tokens 322 and 630).
constexpr int64_t kWalkPairs = 4096;
// A walk takes as long as its sequence, so one much longer than the others would
// be left over: those of more than 3 times the mean length go in segments.
constexpr int64_t kWalkTimesMean = 3;

// A step takes this many sequences to a workgroup where that still makes 8 workgroups for every CU (256 sequences of
// 5120 channels, 16 states: 1 / 2 / 4 / 8 sequences 41.8 / 39.7 / 40.9 / 98 us; 179 MB, so 4.5 TB/s).
constexpr int kStepSeqs = 2;
constexpr int64_t kStepFill = 2048;

template <typename T, typename DT, int N> struct SelectiveLaunch {
    // Sequences of more than a.walk_to tokens, among the `ranks` longest, in segments.
    static hipError_t segments(const SelectiveArgs &a, int64_t ranks, hipStream_t stream) {
        const int64_t blocks = ranks * a.G * ((a.C_total / a.G + kCh - 1) / kCh);
        const int waves = segment_waves(blocks);
        if (!fits_grid(blocks, 64 * waves)) return hipErrorInvalidConfiguration;
        constexpr int NBLK = N / 16;
        const size_t lds = sizeof(float) * (NBLK * 256 + ((2 * NBLK + 3) & ~3) + (size_t)waves * kSeg * 64);
        hipLaunchKernelGGL((ssd_selective_scan_kernel<T, DT, N>), dim3((unsigned)blocks), dim3(64 * waves), lds,
                           stream, a);
        return hipGetLastError();
    }
    static hipError_t scan(SelectiveArgs a, hipStream_t stream) {
        a.walk_to = -1;
        if constexpr (N <= 32) {
            const int64_t walks = (int64_t)a.S * a.G * ((a.C_total / a.G + 63) / 64);
            const bool scalar_rows = sizeof(T) == 4 || ((a.B_stride | a.C_stride) % 2 == 0 &&
                (reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C)) % 4 == 0);
            if (scalar_rows && walks >= kWalkPairs) {
                if (!fits_grid(walks, 64)) return hipErrorInvalidConfiguration;
                const int64_t limit = kWalkTimesMean * ((a.T + (int64_t)a.S - 1) / a.S);
                a.walk_to = (int32_t)(limit < a.T ? limit : a.T);
                const int64_t ranks = a.T / (a.walk_to + 1);   // no more sequences are that long
                if (ranks > 0) {
                    const hipError_t e = segments(a, ranks, stream);
                    if (e != hipSuccess) return e;
                }
                hipLaunchKernelGGL((ssd_selective_walk_kernel<T, DT, N, 2>), dim3((unsigned)walks), dim3(64), 0, stream,
                                   a);
                return hipGetLastError();
            }
        }
        return segments(a, a.S, stream);
    }
    template <int SEQS> static hipError_t steps(const SelectiveArgs &a, int64_t blocks, hipStream_t stream) {
        if (!fits_grid(blocks, kSelStepThreads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((ssd_selective_step_kernel<T, DT, N, SEQS>), dim3((unsigned)blocks), dim3(kSelStepThreads), 0,
                           stream, a);
        return hipGetLastError();
    }
    static hipError_t step(const SelectiveArgs &a, hipStream_t stream) {
        constexpr int CH = kSelStepThreads / (N / 4);
        const int64_t cblocks = (a.C_total + CH - 1) / CH;
        const int64_t groups = ((int64_t)a.S + kStepSeqs - 1) / kStepSeqs;
        if (groups * cblocks >= kStepFill) return steps<kStepSeqs>(a, groups * cblocks, stream);
        return steps<1>(a, a.S * cblocks, stream);
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
