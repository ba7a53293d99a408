// Attention of new tokens over a paged cache of keys and values, its split plan,
// and the write of new keys and values to the cache.
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r . k_j),
// over the keys j <= position of r's token (and > position - window).
//
// One pass with a running maximum and sum. A workgroup takes a part of one
// sequence's keys for one kv head and 16 of its rows (tokens x query heads of the
// kv head), its waves take steps of 64 keys (32 in float32) in turn, and the
// parts of a sequence are joined by a second kernel. The split is planned on the
// device from the lengths: parts of equal length over the whole batch, so that
// there are enough of them whatever the lengths are.
//
// On the matrix cores both products are transposed, S^T = K Q^T and
// O^T = V^T P^T, so that a row of the softmax is a column of the accumulators (its
// maximum takes two lane exchanges, its factor none) and S^T is already the second
// product's right operand: lane (g, q) of S^T holds keys W g .. W g + W - 1 of row q
// (W: values of 16 bytes) once the rows of K are taken in the order key = W (q / 4) +
// 4 u + q mod 4 for the W / 4 tiles u of half a step. The cache holds values as (head dim, keys) so that the
// left operand V^T is contiguous in memory too: keys and values go from memory to
// the matrix cores without a transposition.
//
// What bounds it: memory. 64 sequences of 276 K keys, 8 kv heads of 128 bf16, take
// 190 us, 6.0 TB/s of keys and values (a copy reaches 5.1, reading alone 6 to 7);
// with head dim 64 and 256 the loads alone take as long as the whole. A wave holds
// the next step's loads (16 KB of keys, 8 of values) in registers while it
// computes one, two waves a SIMD.
#include <algorithm>

#include "ssd_elem.hpp"

namespace ssd {

namespace {

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kPartUnit = 256;       // parts are multiples of this many keys, a step of each wave (one sequence of 2000: 12.1 us, 15.2 with 512)
constexpr int kPartCost = 1;       // what a part's start and end cost, in such steps
constexpr int kPlanSearch = 1024;  // sequences among which the best length of the parts is looked for
constexpr int kPartsPerSlot = 8;   // workgroups aimed at (2048), over as many as there are CUs

template <typename T> struct Mma;
template <> struct Mma<__bf16> {
    // An exponent of all ones (infinities, NaN) carries into the sign's place.
    static constexpr uint32_t EXPONENT = 0x7f807f80u, CARRY = 0x00800080u, CARRIED = 0x80008000u;
    __device__ static f32x4 mac(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    // Probabilities are rounded to bf16 for the second product (a relative 2^-8 at most, as the output itself is); their sum
    // is taken before. A second product with what the rounding leaves off would make the error against float64 that of the
    // output's rounding alone (0.0016 relative where it is 0.0021) and takes 4 % longer: its registers do not fit.
    __device__ static u32x4 operand(const f32x4 (&p)[2]) {
        return u32x4{pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]), pack_bf16(p[1][0], p[1][1]),
                     pack_bf16(p[1][2], p[1][3])};
    }
};
template <> struct Mma<float> {
    static constexpr uint32_t EXPONENT = 0x7f800000u, CARRY = 0x00800000u, CARRIED = 0x80000000u;
    __device__ static f32x4 mac(const u32x4 &a, const u32x4 &b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
        return c;
    }
    __device__ static u32x4 operand(const f32x4 (&p)[1]) { return __builtin_bit_cast(u32x4, p[0]); }
};

template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Raw16 { uint32_t w[4]; };

constexpr int kMostKeys = 1 << 30;   // of a sequence: positions stay in 32 bits past a step's end

// Tokens and keys of one sequence, as the plan and the kernels see them.
struct Span {
    int t0, n, len, lo;   // first token, tokens, keys, first key that any token sees (a multiple of 32)
    bool bad;
};

__device__ __forceinline__ Span span_of(const int32_t *cu, const int32_t *lens, int s, int T, int max_new, int window) {
    Span r;
    r.t0 = cu != nullptr ? cu[s] : s;
    const int t1 = cu != nullptr ? cu[s + 1] : s + 1;
    r.bad = r.t0 < 0 || t1 < r.t0 || t1 > T || t1 - r.t0 > max_new || lens[s] > kMostKeys;
    r.n = r.bad ? 0 : t1 - r.t0;
    r.len = max(lens[s], 0);
    const int64_t lo = window > 0 ? (int64_t)r.len - r.n - window + 1 : 0;
    r.lo = lo > 0 ? (int)lo & ~31 : 0;
    return r;
}

__global__ __launch_bounds__(1024) void ssd_attention_plan_kernel(AttnPlanArgs a) {
    __shared__ int64_t wave_sum[16];
    __shared__ int keys_of[kPlanSearch];
    __shared__ unsigned long long best;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto scan = [&](int64_t v, int64_t &total) {   // inclusive
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t o = __shfl_up(v, off, 64);
            if (lane >= off) v += o;
        }
        __syncthreads();
        if (lane == 63) wave_sum[wave] = v;
        __syncthreads();
        total = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) v += wave_sum[w];
            total += wave_sum[w];
        }
        return v;
    };
    int64_t keys = 0;
    for (int s = tid; s < a.S; s += 1024) {
        const Span r = span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window);
        if (r.bad) atomicOr(a.error_flag, SSD_DATA_BAD_CU_SEQLENS);
        if (r.n > 0) keys += r.len - r.lo;
        if (a.S <= kPlanSearch) keys_of[s] = r.n > 0 ? r.len - r.lo : -1;
    }
    if (tid == 0) best = ~0ull;
    int64_t total;
    scan(keys, total);
    // At most max_parts - S parts (`least` units each, or more) and, by their remainders, one a sequence more.
    constexpr int kMostUnits = kMostKeys / kPartUnit;
    const uint32_t target = a.max_parts - a.S;
    const int64_t most = (total >> 31) == 0 ? ((uint32_t)total + target - 1) / target : (total + target - 1) / target;
    const int least = (int)min(max((most + kPartUnit - 1) / kPartUnit, (int64_t)1), (int64_t)kMostUnits), step = (7 * least + 63) / 64;
    auto units = [&](int candidate) { return min(least + candidate * step, kMostUnits); };
    // Of 64 lengths up to 8 times the shortest (or 64 units), the one by which the fullest CU has least to do: its workgroups, times their
    // steps and one more for start and end. One workgroup a CU reads a little slower than two (an eighth more), and
    // short parts even out what this leaves out (1/64 for each time the shortest). 8 kv heads of 128 bf16, parts of 1024
    // keys or, with more of them than 8 for each CU, longer / of this length, us: 30000 keys 27.9 / 27.7 (1024), 4
    // sequences of 10000 39.4 / 33.2 (1280), 100000 83.3 / 76.1, 64 of 48 to 7900 200 / 201 (1280 both), 32 with a window of
    // 4096 104 / 99, 8 tokens each of 16 of 3000 (64 heads, four tiles) 90 / 73.
    // (Not looked for where the shortest ones leave no CU two workgroups; the plan then takes 5 us instead of 8 to 11.)
    const bool search = a.S <= kPlanSearch && kPartsPerSlot * (total / kPartUnit + a.S) > target;
    if (search) {
        int parts[4] = {};
        for (int s = lane; s < a.S; s += 64)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // (whole units over units: short operands)
                const uint32_t keys = keys_of[s], of = (keys + kPartUnit - 1) / kPartUnit, k = units(4 * wave + c);
                parts[c] += keys_of[s] < 0 ? 0 : max((int)((of + k - 1) / k), 1);
            }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int x = 32; x >= 1; x >>= 1) parts[c] += __shfl_xor(parts[c], x);
            const uint32_t k = units(4 * wave + c), rounds = ((uint32_t)kPartsPerSlot * parts[c] + target - 1) / target;
            const uint64_t cost = (uint64_t)(rounds == 1 ? 9 : 8 * rounds) * ((k + kPartCost) * (64 + k / least));
            if (lane == 0) atomicMin(&best, (unsigned long long)(cost << 6 | (uint64_t)(4 * wave + c)));
        }
        __syncthreads();
    }
    const int part = kPartUnit * units(search ? (int)(best & 63) : 0);
    int64_t carry = 0;
    for (int base = 0; base < a.S; base += 1024) {
        const int s = base + tid;
        int64_t n = 0;
        if (s < a.S) {
            const Span r = span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window);
            if (r.n > 0) n = max(((int64_t)r.len - r.lo + part - 1) / part, (int64_t)1);
        }
        const int64_t incl = scan(n, total);
        if (s < a.S) a.part_start[s] = (int)(carry + incl - n);
        carry += total;
    }
    if (tid == 0) {
        a.part_start[a.S] = (int)carry;
        *a.part_keys = part;
    }
    __syncthreads();
    for (int p = tid; p < a.max_parts; p += 1024) {
        int seq = -1;
        if (p < carry) {
            int lo = 0, hi = a.S;   // part_start[lo] <= p < part_start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.part_start[mid] <= p) lo = mid; else hi = mid;
            }
            seq = lo;
        }
        a.part_seq[p] = seq;
    }
}

// How a step's keys and values pass from memory through registers and a wave's own LDS to its matrix operands. Memory is
// read in whole lines by neighbouring lanes (a key row is contiguous, a value row's keys of a step fill a line), which
// operands in the matrix layout are not: 16 rows, 64 bytes of each. Loads of those, straight to the operands, took 217
// us where these take 190 (64 sequences of 276 K keys, 8 kv heads of 128, bf16: 6.0 TB/s), as long as the same loads
// without any arithmetic: half lines do not go with the streaming policy that whole lines gain 10 % from.
template <typename T, int D> struct AttnShape {
    static constexpr int SZ = sizeof(T), W = 16 / SZ, U = W / 4;   // elements of 16 bytes; tiles of 16 keys of a half step
    static constexpr int KEYS = 16 * U, SK = 2 * KEYS;             // keys of a half step and of a step (128 bytes of a value row)
    static constexpr int CH = D / (4 * W), DB = D / 16;            // 16-byte pieces of a key row and lane; blocks of 16 of D
    static constexpr int KPARTS = D > 128 ? 2 : 1, VPARTS = D / 64;   // stages that a step's keys, and its values, pass in
    static constexpr int RB = D * SZ, KROWS = SK / KPARTS, DV = D / VPARTS;   // bytes of a key row; rows of a stage of keys, of values
    static constexpr int NK = KROWS * RB / 1024, NV = DV * 128 / 1024;      // loads of a stage
    // Rows lie 16 bytes further apart than they are long, so that the 16-byte pieces that a fragment read takes at once
    // fall on all banks (those of keys twice on half of them), and so that all offsets from a lane's first are constants.
    static constexpr int KPITCH = RB + 16, VPITCH = 128 + 16;
    static constexpr int STAGE = KROWS * KPITCH > DV * VPITCH ? KROWS * KPITCH : DV * VPITCH;
};

// STREAM: no other workgroup of the same sequence reads the keys and values that this one does (one tile of rows). Those of
// other sequences may, where tables share the blocks of a prefix; the host does not see that, and the policy then costs
// what it gains elsewhere, or more. With / without it, 32 heads of 128 on 8, bf16, us: 64 sequences of 4096 shared keys and
// some 300 of their own 84 / 81 (no block shared 187 / 211), 256 of 2048 and 100 154 / 137 (355 / 397), 16 of 16384 and
// 500 106 / 76 (180 / 204).
template <typename T, int D, bool STREAM>
__global__ __launch_bounds__(kAttnThreads) __attribute__((amdgpu_waves_per_eu(D > 128 ? 1 : 2))) void ssd_attention_kernel(AttnArgs a) {
    using SH = AttnShape<T, D>;
    using M = Mma<T>;
    constexpr int W = SH::W, U = SH::U, KEYS = SH::KEYS, SK = SH::SK, CH = SH::CH, DB = SH::DB, KPARTS = SH::KPARTS, VPARTS = SH::VPARTS, RB = SH::RB;
    constexpr int LDS = kAttnWaves * SH::STAGE > kAttnWaves * 16 * D * 4 ? kAttnWaves * SH::STAGE : kAttnWaves * 16 * D * 4;
    __shared__ __attribute__((aligned(16))) char lds[LDS];   // the waves' stages, then what they hand to the join
    __shared__ float wave_m[kAttnWaves][16], wave_l[kAttnWaves][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, q = lane & 15;
    // Workgroups go to the 8 XCDs in turn: the tiles of one part and head to the same one, one after the other, so that all
    // but the first find its lines in that L2 (64 sequences of 2000 to 4331 keys, 4 tokens, 4 kv heads with 8 query heads
    // each: 119 us, 168 with the tiles on any XCD; two tiles to a workgroup leave one wave a SIMD, 123 us).
    const int in = blockIdx.x % (8 * a.tiles), x = blockIdx.x / (8 * a.tiles) * 8 + in % 8;
    const int tile = in / 8, h = x % a.Hkv, p = x / a.Hkv;
    if (p >= a.max_parts) return;
    const int s = a.part_seq[p];
    if (s < 0) return;
    const Span sp = span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window);
    const int rows = sp.n * a.group;
    if (tile * 16 >= rows) return;
    const int first_part = a.part_start[s], nparts = a.part_start[s + 1] - first_part, part = *a.part_keys;
    // keys that the table holds
    const int trow = a.rows != nullptr ? a.rows[s] : s;
    const bool row_ok = trow >= 0 && trow < a.table_rows;
    const int64_t cap = row_ok ? (int64_t)a.max_blocks * a.block : 0;
    const int len = (int)min((int64_t)sp.len, cap);
    if (len < sp.len && p == first_part && h == 0 && tile == 0 && threadIdx.x == 0 && a.error_flag != nullptr)
        atomicOr(a.error_flag, row_ok ? SSD_DATA_BAD_BLOCK : SSD_DATA_BAD_SLOT);
    const int32_t *table = a.block_table + (int64_t)(row_ok ? trow : 0) * a.max_blocks;
    const int64_t begin64 = sp.lo + (int64_t)(p - first_part) * part;
    const int begin = (int)min(begin64, (int64_t)len), end = (int)min(begin64 + part, (int64_t)len);

    // this lane's row (a column of the accumulators)
    const int r = tile * 16 + q, token = min(r, rows - 1) / a.group;
    const int token0 = tile * 16 / a.group, token1 = min(tile * 16 + 15, rows - 1) / a.group;
    const int all_hi = sp.len - sp.n + token0, all_low = a.window > 0 ? sp.len - sp.n + token1 - a.window + 1 : 0;
    u32x4 qf[CH];
    {
        const int head = h * a.group + min(r, rows - 1) % a.group;
        const T *at = reinterpret_cast<const T *>(a.q) + (sp.t0 + token) * a.q_stride + (int64_t)head * D + W * g;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const Raw16<T> v = *reinterpret_cast<const Raw16<T> *>(at + 4 * W * c);
            qf[c] = r < rows ? u32x4{v.w[0], v.w[1], v.w[2], v.w[3]} : u32x4{0, 0, 0, 0};
        }
    }

    // Where a step's 16-key groups lie: every lane looks up the group of its 16 bytes of a value row (piece lane mod 8),
    // the groups of the keys are read from lanes. Keys past the end take the last group's place.
    const int group = W * (lane & 7) / 16, last = (len - 1) & ~15;
    auto block_of = [&](int key) { return (int)(__umulhi((uint32_t)key, a.block_magic) >> a.block_shift); };
    struct Place { int key, id; };   // first key of the lane's group, its block (not yet checked)
    auto place = [&](int key0) {
        const int key = min(key0 + 16 * group, last);
        return Place{key, table[block_of(key)]};
    };
    const int64_t head_bytes = (int64_t)a.block * RB;   // a kv head's keys, or values, of a block
    char *stage = lds + wave * SH::STAGE;
    char *put_key = stage + lane / (RB / 16) * SH::KPITCH + lane % (RB / 16) * 16;
    char *put_value = stage + (lane >> 3) * SH::VPITCH + (lane & 7) * 16;
    const char *get_key = stage + (W * (q >> 2) + (q & 3)) * SH::KPITCH + 16 * g, *get_value = stage + q * SH::VPITCH + 16 * g;
    u32x4 kr[SH::NK], vr[SH::NV];
    auto stream = [](const u32x4 *at) {
        if constexpr (STREAM) return __builtin_nontemporal_load(at);
        else return *at;
    };
    auto load_keys = [&](int key0, const Place &at, int part) {
        const int id = (uint32_t)at.id < (uint32_t)a.num_blocks ? at.id : 0;
        const uint64_t base = ((uint64_t)((int64_t)id * a.Hkv + h) * head_bytes) + (uint64_t)(at.key - block_of(at.key) * a.block) * RB;
        const int lrow = lane / (RB / 16), lpiece = lane % (RB / 16) * 16;
#pragma unroll
        for (int j = 0; j < SH::NK; ++j) {
            const int row0 = part * SH::KROWS + j * 1024 / RB, from = row0 / 16 * (16 / W);   // first row; a lane of its group
            const uint64_t gb = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)base, from) |
                                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(base >> 32), from) << 32;
            const int gkey = __builtin_amdgcn_readlane(at.key, from);
            const int row = min(key0 + row0 + lrow, len - 1) - gkey;
            kr[j] = stream(reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(a.k_cache) + gb + (uint32_t)(row * RB + lpiece)));
        }
    };
    auto load_values = [&](const Place &at, int part) {
        const int id = (uint32_t)at.id < (uint32_t)a.num_blocks ? at.id : 0;
        const int in = at.key - block_of(at.key) * a.block + W * (lane & 7) % 16;
        const char *from = reinterpret_cast<const char *>(a.v_cache) + ((int64_t)id * a.Hkv + h) * head_bytes +
                           ((int64_t)(part * SH::DV + (lane >> 3)) * a.block + in) * SH::SZ;
        const int64_t step = (int64_t)8 * a.block * SH::SZ;
#pragma unroll
        for (int j = 0; j < SH::NV; ++j) vr[j] = stream(reinterpret_cast<const u32x4 *>(from + j * step));
    };

    // The bits of 4 bytes of a value row, from key `at` on, that one of the tokens t0 .. t1 sees.
    auto seen_bits = [&](bool there, int at, int t0, int t1) {
        const int most = min(sp.len - sp.n + t1, len - 1), least = a.window > 0 ? sp.len - sp.n + t0 - a.window + 1 : 0;
        auto one = [&](int k) { return there && k <= most && k >= least; };
        return W == 4 ? (one(at) ? 0xffffffffu : 0u) : (one(at) ? 0x0000ffffu : 0u) | (one(at + 1) ? 0xffff0000u : 0u);
    };

    f32x4 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;   // of this lane's row; l over this lane's keys only
    constexpr int STRIDE = SK * kAttnWaves;
    int key = begin + wave * SK;
    Place now{0, 0}, next{0, 0};
    if (key < end) {
        now = place(key);
        load_keys(key, now, 0);
        load_values(now, 0);
        next = place(key + STRIDE);
    }
    for (; key < end; key += STRIDE) {
        const bool more = key + STRIDE < end;
        const uint64_t there = __ballot((uint32_t)now.id < (uint32_t)a.num_blocks);   // lane 16 / W i: the block of group i
        f32x4 sc[2][U];
#pragma unroll
        for (int part = 0; part < KPARTS; ++part) {
#pragma unroll
            for (int j = 0; j < SH::NK; ++j) {
                *reinterpret_cast<u32x4 *>(put_key + j * 1024 / RB * SH::KPITCH) = kr[j];
            }
            __builtin_amdgcn_sched_barrier(0);   // (loads ahead of the stores would need registers of their own)
            if (part + 1 < KPARTS) load_keys(key, now, part + 1);
            else if (more) load_keys(key + STRIDE, next, 0);
#pragma unroll
            for (int n = part; n < 2; n += KPARTS)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int row = (KPARTS == 1 ? KEYS * n : 0) + 4 * u;
                    sc[n][u] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        sc[n][u] = M::mac(*reinterpret_cast<const u32x4 *>(get_key + row * SH::KPITCH + 64 * c), qf[c], sc[n][u]);
                    sc[n][u] *= a.scale_log2;
                    __builtin_amdgcn_sched_barrier(0);   // (all fragments at once do not fit the registers)
                }
        }
        auto ok = [&](int n) { return (there >> ((KEYS * n + W * g) / W & ~(16 / W - 1)) & 1) != 0; };   // the block of this lane's keys
        const bool masked = key + SK - 1 > all_hi || key + SK > len || key < all_low || ~there != 0;   // uniform
        if (masked) {
            if (~there != 0 && a.error_flag != nullptr) {
                // (a block of which no token sees a key, before the first one's window, may be gone)
                const bool gone = (uint32_t)now.id >= (uint32_t)a.num_blocks &&
                                  (a.window == 0 || (int64_t)now.key + 15 + a.window > (int64_t)sp.len - sp.n);
                if (__any(gone) && lane == 0) atomicOr(a.error_flag, SSD_DATA_BAD_BLOCK);
            }
            int of = token;
            asm("" : "+v"(of));   // (no registers for the borders outside)
            const int hi = min(sp.len - sp.n + of, len - 1), low = a.window > 0 ? sp.len - sp.n + of - a.window + 1 : 0;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = key + KEYS * n + W * g + 4 * u + i;
                        if (!(ok(n) && at <= hi && at >= low)) sc[n][u][i] = -INFINITY;
                    }
        }
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[n][u][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > m)) {
            const float best = fmaxf(m, top), f = best == -INFINITY ? 1.0f : fast_exp2(m - best);
            m = best;
            l *= f;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        u32x4 pf[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[n][u][i] = fast_exp2(sc[n][u][i] - base);
                    l += sc[n][u][i];
                }
            pf[n] = M::operand(sc[n]);
        }
#pragma unroll
        for (int part = 0; part < VPARTS; ++part) {
#pragma unroll
            for (int j = 0; j < SH::NV; ++j) *reinterpret_cast<u32x4 *>(put_value + 8 * j * SH::VPITCH) = vr[j];
            __builtin_amdgcn_sched_barrier(0);
            bool apart = false;   // uniform
            if (masked && token0 < token1) {
                uint32_t odd = 0;
                int from_key = key;
                asm("" : "+s"(from_key));   // (no registers for the masks outside)
                const bool here = (uint32_t)now.id < (uint32_t)a.num_blocks;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t of = seen_bits(here, from_key + W * (lane & 7) + i * (W / 4), token0, token1) & M::EXPONENT;
#pragma unroll
                    for (int j = 0; j < SH::NV; ++j) odd |= (vr[j][i] & of) + M::CARRY;
                }
                apart = __any((odd & M::CARRIED) != 0);
            }
            if (part + 1 < VPARTS) load_values(now, part + 1);
            else if (more) load_values(next, 0);
            uint32_t from = lds_addr(get_value);
            auto value = [&](int db, int n) { return *(const __attribute__((address_space(3))) u32x4 *)(uintptr_t)(from + 16 * db * SH::VPITCH + 64 * n); };
            if (!masked) {
#pragma unroll
                for (int db = 0; db < DB / VPARTS; ++db)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        o[part * DB / VPARTS + db] = M::mac(value(db, n), pf[n], o[part * DB / VPARTS + db]);
                        if (n == 1 && db % 2 == 1) __builtin_amdgcn_sched_barrier(0);
                    }
            } else {
                // What a token does not see may hold anything, and 0 x infinity is no 0: values that no token of the tile
                // sees are cleared. Where one that some see is not finite, that is done token by token, and only that
                // token's rows take the sum (always doing so: 8 sequences of 4000 keys, 4 tokens each, 32 heads of 128 on 8
                // bf16, 34.5 us for 31.6; the look costs single tokens at most 0.6 us of 12, none at head dim 128).
                for (int t = apart ? token0 : token1; t <= token1; ++t) {
                    asm("" : "+v"(from));   // (the values are read again for every token: all of them do not fit the registers)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint32_t seen[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) seen[i] = seen_bits(ok(n), key + KEYS * n + W * g + i * (W / 4), apart ? t : token0, t);
#pragma unroll
                        for (int db = 0; db < DB / VPARTS; ++db) {
                            const u32x4 v = value(db, n);
                            f32x4 &to = o[part * DB / VPARTS + db];
                            const f32x4 with = M::mac(u32x4{v[0] & seen[0], v[1] & seen[1], v[2] & seen[2], v[3] & seen[3]}, pf[n], to);
                            if (token == t || !apart) to = with;
                        }
                    }
                }
            }
        }
        now = next;
        if (more) next = place(key + 2 * STRIDE);
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the waves
    if (g == 0) {
        wave_m[wave][q] = m;
        wave_l[wave][q] = l;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, wave_m[w][q]);
    const float f = top == -INFINITY ? 0.0f : fast_exp2(m - top);
    float *red = reinterpret_cast<float *>(lds);   // (wave, row, D), four values of a row at a time in the row's own order
    auto red_at = [&](int w, int row, int d4) { return ((w * 16 + row) * (D / 4) + (d4 ^ (row & 15))) * 4; };
#pragma unroll
    for (int db = 0; db < DB; ++db) *reinterpret_cast<f32x4 *>(red + red_at(wave, q, 4 * db + g)) = o[db] * f;
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += kAttnThreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4, rr = tile * 16 + row;
        if (rr >= rows) break;
        float best = -INFINITY, sum = 0.0f;
        for (int w = 0; w < kAttnWaves; ++w) best = fmaxf(best, wave_m[w][row]);
        f32x4 v{0, 0, 0, 0};
        for (int w = 0; w < kAttnWaves; ++w) {
            // (where no product is above -infinity the waves' sums are 0, or NaN if one is NaN, which no maximum shows)
            sum += best == -INFINITY ? wave_l[w][row] : wave_l[w][row] * fast_exp2(wave_m[w][row] - best);
            v += *reinterpret_cast<const f32x4 *>(red + red_at(w, row, d / 4));
        }
        if (nparts == 1) {
            const int64_t t = sp.t0 + rr / a.group;
            const int head = h * a.group + rr % a.group;
            T *out = reinterpret_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D + d;
            const float inv = best == -INFINITY ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = (T)(v[k] * inv);
            if (a.lse != nullptr && d == 0) a.lse[t * a.Hq + head] = (best + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
        } else {
            const int64_t at = ((int64_t)p * a.Hkv + h) * a.max_new * a.group + rr;
            *reinterpret_cast<f32x4 *>(a.part_o + at * D + d) = v;
            if (d == 0) {
                a.part_ml[2 * at] = best;
                a.part_ml[2 * at + 1] = sum;
            }
        }
    }
}

// Joins the parts of sequences that have several: blocks_per_token workgroups a token take its heads in turn.
template <typename T, int D>
__global__ __launch_bounds__(256) void ssd_attention_join_kernel(AttnArgs a, int blocks_per_token) {
    constexpr int LANES = D / 4, GROUPS = 256 / LANES;
    __shared__ float red[GROUPS][D], red_m[4], red_l[GROUPS];
    __shared__ int found;
    const int t = blockIdx.x / blocks_per_token;
    int s = t;
    if (a.cu_seqlens != nullptr) {
        int lo = 0, hi = a.S;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
        }
        s = lo;
    }
    Span sp = span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window);
    auto has = [t](const Span &r) { return t >= r.t0 && t < r.t0 + r.n; };
    if (!has(sp)) {   // behind the last sequence, or sequences left out have misled the search: look at each
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        for (s = threadIdx.x; s < a.S; s += 256)
            if (has(span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window))) atomicMax(&found, s);
        __syncthreads();
        s = found;
        if (s < 0) return;
        sp = span_of(a.cu_seqlens, a.seq_lens, s, a.T, a.max_new, a.window);
    }
    const int first = a.part_start[s], nparts = a.part_start[s + 1] - first;
    if (nparts <= 1) return;
    const int rows = a.max_new * a.group;
    for (int head = blockIdx.x % blocks_per_token; head < a.Hq; head += blocks_per_token) {
        const int r = (t - sp.t0) * a.group + head % a.group, h = head / a.group;
        // the largest maximum, then the sums: independent loads, so that all of a lane's are on their way at once
        const int64_t at0 = ((int64_t)first * a.Hkv + h) * rows + r, step = (int64_t)a.Hkv * rows;
        float best = -INFINITY;
        for (int k = threadIdx.x; k < nparts; k += 256) best = fmaxf(best, a.part_ml[2 * (at0 + k * step)]);
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1) best = fmaxf(best, __shfl_xor(best, x));
        __syncthreads();   // the head before has been read
        if ((threadIdx.x & 63) == 0) red_m[threadIdx.x >> 6] = best;
        __syncthreads();
        best = fmaxf(fmaxf(red_m[0], red_m[1]), fmaxf(red_m[2], red_m[3]));
        const float base = best == -INFINITY ? 0.0f : best;
        const int grp = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
        float l = 0.0f;
        f32x4 v{0, 0, 0, 0};
#pragma unroll 4
        for (int k = grp; k < nparts; k += GROUPS) {
            const int64_t at = at0 + k * step;
            const float e = fast_exp2(a.part_ml[2 * at] - base);
            l += a.part_ml[2 * at + 1] * e;
            v += *reinterpret_cast<const f32x4 *>(a.part_o + at * D + d) * e;
        }
        *reinterpret_cast<f32x4 *>(&red[grp][d]) = v;
        if (d == 0) red_l[grp] = l;
        __syncthreads();
        if (grp != 0) continue;
        l = 0.0f;
        v = f32x4{0, 0, 0, 0};
        for (int k = 0; k < GROUPS; ++k) {
            l += red_l[k];
            v += *reinterpret_cast<const f32x4 *>(&red[k][d]);
        }
        T *out = reinterpret_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D + d;
        const float inv = best == -INFINITY ? 0.0f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = (T)(v[k] * inv);
        if (a.lse != nullptr && d == 0) a.lse[(int64_t)t * a.Hq + head] = (best + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
}

// Copies the rows of new tokens to their slots: keys as they are, values turned. One token and 16 bytes of its row a lane:
// for few tokens, whose slots lie apart anyway.
template <typename T>
__global__ __launch_bounds__(256) void ssd_kv_write_kernel(KvWriteArgs a) {
    constexpr int W = 16 / sizeof(T);
    const int per = a.Hkv * a.D / W;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / per;
    if (t >= a.T) return;
    const int e = (int)(i - t * per) * W, h = e / a.D, d = e % a.D;
    const int slot = a.slots[t];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (e == 0 && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
        return;
    }
    const int block = slot / a.block, at = slot - block * a.block;
    const Raw16<T> k = *reinterpret_cast<const Raw16<T> *>(reinterpret_cast<const T *>(a.k) + t * a.k_stride + e);
    const T *v = reinterpret_cast<const T *>(a.v) + t * a.v_stride + e;
    const int64_t head = ((int64_t)block * a.Hkv + h) * a.block * a.D;
    *reinterpret_cast<Raw16<T> *>(reinterpret_cast<T *>(a.k_cache) + head + (int64_t)at * a.D + d) = k;
    T *vc = reinterpret_cast<T *>(a.v_cache) + head + (int64_t)d * a.block + at;
#pragma unroll
    for (int j = 0; j < W; ++j) vc[(int64_t)j * a.block] = v[j];
}

// The same for many tokens: 64 tokens of one head a workgroup, the values turned in LDS, so that a store's lanes are
// tokens, whose places in a prompt's block follow each other: a store writes whole lines of the values (single values
// scattered took 6 times as long). 35576 tokens x 8 heads x 128 bf16 take 55 us, 5.3 TB/s, a large copy's rate; 69 without
// the streaming policy on what is read and on the keys, 80 with it on the values too, whose lines two stores fill. Other
// rows, times a copy's: 1.1 (64 values bf16), 1.0 (64 and 256 float32), but 1.8 to 1.9 for 256 bf16 and 128 float32 (219 and
// 207 us for 35576 x 8), whose two tiles, wholly in registers, leave one wave a SIMD.
template <typename T, int D>
__global__ __launch_bounds__(256) void ssd_kv_write_tile_kernel(KvWriteArgs a) {
    constexpr int W = 16 / sizeof(T), PER = D / W, ROW = D * sizeof(T) + 8;   // 16-byte pieces of a row; its bytes in LDS
    constexpr int ROUNDS = 64 * PER / 256, WORDS = D * sizeof(T) / 4;
    __shared__ __attribute__((aligned(16))) char tile[64 * ROW];
    __shared__ int slots[64];
    const int h = blockIdx.x % a.Hkv;
    const int64_t t0 = (int64_t)(blockIdx.x / a.Hkv) * 64;
    if (threadIdx.x < 64) {
        int slot = t0 + threadIdx.x < a.T ? a.slots[t0 + threadIdx.x] : -1;
        if (slot >= a.num_slots) {
            if (h == 0 && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_SLOT);
            slot = -1;
        }
        slots[threadIdx.x] = slot;
    }
    typedef u32x4 Vec __attribute__((aligned(2)));   // (rows start on any element)
    u32x4 k[ROUNDS], v[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = r * 256 + threadIdx.x;
        const int64_t t = t0 + i / PER, e = (int64_t)h * D + i % PER * W;
        if (t < a.T) {
            k[r] = __builtin_nontemporal_load(reinterpret_cast<const Vec *>(reinterpret_cast<const T *>(a.k) + t * a.k_stride + e));
            v[r] = __builtin_nontemporal_load(reinterpret_cast<const Vec *>(reinterpret_cast<const T *>(a.v) + t * a.v_stride + e));
        }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = r * 256 + threadIdx.x;
        u32x2 *to = reinterpret_cast<u32x2 *>(tile + i / PER * ROW + i % PER * 16);
        to[0] = u32x2{v[r][0], v[r][1]};
        to[1] = u32x2{v[r][2], v[r][3]};
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = r * 256 + threadIdx.x, slot = slots[i / PER];
        if (slot < 0) continue;
        const int block = slot / a.block, at = slot - block * a.block;
        T *to = reinterpret_cast<T *>(a.k_cache) + (((int64_t)block * a.Hkv + h) * a.block + at) * D + i % PER * W;
        __builtin_nontemporal_store(k[r], reinterpret_cast<u32x4 *>(to));
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, slot = slots[lane];
    if (slot < 0) return;
    const int block = slot / a.block, at = slot - block * a.block;
    T *to = reinterpret_cast<T *>(a.v_cache) + ((int64_t)block * a.Hkv + h) * a.block * D + at;
#pragma unroll 8
    for (int w = wave; w < WORDS; w += 4) {
        const uint32_t word = *reinterpret_cast<const uint32_t *>(tile + lane * ROW + 4 * w);
        if constexpr (sizeof(T) == 4) {
            to[(int64_t)w * a.block] = __uint_as_float(word);
        } else {
            uint16_t *at2 = reinterpret_cast<uint16_t *>(to) + (int64_t)2 * w * a.block;
            at2[0] = (uint16_t)word;
            at2[a.block] = (uint16_t)(word >> 16);
        }
    }
}

constexpr int kJoinWorkgroups = 2048;

template <typename T, int D> hipError_t launch_attention_d(const AttnArgs &a, hipStream_t stream) {
    // (many tokens have few parts each, or none: no more workgroups than see to that at once)
    const int per_token = std::max(1, std::min(a.Hq, (kJoinWorkgroups + a.T - 1) / a.T));
    const int64_t blocks = ((int64_t)a.max_parts * a.Hkv + 7) / 8 * 8 * a.tiles, joins = (int64_t)a.T * per_token;
    if (!fits_grid(blocks, kAttnThreads) || !fits_grid(joins, 256)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kAttnThreads);
    if (a.tiles == 1) hipLaunchKernelGGL((ssd_attention_kernel<T, D, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((ssd_attention_kernel<T, D, false>), grid, block, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssd_attention_join_kernel<T, D>), dim3((unsigned)joins), dim3(256), 0, stream, a, per_token);
    return hipGetLastError();
}

template <typename T> hipError_t launch_attention_t(const AttnArgs &a, int D, hipStream_t stream) {
    switch (D) {
        case 64: return launch_attention_d<T, 64>(a, stream);
        case 128: return launch_attention_d<T, 128>(a, stream);
        case 256: return launch_attention_d<T, 256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_attention_plan(const AttnPlanArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL(ssd_attention_plan_kernel, dim3(1), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs &a, bool bf16, int D, hipStream_t stream) {
    return bf16 ? launch_attention_t<__bf16>(a, D, stream) : launch_attention_t<float>(a, D, stream);
}

// From this many rows of heads on the values are turned in LDS (128 bf16: a prompt of 512 / 1024 tokens x 8 heads 5.6 / 6.5
// us, 6.2 / 10.2 without; 2048 / 4096 x 2 heads 5.5 / 6.1, 4.5 / 6.6 without; 512 / 1024 single tokens x 8 heads 14.0 / 16.3,
// 7.9 / 23.2 without. Prompts of 1024 x 8 of the other rows, 64 and 256 bf16, 64, 128 and 256 float32: 3.7, 10.7, 4.7, 9.9 and
// 9.5; 6.7, 15.9, 7.7, 12.7 and 19.0 without).
constexpr int64_t kTileRows = 8192;

template <typename T> static hipError_t launch_kv_write_t(const KvWriteArgs &a, hipStream_t stream) {
    const bool tiles = (int64_t)a.T * a.Hkv >= kTileRows;
    const int64_t lanes = (int64_t)a.T * a.Hkv * a.D * sizeof(T) / 16;
    const int64_t blocks = tiles ? ((int64_t)a.T + 63) / 64 * a.Hkv : (lanes + 255) / 256;
    if (!fits_grid(blocks, 256)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(256);
    if (!tiles) hipLaunchKernelGGL((ssd_kv_write_kernel<T>), grid, block, 0, stream, a);
    else if (a.D == 64) hipLaunchKernelGGL((ssd_kv_write_tile_kernel<T, 64>), grid, block, 0, stream, a);
    else if (a.D == 128) hipLaunchKernelGGL((ssd_kv_write_tile_kernel<T, 128>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((ssd_kv_write_tile_kernel<T, 256>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_kv_write(const KvWriteArgs &a, bool bf16, hipStream_t stream) {
    return bf16 ? launch_kv_write_t<__bf16>(a, stream) : launch_kv_write_t<float>(a, stream);
}

}  // namespace ssd
