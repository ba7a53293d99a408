// Block tables and slot maps of one step: which blocks the new tokens of every
// request take, where each token's keys and values go, which state slot a request
// reads and where the states after its tokens go. Request s has c = num_computed
// tokens and gets n = num_new more; with `block` tokens per block it needs
// ceil((c + n) / block) - ceil(c / block) new blocks, which come from the end of
// the free list in the order of the requests.
//
// Latency is all there is: a few integers per request and token. One workgroup
// scans the requests (two sums: tokens and blocks); where there are few tokens it
// writes their maps too, else a second kernel does.
#include "ssd_internal.h"

namespace ssd {

namespace {

constexpr int kTablesThreads = 1024;
// A step of no more tokens than this, and of no more requests than threads, is one launch.
constexpr int kTablesOneLaunch = 4096;

struct Scan2 {
    int tokens, blocks;
};

// Inclusive sums over the workgroup; `total` gets the sums of all.
__device__ __forceinline__ Scan2 workgroup_scan(Scan2 v, Scan2 *wave_total, Scan2 &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(v.tokens, off, 64), b = __shfl_up(v.blocks, off, 64);
        if (lane >= off) {
            v.tokens += t;
            v.blocks += b;
        }
    }
    __syncthreads();   // the totals before have been read
    if (lane == 63) wave_total[wave] = v;
    __syncthreads();
    total = Scan2{0, 0};
    for (int w = 0; w < kTablesThreads / 64; ++w) {
        if (w < wave) {
            v.tokens += wave_total[w].tokens;
            v.blocks += wave_total[w].blocks;
        }
        total.tokens += wave_total[w].tokens;
        total.blocks += wave_total[w].blocks;
    }
    return v;
}

// What the maps need of a request. Refused: end is 0.
struct Request {
    int start, computed, end, row;   // its first token in the batch; its tokens before and after the step; its table row
};

// The maps of token t, the j-th of request `seq`; `id` gives a block of its table.
template <typename F> __device__ __forceinline__ void map_token(const TablesArgs &a, int t, int seq, const Request &r, F &&id_of) {
    int pos = -1, slot = -1, state = -1;
    const int64_t p = (int64_t)r.computed + (t - r.start);
    if (r.end > 0 && t >= r.start && p < r.end) {
        pos = (int)p;
        const int at = pos / a.block, in = pos - at * a.block, id = id_of(at);
        if (id >= a.num_blocks) {
            if (a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_BLOCK);
        } else if (id >= 0) {
            slot = id * a.block + in;
            if (pos + 1 == r.end || in + 1 == a.block) state = id;
        }
    }
    a.token_seq[t] = seq;
    a.positions[t] = pos;
    a.slots[t] = slot;
    a.state_slot[t] = state;
}

// The request of token t: start(lo) <= t < start(hi).
template <typename F> __device__ __forceinline__ int request_of(int t, int lo, int hi, F &&start) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kTablesThreads) void ssd_step_tables_kernel(TablesArgs a, int tokens_here) {
    __shared__ Scan2 wave_total[kTablesThreads / 64];
    __shared__ Request requests[kTablesThreads];
    __shared__ struct { int first, before, need; } takes[kTablesThreads];
    __shared__ int left_s;
    const int tid = threadIdx.x;
    const int free_count = a.free_blocks != nullptr ? min(max(*a.free_count, 0), a.num_free) : 0;
    if (tid == 0) left_s = free_count;
    Scan2 carry{0, 0};
    bool bad_tokens = false;
    for (int base = 0; base < a.S; base += kTablesThreads) {
        const int s = base + tid;
        int c = 0, n = 0, row = 0, bits = 0, need = 0, first = 0;
        bool taken = false;
        if (s < a.S) {
            c = a.num_computed[s];
            n = a.num_new[s];
            row = a.rows != nullptr ? a.rows[s] : s;
            const int64_t end = (int64_t)c + n;
            if (n < 0 || n > a.T) {
                bits = SSD_DATA_BAD_CU_SEQLENS;
                n = 0;
            } else if (c < 0 || end > INT32_MAX) {
                bits = SSD_DATA_BAD_CU_SEQLENS;
            } else if (row < 0 || row >= a.table_rows) {
                bits = SSD_DATA_BAD_SLOT;
            } else if ((end + a.block - 1) / a.block > a.max_blocks) {
                bits = SSD_DATA_BAD_BLOCK;
            }
            taken = bits == 0;
            if (taken && a.free_blocks != nullptr) {
                first = (int)(((int64_t)c + a.block - 1) / a.block);
                need = (int)((end + a.block - 1) / a.block) - first;
            }
        }
        // the table's block of the last computed token, on its way during the sums
        int32_t *table = a.block_table + (int64_t)(taken ? row : 0) * a.max_blocks;
        int read = taken && c > 0 ? table[(c - 1) / a.block] : -1;
        Scan2 total;
        // (a request of more blocks than there are counts as one more than there are, so that the sums stay in 32 bits)
        const Scan2 incl = workgroup_scan(Scan2{n, min(need, free_count + 1)}, wave_total, total);
        const int before = carry.blocks + incl.blocks - min(need, free_count + 1), upto = carry.blocks + incl.blocks;
        if (s < a.S) {
            if (need > 0 && upto > free_count) {
                bits |= SSD_DATA_NO_BLOCK;
                taken = false;
                need = 0;
            }
            if (need > 0) atomicMin(&left_s, free_count - upto);
            if (!taken) read = -1;
            if (read >= a.num_blocks) {
                bits |= SSD_DATA_BAD_BLOCK;
                read = -1;
            }
            const int start = carry.tokens + incl.tokens - n, end = taken ? c + n : 0;
            a.cu_seqlens[s] = start;
            a.seq_lens[s] = end;
            a.read_slot[s] = max(read, -1);
            requests[tid] = Request{start, c, end, row};
            takes[tid].first = first;
            takes[tid].before = before;
            takes[tid].need = need;
            if (carry.tokens + incl.tokens > a.T) bad_tokens = true;
            if (bits != 0 && a.error_flag != nullptr) atomicOr(a.error_flag, bits);
        }
        const int from = carry.blocks, to = min(carry.blocks + total.blocks, free_count);
        carry.tokens = min(carry.tokens + total.tokens, (1 << 30) - 1);   // (so the next sums stay in 32 bits)
        carry.blocks = min(carry.blocks + total.blocks, free_count + 1);
        __syncthreads();
        // a thread per block taken, whatever request it belongs to
        for (int k = from + tid; k < to; k += kTablesThreads) {
            const int i = request_of(k, 0, min(kTablesThreads, a.S - base), [&](int j) { return takes[j].before; });
            const int j = k - takes[i].before;
            if (j < takes[i].need)
                a.block_table[(int64_t)requests[i].row * a.max_blocks + takes[i].first + j] = a.free_blocks[free_count - 1 - k];
        }
    }
    if (tid == 0) {
        a.cu_seqlens[a.S] = carry.tokens;
        if (a.free_count_out != nullptr) *a.free_count_out = left_s;
    }
    if (bad_tokens && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_CU_SEQLENS);
    // (one launch: all requests are in LDS)
    for (int t = tid; t < tokens_here; t += kTablesThreads) {
        int seq = -1;
        Request r{0, 0, 0, 0};
        if (t < carry.tokens) {
            seq = request_of(t, 0, a.S, [&](int i) { return requests[i].start; });
            r = requests[seq];
        }
        map_token(a, t, seq, r, [&](int at) {
            // (a new block from the list: what this launch writes to the table need not have arrived)
            const auto k = takes[seq];
            return at >= k.first && at - k.first < k.need ? a.free_blocks[free_count - 1 - (k.before + at - k.first)]
                                                          : a.block_table[(int64_t)r.row * a.max_blocks + at];
        });
    }
}

// The same as request_of by a whole wave, 64 places at a time.
__device__ __forceinline__ int request_of_wave(int t, int n, const int32_t *start) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = n;   // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, at = lo + lane * step;
        const uint64_t below = __ballot(at < hi && start[min(at, n)] <= t);   // lanes 0 .. k
        lo += (63 - __clzll(below)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The maps of many tokens, from what the first launch wrote. A workgroup's 256 tokens belong to a few requests: the
// first and the last bound every lane's search.
__global__ __launch_bounds__(256) void ssd_token_maps_kernel(TablesArgs a) {
    __shared__ int bound[2];
    const int t0 = (int)blockIdx.x * 256, t = t0 + (int)threadIdx.x, tokens = a.cu_seqlens[a.S];
    if (threadIdx.x < 128) {
        const int at = min(threadIdx.x < 64 ? t0 : t0 + 255, tokens - 1);
        const int seq = at >= 0 ? request_of_wave(at, a.S, a.cu_seqlens) : 0;
        if ((threadIdx.x & 63) == 0) bound[threadIdx.x >> 6] = seq;
    }
    __syncthreads();
    if (t >= a.T) return;
    int seq = -1;
    Request r{0, 0, 0, 0};
    if (t < tokens) {
        seq = request_of(t, bound[0], bound[1] + 1, [&](int i) { return a.cu_seqlens[i]; });
        r = Request{a.cu_seqlens[seq], a.num_computed[seq], a.seq_lens[seq], a.rows != nullptr ? a.rows[seq] : seq};
    }
    map_token(a, t, seq, r, [&](int at) { return a.block_table[(int64_t)r.row * a.max_blocks + at]; });
}

}  // namespace

hipError_t launch_step_tables(const TablesArgs &a, hipStream_t stream) {
    const bool one = a.T <= kTablesOneLaunch && a.S <= kTablesThreads;
    hipLaunchKernelGGL(ssd_step_tables_kernel, dim3(1), dim3(kTablesThreads), 0, stream, a, one ? a.T : 0);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || one || a.T == 0) return e;   // (no tokens, no maps)
    hipLaunchKernelGGL(ssd_token_maps_kernel, dim3((unsigned)((a.T + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ssd
