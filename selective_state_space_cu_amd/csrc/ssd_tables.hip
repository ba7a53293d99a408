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
// A step of no more tokens than this is one launch.
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

// The maps of token t, from the requests' sums and tables.
__device__ __forceinline__ void map_token(const TablesArgs &a, int t) {
    int seq = -1, pos = -1, slot = -1, state = -1;
    if (t < a.cu_seqlens[a.S]) {
        int lo = 0, hi = a.S;   // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
        }
        seq = lo;
        const int end = a.seq_lens[seq];   // 0 where the request was refused
        const int64_t p = (int64_t)a.num_computed[seq] + (t - a.cu_seqlens[seq]);
        if (end > 0 && p < end) {
            pos = (int)p;
            const int at = pos / a.block, in = pos - at * a.block;
            const int id = a.block_table[(int64_t)(a.rows != nullptr ? a.rows[seq] : seq) * a.max_blocks + at];
            if (id >= a.num_blocks) {
                if (a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_BLOCK);
            } else if (id >= 0) {
                slot = id * a.block + in;
                if (pos + 1 == end || in + 1 == a.block) state = id;
            }
        }
    }
    a.token_seq[t] = seq;
    a.positions[t] = pos;
    a.slots[t] = slot;
    a.state_slot[t] = state;
}

__global__ __launch_bounds__(kTablesThreads) void ssd_step_tables_kernel(TablesArgs a, int tokens_here) {
    __shared__ Scan2 wave_total[kTablesThreads / 64];
    __shared__ struct { int row, first, before, need; } take[kTablesThreads];
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
            a.cu_seqlens[s] = carry.tokens + incl.tokens - n;
            a.seq_lens[s] = taken ? c + n : 0;
            int read = -1;
            if (taken && c > 0) {
                read = max(a.block_table[(int64_t)row * a.max_blocks + (c - 1) / a.block], -1);
                if (read >= a.num_blocks) {
                    bits |= SSD_DATA_BAD_BLOCK;
                    read = -1;
                }
            }
            a.read_slot[s] = read;
            if (carry.tokens + incl.tokens > a.T) bad_tokens = true;
            if (bits != 0 && a.error_flag != nullptr) atomicOr(a.error_flag, bits);
        }
        carry.tokens = min(carry.tokens + total.tokens, (1 << 30) - 1);   // (so the next sums stay in 32 bits)
        carry.blocks = min(carry.blocks + total.blocks, free_count + 1);
        take[tid].row = row;
        take[tid].first = first;
        take[tid].before = before;
        take[tid].need = need;
        __syncthreads();
        for (int i = tid >> 6; i < kTablesThreads && base + i < a.S; i += kTablesThreads / 64) {   // a wave per request
            int32_t *table = a.block_table + (int64_t)take[i].row * a.max_blocks + take[i].first;
            for (int j = tid & 63; j < take[i].need; j += 64) table[j] = a.free_blocks[free_count - 1 - (take[i].before + j)];
        }
    }
    __syncthreads();
    if (tid == 0) {
        a.cu_seqlens[a.S] = carry.tokens;
        if (a.free_count_out != nullptr) *a.free_count_out = left_s;
    }
    if (bad_tokens && a.error_flag != nullptr) atomicOr(a.error_flag, SSD_DATA_BAD_CU_SEQLENS);
    __syncthreads();   // the sums and tables in memory are visible to the whole workgroup
    for (int t = tid; t < tokens_here; t += kTablesThreads) map_token(a, t);
}

__global__ __launch_bounds__(256) void ssd_token_maps_kernel(TablesArgs a) {
    const int t = (int)(blockIdx.x * 256 + threadIdx.x);
    if (t < a.T) map_token(a, t);
}

}  // namespace

hipError_t launch_step_tables(const TablesArgs &a, hipStream_t stream) {
    const bool one = a.T <= kTablesOneLaunch;
    hipLaunchKernelGGL(ssd_step_tables_kernel, dim3(1), dim3(kTablesThreads), 0, stream, a, one ? a.T : 0);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
    hipLaunchKernelGGL(ssd_token_maps_kernel, dim3((unsigned)((a.T + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ssd
