// tables.cu -- a step's block tables, slot map, query starts and lengths from request lengths (sm_103a).
//
// What pkv_mgr_extend does row after row on the host is a prefix sum on the device: with need_i = the blocks that
// row i's new tokens take beyond its last one, row i gets the free blocks behind those of the rows before it, and its
// tokens the places behind theirs. A row is served if the sums up to it fit; sums only grow, so the rows served are
// those before the first that does not fit. Sums saturate at 2^31 - 1, above the largest max_tokens: a row whose tokens saturate
// fails, and blocks, never more than tokens, saturate no earlier.
//
// Everything that a row decides (its first token, its first free block) is worked out by every CTA for itself, 1,024
// rows at a time, and kept in shared memory; the tokens are then shared out by warps, 32 at a time, each finding its
// row by bisection (once for the whole warp where the 32 lie in one row). A fresh block's table entry is written
// with its first token, which this call always holds. Lengths and totals may be written over what they were read
// from, so one CTA alone writes them: behind its tokens where it does the whole call, in a launch of its own behind the
// CTAs that share many tokens, which counts while they work and writes when they are done.
//
// Bound by latency: the counts, the scan, free ids, stores one after the other. Calls behind one another in a graph take 3.5 us for
// 64 rows of a token each and 6.0 for 1,000 rows of 288,070 tokens (on the device alone 5.6; 41 by one CTA, 7.4 where the rows'
// launch does not begin early); launched one by one from the host 8.4 to 10 and 12 to 15.
#include "common.cuh"
#include "linear.h"

namespace pkv {
namespace {

constexpr int kRows = 1024;  // rows of a tile, one a thread
constexpr unsigned kMost = 0x7fffffffu;
constexpr int kShared = 8 * kRows;  // up to this many tokens one CTA does the whole call
constexpr int kEach = 2 * kRows;    // tokens of a CTA beyond that

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kMost); }

// Inclusive sums of two values over the block's threads (kRows of them); part: [2][32].
__device__ __forceinline__ void block_scan(unsigned& x, unsigned& y, unsigned (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x = sat_add(x, u), y = sat_add(y, v);
    }
    if (lane == 31) part[0][warp] = x, part[1][warp] = y;
    __syncthreads();
    if (warp < 2) {
        unsigned p = part[warp][lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned u = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) p = sat_add(p, u);
        }
        part[warp][lane] = p;
    }
    __syncthreads();
    if (warp > 0) x = sat_add(x, part[0][warp - 1]), y = sat_add(y, part[1][warp - 1]);
}

// TOKENS: tables and slots of the new tokens, shared by the grid. ROWS (one CTA): starts, lengths, totals.
template <bool TOKENS, bool ROWS>
__global__ void __launch_bounds__(kRows) extend_tables_kernel(const ExtendArgs a) {
    __shared__ unsigned s_part[2][32];
    __shared__ int s_start[kRows + 1];  // first token of each row of the tile
    __shared__ int s_len[kRows];        // its length before the call
    __shared__ unsigned s_block[kRows]; // its first free block, counted from `used`
    __shared__ int s_first;             // the tile's first row that does not fit
    __shared__ unsigned s_tok, s_blk;   // tokens and blocks up to the tile's end
    if (!ROWS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the rows' launch may begin to count
    const int tid = threadIdx.x, lane = tid & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    const unsigned warp_of_all = cta * (kRows / 32) + (tid >> 5), warps = ctas * (kRows / 32);
    const int used = *a.used;
    const bool bad_used = used < 0 || used > a.n_free;
    const unsigned avail = bad_used ? 0u : (unsigned)(a.n_free - used);
    unsigned flags = bad_used ? (unsigned)PKV_DEV_BAD_FREE_LIST : 0u;
    constexpr unsigned row_flags = PKV_DEV_BAD_CONTEXT_LEN | PKV_DEV_BAD_QUERY_RANGE;  // which every CTA finds
    unsigned tok = 0, blk = 0;  // before this tile
    int served = 0;
    bool open = true;
    int my_len = 0, my_new = 0;  // of this thread's row in the last tile
    for (int row0 = 0; row0 < a.n_seqs; row0 += kRows) {
        const int rows = min(kRows, a.n_seqs - row0);
        const int row = row0 + tid;
        int len = 0, count = 0, want = 0;
        if (tid < rows) {
            len = a.lens[row];
            count = a.new_tokens ? a.new_tokens[row] : 1;
            if (len < 0 || len > a.max_blocks * kBlock) flags |= PKV_DEV_BAD_CONTEXT_LEN, count = 0;
            else if (count < 0) flags |= PKV_DEV_BAD_QUERY_RANGE, count = 0;
        }
        my_len = len;
        if (tid == 0) s_first = kRows;
        const unsigned n_new = (unsigned)count;
        unsigned need = 0;
        if (count > 0) {
            want = (int)(((unsigned)len + n_new + kBlock - 1) / kBlock);  // (both below 2^31)
            need = (unsigned)(want - (len + kBlock - 1) / kBlock);
        }
        unsigned x = n_new, y = need;
        if (tid == 0) x = sat_add(x, tok), y = sat_add(y, blk);
        block_scan(x, y, s_part);  // (its barriers stand between s_first's two writers)
        if (!open || x > (unsigned)a.max_tokens || y > avail || want > a.max_blocks) atomicMin(&s_first, tid);
        __syncthreads();
        const int first = min(s_first, rows);
        const bool ok = tid < first;
        my_new = ok ? count : 0;
        if (first == 0) {
            if (tid == 0) s_tok = tok, s_blk = blk;
        } else if (tid == first - 1) {
            s_tok = x, s_blk = y;
        }
        __syncthreads();
        const unsigned end = s_tok;
        s_start[tid] = (int)(ok ? x - n_new : end);
        s_len[tid] = len;
        s_block[tid] = y - need;
        if (tid == 0) s_start[kRows] = (int)end;
        if (ROWS && tid < rows) a.query_start[row] = s_start[tid];
        served += first;
        open = open && first == rows;
        __syncthreads();
        // tokens tok .. end - 1 lie in rows 0 .. first - 1 of the tile
        for (unsigned t0 = TOKENS ? tok + warp_of_all * 32 : end; t0 < end; t0 += warps * 32) {
            const unsigned t = t0 + lane;
            int lo = 0, hi = first;  // s_start[lo] <= t0, and t0 < s_start[hi] or hi == first
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((unsigned)s_start[mid] <= t0) lo = mid; else hi = mid;
            }
            if (hi < first && (unsigned)s_start[hi] <= min(t0 + 31, end - 1)) {  // the 32 lie in several rows
                hi = first;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if ((unsigned)s_start[mid] <= t) lo = mid; else hi = mid;
                }
            }
            if (t < end) {
                const int pos = s_len[lo] + (int)(t - (unsigned)s_start[lo]);
                const int b = pos / kBlock, old = (s_len[lo] + kBlock - 1) / kBlock;
                int32_t* entry = a.tables + (size_t)(row0 + lo) * a.max_blocks + b;
                int id;
                if (b >= old) {
                    id = a.free_blocks[(size_t)used + s_block[lo] + (unsigned)(b - old)];
                    if (pos % kBlock == 0) *entry = id;
                    if ((unsigned)id >= (unsigned)a.num_blocks) flags |= PKV_DEV_BAD_FREE_LIST;
                } else {
                    id = *entry;
                    if ((unsigned)id >= (unsigned)a.num_blocks) flags |= PKV_DEV_BAD_BLOCK_ID;
                }
                a.slots[t] = (unsigned)id < (unsigned)a.num_blocks ? (int64_t)id * kBlock + pos % kBlock : -1;
            }
        }
        tok = end;
        blk = s_blk;
        __syncthreads();  // the tile's shared values have been read
    }
    if (TOKENS)
        for (unsigned t = tok + warp_of_all * 32 + lane; t < (unsigned)a.max_tokens; t += warps * 32) a.slots[t] = -1;
    if (flags && (cta == 0 || (flags & ~row_flags))) atomicOr(a.status, flags);
    if constexpr (ROWS) {
        if (tid == 0) a.query_start[a.n_seqs] = (int)tok;
        if (!TOKENS) grid_dependency_wait();  // the tokens' CTAs have read the lengths and `used`
        __syncthreads();  // the lengths and `used` have been read, query_start is written
        if (a.n_seqs <= kRows) {
            if (tid < a.n_seqs) a.new_lens[tid] = my_len + my_new;
        } else {
            for (int row = tid; row < a.n_seqs; row += kRows)
                a.new_lens[row] = a.lens[row] + (a.query_start[row + 1] - a.query_start[row]);
        }
        if (tid == 0) {
            a.totals[0] = used + (int)blk;
            a.totals[1] = served;
            a.totals[2] = (int)tok;
        }
    }
}

}  // namespace

cudaError_t launch_extend_tables(const ExtendArgs& a, cudaStream_t stream, int sms, int* n_launches) {
    *n_launches = 1;
    if (a.max_tokens <= kShared) {
        extend_tables_kernel<true, true><<<1, kRows, 0, stream>>>(a);
    } else {
        const long long ctas = ((long long)a.max_tokens + kEach - 1) / kEach;
        extend_tables_kernel<true, false><<<(unsigned)(ctas < sms ? ctas : sms), kRows, 0, stream>>>(a);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(kRows);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t err = cudaLaunchKernelEx(&cfg, extend_tables_kernel<false, true>, a);
        if (err != cudaSuccess) return err;
        *n_launches = 2;
    }
    return cudaGetLastError();
}

}  // namespace pkv
