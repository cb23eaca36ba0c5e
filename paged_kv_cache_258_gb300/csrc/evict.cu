// evict.cu -- eviction from the cache by accumulated attention weight (sm_103a).
//
// For every (layer, sequence s, KV head g), c = lens[s], k = min(keep[s], c), R = min(recent, k): the
// last R positions stay, and of the first c - R the k - R with the largest score (ties: the lower
// position; NaN counts as largest). The kept rows of K and V move, in order of position, to logical
// positions 0 .. k-1 of the destination table, their scores with them; scores in [k, c) become 0.
// Heads and layers choose for themselves: a table is shared by all of them, but each has its own rows.
//
// Two launches. Both are bound by memory when they have enough (sequence, head, layer) triples, the
// second by far the larger: 2 k row bytes each way against 8 c + 4 k of the first.
//  1. select: one CTA per triple. The (k - R)-th largest score is found by a radix select over the
//     scores' ordered bits (11 + 11 + 10 bits, histograms in shared memory), then one ordered sweep
//     numbers the kept positions with a block-wide scan and writes them and their scores. The sweep may
//     run in place: it writes index i only after every score up to that position has been read, and the
//     i-th kept position is never below i.
//     For 8-bit pools it also reads the old scales of all the sequence's blocks aside and writes each
//     destination block's new scale, the largest among its rows' (a power of two like them, so the
//     codes only shift).
//  2. move: CTAs own column slices of a triple's rows, so two CTAs never touch the same bytes and a
//     sequence can be compacted in place without any order between CTAs. A CTA walks the kept list in
//     chunks; the loads of a chunk are all done before its stores (a barrier). Row i of chunk n is read
//     from a position >= i, so loads of later chunks never see an earlier chunk's stores.
#include <math.h>

#include "common.cuh"
#include "shrink.h"

namespace pkv {
namespace {

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;

// Scores as integers in the same order; NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sums of two counts packed as (a in the low, b in the high half) over the CTA; *total gets
// the whole sum. Counts stay below 2^16.
__device__ __forceinline__ uint32_t scan2(uint32_t v, uint32_t* s_warp, uint32_t* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's reads are done
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        const uint32_t y = s_warp[w];
        if (w < warp) before += y;
        all += y;
    }
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
    __shared__ uint32_t s_hist[kBins];
    __shared__ uint32_t s_warp[kSelThreads / 32];
    __shared__ uint32_t s_pick[2];
    const long long pair = blockIdx.x;  // s * n_kv + g
    const int s = (int)(pair / a.n_kv), g = (int)(pair % a.n_kv), layer = blockIdx.y;
    const int cap = a.max_blocks * kBlock;
    grid_launch_dependents();
    grid_dependency_wait();
    const int c = a.lens[s], want = a.keep[s];
    if (c < 0 || c > cap || want < 0 || min(want, c) > a.max_keep) {
        if (threadIdx.x == 0 && g == 0 && layer == 0)
            atomicOr(a.status, (unsigned)(c < 0 || c > cap ? PKV_DEV_BAD_CONTEXT_LEN : PKV_DEV_BAD_KEEP));
        return;
    }
    const int k = min(want, c);
    const int recent = min(a.recent, k);
    const int older = c - recent;
    const int pick = k - recent;  // of the first `older` positions
    const size_t triple = (size_t)layer * a.n_seqs * a.n_kv + pair;
    const float* score = a.scores + triple * a.stride;
    float* out = a.new_scores + triple * a.stride;
    int32_t* kept = a.kept + triple * a.max_keep;

    // threshold: positions above it are kept, of those equal to it the first `ties`
    uint32_t threshold = 0xffffffffu, ties = 0;
    if (pick == older) {
        threshold = 0;
        ties = (uint32_t)older;
    } else if (pick > 0) {
        uint32_t prefix = 0, mask = 0, left = (uint32_t)pick;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            for (int i = threadIdx.x; i < kBins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < older; j += kSelThreads) {
                const uint32_t key = order_key(score[j]);
                if ((key & mask) == prefix) atomicAdd(&s_hist[(key >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // bins from the top: thread t sums bins (kBins-1-4t .. kBins-4-4t)
            constexpr int PER = kBins / kSelThreads;
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += s_hist[kBins - 1 - (threadIdx.x * PER + i)];
            uint32_t above = mine;
            {
                const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
                    if (lane >= o) above += y;
                }
                if (lane == 31) s_warp[warp] = above;
                __syncthreads();
                for (int w = 0; w < warp; ++w) above += s_warp[w];
                above -= mine;
            }
            if (above < left && above + mine >= left) {  // the bin that holds the left-th largest is here
                uint32_t n = above;
                for (int i = 0; i < PER; ++i) {
                    const int bin = kBins - 1 - (threadIdx.x * PER + i);
                    const uint32_t h = s_hist[bin];
                    if (n + h >= left) {
                        s_pick[0] = (uint32_t)bin;
                        s_pick[1] = left - n;
                        break;
                    }
                    n += h;
                }
            }
            __syncthreads();
            prefix |= s_pick[0] << shift;
            mask |= ((1u << bits) - 1) << shift;
            left = s_pick[1];
            __syncthreads();
        }
        threshold = prefix;
        ties = left;
    }

    // ordered sweep: number the kept positions, move their scores
    uint32_t n_above = 0, n_equal = 0;  // kept above the threshold and equal to it, so far
    for (int j0 = 0; j0 < c; j0 += kSelThreads) {
        const int j = j0 + threadIdx.x;
        float x = 0.f;
        uint32_t above = 0, equal = 0;
        if (j < c) {
            x = score[j];
            const uint32_t key = order_key(x);
            if (j >= older) above = 1;
            else if (key > threshold) above = 1;
            else if (key == threshold) equal = 1;
        }
        uint32_t total;
        const uint32_t at = scan2(above | (equal << 16), s_warp, &total);  // its barriers end the reads of this chunk
        const uint32_t eq_before = n_equal + (at >> 16), ab_before = n_above + (at & 0xffffu);
        if (above || (equal && eq_before < ties)) {
            const uint32_t i = ab_before + min(eq_before, ties);
            kept[i] = j;
            out[i] = x;
        }
        n_above += total & 0xffffu;
        n_equal += total >> 16;
    }
    __syncthreads();
    for (int j = k + threadIdx.x; j < c; j += kSelThreads) out[j] = 0.f;

    if (a.k_scales != nullptr) {
        const int nb = (c + kBlock - 1) / kBlock, kb = (k + kBlock - 1) / kBlock;
        const int32_t* src = a.src + (size_t)s * a.max_blocks;
        const int32_t* dst = a.dst + (size_t)s * a.max_blocks;
        const size_t triples = (size_t)a.n_layers * a.n_seqs * a.n_kv;
        float* old_k = a.old_scales + triple * a.max_blocks;
        float* old_v = a.old_scales + (triples + triple) * a.max_blocks;
        float* ks = a.k_scales + (size_t)layer * a.num_blocks * a.n_kv + g;
        float* vs = a.v_scales + (size_t)layer * a.num_blocks * a.n_kv + g;
        for (int b = threadIdx.x; b < nb; b += kSelThreads) {
            const int phys = src[b];
            const bool ok = (unsigned)phys < (unsigned)a.num_blocks;
            old_k[b] = ok ? ks[(size_t)phys * a.n_kv] : 0.f;
            old_v[b] = ok ? vs[(size_t)phys * a.n_kv] : 0.f;
        }
        __syncthreads();  // the old scales are read, the kept list is written
        for (int b = threadIdx.x; b < kb; b += kSelThreads) {
            const int phys = dst[b];
            if ((unsigned)phys >= (unsigned)a.num_blocks) continue;
            float mk = 0.f, mv = 0.f;
            for (int i = b * kBlock; i < min(k, (b + 1) * kBlock); ++i) {
                const int sb = kept[i] / kBlock;
                mk = fmaxf(mk, old_k[sb]);
                mv = fmaxf(mv, old_v[sb]);
            }
            ks[(size_t)phys * a.n_kv] = mk;
            vs[(size_t)phys * a.n_kv] = mv;
        }
    }
}

// Sixteen codes * f, back to codes.
__device__ __forceinline__ uint4 rescale16(uint4 c, float f) {
    uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        const uint16_t lo = (uint16_t)w[i], hi = (uint16_t)(w[i] >> 16);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(lo));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(hi));
        const float2 x = __half22float2(*reinterpret_cast<__half2*>(&h[0]));
        const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h[1]));
        uint16_t r0, r1;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r0) : "f"(x.y * f), "f"(x.x * f));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r1) : "f"(y.y * f), "f"(y.x * f));
        w[i] = (uint32_t)r0 | ((uint32_t)r1 << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kMoveThreads = 256;

// grid ((sequence, head) x slices, layer, K/V)
template <bool Q8>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    constexpr int U = 4;  // rows of a thread per chunk
    const long long pair = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x % a.slices);
    const int s = (int)(pair / a.n_kv), g = (int)(pair % a.n_kv), layer = blockIdx.y;
    const int cap = a.max_blocks * kBlock;
    grid_launch_dependents();
    grid_dependency_wait();
    const int c = a.lens[s], want = a.keep[s];
    if (c < 0 || c > cap || want < 0 || min(want, c) > a.max_keep) return;  // flagged by the selection
    const int k = min(want, c);
    const int lanes = a.row_bytes / a.slices / 16;  // threads that share a row
    const int rows = kMoveThreads / lanes;          // rows the CTA covers at once
    const int sub = threadIdx.x / lanes;
    const size_t col = (size_t)slice * lanes * 16 + (threadIdx.x % lanes) * 16;
    const size_t triple = (size_t)layer * a.n_seqs * a.n_kv + pair;
    const size_t triples = (size_t)a.n_layers * a.n_seqs * a.n_kv;
    const int32_t* kept = a.kept + triple * a.max_keep;
    const int32_t* src = a.src + (size_t)s * a.max_blocks;
    const int32_t* dst = a.dst + (size_t)s * a.max_blocks;
    const bool is_v = blockIdx.z != 0;
    const size_t layer_rows = (size_t)a.num_blocks * a.n_kv * kBlock;
    char* pool = reinterpret_cast<char*>(is_v ? a.v_pool : a.k_pool) + (size_t)layer * layer_rows * a.row_bytes;
    const float* old_scale = Q8 ? a.old_scales + ((is_v ? triples : 0) + triple) * a.max_blocks : nullptr;
    const float* new_scale = Q8 ? (is_v ? a.v_scales : a.k_scales) + (size_t)layer * a.num_blocks * a.n_kv + g : nullptr;

    for (int i0 = 0; i0 < k; i0 += rows * U) {
        uint4 x[U];
        char* to[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * rows + sub;
            to[u] = nullptr;
            if (i < k) {
                const int j = kept[i];
                const int ps = src[j / kBlock], pd = dst[i / kBlock];
                if ((unsigned)ps >= (unsigned)a.num_blocks || (unsigned)pd >= (unsigned)a.num_blocks) {
                    atomicOr(a.status, (unsigned)PKV_DEV_BAD_BLOCK_ID);
                } else {
                    f[u] = 1.f;
                    if (Q8) {
                        const float o = old_scale[j / kBlock], n = new_scale[(size_t)pd * a.n_kv];
                        f[u] = o == n ? 1.f : o / n;
                    }
                    const size_t from_row = ((size_t)ps * a.n_kv + g) * kBlock + j % kBlock;
                    const size_t to_row = ((size_t)pd * a.n_kv + g) * kBlock + i % kBlock;
                    if (from_row != to_row || f[u] != 1.f) {
                        to[u] = pool + to_row * a.row_bytes + col;
                        x[u] = *reinterpret_cast<const uint4*>(pool + from_row * a.row_bytes + col);
                    }
                }
            }
        }
        __syncthreads();  // the chunk's rows are in registers before any of its places is written
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (to[u]) *reinterpret_cast<uint4*>(to[u]) = Q8 && f[u] != 1.f ? rescale16(x[u], f[u]) : x[u];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    const unsigned pairs = (unsigned)a.n_seqs * (unsigned)a.n_kv;
    cudaError_t err = launch_dependent(evict_select_kernel, dim3(pairs, a.n_layers), kSelThreads, 0, stream, 1, a);
    if (err != cudaSuccess) return err;
    const dim3 grid(pairs * (unsigned)a.slices, a.n_layers, 2);
    return launch_dependent(a.k_scales ? evict_move_kernel<true> : evict_move_kernel<false>, grid, kMoveThreads, 0, stream, 1, a);
}

}  // namespace pkv
