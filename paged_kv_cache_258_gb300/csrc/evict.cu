// evict.cu -- eviction from the cache by accumulated attention weight (sm_103a).
//
// For every (layer, sequence s, KV head g), c = lens[s], k = min(keep[s], c), R = min(recent, k): the
// last R positions stay, and of the first c - R the k - R with the largest score (ties: the lower
// position; NaN counts as largest). The kept rows of K and V move, in order of position, to logical
// positions 0 .. k-1 of the destination table, their scores with them; scores in [k, c) become 0.
// Heads and layers choose for themselves: a table is shared by all of them, but each has its own rows.
//
// Two launches; the second moves 2 k row bytes each way for K and V against 8 c + 4 k bytes of the first.
//  1. select: one CTA per triple. A thread holds up to 16 scores as ordered integers in registers (all
//     its loads in flight at once); a radix select over 11 + 11 + 10 bits, with histograms in shared
//     memory, finds the (k - R)-th largest. Then every warp counts what it keeps of its consecutive
//     positions, a scan over the warps numbers them, and ballots place each one. The scores are rebuilt
//     from the registers, so they may move in place: what is written at index i was read, as were all
//     scores up to the i-th kept position, which is never below i. Contexts longer than the CTA's
//     registers go by in pieces, in order.
//     For 8-bit pools it also reads the old scales of all the sequence's blocks aside and writes each
//     destination block's new scale, the largest among its rows' (a power of two like them, so the
//     codes only shift).
//  2. move: `parts` CTAs share the rows of a triple (K or V). Where all of a sequence's destinations are
//     blocks of their own, a CTA takes a run of whole rows. Where some are the blocks the rows come from,
//     the CTAs take column slices instead, so that no two touch the same bytes and rows can move up in
//     place without any order between CTAs: a CTA works through its rows in chunks, the next chunk's
//     loads in flight, a chunk's stores behind a barrier behind all its loads; row i is read from a
//     position >= i, so loads of later chunks never see an earlier chunk's stores. The places of kIndex
//     rows at a time are worked out in shared memory.
#include <math.h>

#include "common.cuh"
#include "shrink.h"

namespace pkv {
namespace {

constexpr int kBins = 2048;
constexpr int kKeys = 16;  // scores of a thread

// Scores as integers in the same order; NaN above everything, -0 equal to 0. And back (NaN to a NaN).
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int NT>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
    constexpr int NW = NT / 32;
    __shared__ uint32_t s_hist[kBins];
    __shared__ uint32_t s_warp[NW], s_warp2[NW];
    __shared__ uint32_t s_pick[3];
    __shared__ float s_old[2][NT];  // old scales of K and V by block, while the CTA has a thread for each
    const long long pair = blockIdx.x;  // s * n_kv + g
    const int s = (int)(pair / a.n_kv), g = (int)(pair % a.n_kv), layer = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = a.max_blocks * kBlock;
    grid_dependency_wait();
    grid_launch_dependents();
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

    // Positions go by in pieces of NT * rounds; warp w holds `rounds` * 32 consecutive ones.
    const int rounds = min(kKeys, (c + NT - 1) / NT);
    const int piece = NT * rounds;
    const int pieces = c > 0 ? (c + piece - 1) / piece : 0;
    uint32_t key[kKeys] = {};
    auto at = [&](int p, int r) -> int { return p * piece + (warp * rounds + r) * 32 + lane; };
    auto load = [&](int p) {
        float x[kKeys];
#pragma unroll
        for (int r = 0; r < kKeys; ++r)
            if (r < rounds) x[r] = at(p, r) < c ? score[at(p, r)] : 0.f;
#pragma unroll
        for (int r = 0; r < kKeys; ++r)
            if (r < rounds) key[r] = order_key(x[r]);
    };
    // bit r: this thread's r-th position of piece p lies before `end`
    auto before = [&](int p, int end) -> uint32_t {
        const int n = (end - at(p, 0) + 31) / 32;
        return n <= 0 ? 0u : (1u << min(n, rounds)) - 1;
    };
    // 8-bit pools: the old scales are on their way while the selection runs
    const int nb = (c + kBlock - 1) / kBlock;
    const size_t triples = (size_t)a.n_layers * a.n_seqs * a.n_kv;
    float* ks = a.k_scales ? a.k_scales + (size_t)layer * a.num_blocks * a.n_kv + g : nullptr;
    float* vs = a.k_scales ? a.v_scales + (size_t)layer * a.num_blocks * a.n_kv + g : nullptr;
    auto old_scale = [&](int b, float* k_old, float* v_old) {
        const int phys = a.src[(size_t)s * a.max_blocks + b];
        const bool ok = (unsigned)phys < (unsigned)a.num_blocks;
        *k_old = ok ? ks[(size_t)phys * a.n_kv] : 0.f;
        *v_old = ok ? vs[(size_t)phys * a.n_kv] : 0.f;
    };
    float k_old = 0.f, v_old = 0.f;
    if (ks && (int)threadIdx.x < nb) old_scale(threadIdx.x, &k_old, &v_old);
    if (pieces == 1) load(0);

    // threshold: positions above it are kept, of those equal to it the first `ties`
    uint32_t threshold = 0xffffffffu, ties = 0;
    if (pick == older) {
        threshold = 0;  // (no score has key 0)
    } else if (pick > 0) {
        uint32_t prefix = 0, mask = 0, left = (uint32_t)pick;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            for (int i = threadIdx.x; i < kBins; i += NT) s_hist[i] = 0;
            __syncthreads();
            for (int p = 0; p < pieces; ++p) {
                if (pieces > 1) load(p);
                const uint32_t old = before(p, older);
#pragma unroll
                for (int r = 0; r < kKeys; ++r)
                    if ((old >> r) & 1u && (key[r] & mask) == prefix)
                        atomicAdd(&s_hist[(key[r] >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // thread t takes PER bins from the top: the scan counts what lies above them
            constexpr int PER = kBins / NT;
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += s_hist[kBins - 1 - (threadIdx.x * PER + i)];
            uint32_t above = warp_scan(mine);
            if (lane == 31) s_warp[warp] = above;
            __syncthreads();
            if (warp == 0) {
                const uint32_t v = lane < NW ? s_warp[lane] : 0u;
                const uint32_t before = warp_scan(v) - v;
                if (lane < NW) s_warp[lane] = before;
            }
            __syncthreads();
            above += s_warp[warp] - mine;
            if (above < left && above + mine >= left) {  // the bin that holds the left-th largest is here
                uint32_t n = above;
                for (int i = 0; i < PER; ++i) {
                    const int bin = kBins - 1 - (threadIdx.x * PER + i);
                    const uint32_t h = s_hist[bin];
                    if (n + h >= left) {
                        s_pick[0] = (uint32_t)bin;
                        s_pick[1] = left - n;
                        s_pick[2] = h;
                        break;
                    }
                    n += h;
                }
            }
            __syncthreads();
            prefix |= s_pick[0] << shift;
            mask |= ((1u << bits) - 1) << shift;
            left = s_pick[1];
            if (left == s_pick[2]) break;  // the whole bin is kept: its lower bits do not matter
        }
        // keys from the bin's first on; or, where not all of it is kept, the first `left` of one value
        const bool whole = left == s_pick[2];
        threshold = whole && prefix > 0 ? prefix - 1 : prefix;
        ties = whole ? 0u : left;
    }

    uint32_t n_above = 0, n_equal = 0;  // positions above the threshold and equal to it, in earlier pieces
    for (int p = 0; p < pieces; ++p) {
        if (pieces > 1) load(p);
        uint32_t is_above = 0, is_equal = 0;  // bit r: the thread's r-th position
#pragma unroll
        for (int r = 0; r < kKeys; ++r) {
            is_above |= (key[r] > threshold ? 1u : 0u) << r;
            is_equal |= (key[r] == threshold ? 1u : 0u) << r;
        }
        const uint32_t old = before(p, older);
        is_above = (is_above & old) | (before(p, c) & ~old);  // the recent window counts as above
        is_equal &= old;
        const uint32_t above = __reduce_add_sync(0xffffffffu, __popc(is_above));
        const uint32_t equal = __reduce_add_sync(0xffffffffu, __popc(is_equal));
        __syncthreads();  // the piece's scores are read by all; the counts of the last piece are consumed
        if (lane == 0) {
            s_warp[warp] = above;
            s_warp2[warp] = equal;
        }
        __syncthreads();
        if (warp == 0) {  // sums over the warps before, and over all
            const uint32_t va = lane < NW ? s_warp[lane] : 0u, ve = lane < NW ? s_warp2[lane] : 0u;
            const uint32_t ia = warp_scan(va), ie = warp_scan(ve);
            if (lane < NW) {
                s_warp[lane] = ia - va;
                s_warp2[lane] = ie - ve;
            }
            if (lane == 31) {
                s_pick[0] = ia;
                s_pick[1] = ie;
            }
        }
        __syncthreads();
        uint32_t ab = n_above + s_warp[warp], eq = n_equal + s_warp2[warp];
        n_above += s_pick[0];
        n_equal += s_pick[1];
        const uint32_t below = (1u << lane) - 1;
        if (ties == 0) {
#pragma unroll
            for (int r = 0; r < kKeys; ++r) {
                if (r < rounds) {
                    const uint32_t ba = __ballot_sync(0xffffffffu, (is_above >> r) & 1u);
                    if ((is_above >> r) & 1u) {
                        const uint32_t i = ab + __popc(ba & below);
                        kept[i] = at(p, r);
                        out[i] = key_score(key[r]);
                    }
                    ab += __popc(ba);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < kKeys; ++r) {
                if (r < rounds) {
                    const uint32_t ba = __ballot_sync(0xffffffffu, (is_above >> r) & 1u);
                    const uint32_t be = __ballot_sync(0xffffffffu, (is_equal >> r) & 1u);
                    const uint32_t eq_before = eq + __popc(be & below);
                    if ((is_above >> r) & 1u || ((is_equal >> r) & 1u && eq_before < ties)) {
                        const uint32_t i = ab + __popc(ba & below) + min(eq_before, ties);
                        kept[i] = at(p, r);
                        out[i] = key_score(key[r]);
                    }
                    ab += __popc(ba);
                    eq += __popc(be);
                }
            }
        }
    }
    __syncthreads();
    for (int j = k + threadIdx.x; j < c; j += NT) out[j] = 0.f;

    if (ks) {
        const int kb = (k + kBlock - 1) / kBlock;
        const int32_t* dst = a.dst + (size_t)s * a.max_blocks;
        float* old_k = a.old_scales + triple * a.max_blocks;  // kept for the move
        float* old_v = a.old_scales + (triples + triple) * a.max_blocks;
        for (int b = threadIdx.x; b < nb; b += NT) {
            if (b >= NT) old_scale(b, &k_old, &v_old);
            old_k[b] = k_old;
            old_v[b] = v_old;
            if (b < NT) {
                s_old[0][b] = k_old;
                s_old[1][b] = v_old;
            }
        }
        __syncthreads();  // the old scales are read, the kept list is written
        for (int b = warp * 2 + (lane >> 4); b < (kb + 1) / 2 * 2; b += 2 * NW) {  // half a warp a block
            const int i = b * kBlock + (lane & 15);
            float mk = 0.f, mv = 0.f;
            if (i < k) {
                const int sb = kept[i] / kBlock;
                mk = nb <= NT ? s_old[0][sb] : old_k[sb];
                mv = nb <= NT ? s_old[1][sb] : old_v[sb];
            }
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) {
                mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
                mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
            }
            if ((lane & 15) == 0 && b < kb) {
                const int phys = dst[b];
                if ((unsigned)phys < (unsigned)a.num_blocks) {
                    ks[(size_t)phys * a.n_kv] = mk;
                    vs[(size_t)phys * a.n_kv] = mv;
                }
            }
        }
    }
}

// Sixteen codes * f, back to codes (round to nearest even). A power of two f <= 1 multiplies in fp16: what
// lies at or above 2^-10, half the least code, is exact there, and what lies below becomes 0 either way.
__device__ __forceinline__ uint4 rescale16(uint4 c, float f) {
    uint32_t w[4] = {c.x, c.y, c.z, c.w};
    const bool half_exact = f <= 1.f && (__float_as_uint(f) & 0x7fffffu) == 0;
    const __half2 f2 = __float2half2_rn(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        uint16_t r[2];
        const uint16_t lo = (uint16_t)w[i], hi = (uint16_t)(w[i] >> 16);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(lo));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(hi));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            __half2 v = *reinterpret_cast<__half2*>(&h[e]);
            if (half_exact) {
                v = __hmul2(v, f2);
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[e]) : "r"(*reinterpret_cast<uint32_t*>(&v)));
            } else {
                const float2 x = __half22float2(v);
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r[e]) : "f"(x.y * f), "f"(x.x * f));
            }
        }
        w[i] = (uint32_t)r[0] | ((uint32_t)r[1] << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kMoveThreads = 256;
// Sequences up to which the move starts with those that keep most: a thread each works out its rank. 100 to 8,192
// tokens, 2 layers, 4 heads x 128 of 16 bits: 64 sequences 198 us against 215 in their own order, 100 309 against
// 338, 200 596 against 624; 16 and fewer the same.
constexpr int kRanked = kMoveThreads;
constexpr int kIndex = 512;  // kept rows whose places are worked out at a time
static_assert(2 * kRanked * sizeof(int) <= kIndex * sizeof(long long), "ranks and order fit where the places go");

// Little in flight is best here: reads and writes share DRAM, and CTAs that share rows or blocks should not
// drift apart. 8-bit pools, 128 triples of 2,250 to 4,096 kept rows: U = 2 79 us, 4 94, 8 101; a pipeline that
// runs on over the index instead of stopping every kIndex rows 103 against 100.
template <bool Q8>
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictArgs a) {
    constexpr int U = 2;  // rows of a thread per chunk
    __shared__ long long s_from[kIndex], s_to[kIndex];  // row numbers in the layer; s_to < 0: stays where it is
    __shared__ float s_f[Q8 ? kIndex : 1];              // what the row's codes are multiplied with
    // grid x: (sequence, layer, K or V, head, part), so that the sequences that keep most start first
    long long rest = blockIdx.x;
    const int part = (int)(rest % a.parts);
    rest /= a.parts;
    const int g = (int)(rest % a.n_kv);
    rest /= a.n_kv;
    const bool is_v = rest % 2 != 0;
    rest /= 2;
    const int layer = (int)(rest % a.n_layers);
    int s = (int)(rest / a.n_layers);
    const int cap = a.max_blocks * kBlock;
    grid_dependency_wait();
    grid_launch_dependents();
    if (a.n_seqs > 1 && a.n_seqs <= kRanked) {
        int* rank_k = reinterpret_cast<int*>(s_from);
        int* by_rank = rank_k + kRanked;
        if (threadIdx.x < a.n_seqs) rank_k[threadIdx.x] = min(a.keep[threadIdx.x], a.lens[threadIdx.x]);
        __syncthreads();
        if (threadIdx.x < a.n_seqs) {
            const int mine = rank_k[threadIdx.x];
            int r = 0;
            for (int i = 0; i < a.n_seqs; ++i) r += rank_k[i] > mine || (rank_k[i] == mine && i < (int)threadIdx.x);
            by_rank[r] = threadIdx.x;
        }
        __syncthreads();
        s = by_rank[s];
        __syncthreads();  // the index overwrites the ranks
    }
    const long long pair = (long long)s * a.n_kv + g;
    const int c = a.lens[s], want = a.keep[s];
    if (c < 0 || c > cap || want < 0 || min(want, c) > a.max_keep) return;  // flagged by the selection
    const int k = min(want, c);
    const size_t triple = (size_t)layer * a.n_seqs * a.n_kv + pair;
    const size_t triples = (size_t)a.n_layers * a.n_seqs * a.n_kv;
    const int32_t* kept = a.kept + triple * a.max_keep;
    const int32_t* src = a.src + (size_t)s * a.max_blocks;
    const int32_t* dst = a.dst + (size_t)s * a.max_blocks;
    const int kb = (k + kBlock - 1) / kBlock;
    bool same = false;
    for (int b = threadIdx.x; b < kb; b += kMoveThreads) same = same || src[b] == dst[b];
    int lo = 0, hi = k, lanes = a.row_bytes / 16;  // the CTA's rows; threads that share a row
    size_t column = 0;
    if (__syncthreads_or(same)) {
        const int slices = min(a.parts, a.slices);
        if (part >= slices) return;
        lanes /= slices;
        column = (size_t)part * lanes * 16;
    } else {
        lo = (int)((long long)kb * part / a.parts) * kBlock;
        hi = min(k, (int)((long long)kb * (part + 1) / a.parts) * kBlock);
    }
    const int rows = kMoveThreads / lanes;  // rows the CTA covers at once
    const int sub = threadIdx.x / lanes;
    const size_t layer_rows = (size_t)a.num_blocks * a.n_kv * kBlock;
    char* pool = reinterpret_cast<char*>(is_v ? a.v_pool : a.k_pool) + (size_t)layer * layer_rows * a.row_bytes + column +
                 (threadIdx.x % lanes) * 16;
    const float* old_scale = Q8 ? a.old_scales + ((is_v ? triples : 0) + triple) * a.max_blocks : nullptr;
    const float* new_scale = Q8 ? (is_v ? a.v_scales : a.k_scales) + (size_t)layer * a.num_blocks * a.n_kv + g : nullptr;

    // The places of the next kIndex rows are on their way while these are moved: first the positions,
    // one step ahead the blocks (and scales) they lie in.
    constexpr int PER = kIndex / kMoveThreads;
    int j_next[PER], ps[PER], pd[PER];
    float so[PER], sn[PER];
    auto fetch_kept = [&](int i0) {
#pragma unroll
        for (int t = 0; t < PER; ++t) {
            const int i = i0 + t * kMoveThreads + threadIdx.x;
            j_next[t] = i < hi ? kept[i] : 0;
        }
    };
    auto fetch_blocks = [&](int i0) {
#pragma unroll
        for (int t = 0; t < PER; ++t) {
            const int i = i0 + t * kMoveThreads + threadIdx.x;
            ps[t] = i < hi ? src[j_next[t] / kBlock] : 0;
            pd[t] = i < hi ? dst[i / kBlock] : 0;
        }
        if (Q8) {
#pragma unroll
            for (int t = 0; t < PER; ++t) {
                const int i = i0 + t * kMoveThreads + threadIdx.x;
                so[t] = i < hi ? old_scale[j_next[t] / kBlock] : 0.f;
                sn[t] = i < hi && (unsigned)pd[t] < (unsigned)a.num_blocks ? new_scale[(size_t)pd[t] * a.n_kv] : 0.f;
            }
        }
    };
    fetch_kept(lo);
    fetch_blocks(lo);
    for (int i0 = lo; i0 < hi; i0 += kIndex) {
        const int n = min(kIndex, hi - i0);
        __syncthreads();  // the last index has been read
#pragma unroll
        for (int t = 0; t < PER; ++t) {
            const int e = t * kMoveThreads + threadIdx.x, i = i0 + e;
            long long from = 0, to = -1;
            float f = 1.f;
            if (i < hi) {
                if ((unsigned)ps[t] >= (unsigned)a.num_blocks || (unsigned)pd[t] >= (unsigned)a.num_blocks) {
                    atomicOr(a.status, (unsigned)PKV_DEV_BAD_BLOCK_ID);
                } else {
                    if (Q8) f = so[t] == sn[t] ? 1.f : so[t] / sn[t];
                    from = ((long long)ps[t] * a.n_kv + g) * kBlock + j_next[t] % kBlock;
                    to = ((long long)pd[t] * a.n_kv + g) * kBlock + i % kBlock;
                    if (from == to && f == 1.f) to = -1;
                }
            }
            s_from[e] = from;
            s_to[e] = to;
            if (Q8) s_f[e] = f;
        }
        __syncthreads();
        fetch_kept(i0 + kIndex);
        uint4 x[2][U];
        auto load = [&](int e0, uint4* v) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * rows + sub;
                if (e < n && s_to[e] >= 0) v[u] = *reinterpret_cast<const uint4*>(pool + (size_t)s_from[e] * a.row_bytes);
            }
        };
        auto store = [&](int e0, const uint4* v) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * rows + sub;
                if (e < n && s_to[e] >= 0)
                    *reinterpret_cast<uint4*>(pool + (size_t)s_to[e] * a.row_bytes) =
                        Q8 && s_f[e] != 1.f ? rescale16(v[u], s_f[e]) : v[u];
            }
        };
        const int chunk = rows * U;
        load(0, x[0]);
        for (int e0 = 0; e0 < n; e0 += 2 * chunk) {
            load(e0 + chunk, x[1]);
            if (e0 == 0) fetch_blocks(i0 + kIndex);  // the positions have arrived
            __syncthreads();  // all of this chunk is in registers before any of its places is written
            store(e0, x[0]);
            load(e0 + 2 * chunk, x[0]);
            __syncthreads();
            store(e0 + chunk, x[1]);
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    const unsigned pairs = (unsigned)a.n_seqs * (unsigned)a.n_kv;
    // the fewest threads whose registers hold a context: more CTAs an SM, cheaper barriers
    const int cap = a.max_blocks * kBlock;
    cudaError_t err = cap <= 256 * kKeys
                          ? launch_dependent(evict_select_kernel<256>, dim3(pairs, a.n_layers), 256, 0, stream, 1, a)
                      : cap <= 512 * kKeys
                          ? launch_dependent(evict_select_kernel<512>, dim3(pairs, a.n_layers), 512, 0, stream, 1, a)
                          : launch_dependent(evict_select_kernel<1024>, dim3(pairs, a.n_layers), 1024, 0, stream, 1, a);
    if (err != cudaSuccess) return err;
    const dim3 grid(pairs * (unsigned)a.parts * (unsigned)a.n_layers * 2u);
    return launch_dependent(a.k_scales ? evict_move_kernel<true> : evict_move_kernel<false>, grid, kMoveThreads, 0, stream, 1, a);
}

}  // namespace pkv
