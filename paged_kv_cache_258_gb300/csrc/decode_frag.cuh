// decode_frag.cuh -- decode attention over 8-bit pools, and over 16-bit pools with the attention
// weights summed (sm_103a).
//
// For sequence s, query head h of KV head g, position j in block b (16 tokens):
//   z_j = scale log2(e) S_K(b) (q . cK_j),   out = sum_j 2^(z_j - m) S_V(b) cV_j / sum_j 2^(z_j - m),
// c the stored codes, S the block's scale (1 for 16-bit pools). One pass over the cache: 2 D bytes a
// token and head for codes, against 4 D for 16-bit rows, so a kernel that keeps up with memory takes
// half the time -- and has half as long for the arithmetic of each token.
//
// Work is cut by blocks, not by sequences: the blocks of all (sequence, KV head) pairs form one list,
// and each of the CTAs the GPU holds at once takes an equal run of it, whatever the lengths are (a pair
// counts kPairCost blocks on top of its own, what starting and ending it costs). A run covers the end
// of one pair, some whole pairs and the start of another; only its first and its last pair can be
// shared with other CTAs, so two partial results a CTA are all that is kept in memory, and the CTA that
// arrives last at a shared pair joins its partials. (A grid over table-width partitions gave a ragged
// batch -- 32 sequences of 0..8,192 tokens, 8 heads x 8 queries -- 70 us, of which a third were starts,
// joins and a tail of half-empty SMs; runs take 50.) Calls of a few small contexts take a grid of
// (partition, head, sequence) instead, the partitions of a context being a thread-block cluster that
// joins through shared memory (one sequence of 301 tokens: 10.2 us with partials in memory, 5.4).
// Bound by memory: 10 x 30,000 tokens read at 6.4 TB/s (d = 256) and 6.5 (d = 128), 94 % of the copy
// rate; the GPT-style batch at 6.0, its many short pairs' ends not wholly hidden.
//
// Short prompt chunks over an 8-bit pool run here too (MULTI): the query columns (8, or 16 and 32 as two and
// four column tiles at D = 128 and 64) hold tokens x G heads, a "sequence" of the list is such a group of
// tokens, and each column has its own causal limit. Every group reads the context again, mostly from L2; wide
// ones do so less often and convert each code once for all tiles. Bound by issue and the tensor pipe: a block of
// 16 tokens x 16 columns at D = 128 costs a scheduler 460 cycles. A second stage in flight is no faster, one
// block an iteration (3 stages or 3 CTAs an SM) 30 % slower.
//
// Per-warp rings of TMA copies feed the warps as in decode_mma.cuh. What differs is how a 16-token tile
// gets from shared memory into fragments:
//  * The contraction of S = K Q^T runs over head dims in any order, as long as Q's fragment uses the
//    same one. A lane therefore takes whole 16-byte chunks of a K row (one 128-bit read) and the dims
//    that lie in them become its k indices: 16 codes are the k indices of four m16n8k16 steps.
//  * O^T = V^T P^T has head dims as rows, also in any order: lane group gid owns the 16-byte chunk
//    gid of every row, and byte permutes (prmt) pair the same dim of two tokens. No ldmatrix, which
//    cannot transpose single bytes.
//  * Chunk choice and the 128-byte swizzle put the eight lanes of a read phase on eight different
//    16-byte columns: K takes chunks 2 tig + i (rows gid), V chunk gid (rows 2 tig + j).
//  * Codes become fp16 by cvt.rn.f16x2.e4m3x2, which is exact (e4m3 is a subset of fp16, NaN stays
//    NaN). q is brought to fp16 with a power of two of its own row, so bf16's range cannot overflow:
//    a query element keeps at least 11 bits unless it is 2^-29 of its row's largest, where what is
//    lost is below fp32's own rounding of the dot product.
//  * Weights for the PV product are fp16 too (11 bits; over 16-bit pools they have the pool's type, because both
//    operands of an instruction have one type and V's range is bf16's: 8 bits there, each weight off by at most 2^-8 of
//    itself; fp16 ones times 2^15: its subnormals begin at 2^-14, and many small weights may make up a large sum):
//    w_j = 2^(z_j + log2 S_V(b) + 15 - m'), m' the running maximum of z + log2 S_V. So the largest w is
//    2^15 whatever the blocks' scales, and one keeps 11 bits down to 2^-29 of it (below 2^-40 it is 0:
//    2^28 tokens of those make up 2^-12). The sum of weights runs in fp32 beside it with its own maximum m.
//  * Positions past the length are removed by selection (logits) and by zeroing V's words, so NaN in
//    unused rows cannot reach the result.
// With `z` set every logit is also written out (fp32, G per position, 64 G contiguous bytes a block);
// the launch of scores.cu that follows turns them into weights once the row's final maximum and sum
// are known. Storing them costs 4 G bytes a token and head, reading K again would cost 2 D or 4 D.
#pragma once

#include <type_traits>

#include "decode.cuh"
#include "decode_mma.cuh"
#include "shrink.h"

namespace pkv {

// Two e4m3 codes (low 16 bits) -> two halves.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w) {
    uint32_t r;
    const uint16_t c = (uint16_t)w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// What a pair costs a CTA beside its blocks, in blocks: 4.7 us (loads of the table, the query and the
// first tiles, the warps' join, the output) against 0.19 us a block of codes. Without it a CTA whose run
// holds 34 short contexts ended 66 us after one with long ones.
template <bool Q8>
constexpr int kPairCost = Q8 ? 24 : 12;

constexpr int kJoinChunk = 128;  // partials whose weights are worked out at a time

// Shared-memory floats the join of partials needs (flag, row maxima, sums, factors, a chunk's weights).
template <int G>
struct JoinScratch {
    static constexpr size_t BYTES = (4 + 3 * G + G * kJoinChunk) * sizeof(float);
};

// NW warps, each with a ring of ST stages of BPI blocks (K tiles, then V tiles).
template <bool Q8, int D, int G, int NW, int ST, int BPI>
struct FragGeom {
    static constexpr int ROWB = D * (Q8 ? 1 : 2);            // bytes of a row
    static constexpr int PANB = ROWB < 128 ? ROWB : 128;     // bytes of a panel's row (one TMA box)
    static constexpr int PANELS = ROWB / PANB;
    static constexpr int PANEL = kBlock * PANB;
    static constexpr uint32_t TILE = kBlock * ROWB;
    static constexpr uint32_t STAGE = 2 * BPI * TILE;
    static constexpr int KCH = ROWB / 64;                    // 16-byte chunks of a K row per lane
    static constexpr int COLS = (G + 7) / 8 * 8;             // query columns of the instructions
    static constexpr size_t MERGE = (size_t)NW * G * D * 4;  // join scratch, after the combine buffer
    static constexpr size_t RINGS = (size_t)NW * ST * STAGE;
    static constexpr size_t AFTER = MERGE + (JoinScratch<G>::BYTES > G * (D + 2) * 4 ? JoinScratch<G>::BYTES : G * (D + 2) * 4);
    static constexpr size_t STAGES = RINGS > AFTER ? RINGS : (AFTER + 15) / 16 * 16;  // rings, then the join
    static constexpr size_t BARS = STAGES;                            // uint64 [NW][ST][K, V]
    static constexpr size_t ML = BARS + (size_t)NW * ST * 16;            // float2 [NW][COLS]: (max, sum) of a warp's rows
    static constexpr size_t JOIN = ML + (size_t)NW * COLS * 8;           // float [COLS][NW] weights, [COLS] maxima, [COLS] sums
    static constexpr size_t FIND = JOIN + (size_t)COLS * (NW + 2) * 4;   // long long [NW + 2]
    static constexpr size_t TOTAL = (FIND + (size_t)(NW + 2) * 8 + 15) / 16 * 16;
    static constexpr size_t ALLOC = TOTAL + 1024;             // room to align the base
    static_assert(TOTAL % 16 == 0, "the logits of a partition follow");
    // byte of 16-byte chunk `c` of row `r`: the copy's swizzle XORs the chunk with the 128-byte line's
    // number modulo the pattern (8 rows of 128 bytes, or 4 lines of two 64-byte rows)
    __device__ __forceinline__ static uint32_t at(int r, int c) {
        if constexpr (PANB == 128)
            return (uint32_t)((c >> 3) * PANEL + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        else
            return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
    // the chunk a lane of column tig takes as its i-th
    __device__ __forceinline__ static int k_chunk(int tig, int i) {
        return PANB == 128 ? (i >> 1) * 8 + 2 * tig + (i & 1) : tig;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// An output before its rounding. Rows near 65,504 are held as 65,536, which fp16 has no room for: means up
// to there (and the 2^-11 that rounded weights may add) come out as the largest half.
template <typename T>
__device__ __forceinline__ float in_range(float x) {
    if constexpr (std::is_same<T, __half>::value) return fabsf(x) <= 65600.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
    return x;
}

// f * v, rounded, to four consecutive elements.
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v, float f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(MmaType<T>::pack(in_range<T>(v.x * f), in_range<T>(v.y * f)),
                                              MmaType<T>::pack(in_range<T>(v.z * f), in_range<T>(v.w * f)));
}

// The pair's rows in q or out: row r is head r of the sequence's row, or (MULTI) head r mod 2^shift of
// token r / 2^shift, for r < rows.
template <typename P, int D, bool MULTI>
struct PairRows {
    P* base;
    int n_q, shift, rows;
    __device__ __forceinline__ bool has(int r) const { return !MULTI || r < rows; }
    __device__ __forceinline__ P* row(int r) const {
        if constexpr (!MULTI) return base + (size_t)r * D;
        return base + ((size_t)(r >> shift) * n_q + (r & ((1 << shift) - 1))) * D;
    }
};

// Four consecutive elements of a query row, widened.
template <typename T>
__device__ __forceinline__ void load4(const T* p, float* f) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = MmaType<T>::unpack(u.x), b = MmaType<T>::unpack(u.y);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// 2^x, x <= 0 in every use or a rounding above it; 2 ulp, results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kWeightExp = 15.f;  // exponent of the largest fp16 weight

// (max, sum) pairs and partial outputs a run leaves in memory: slot 0 for a pair it did not start, slot 1
// for one it does not end. Partial i of a pair whose first CTA is `first` lies in:
__device__ __forceinline__ int partial_slot(int first, int i) { return i == 0 ? 2 * first + 1 : 2 * (first + i); }

// Ends a shared pair in the CTA that arrives last: joins the np partials in order,
//   out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),  M = max_i m_i.
// The arrival counter wraps to 0 with the last arrival (atomicInc), so it is ready for the next call; it
// belongs to the pair's first CTA and always lies at the same place of the workspace. An addition, not a
// compare-and-swap: the CTAs of one wave end together, and retries would queue at an L2 round trip each.
template <typename T, int D, int G, int NT, bool MULTI>
__device__ __forceinline__ void join_if_last(const FragArgs& fa, const PairRows<T, D, MULTI>& out, float2* row_ml, int first,
                                             int np, float* scratch) {
    const DecodeArgs& a = fa.d;
    constexpr int NWARP = NT / 32;
    constexpr int PER = (G * D / 4 + NT - 1) / NT;  // groups of four outputs of a thread
    constexpr int MQ = 16 / PER;                     // partials of each in flight at once
    int* flag = reinterpret_cast<int*>(scratch);
    float* sM = scratch + 4;  // [G]
    float* sL = sM + G;       // [G]
    float* sF = sL + G;       // [G]
    float* sW = sF + G;       // [G][kJoinChunk]
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        *flag = atomicInc(fa.arrivals + first, (unsigned)np - 1) == (unsigned)np - 1;
        __threadfence();
    }
    __syncthreads();
    if (!*flag) return;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    // a warp per row: every pair is read once, a chunk's at the same time
    float4 O[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < np; c0 += kJoinChunk) {
        const int nq = min(kJoinChunk, np - c0);
        if (c0 > 0) __syncthreads();  // the previous chunk's weights are consumed
        for (int r = warp; r < G; r += NWARP) {
            float2 u[kJoinChunk / 32];
            float m = c0 > 0 ? sM[r] : -INFINITY;
            const float before = m;
#pragma unroll
            for (int i = 0; i < kJoinChunk / 32; ++i) {
                const int q = i * 32 + lane;
                u[i] = make_float2(-INFINITY, 0.f);
                if (q < nq) u[i] = __ldcg(ml + (size_t)partial_slot(first, c0 + q) * G + r);
            }
#pragma unroll
            for (int i = 0; i < kJoinChunk / 32; ++i) m = fmaxf(m, u[i].x);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < kJoinChunk / 32; ++i) {
                const float w = u[i].x == -INFINITY ? 0.f : ex2(u[i].x - m);
                sW[r * kJoinChunk + i * 32 + lane] = w;
                l = fmaf(u[i].y, w, l);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) {
                const float f = before == -INFINITY ? 0.f : ex2(before - m);
                sL[r] = c0 > 0 ? fmaf(sL[r], f, l) : l;
                sF[r] = f;
                sM[r] = m;
            }
        }
        __syncthreads();
        if (c0 > 0) {
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const float f = sF[min((int)threadIdx.x + k * NT, G * D / 4 - 1) / (D / 4)];
                O[k] = make_float4(O[k].x * f, O[k].y * f, O[k].z * f, O[k].w * f);
            }
        }
        for (int q0 = 0; q0 < nq; q0 += MQ) {
            float4 v[PER][MQ];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int i4 = threadIdx.x + k * NT;
#pragma unroll
                for (int u = 0; u < MQ; ++u) {
                    v[k][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i4 < G * D / 4 && q0 + u < nq)
                        v[k][u] = __ldcg(reinterpret_cast<const float4*>(
                                             a.part_o + (size_t)partial_slot(first, c0 + q0 + u) * G * D) + i4);
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int i4 = threadIdx.x + k * NT;
                if (i4 < G * D / 4) {
                    const float* w = sW + (i4 / (D / 4)) * kJoinChunk + q0;
#pragma unroll
                    for (int u = 0; u < MQ; ++u) {
                        if (q0 + u < nq) {
                            O[k].x = fmaf(w[u], v[k][u].x, O[k].x);
                            O[k].y = fmaf(w[u], v[k][u].y, O[k].y);
                            O[k].z = fmaf(w[u], v[k][u].z, O[k].z);
                            O[k].w = fmaf(w[u], v[k][u].w, O[k].w);
                        }
                    }
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i4 = threadIdx.x + k * NT;
        if (i4 < G * D / 4) {
            const int r = i4 / (D / 4);
            const float L = sL[r];
            if (out.has(r)) store4(out.row(r) + 4 * (i4 % (D / 4)), O[k], L == 0.f ? 0.f : 1.f / L);
        }
    }
    if (row_ml && threadIdx.x < G) row_ml[threadIdx.x] = make_float2(sM[threadIdx.x], sL[threadIdx.x]);
}

// The same join for a cluster of a pair's partitions, through the CTAs' shared memory: no trip to L2 for
// the partials and none for a counter. Every CTA p < np has its (max, sum) pairs in ml [G][2] and its
// partial outputs in po [G * D], and writes every np-th piece of the output.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_load(uint32_t a) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
    return r;
}
// All threads of the cluster's CTAs that have not left (CTAs past the context leave at once and count
// as arrived).
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <typename T, int D, int G, int NT, bool MULTI>
__device__ __forceinline__ void cluster_join(const PairRows<T, D, MULTI>& out, int p, int np, const float* ml, const float* po, float* s_max,
                                             float* s_sum) {
    cluster_barrier();
    const uint32_t ml0 = smem_addr(ml), po0 = smem_addr(po);
    auto row = [&](int r, float* w, float* M, float* L) {  // the partials' weights, the row's maximum and sum
        float m[kMaxCluster], l[kMaxCluster];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            m[q] = -INFINITY;
            l[q] = 0.f;
            if (q < np) {
                m[q] = cluster_load(cluster_addr(ml0 + (2 * r) * 4, q));
                l[q] = cluster_load(cluster_addr(ml0 + (2 * r + 1) * 4, q));
            }
        }
        *M = -INFINITY;
        *L = 0.f;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) *M = fmaxf(*M, m[q]);
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            w[q] = m[q] == -INFINITY ? 0.f : ex2(m[q] - *M);
            *L = fmaf(l[q], w[q], *L);
        }
    };
    float w[kMaxCluster], M, L;
    for (int idx = p * NT + threadIdx.x; idx < G * D; idx += np * NT) {
        float o[kMaxCluster], O = 0.f;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) o[q] = q < np ? cluster_load(cluster_addr(po0 + idx * 4, q)) : 0.f;
        row(idx / D, w, &M, &L);
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) O = fmaf(o[q], w[q], O);
        if (out.has(idx / D)) out.row(idx / D)[idx % D] = from_float<T>(in_range<T>(L == 0.f ? 0.f : O / L));
    }
    if (s_max && threadIdx.x < G) {
        row(threadIdx.x, w, &M, &L);
        s_max[threadIdx.x] = M;
        s_sum[threadIdx.x] = L;
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory; the statistics are written
}

template <typename T, bool Q8, int D, int G, int NW, int ST, int BPI, int CTAS, bool MULTI>
__global__ void __launch_bounds__(NW * 32, CTAS) frag_decode_kernel(const FragArgs fa,
                                                                    const __grid_constant__ CUtensorMap tm_k,
                                                                    const __grid_constant__ CUtensorMap tm_v) {
    static_assert(MULTI ? Q8 && G % 8 == 0 && G <= 32 : G <= 8, "one column tile, or whole ones over codes");
    static_assert(BPI == 1 || BPI == 2 || BPI == 4, "blocks per iteration");
    using S = FragGeom<Q8, D, G, NW, ST, BPI>;
    using MT = typename std::conditional<Q8, __half, T>::type;  // type of the matrix instructions' operands
    using M = MmaType<MT>;
    constexpr int KSTEPS = D / 16;  // QK k-steps = PV m-tiles
    constexpr uint32_t TILE = S::TILE;
    constexpr int NT = S::COLS / 8;  // column tiles: query rows 8 nt + 2 tig, + 1 are this lane's
    // what weights over 16-bit pools are multiplied with before their rounding; bf16 has fp32's range
    constexpr float kUp = std::is_same<T, __half>::value ? 32768.f : 1.f;
    static_assert(kWeightExp == 15.f, "both kinds of pools use the same room");
    const DecodeArgs& a = fa.d;

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int gid = lane >> 2;  // token row of S, chunk of V
    const int tig = lane & 3;   // owns query rows 2 tig, 2 tig + 1 of every column tile
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
    if (threadIdx.x < 2 * NW * ST) mbar_init(&bars[threadIdx.x], 1);
    fence_mbar_init();
    __syncthreads();
    // Nothing in global memory has been touched so far. Loads behind the wait are plain ones: the read-only
    // path is for data that nobody writes while this grid lives, and the grid before may still be writing.
    grid_dependency_wait();
    grid_launch_dependents();

    const int cap = a.max_blocks * kBlock;
    uint64_t* wbars = bars + warp * ST * 2;  // [ST][K, V]
    const uint32_t wstage = smem_addr(smem) + (uint32_t)(warp * ST) * S::STAGE;
    const uint64_t policy = l2_evict_first_policy();
    // Sequence s of the list: its row of the table, the positions it sees; MULTI: its first token (a row of
    // q and out), how many it has, and how many positions the first one sees.
    struct Seq {
        int ctx, row, tok0, tokens, first;
    };
    auto seq_of = [&](int i) -> Seq {
        if constexpr (!MULTI) {
            return Seq{min(max(a.lens[i], 0), cap), i, i, 1, 0};
        } else {
            const int row = i / fa.groups, j0 = i % fa.groups * (G >> fa.shift);
            const int c = a.lens[row];
            const long long q0 = fa.q_start[row], n = fa.q_start[row + 1] - q0;
            const bool bad = q0 < 0 || n < 0 || n > fa.max_query || q0 + n > fa.n_tokens || n > c || c > cap;
            if (bad && j0 == 0 && blockIdx.x == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_QUERY_RANGE);
            if (bad || j0 >= n) return Seq{0, row, 0, 0, 0};
            const int tokens = min(G >> fa.shift, (int)n - j0), first = c - (int)n + j0 + 1;
            return Seq{first + tokens - 1, row, (int)q0 + j0, tokens, first};
        }
    };
    auto length = [&](int i) -> int { return seq_of(i).ctx; };
    auto blocks_of = [&](int len) -> int { return (len + kBlock - 1) / kBlock; };
    // places a pair of so many blocks takes in the list: first its cost, then its blocks
    auto span_of = [](int blocks) -> int { return blocks > 0 ? blocks + kPairCost<Q8> : 0; };
    auto zero_row = [&](size_t row0, int n) {
        for (int i = threadIdx.x; i < n * D / 8; i += NW * 32)
            reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + row0 * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    };

    // The run: [x, x_end) of the list, x lying at block `b` of pair (s, g). In a grid of partitions it is
    // one partition of a context.
    long long x, x_end, per = 0;
    int s, g, b, ctx;
    if (fa.partition > 0) {
        s = blockIdx.z;
        g = blockIdx.y;
        b = blockIdx.x * fa.partition;
        if (!MULTI && threadIdx.x == 0 && blockIdx.x == 0 && g == 0 && (a.lens[s] < 0 || a.lens[s] > cap))
            atomicOr(a.status, (unsigned)PKV_DEV_BAD_CONTEXT_LEN);
        ctx = length(s);
        const int nb = blocks_of(ctx);
        if (b >= nb) {
            if (!MULTI && b == 0) zero_row((size_t)s * a.n_q + (size_t)g * G, G);
            return;
        }
        x = b;
        x_end = min(b + fa.partition, nb);
    } else {
        // thread t sums the blocks of sequences [t per_t, (t + 1) per_t); a scan gives where they lie
        long long* s_find = reinterpret_cast<long long*>(smem + S::FIND);
        const int per_t = (a.n_seqs + NW * 32 - 1) / (NW * 32);
        const int i0 = min((int)threadIdx.x * per_t, a.n_seqs), i1 = min(i0 + per_t, a.n_seqs);
        long long mine = 0;
        for (int i = i0; i < i1; ++i) {
            if (!MULTI && blockIdx.x == 0 && (a.lens[i] < 0 || a.lens[i] > cap))
                atomicOr(a.status, (unsigned)PKV_DEV_BAD_CONTEXT_LEN);
            mine += span_of(blocks_of(length(i)));
        }
        long long before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31) s_find[warp] = before;
        __syncthreads();
        long long total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += s_find[w];
            total += s_find[w];
        }
        before -= mine;
        total *= a.n_kv;
        // equal runs, but of 24 places at least: shorter ones of a small call are more partials to join than
        // they save (2 heads of 16,000 tokens: 8 places 31 us, 16 22.7, 24 21.0, 32 21.1)
        per = max((total + gridDim.x - 1) / gridDim.x, 24LL);
        x = per * blockIdx.x;
        x_end = min(x + per, total);
        if (x >= before * a.n_kv && x < (before + mine) * a.n_kv) {  // one thread, if the run is not empty
            int i = i0;
            while (true) {
                const int n = span_of(blocks_of(length(i)));
                if (x < (before + n) * a.n_kv) break;
                before += n;
                ++i;
            }
            s_find[NW] = i;
            s_find[NW + 1] = x - before * a.n_kv;
        }
        for (int i = blockIdx.x; !MULTI && i < a.n_seqs; i += gridDim.x)
            if (a.lens[i] <= 0) zero_row((size_t)i * a.n_q, a.n_q);
        __syncthreads();
        if (x >= x_end) return;
        s = (int)s_find[NW];
        ctx = length(s);
        const long long off = s_find[NW + 1];
        const int span = span_of(blocks_of(ctx));
        g = (int)(off / span);
        b = (int)(off - (long long)g * span) - kPairCost<Q8>;
        if (b < 0) {  // the run starts before the pair's first block
            x -= b;
            b = 0;
            if (x >= x_end) return;
        }
    }

    float* s_join = reinterpret_cast<float*>(smem + S::JOIN);  // [COLS][NW] weights, [COLS] maxima, [COLS] sums
    float2* s_ml = reinterpret_cast<float2*>(smem + S::ML);    // [NW][COLS]
    int t_next = 0;     // this warp's first chunk of the next pair's table, read ahead
    bool ahead = false; // and whether it has been
    bool lost = false;  // a wait gave up
    int done = 0;  // iterations of this warp in earlier pairs: the ring and its phases run on
    while (true) {  // one pair (s, g), blocks [b, b + nblk) of its nb
        const int nb = blocks_of(ctx);
        const int nblk = (int)min(x_end - x, (long long)(nb - b));
        const Seq seq = seq_of(s);
        const size_t row0 = MULTI ? (size_t)seq.tok0 * a.n_q + (size_t)g * (1 << fa.shift) : (size_t)s * a.n_q + (size_t)g * G;
        const PairRows<const T, D, MULTI> q_rows{reinterpret_cast<const T*>(a.q) + row0 * D, a.n_q, fa.shift,
                                                 seq.tokens << fa.shift};
        const PairRows<T, D, MULTI> out_rows{reinterpret_cast<T*>(a.out) + row0 * D, a.n_q, fa.shift, q_rows.rows};

        // This warp's i-th block (i = BPI k + u) is block BPI (warp + k NW) + u of the run's share. Table
        // entries come in chunks of 32 held in registers (lane l: entry 32 c + l): the chunk whose copies
        // are being issued, the next, and the one after; scales follow a chunk behind the tables.
        auto local_block = [&](int i) -> int { return (i / BPI) * (NW * BPI) + warp * BPI + i % BPI; };
        const int32_t* table = a.tables + (size_t)seq.row * a.max_blocks + b;
        auto load_chunk = [&](int c) -> int {
            const int lb = local_block(c * 32 + lane);
            return lb < nblk ? table[lb] : -1;
        };
        int t0 = ahead ? t_next : load_chunk(0);
        int t1 = nblk > 32 * NW ? load_chunk(1) : -1;
        int t2 = nblk > 64 * NW ? load_chunk(2) : -1;
        constexpr int PER = KSTEPS / S::KCH;  // k-steps per chunk of a K row
        uint2 qraw[NT][KSTEPS];               // the query rows' words, on their way while the first tiles are
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + gid;
            const T* qrow = q_rows.row(r);
#pragma unroll
            for (int i = 0; i < KSTEPS; ++i) {
                qraw[nt][i] = make_uint2(0u, 0u);
                if (r < G && q_rows.has(r))
                    qraw[nt][i] = *reinterpret_cast<const uint2*>(qrow + S::k_chunk(tig, i / PER) * (Q8 ? 16 : 8) +
                                                              (i % PER) * 4);
            }
        }
        // iterations of this warp, and its blocks (the last iteration may have one less than BPI)
        const int nk = nblk > warp * BPI ? (nblk - warp * BPI + NW * BPI - 1) / (NW * BPI) : 0;
        const int ni = nk == 0 ? 0 : (nk - 1) * BPI + min(BPI, nblk - local_block((nk - 1) * BPI));

        // the pair after this one, if the run holds any of it
        int s_next = s, g_next = g + 1, ctx_next = ctx;
        ahead = fa.partition == 0 && x + nblk + kPairCost<Q8> < x_end;
        if (ahead) {
            if (g_next == a.n_kv) {
                g_next = 0;
                do ctx_next = length(++s_next);
                while (ctx_next == 0);
            }
            const int n = blocks_of(ctx_next), lb = local_block(lane);
            t_next = lb < n ? a.tables[(size_t)(MULTI ? s_next / fa.groups : s_next) * a.max_blocks + lb] : -1;
        }

        struct Blocks {
            int phys[BPI];
        };
        // Every lane: the blocks of iteration k (-1: none), for k = 0, 1, 2, ... in order (each once).
        auto entries = [&](int k) -> Blocks {
            const int i = k * BPI;
            if ((i & 31) == 0 && i > 0) {
                t0 = t1;
                t1 = t2;
                t2 = load_chunk((i >> 5) + 2);
            }
            Blocks e;
#pragma unroll
            for (int u = 0; u < BPI; ++u) {
                e.phys[u] = __shfl_sync(0xffffffffu, t0, (i & 31) + u);
                const bool inside = (unsigned)e.phys[u] < (unsigned)a.num_blocks;
                if (i + u < ni && !inside && lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_BLOCK_ID);
                if (i + u >= ni || !inside) e.phys[u] = -1;
            }
            return e;
        };
        // lane 0: start the copies of the K (v = 0) or V (v = 1) tiles of iteration k; none: the phase
        // completes with nothing copied
        auto issue = [&](int k, int v, const Blocks& e) {
            const int st = (done + k) % ST;
            uint64_t* bar = &wbars[st * 2 + v];
            uint32_t bytes = 0;
#pragma unroll
            for (int u = 0; u < BPI; ++u) bytes += e.phys[u] >= 0 ? TILE : 0u;
            if (bytes > 0) mbar_arrive_expect_tx(bar, bytes);
            else mbar_arrive(bar);
#pragma unroll
            for (int u = 0; u < BPI; ++u) {
                if (e.phys[u] < 0) continue;
                const int row = (int)(((long long)e.phys[u] * a.n_kv + g) * kBlock);
                const uint32_t dst = wstage + (uint32_t)st * S::STAGE + (uint32_t)(v * BPI + u) * TILE;
#pragma unroll
                for (int pn = 0; pn < S::PANELS; ++pn)
                    tma_load_2d(dst + pn * S::PANEL, v ? &tm_v : &tm_k, pn * (Q8 ? S::PANB : S::PANB / 2), row, bar, policy);
            }
        };
        auto phase = [&](int k) -> uint32_t { return (uint32_t)((done + k) / ST) & 1u; };
        // after a timed-out wait: wait (bounded) for the tiles of iterations [k0, k1) of kind v still in flight
        auto drain = [&](int k0, int k1, int v) {
            for (int kk = k0; kk < k1 && kk < nk; ++kk) mbar_wait_bounded(&wbars[((done + kk) % ST) * 2 + v], phase(kk));
        };
        // Valid blocks of the iterations in the ring, as bits (iteration k: bits BPI (k % ST) ..).
        unsigned ring = 0;
        auto note = [&](int k, const Blocks& e) {
            const int at = (k % ST) * BPI;
#pragma unroll
            for (int u = 0; u < BPI; ++u) ring = (ring & ~(1u << (at + u))) | ((e.phys[u] >= 0 ? 1u : 0u) << (at + u));
        };
        static_assert(ST * BPI <= 16, "a ring's blocks fit the bits and one chunk of the table");
        // Scales of the blocks of t0's chunk at the time, lane l: entry 32 c + l. They are consumed up to ST
        // iterations behind the copies, so their chunk moves when the consumer enters it: t0 has entered it
        // already (ST BPI <= 16 entries ago) and not left it.
        auto load_scales = [&](int c, int phys) -> float2 {
            if (!Q8 || c * 32 + lane >= ni || (unsigned)phys >= (unsigned)a.num_blocks) return make_float2(0.f, 0.f);
            const size_t i = (size_t)phys * a.n_kv + g;
            return make_float2(fa.k_scales[i], fa.v_scales[i]);
        };
        float2 s0 = load_scales(0, t0), s1 = load_scales(1, t1);
        for (int k = 0; k < ST && k < nk; ++k) {
            const Blocks e = entries(k);
            note(k, e);
            if (lane == 0) {
                issue(k, 0, e);
                issue(k, 1, e);
            }
        }

        // Q^T fragments: k-step `ks` of row gid takes four dims of one of the lane's K chunks (one 32-bit
        // word of codes, two words of halves); rows >= G are 0.
        uint32_t qb[NT][KSTEPS][2];
        float zf[NT][2];  // factor of the logits of the lane's query rows
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (Q8) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < KSTEPS; ++i) {
                    const float2 lo = MmaType<T>::unpack(qraw[nt][i].x), hi = MmaType<T>::unpack(qraw[nt][i].y);
                    const float f[4] = {fabsf(lo.x), fabsf(lo.y), fabsf(hi.x), fabsf(hi.y)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (f[e] <= 3.4028234e38f) amax = fmaxf(amax, f[e]);
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^-eq brings the row's largest element into [2^14, 2^15)
                const int eq = max(amax > 0.f ? ilogbf(amax) - 14 : 0, -126);
                const float down = pow2(-eq);
#pragma unroll
                for (int i = 0; i < KSTEPS; ++i) {
                    const float2 lo = MmaType<T>::unpack(qraw[nt][i].x), hi = MmaType<T>::unpack(qraw[nt][i].y);
                    qb[nt][i][0] = M::pack(lo.x * down, lo.y * down);
                    qb[nt][i][1] = M::pack(hi.x * down, hi.y * down);
                }
                const float f = a.scale_log2 * pow2(eq);
                zf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
                zf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
            } else {
#pragma unroll
                for (int i = 0; i < KSTEPS; ++i) {
                    qb[nt][i][0] = qraw[nt][i].x;
                    qb[nt][i][1] = qraw[nt][i].y;
                }
                zf[nt][0] = zf[nt][1] = a.scale_log2;
            }
        }

        float acc[NT][KSTEPS][4];  // m-tile mt: (dims dA, dA + 1) x (row 2tig | 2tig+1)
        float m_run[NT][2];        // of z
        float m_out[NT][2];        // of z + log2 S_V (8-bit pools)
        float l_run[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < KSTEPS; ++mt) acc[nt][mt][0] = acc[nt][mt][1] = acc[nt][mt][2] = acc[nt][mt][3] = 0.f;
            m_run[nt][0] = m_run[nt][1] = m_out[nt][0] = m_out[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.f;
        }

        // where logits go: memory, or behind the rings in a grid of partitions
        float* zrow = nullptr;
        int z0 = 0;  // the position it starts with
        if (fa.partition > 0 && fa.scores) {
            zrow = reinterpret_cast<float*>(smem + S::TOTAL);
            z0 = b * kBlock;
        } else if (fa.z) {
            zrow = fa.z + ((size_t)s * a.n_kv + g) * cap * G;
        }
        const int z_end = min(ctx, (b + nblk) * kBlock);  // positions behind belong to the next run

        for (int k = 0; k < nk; ++k) {
            const int st = (done + k) % ST;
            const uint32_t par = phase(k);
            const unsigned have = (ring >> ((k % ST) * BPI)) & ((1u << BPI) - 1);
            Blocks next;
            if (k + ST < nk) {  // the blocks whose copies go next
                next = entries(k + ST);
                note(k + ST, next);
            }
            float2 sc2[BPI];
#pragma unroll
            for (int u = 0; u < BPI; ++u) {
                const int i = k * BPI + u;
                if (Q8) {
                    if ((i & 31) == 0 && i > 0) {
                        s0 = s1;
                        s1 = load_scales((i >> 5) + 1, t1);
                    }
                    sc2[u] = make_float2(__shfl_sync(0xffffffffu, s0.x, i & 31), __shfl_sync(0xffffffffu, s0.y, i & 31));
                } else {
                    sc2[u] = make_float2(1.f, 1.f);
                }
            }
            if (!mbar_wait_bounded(&wbars[st * 2], par)) {
                if (lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
                drain(k, k + ST, 0);  // K tiles of iterations k .. k+ST-1 may be in flight
                drain(k, k + ST, 1);  // and their V tiles
                lost = true;
                break;
            }
            const int jb = (b + local_block(k * BPI)) * kBlock;
            const uint32_t sK = wstage + (uint32_t)st * S::STAGE;
            const uint32_t sV = sK + BPI * TILE;
            int nvalid[BPI];
#pragma unroll
            for (int u = 0; u < BPI; ++u) nvalid[u] = (have >> u) & 1 ? min(kBlock, ctx - jb - u * kBlock) : 0;
            uint32_t b0f[NT][BPI], b1f[NT][BPI];
            if (have) {
                // ---- S = K Q^T (16 tokens x 8 rows a block and column tile), fp32; two chains hide the
                // instruction's latency where there is one tile ----
                float z[NT][BPI][4];  // tokens gid (0, 1) and gid + 8 (2, 3) x the lane's rows
#pragma unroll
                for (int u = 0; u < BPI; ++u) {
                    float sa[NT][4], sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sa[nt][0] = sa[nt][1] = sa[nt][2] = sa[nt][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < S::KCH; ++i) {
                        const int c = S::k_chunk(tig, i);
                        const uint32_t tile = sK + u * TILE;
                        const uint4 lo = lds128(tile + S::at(gid, c)), hi = lds128(tile + S::at(gid + 8, c));
                        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
                        if constexpr (Q8) {
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint32_t af[4] = {e4m3x2_to_half2(wl[w]), e4m3x2_to_half2(wh[w]),
                                                        e4m3x2_to_half2(wl[w] >> 16), e4m3x2_to_half2(wh[w] >> 16)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    M::mma(NT == 1 && (w & 1) ? sb : sa[nt], af, qb[nt][i * 4 + w][0], qb[nt][i * 4 + w][1]);
                            }
                        } else {
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const uint32_t af[4] = {wl[2 * w], wh[2 * w], wl[2 * w + 1], wh[2 * w + 1]};
                                M::mma(w ? sb : sa[0], af, qb[0][i * 2 + w][0], qb[0][i * 2 + w][1]);
                            }
                        }
                    }
                    const bool v0 = gid < nvalid[u], v1 = gid + 8 < nvalid[u];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* x = z[nt][u];
                        const float f0 = zf[nt][0] * sc2[u].x, f1 = zf[nt][1] * sc2[u].x;
                        x[0] = v0 ? (NT == 1 ? sa[nt][0] + sb[0] : sa[nt][0]) * f0 : -INFINITY;
                        x[1] = v0 ? (NT == 1 ? sa[nt][1] + sb[1] : sa[nt][1]) * f1 : -INFINITY;
                        x[2] = v1 ? (NT == 1 ? sa[nt][2] + sb[2] : sa[nt][2]) * f0 : -INFINITY;
                        x[3] = v1 ? (NT == 1 ? sa[nt][3] + sb[3] : sa[nt][3]) * f1 : -INFINITY;
                        if constexpr (MULTI) {  // each column's token sees the positions up to its own
                            const int pos = jb + u * kBlock + gid, r = nt * 8 + 2 * tig;
                            const int e0 = seq.first + (r >> fa.shift), e1 = seq.first + (r + 1 >> fa.shift);
                            if (pos >= e0) x[0] = -INFINITY;
                            if (pos >= e1) x[1] = -INFINITY;
                            if (pos + 8 >= e0) x[2] = -INFINITY;
                            if (pos + 8 >= e1) x[3] = -INFINITY;
                        }
                    }
                }
                float ev[BPI];  // log2 S_V of the blocks (of a power of two; -inf for 0)
#pragma unroll
                for (int u = 0; u < BPI; ++u) ev[u] = Q8 && nvalid[u] > 0 ? __log2f(sc2[u].y) : 0.f;
                if constexpr (!MULTI) {
                    if (zrow != nullptr && 2 * tig < G) {
#pragma unroll
                        for (int u = 0; u < BPI; ++u) {
                            const float* x = z[0][u];
                            float* zt = zrow + (size_t)(jb - z0 + u * kBlock + gid) * G + 2 * tig;
                            const bool v0 = jb + u * kBlock + gid < z_end, v1 = jb + u * kBlock + gid + 8 < z_end;
                            if constexpr (G == 1) {
                                if (v0) zt[0] = x[0];
                                if (v1) zt[8] = x[2];
                            } else {
                                if (v0) *reinterpret_cast<float2*>(zt) = make_float2(x[0], x[1]);
                                if (v1) *reinterpret_cast<float2*>(zt + 8 * G) = make_float2(x[2], x[3]);
                            }
                        }
                    }
                }
                // ---- online softmax ----
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float mx0 = -INFINITY, mx1 = -INFINITY, mo0 = m_out[nt][0], mo1 = m_out[nt][1];
#pragma unroll
                    for (int u = 0; u < BPI; ++u) {
                        const float a0 = fmaxf(z[nt][u][0], z[nt][u][2]), a1 = fmaxf(z[nt][u][1], z[nt][u][3]);
                        mx0 = fmaxf(mx0, a0);
                        mx1 = fmaxf(mx1, a1);
                        if constexpr (Q8) {  // the largest z + log2 S_V of the iteration needs each block's own maximum
                            mo0 = fmaxf(mo0, a0 + ev[u]);
                            mo1 = fmaxf(mo1, a1 + ev[u]);
                        }
                    }
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) {
                        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
                        if constexpr (Q8) {
                            mo0 = fmaxf(mo0, __shfl_xor_sync(0xffffffffu, mo0, o));
                            mo1 = fmaxf(mo1, __shfl_xor_sync(0xffffffffu, mo1, o));
                        }
                    }
                    // A maximum of -inf (nothing but -inf or NaN logits so far) stands for 0: 2^(-inf - 0) is 0.
                    const float mn0 = fmaxf(m_run[nt][0], mx0), mn1 = fmaxf(m_run[nt][1], mx1);
                    const float ms0 = mn0 == -INFINITY ? 0.f : mn0, ms1 = mn1 == -INFINITY ? 0.f : mn1;
                    const float al0 = ex2(m_run[nt][0] - ms0), al1 = ex2(m_run[nt][1] - ms1);
                    m_run[nt][0] = mn0;
                    m_run[nt][1] = mn1;
                    float sum0 = 0.f, sum1 = 0.f;
                    float c0 = 0.f, c1 = 0.f, be0 = al0, be1 = al1;
                    if constexpr (Q8) {
                        const float os0 = mo0 == -INFINITY ? 0.f : mo0, os1 = mo1 == -INFINITY ? 0.f : mo1;
                        be0 = ex2(m_out[nt][0] - os0);
                        be1 = ex2(m_out[nt][1] - os1);
                        m_out[nt][0] = mo0;
                        m_out[nt][1] = mo1;
                        c0 = kWeightExp - os0;
                        c1 = kWeightExp - os1;
                    }
#pragma unroll
                    for (int u = 0; u < BPI; ++u) {
                        // the sum is of the weights before rounding: the scores divide by it in fp32
                        const float* x = z[nt][u];
                        const float p0 = ex2(x[0] - ms0), p1 = ex2(x[1] - ms1), p2 = ex2(x[2] - ms0), p3 = ex2(x[3] - ms1);
                        sum0 += p0 + p2;
                        sum1 += p1 + p3;
                        uint32_t pa, pb;  // tokens gid, gid + 8: the lane's rows
                        if constexpr (Q8) {
                            const float e0 = ev[u] + c0, e1 = ev[u] + c1;
                            pa = M::pack(ex2(x[0] + e0), ex2(x[1] + e1));
                            pb = M::pack(ex2(x[2] + e0), ex2(x[3] + e1));
                        } else {
                            pa = M::pack(p0 * kUp, p1 * kUp);
                            pb = M::pack(p2 * kUp, p3 * kUp);
                        }
                        b0f[nt][u] = movmatrix_trans(pa);  // P^T: tokens 2tig, 2tig+1 of row gid
                        b1f[nt][u] = movmatrix_trans(pb);  // tokens 8+2tig, 9+2tig of row gid
                    }
                    l_run[nt][0] = fmaf(l_run[nt][0], al0, sum0);
                    l_run[nt][1] = fmaf(l_run[nt][1], al1, sum1);
                    if (__any_sync(0xffffffffu, be0 != 1.f || be1 != 1.f)) {
#pragma unroll
                        for (int mt = 0; mt < KSTEPS; ++mt) {
                            acc[nt][mt][0] *= be0;
                            acc[nt][mt][1] *= be1;
                            acc[nt][mt][2] *= be0;
                            acc[nt][mt][3] *= be1;
                        }
                    }
                }
            } else if (zrow != nullptr) {  // blocks outside the pool: their positions weigh nothing
                for (int x = lane; x < BPI * kBlock * G; x += 32)
                    if (jb + x / G < z_end) zrow[(size_t)(jb - z0) * G + x] = -INFINITY;
            }
            __syncwarp();  // the K tiles have been read by every lane
            if (lane == 0 && k + ST < nk) {
                fence_proxy_async_smem();
                issue(k + ST, 0, next);
            }
            if (!mbar_wait_bounded(&wbars[st * 2 + 1], par)) {
                if (lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
                drain(k + 1, k + ST + 1, 0);  // K tiles of iterations k+1 .. k+ST may be in flight
                drain(k, k + ST, 1);          // V tiles of iterations k .. k+ST-1
                lost = true;
                break;
            }
            // ---- O^T += V^T P^T: this lane's tokens are 2tig, 2tig+1, 2tig+8, 2tig+9 ----
#pragma unroll
            for (int u = 0; u < BPI; ++u) {
                if (nvalid[u] <= 0) continue;
                const uint32_t tile = sV + u * TILE;
#pragma unroll
                for (int pn = 0; pn < S::PANELS; ++pn) {
                    constexpr int WORDS = S::PANB / 32;  // 32-bit words of a row and panel per lane
                    uint32_t w[4][WORDS];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tok = 2 * tig + (j & 1) + 8 * (j >> 1);
                        if constexpr (WORDS == 4) {
                            const uint4 x = lds128(tile + S::at(tok, pn * 8 + gid));
                            w[j][0] = x.x;
                            w[j][1] = x.y;
                            w[j][2] = x.z;
                            w[j][3] = x.w;
                        } else {
                            const uint2 x = lds64(tile + S::at(tok, gid >> 1) + (gid & 1) * 8);
                            w[j][0] = x.x;
                            w[j][1] = x.y;
                        }
                    }
                    if (nvalid[u] < kBlock) {  // rows past the context may hold anything
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int x = 0; x < WORDS; ++x)
                                w[j][x] = 2 * tig + (j & 1) + 8 * (j >> 1) < nvalid[u] ? w[j][x] : 0u;
                    }
                    if constexpr (MULTI) {
                        // A NaN in a row that only some of the group's tokens see would reach the others as 0 x NaN:
                        // such a panel goes token by token, each with the rows behind its own removed.
                        bool nan = false;
                        if (jb + (u + 1) * kBlock > seq.first) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int x = 0; x < WORDS; ++x)
                                    nan = nan || __vcmpeq4(w[j][x] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
                        }
                        if (__any_sync(0xffffffffu, nan)) {
                            for (int i = 0; i < seq.tokens; ++i) {
                                const int seen = seq.first + i - (jb + u * kBlock);  // rows of the block that token i sees
#pragma unroll
                                for (int x = 0; x < WORDS; ++x) {
                                    uint32_t v[4];
#pragma unroll
                                    for (int j = 0; j < 4; ++j) v[j] = 2 * tig + (j & 1) + 8 * (j >> 1) < seen ? w[j][x] : 0u;
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const uint32_t sel = h ? 0x7362u : 0x5140u;
                                        const uint32_t x01 = __byte_perm(v[0], v[1], sel), x23 = __byte_perm(v[2], v[3], sel);
                                        const uint32_t af[4] = {e4m3x2_to_half2(x01), e4m3x2_to_half2(x01 >> 16),
                                                                e4m3x2_to_half2(x23), e4m3x2_to_half2(x23 >> 16)};
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt) {
                                            const int r = nt * 8 + 2 * tig;
                                            float part[4] = {0.f, 0.f, 0.f, 0.f};
                                            M::mma(part, af, b0f[nt][u], b1f[nt][u]);
                                            float* to = acc[nt][(pn * WORDS + x) * 2 + h];
                                            if (r >> fa.shift == i) {
                                                to[0] += part[0];
                                                to[2] += part[2];
                                            }
                                            if (r + 1 >> fa.shift == i) {
                                                to[1] += part[1];
                                                to[3] += part[3];
                                            }
                                        }
                                    }
                                }
                            }
                            continue;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < WORDS; ++x) {
                        if constexpr (Q8) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t sel = h ? 0x7362u : 0x5140u;  // bytes (t0.d, t1.d, t0.d+1, t1.d+1)
                                const uint32_t x01 = __byte_perm(w[0][x], w[1][x], sel);
                                const uint32_t x23 = __byte_perm(w[2][x], w[3][x], sel);
                                const uint32_t af[4] = {e4m3x2_to_half2(x01), e4m3x2_to_half2(x01 >> 16),
                                                        e4m3x2_to_half2(x23), e4m3x2_to_half2(x23 >> 16)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    M::mma(acc[nt][(pn * WORDS + x) * 2 + h], af, b0f[nt][u], b1f[nt][u]);
                            }
                        } else {
                            const uint32_t af[4] = {__byte_perm(w[0][x], w[1][x], 0x5410u), __byte_perm(w[0][x], w[1][x], 0x7632u),
                                                    __byte_perm(w[2][x], w[3][x], 0x5410u), __byte_perm(w[2][x], w[3][x], 0x7632u)};
                            M::mma(acc[0][pn * WORDS + x], af, b0f[0][u], b1f[0][u]);
                        }
                    }
                }
            }
            __syncwarp();  // the V tiles have been read by every lane
            if (lane == 0 && k + ST < nk) {
                fence_proxy_async_smem();
                issue(k + ST, 1, next);
            }
        }

        // ---- row sums over the 8 lanes sharing a row; the accumulator in units of 2^m_run ----
        float fo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l_run[nt][r] += __shfl_xor_sync(0xffffffffu, l_run[nt][r], o);
                fo[nt][r] = 1.f / kUp;
                if constexpr (Q8)
                    fo[nt][r] = m_out[nt][r] == -INFINITY ? 0.f : exp2f(m_out[nt][r] - kWeightExp - m_run[nt][r]);
            }
        }

        // ---- join the warps ----
        __syncthreads();  // the rings have been read
        float* s_acc = reinterpret_cast<float*>(smem);  // [NW][G][D]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r0 = nt * 8 + 2 * tig;
#pragma unroll
            for (int mt = 0; mt < KSTEPS; ++mt) {
                constexpr int WORDS = S::PANB / 32;
                constexpr int PER_PANEL = Q8 ? 2 * WORDS : WORDS;       // m-tiles per panel
                constexpr int PAN_D = S::PANB / (Q8 ? 1 : 2);           // dims per panel
                const int d0 = (mt / PER_PANEL) * PAN_D + gid * (2 * PER_PANEL) + 2 * (mt % PER_PANEL);
                const float* x = acc[nt][mt];
                float* base = s_acc + (size_t)warp * G * D;
                if (r0 < G) *reinterpret_cast<float2*>(base + r0 * D + d0) = make_float2(x[0] * fo[nt][0], x[2] * fo[nt][0]);
                if (r0 + 1 < G)
                    *reinterpret_cast<float2*>(base + (r0 + 1) * D + d0) = make_float2(x[1] * fo[nt][1], x[3] * fo[nt][1]);
            }
            if (gid == 0) {
                s_ml[warp * S::COLS + r0] = make_float2(m_run[nt][0], l_run[nt][0]);
                s_ml[warp * S::COLS + r0 + 1] = make_float2(m_run[nt][1], l_run[nt][1]);
            }
        }
        __syncthreads();
        float* s_max = s_join + S::COLS * NW;
        float* s_sum = s_max + S::COLS;
        if (threadIdx.x < G) {
            const int r = threadIdx.x;
            float Mx = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) Mx = fmaxf(Mx, s_ml[w * S::COLS + r].x);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                // a warp without a finite maximum adds its sum times zero: nothing, or the NaN of its logits
                const float2 u = s_ml[w * S::COLS + r];
                const float f = u.x == -INFINITY ? 0.f : ex2(u.x - Mx);
                s_join[r * NW + w] = f;
                L = fmaf(u.y, f, L);
            }
            s_max[r] = Mx;
            s_sum[r] = L;
        }
        __syncthreads();
        // partials of this pair: one for each partition, or for each CTA whose run holds a piece of it
        int np, first = 0;
        if (fa.partition > 0) {
            np = (nb + fa.partition - 1) / fa.partition;
        } else {
            const long long start = x - b;
            first = (int)(start / per);
            np = (int)((start + nb - 1) / per) - first + 1;
        }
        const int slot = partial_slot(first, (int)blockIdx.x - first);
        float* s_po = reinterpret_cast<float*>(smem + S::MERGE);  // [G][D], then [G][2]: a cluster's partials
        float* s_pml = s_po + G * D;
        for (int i4 = threadIdx.x; i4 < G * D / 4; i4 += NW * 32) {
            const int r = i4 / (D / 4);
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = s_join[r * NW + w];
                const float4 v = reinterpret_cast<const float4*>(s_acc + (size_t)w * G * D)[i4];
                O.x = fmaf(v.x, f, O.x);
                O.y = fmaf(v.y, f, O.y);
                O.z = fmaf(v.z, f, O.z);
                O.w = fmaf(v.w, f, O.w);
            }
            if (np == 1) {
                const float L = s_sum[r];
                if (out_rows.has(r)) store4(out_rows.row(r) + 4 * (i4 % (D / 4)), O, L == 0.f ? 0.f : 1.f / L);
            } else if (fa.partition > 0) {
                reinterpret_cast<float4*>(s_po)[i4] = O;
            } else {
                reinterpret_cast<float4*>(a.part_o + (size_t)slot * G * D)[i4] = O;
            }
        }
        if (threadIdx.x < G) {
            const float2 u = make_float2(s_max[threadIdx.x], s_sum[threadIdx.x]);
            if (np == 1) {
                if (fa.row_ml) fa.row_ml[row0 + threadIdx.x] = u;
            } else if (fa.partition > 0) {
                reinterpret_cast<float2*>(s_pml)[threadIdx.x] = u;
            } else {
                reinterpret_cast<float2*>(a.part_ml)[(size_t)slot * G + threadIdx.x] = u;
            }
        }
        if (fa.partition > 0) {
            if (np > 1)
                cluster_join<T, D, G, NW * 32, MULTI>(out_rows, (int)blockIdx.x, np, s_pml, s_po,
                                                      fa.scores ? s_max : nullptr, s_sum);
            if (fa.scores) {  // weights of the partition's own positions (the barriers above order the logits)
                float* to = fa.scores + ((size_t)s * a.n_kv + g) * fa.score_stride + z0;
                for (int j = threadIdx.x; j < z_end - z0; j += NW * 32) {
                    float w = 0.f;
#pragma unroll
                    for (int r = 0; r < G; ++r) {
                        const float M = s_max[r], L = s_sum[r];
                        w += ex2(zrow[j * G + r] - (M == -INFINITY ? 0.f : M)) * (L == 0.f ? 0.f : 1.f / L);
                    }
                    to[j] += w;
                }
            }
            return;
        }
        if (np > 1)
            join_if_last<T, D, G, NW * 32, MULTI>(fa, out_rows, fa.row_ml ? fa.row_ml + row0 : nullptr, first, np,
                                                  reinterpret_cast<float*>(smem + S::MERGE));
        x += nblk + kPairCost<Q8>;  // the next pair's first block
        if (x >= x_end) return;
        // the next pair of the run
        done += nk;
        b = 0;
        s = s_next;
        g = g_next;
        ctx = ctx_next;
        if (__syncthreads_or(lost)) return;  // flagged: the ring's phases no longer match; the scratch has been read
        fence_proxy_async_smem();            // before the copies that overwrite it
    }
}

template <typename T, bool Q8, int D, int G, bool MULTI = false>
struct FragKernel {
    // Blocks per iteration, CTAs per SM: 64 to 128 KiB of tiles in flight an SM. More is slower (d = 128
    // codes, 10 x 30,000 tokens, 8 x 4 heads: 64 KiB 105 us, 96 KiB 99, 128 KiB 103, 192 KiB 115).
    static constexpr int NW = 4;
    static constexpr int ST = 1;
    static constexpr int BPI = Q8 && D == 64 && G <= 8 ? 4 : !Q8 && D == 256 ? 1 : 2;
    static constexpr int CTAS = D == 256 || G > 8 ? 2 : !Q8 || D == 128 ? 3 : 4;
    static constexpr size_t smem = FragGeom<Q8, D, G, NW, ST, BPI>::ALLOC;
    static unsigned long long attr_done;
    static int resident[64];
    static constexpr auto kernel = frag_decode_kernel<T, Q8, D, G, NW, ST, BPI, CTAS, MULTI>;
    static cudaError_t prepare() { return allow_dynamic_smem(kernel, smem + kMaxPartition * kBlock * G * sizeof(float), &attr_done); }
    // CTAs one SM of the current device holds at once; asked of the occupancy calculator once per device
    static cudaError_t ctas_per_sm(int* out) {
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        int n = __atomic_load_n(&resident[dev], __ATOMIC_RELAXED);
        if (n == 0) {
            err = prepare();
            if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, NW * 32, smem);
            if (err != cudaSuccess) return err;
            if (n <= 0) return cudaErrorInvalidConfiguration;
            __atomic_store_n(&resident[dev], n, __ATOMIC_RELAXED);
        }
        *out = n;
        return cudaSuccess;
    }
    static cudaError_t launch(const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
        cudaError_t err = prepare();
        if (err != cudaSuccess) return err;
        const dim3 grid = a.partition > 0 ? dim3(a.d.n_parts, a.d.n_kv, a.d.n_seqs) : dim3(a.d.n_parts);
        const size_t logits = a.partition > 0 && a.scores ? (size_t)a.partition * kBlock * G * sizeof(float) : 0;
        return launch_dependent(kernel, grid, NW * 32, smem + logits, stream, a.partition > 0 ? a.d.n_parts : 1, a, tk, tv);
    }
};
template <typename T, bool Q8, int D, int G, bool MULTI>
unsigned long long FragKernel<T, Q8, D, G, MULTI>::attr_done = 0;
template <typename T, bool Q8, int D, int G, bool MULTI>
int FragKernel<T, Q8, D, G, MULTI>::resident[64] = {};

#define PKV_FRAG_CASES                                                  \
    PKV_CASE(64, 1) PKV_CASE(64, 2) PKV_CASE(64, 4) PKV_CASE(64, 8)     \
    PKV_CASE(128, 1) PKV_CASE(128, 2) PKV_CASE(128, 4) PKV_CASE(128, 8) \
    PKV_CASE(256, 1) PKV_CASE(256, 2) PKV_CASE(256, 4) PKV_CASE(256, 8)

template <typename T, bool Q8>
cudaError_t frag_ctas_per_sm_of(int head_dim, int group, int* out) {
#define PKV_CASE(DD, GG) \
    if (head_dim == DD && group == GG) return FragKernel<T, Q8, DD, GG>::ctas_per_sm(out);
    PKV_FRAG_CASES
#undef PKV_CASE
    return cudaErrorInvalidValue;
}

template <typename T, bool Q8>
cudaError_t launch_frag_of(int head_dim, int group, const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t stream) {
#define PKV_CASE(DD, GG) \
    if (head_dim == DD && group == GG) return FragKernel<T, Q8, DD, GG>::launch(a, tk, tv, stream);
    PKV_FRAG_CASES
#undef PKV_CASE
    return cudaErrorInvalidValue;
}

// Prompt chunks (MULTI): `columns` query rows (tokens x heads of the group) a pair, 8 or 2,048 / D.
template <typename T>
cudaError_t frag_multi_ctas_per_sm_of(int head_dim, int columns, int* out) {
    if (columns == 8) switch (head_dim) {
        case 64: return FragKernel<T, true, 64, 8, true>::ctas_per_sm(out);
        case 128: return FragKernel<T, true, 128, 8, true>::ctas_per_sm(out);
        case 256: return FragKernel<T, true, 256, 8, true>::ctas_per_sm(out);
        }
    if (head_dim == 64 && columns == 32) return FragKernel<T, true, 64, 32, true>::ctas_per_sm(out);
    if (head_dim == 128 && columns == 16) return FragKernel<T, true, 128, 16, true>::ctas_per_sm(out);
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_frag_multi_of(int head_dim, int columns, const FragArgs& a, const CUtensorMap& tk,
                                 const CUtensorMap& tv, cudaStream_t stream) {
    if (columns == 8) switch (head_dim) {
        case 64: return FragKernel<T, true, 64, 8, true>::launch(a, tk, tv, stream);
        case 128: return FragKernel<T, true, 128, 8, true>::launch(a, tk, tv, stream);
        case 256: return FragKernel<T, true, 256, 8, true>::launch(a, tk, tv, stream);
        }
    if (head_dim == 64 && columns == 32) return FragKernel<T, true, 64, 32, true>::launch(a, tk, tv, stream);
    if (head_dim == 128 && columns == 16) return FragKernel<T, true, 128, 16, true>::launch(a, tk, tv, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
