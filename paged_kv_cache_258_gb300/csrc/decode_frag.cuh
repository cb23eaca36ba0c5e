// decode_frag.cuh -- decode attention over 8-bit pools, and over 16-bit pools with the attention
// weights summed (sm_103a).
//
// For sequence s, query head h of KV head g, position j in block b (16 tokens):
//   z_j = scale log2(e) S_K(b) (q . cK_j),   out = sum_j 2^(z_j - m) S_V(b) cV_j / sum_j 2^(z_j - m),
// c the stored codes, S the block's scale (1 for 16-bit pools). One pass over the cache: 2 D bytes a
// token and head for codes, against 4 D for 16-bit rows, so a kernel that keeps up with memory takes
// half the time -- and has half as long for the arithmetic of each token.
//
// The grid, the partitions, the split-K merge and the per-warp rings of TMA copies are those of
// decode_mma.cuh. What differs is how a 16-token tile gets from shared memory into fragments:
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
//  * Weights for the PV product are fp16 too (11 bits; the 16-bit pools' kernel rounds to the storage
//    type): w_j = 2^(z_j + log2 S_V(b) + 15 - m'), m' the running maximum of z + log2 S_V. So the
//    largest w is 2^15 whatever the blocks' scales, and one keeps 11 bits down to 2^-29 of it. The
//    sum of weights runs in fp32 beside it with its own maximum m.
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

template <bool Q8, int D, int NW, int ST>
struct FragGeom {
    static constexpr int ROWB = D * (Q8 ? 1 : 2);            // bytes of a row
    static constexpr int PANB = ROWB < 128 ? ROWB : 128;     // bytes of a panel's row (one TMA box)
    static constexpr int PANELS = ROWB / PANB;
    static constexpr int PANEL = kBlock * PANB;
    static constexpr uint32_t TILE = kBlock * ROWB;
    static constexpr int KCH = ROWB / 64;                    // 16-byte chunks of a K row per lane
    static constexpr size_t STAGES = (size_t)NW * ST * 2 * TILE;
    static constexpr size_t BARS = STAGES;                               // uint64 [NW][ST][K, V]
    static constexpr size_t PHYS = BARS + (size_t)NW * ST * 16;          // int [NW][ST]
    static constexpr size_t SCALE = (PHYS + (size_t)NW * ST * 4 + 7) / 8 * 8;  // float2 [NW][ST] (K, V)
    static constexpr size_t ML = (SCALE + (size_t)NW * ST * 8 + 15) / 16 * 16;  // float [NW][8][2]
    static constexpr size_t TOTAL = ML + (size_t)NW * 8 * 2 * 4;
    static constexpr size_t ALLOC = TOTAL + 1024;             // room to align the base
    static constexpr size_t MERGE = (size_t)NW * 8 * D * 4;  // merge scratch, after the combine buffer
    static_assert(MERGE + MergeScratch<8>::BYTES <= STAGES, "combine buffer and merge scratch must fit");
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

constexpr float kWeightExp = 15.f;  // exponent of the largest fp16 weight

// Split-K epilogue of the CTA (s, g, p) of a sequence with np > 1 partitions: the CTA that arrives last
// at the (s, g) counter joins the np partials of every row in partition order,
//   out = sum_p o_p 2^(m_p - M) / sum_p l_p 2^(m_p - M),  M = max_p m_p.
// The counter protocol is splitk_merge_if_last's (decode.cuh): (call tag << 24) | arrivals, any other
// tag reads as zero arrivals, the merging CTA leaves 0. Unlike there, a partial whose sum is NaN makes
// the row NaN instead of being left out.
template <typename T, int D, int G, int NT>
__device__ __forceinline__ void frag_merge_if_last(const DecodeArgs& a, int s, int g, int np, float* scratch) {
    constexpr int NWARP = NT / 32;
    constexpr int PER = (G * D + NT - 1) / NT;
    constexpr int MQ = kMergeLoads / PER < 2 ? 2 : (kMergeLoads / PER > 16 ? 16 : kMergeLoads / PER);
    int* flag = reinterpret_cast<int*>(scratch);
    float* sM = scratch + 4;  // [G]
    float* sL = sM + G;       // [G]
    float* sW = sL + G;       // [G][kMergeChunk]
    unsigned long long* cnt = a.counters + (size_t)s * a.n_kv + g;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        unsigned long long cur = *reinterpret_cast<volatile unsigned long long*>(cnt);
        unsigned long long next;
        while (true) {
            next = ((cur >> 24) == a.call_tag) ? cur + 1 : ((a.call_tag << 24) | 1ull);
            const unsigned long long prev = atomicCAS(cnt, cur, next);
            if (prev == cur) break;
            cur = prev;
        }
        *flag = (next & 0xffffffull) == (unsigned long long)np;
        __threadfence();
    }
    __syncthreads();
    if (!*flag) return;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const size_t row0 = (size_t)s * a.n_q + (size_t)g * G;
    for (int r = warp; r < G; r += NWARP) {
        const float* ml = a.part_ml + (row0 + r) * a.n_parts * 2;
        float m = -INFINITY;
        for (int q = lane; q < np; q += 32) m = fmaxf(m, __ldcg(ml + 2 * q));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) {
            sM[r] = m;
            sL[r] = 0.f;
        }
    }
    float O[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) O[k] = 0.f;
    for (int c0 = 0; c0 < np; c0 += kMergeChunk) {
        __syncthreads();  // maxima visible; the previous chunk's weights consumed
        for (int r = warp; r < G; r += NWARP) {
            const float* ml = a.part_ml + (row0 + r) * a.n_parts * 2;
            const int q = c0 + lane;
            float w = 0.f, lw = 0.f;
            if (q < np) {
                const float m = __ldcg(ml + 2 * q);
                w = m == -INFINITY ? 0.f : exp2f(m - sM[r]);
                lw = __ldcg(ml + 2 * q + 1) * w;
            }
            sW[r * kMergeChunk + lane] = w;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
            if (lane == 0) sL[r] += lw;
        }
        __syncthreads();
        const int nq = min(kMergeChunk, np - c0);
        // groups of MQ partials: all MQ x PER loads of a group in flight before they are folded
        for (int q0 = 0; q0 < nq; q0 += MQ) {
            const int mq = min(MQ, nq - q0);
            float v[PER][MQ];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int idx = threadIdx.x + k * NT;
                const float* po = a.part_o + ((row0 + idx / D) * a.n_parts + c0 + q0) * D + idx % D;
#pragma unroll
                for (int u = 0; u < MQ; ++u) v[k][u] = (idx < G * D && u < mq) ? __ldcg(po + (size_t)u * D) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int idx = threadIdx.x + k * NT;
                if (idx < G * D) {
                    const float* w = sW + (idx / D) * kMergeChunk + q0;
#pragma unroll
                    for (int u = 0; u < MQ; ++u)
                        if (u < mq) O[k] = fmaf(w[u], v[k][u], O[k]);
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int idx = threadIdx.x + k * NT;
        if (idx < G * D) {
            const float L = sL[idx / D];
            reinterpret_cast<T*>(a.out)[row0 * D + idx] = from_float<T>(L == 0.f ? 0.f : O[k] / L);
        }
    }
    if (threadIdx.x == 0) *cnt = 0ull;
}

template <typename T, bool Q8, int D, int G, int NW, int ST>
__global__ void __launch_bounds__(NW * 32) frag_decode_kernel(const FragArgs fa, const __grid_constant__ CUtensorMap tm_k,
                                                              const __grid_constant__ CUtensorMap tm_v) {
    static_assert(G <= 8, "at most 8 query rows per KV head");
    using S = FragGeom<Q8, D, NW, ST>;
    using MT = typename std::conditional<Q8, __half, T>::type;  // type of the matrix instructions' operands
    using M = MmaType<MT>;
    constexpr int KSTEPS = D / 16;  // QK k-steps = PV m-tiles
    constexpr uint32_t TILE = S::TILE;
    const DecodeArgs& a = fa.d;

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);
    float* s_ml = reinterpret_cast<float*>(smem + S::ML);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int gid = lane >> 2;  // token row of S, chunk of V
    const int tig = lane & 3;   // owns query rows 2 tig, 2 tig + 1
    const int p = blockIdx.x;
    const int g = blockIdx.y;
    const int s = blockIdx.z;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Table entries of this warp's blocks, 32 per chunk in registers: the chunk in use, the next one
    // (with its blocks' scales already on their way) and the one after.
    auto load_chunk = [&](int c) -> int {
        const long long kk = (long long)c * 32 + lane;
        const long long idx = (long long)p * a.bpp + warp + kk * NW;
        return kk * NW + warp < a.bpp && idx < a.max_blocks ? a.tables[(size_t)s * a.max_blocks + idx] : -1;
    };
    auto load_scales = [&](int phys) -> float2 {
        if (!Q8 || (unsigned)phys >= (unsigned)a.num_blocks) return make_float2(0.f, 0.f);
        const size_t i = (size_t)phys * a.n_kv + g;
        return make_float2(__ldg(fa.k_scales + i), __ldg(fa.v_scales + i));
    };
    int t0 = load_chunk(0);
    int t1 = a.bpp > 32 * NW ? load_chunk(1) : -1;
    int t2 = a.bpp > 64 * NW ? load_chunk(2) : -1;
    int ctx = a.lens[s];
    const int cap = a.max_blocks * kBlock;
    if (ctx < 0 || ctx > cap) {
        if (p == 0 && threadIdx.x == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_CONTEXT_LEN);
        ctx = ctx < 0 ? 0 : cap;
    }
    const int nb = (ctx + kBlock - 1) / kBlock;
    const int b0 = p * a.bpp;
    if (b0 >= nb) {
        if (p == 0) {
            T* o = reinterpret_cast<T*>(a.out) + ((size_t)s * a.n_q + (size_t)g * G) * D;
            for (int i = threadIdx.x; i < G * D; i += NW * 32) o[i] = from_float<T>(0.f);
        }
        return;
    }
    const int nblk = min(a.bpp, nb - b0);
    const bool single = nb <= a.bpp;
    const int nk = nblk > warp ? (nblk - warp + NW - 1) / NW : 0;
    // entries past the sequence's last block may be anything: their scales are not read
    auto mine = [&](int c, int phys) { return c * 32 + lane < nk ? phys : -1; };
    float2 s0 = load_scales(mine(0, t0));
    float2 s1 = load_scales(mine(1, t1));

    if (threadIdx.x < 2 * NW * ST) mbar_init(&bars[threadIdx.x], 1);
    fence_mbar_init();
    __syncthreads();

    uint64_t* wbars = bars + warp * ST * 2;  // [ST][K, V]
    int* wphys = reinterpret_cast<int*>(smem + S::PHYS) + warp * ST;
    float2* wscale = reinterpret_cast<float2*>(smem + S::SCALE) + warp * ST;
    const uint32_t wstage = smem_addr(smem) + (uint32_t)(warp * ST) * 2 * TILE;
    const uint64_t policy = l2_evict_first_policy();

    struct Entry {
        int phys;
        float ks, vs;
    };
    // Every lane: this warp's k-th block and its scales, for k = 0, 1, 2, ... in order (each once).
    auto entry = [&](int k) -> Entry {
        if ((k & 31) == 0 && k > 0) {
            const int c = k >> 5;
            t0 = t1;
            t1 = t2;
            t2 = load_chunk(c + 2);
            if (Q8) {
                s0 = s1;
                s1 = load_scales(mine(c + 1, t1));
            }
        }
        Entry e;
        e.phys = __shfl_sync(0xffffffffu, t0, k & 31);
        e.ks = Q8 ? __shfl_sync(0xffffffffu, s0.x, k & 31) : 1.f;
        e.vs = Q8 ? __shfl_sync(0xffffffffu, s0.y, k & 31) : 1.f;
        return e;
    };
    // lane 0: start the copy of the K (v = 0) or V (v = 1) tile of this warp's k-th block
    auto issue = [&](int k, int v, const Entry& e) {
        const int st = k % ST;
        const bool ok = (unsigned)e.phys < (unsigned)a.num_blocks;
        uint64_t* bar = &wbars[st * 2 + v];
        if (v == 0) {
            wphys[st] = ok ? e.phys : -1;
            if (Q8) wscale[st] = make_float2(e.ks, e.vs);
        }
        if (ok) {
            const int row0 = (int)(((long long)e.phys * a.n_kv + g) * kBlock);
            const uint32_t dst = wstage + (uint32_t)st * 2 * TILE + (uint32_t)v * TILE;
            mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
            for (int pn = 0; pn < S::PANELS; ++pn)
                tma_load_2d(dst + pn * S::PANEL, v ? &tm_v : &tm_k, pn * (Q8 ? S::PANB : S::PANB / 2), row0, bar, policy);
        } else {
            if (v == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_BLOCK_ID);
            mbar_arrive(bar);  // completes the phase with nothing copied: the block is masked
        }
    };
    // after a timed-out wait: wait (bounded) for the tiles of blocks [k0, k1) of kind v still in flight
    auto drain = [&](int k0, int k1, int v) {
        for (int kk = k0; kk < k1 && kk < nk; ++kk) mbar_wait_bounded(&wbars[(kk % ST) * 2 + v], (uint32_t)(kk / ST) & 1u);
    };
    for (int k = 0; k < ST && k < nk; ++k) {
        const Entry e = entry(k);
        if (lane == 0) {
            issue(k, 0, e);
            issue(k, 1, e);
        }
    }

    // Q^T fragments: k-step `ks` of row gid takes the four dims of one 32-bit (codes) or 64-bit word
    // pair of the lane's K chunks; rows >= G are 0.
    uint32_t qb[KSTEPS][2];
    float zf[2];  // factor of the logits of query rows 2 tig, 2 tig + 1
    {
        const T* qrow = reinterpret_cast<const T*>(a.q) + ((size_t)s * a.n_q + (size_t)g * G + gid) * D;
        constexpr int PER = KSTEPS / S::KCH;  // k-steps per chunk
        if constexpr (Q8) {
            float qf[KSTEPS][4];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < KSTEPS; ++i) {
                if (gid < G) load4(qrow + S::k_chunk(tig, i / PER) * 16 + (i % PER) * 4, qf[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (gid >= G) qf[i][e] = 0.f;
                    const float x = fabsf(qf[i][e]);
                    if (x <= 3.4028234e38f) amax = fmaxf(amax, x);
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^-eq brings the row's largest element into [2^14, 2^15)
            const int eq = max(amax > 0.f ? ilogbf(amax) - 14 : 0, -126);
            const float down = pow2(-eq);
#pragma unroll
            for (int i = 0; i < KSTEPS; ++i) {
                qb[i][0] = M::pack(qf[i][0] * down, qf[i][1] * down);
                qb[i][1] = M::pack(qf[i][2] * down, qf[i][3] * down);
            }
            const float f = a.scale_log2 * pow2(eq);
            zf[0] = __shfl_sync(0xffffffffu, f, 8 * tig);
            zf[1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
        } else {
#pragma unroll
            for (int i = 0; i < KSTEPS; ++i) {
                uint2 u = make_uint2(0u, 0u);
                if (gid < G)
                    u = *reinterpret_cast<const uint2*>(qrow + S::k_chunk(tig, i / PER) * 8 + (i % PER) * 4);
                qb[i][0] = u.x;
                qb[i][1] = u.y;
            }
            zf[0] = zf[1] = a.scale_log2;
        }
    }

    float acc[KSTEPS][4];  // m-tile mt: (dims dA, dA + 1 of dim_of(mt)) x (row 2tig | 2tig+1)
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY};  // of z
    float m_out[2] = {-INFINITY, -INFINITY};  // of z + log2 S_V (8-bit pools)
    float l_run[2] = {0.f, 0.f};

    float* zrow = fa.z ? fa.z + ((size_t)s * a.n_kv + g) * cap * G : nullptr;

    for (int k = 0; k < nk; ++k) {
        const int st = k % ST;
        const uint32_t par = (uint32_t)(k / ST) & 1u;
        Entry next = {-1, 0.f, 0.f};
        if (k + ST < nk) next = entry(k + ST);  // the block whose copies go next
        if (!mbar_wait_bounded(&wbars[st * 2], par)) {
            if (lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
            drain(k, k + ST, 0);  // K tiles of blocks k .. k+ST-1 may be in flight
            drain(k, k + ST, 1);  // and their V tiles
            break;
        }
        const int jb = (b0 + warp + k * NW) * kBlock;
        const int live = min(kBlock, ctx - jb);
        const int nvalid = wphys[st] >= 0 ? live : 0;
        const float2 sc2 = Q8 ? wscale[st] : make_float2(1.f, 1.f);
        const uint32_t sK = wstage + (uint32_t)st * 2 * TILE;
        const uint32_t sV = sK + TILE;
        uint32_t b0f = 0u, b1f = 0u;
        if (nvalid > 0) {
            // ---- S = K Q^T (16 tokens x 8 rows), fp32; two chains hide the instruction's latency ----
            float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < S::KCH; ++i) {
                const int c = S::k_chunk(tig, i);
                const uint4 lo = lds128(sK + S::at(gid, c)), hi = lds128(sK + S::at(gid + 8, c));
                const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
                if constexpr (Q8) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t af[4] = {e4m3x2_to_half2(wl[w]), e4m3x2_to_half2(wh[w]),
                                                e4m3x2_to_half2(wl[w] >> 16), e4m3x2_to_half2(wh[w] >> 16)};
                        M::mma((w & 1) ? sb : sa, af, qb[i * 4 + w][0], qb[i * 4 + w][1]);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t af[4] = {wl[2 * u], wh[2 * u], wl[2 * u + 1], wh[2 * u + 1]};
                        M::mma(u ? sb : sa, af, qb[i * 2 + u][0], qb[i * 2 + u][1]);
                    }
                }
            }
            // ---- online softmax: lane holds tokens gid, gid+8 of rows 2tig, 2tig+1 ----
            const bool v0 = gid < nvalid, v1 = gid + 8 < nvalid;
            const float f0 = zf[0] * sc2.x, f1 = zf[1] * sc2.x;
            const float z0 = v0 ? (sa[0] + sb[0]) * f0 : -INFINITY;  // token gid,   row 2tig
            const float z1 = v0 ? (sa[1] + sb[1]) * f1 : -INFINITY;  // token gid,   row 2tig+1
            const float z2 = v1 ? (sa[2] + sb[2]) * f0 : -INFINITY;  // token gid+8, row 2tig
            const float z3 = v1 ? (sa[3] + sb[3]) * f1 : -INFINITY;  // token gid+8, row 2tig+1
            if (zrow != nullptr && 2 * tig < G) {
                float* zt = zrow + (size_t)(jb + gid) * G + 2 * tig;
                if constexpr (G == 1) {
                    if (v0) zt[0] = z0;
                    if (v1) zt[8] = z2;
                } else {
                    if (v0) *reinterpret_cast<float2*>(zt) = make_float2(z0, z1);
                    if (v1) *reinterpret_cast<float2*>(zt + 8 * G) = make_float2(z2, z3);
                }
            }
            float mx0 = fmaxf(z0, z2), mx1 = fmaxf(z1, z3);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            const float mn0 = fmaxf(m_run[0], mx0), mn1 = fmaxf(m_run[1], mx1);
            float al0 = (m_run[0] == -INFINITY) ? 0.f : exp2f(m_run[0] - mn0);
            float al1 = (m_run[1] == -INFINITY) ? 0.f : exp2f(m_run[1] - mn1);
            m_run[0] = mn0;
            m_run[1] = mn1;
            const float p0 = (z0 == -INFINITY) ? 0.f : exp2f(z0 - mn0);
            const float p1 = (z1 == -INFINITY) ? 0.f : exp2f(z1 - mn1);
            const float p2 = (z2 == -INFINITY) ? 0.f : exp2f(z2 - mn0);
            const float p3 = (z3 == -INFINITY) ? 0.f : exp2f(z3 - mn1);
            uint32_t pa, pb;  // tokens gid, gid + 8: rows 2tig, 2tig+1
            // the sum is of the weights before rounding: the scores divide by it in fp32
            l_run[0] = l_run[0] * al0 + (p0 + p2);
            l_run[1] = l_run[1] * al1 + (p1 + p3);
            if constexpr (Q8) {
                const float ev = log2f(sc2.y);  // exact for the power of two that the scale is; -inf for 0
                const float o0 = fmaxf(m_out[0], mx0 + ev), o1 = fmaxf(m_out[1], mx1 + ev);
                al0 = (m_out[0] == -INFINITY) ? 0.f : exp2f(m_out[0] - o0);
                al1 = (m_out[1] == -INFINITY) ? 0.f : exp2f(m_out[1] - o1);
                m_out[0] = o0;
                m_out[1] = o1;
                const float c0 = o0 == -INFINITY ? -INFINITY : ev + (kWeightExp - o0);
                const float c1 = o1 == -INFINITY ? -INFINITY : ev + (kWeightExp - o1);
                pa = M::pack(z0 == -INFINITY ? 0.f : exp2f(z0 + c0), z1 == -INFINITY ? 0.f : exp2f(z1 + c1));
                pb = M::pack(z2 == -INFINITY ? 0.f : exp2f(z2 + c0), z3 == -INFINITY ? 0.f : exp2f(z3 + c1));
            } else {
                pa = M::pack(p0, p1);
                pb = M::pack(p2, p3);
            }
            b0f = movmatrix_trans(pa);  // P^T: tokens 2tig, 2tig+1 of row gid
            b1f = movmatrix_trans(pb);  // tokens 8+2tig, 9+2tig of row gid
            if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
                for (int mt = 0; mt < KSTEPS; ++mt) {
                    acc[mt][0] *= al0;
                    acc[mt][1] *= al1;
                    acc[mt][2] *= al0;
                    acc[mt][3] *= al1;
                }
            }
        } else if (zrow != nullptr && 2 * tig < G) {  // a block outside the pool: its positions weigh nothing
            for (int r = gid; r < live; r += 8)
                for (int x = 2 * tig; x < min(G, 2 * tig + 2); ++x) zrow[(size_t)(jb + r) * G + x] = -INFINITY;
        }
        __syncwarp();  // the K tile has been read by every lane
        if (lane == 0 && k + ST < nk) {
            fence_proxy_async_smem();
            issue(k + ST, 0, next);
        }
        if (!mbar_wait_bounded(&wbars[st * 2 + 1], par)) {
            if (lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
            drain(k + 1, k + ST + 1, 0);  // K tiles of blocks k+1 .. k+ST may be in flight
            drain(k, k + ST, 1);          // V tiles of blocks k .. k+ST-1
            break;
        }
        if (nvalid > 0) {
            // ---- O^T += V^T P^T: this lane's tokens are 2tig, 2tig+1, 2tig+8, 2tig+9 ----
            const bool keep[4] = {2 * tig < nvalid, 2 * tig + 1 < nvalid, 2 * tig + 8 < nvalid, 2 * tig + 9 < nvalid};
#pragma unroll
            for (int pn = 0; pn < S::PANELS; ++pn) {
                constexpr int WORDS = S::PANB / 32;  // 32-bit words of a row and panel per lane
                uint32_t w[4][WORDS];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = 2 * tig + (j & 1) + 8 * (j >> 1);
                    if constexpr (WORDS == 4) {
                        const uint4 u = lds128(sV + S::at(tok, pn * 8 + gid));
                        w[j][0] = u.x;
                        w[j][1] = u.y;
                        w[j][2] = u.z;
                        w[j][3] = u.w;
                    } else {
                        const uint2 u = lds64(sV + S::at(tok, gid >> 1) + (gid & 1) * 8);
                        w[j][0] = u.x;
                        w[j][1] = u.y;
                    }
                }
                if (nvalid < kBlock) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < WORDS; ++x) w[j][x] = keep[j] ? w[j][x] : 0u;
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
                            M::mma(acc[(pn * WORDS + x) * 2 + h], af, b0f, b1f);
                        }
                    } else {
                        const uint32_t af[4] = {__byte_perm(w[0][x], w[1][x], 0x5410u), __byte_perm(w[0][x], w[1][x], 0x7632u),
                                                __byte_perm(w[2][x], w[3][x], 0x5410u), __byte_perm(w[2][x], w[3][x], 0x7632u)};
                        M::mma(acc[pn * WORDS + x], af, b0f, b1f);
                    }
                }
            }
        }
        __syncwarp();  // the V tile has been read by every lane
        if (lane == 0 && k + ST < nk) {
            fence_proxy_async_smem();
            issue(k + ST, 1, next);
        }
    }

    // ---- row sums over the 8 lanes sharing a row; the accumulator in units of 2^m_run ----
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
        l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], o);
        l_run[1] += __shfl_xor_sync(0xffffffffu, l_run[1], o);
    }
    float fo[2] = {1.f, 1.f};
    if constexpr (Q8) {
#pragma unroll
        for (int r = 0; r < 2; ++r) fo[r] = m_out[r] == -INFINITY ? 0.f : exp2f(m_out[r] - kWeightExp - m_run[r]);
    }

    // ---- merge the warps ----
    __syncthreads();
    float* s_acc = reinterpret_cast<float*>(smem);  // [NW][8][D]
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) {
        constexpr int WORDS = S::PANB / 32;
        constexpr int PER_PANEL = Q8 ? 2 * WORDS : WORDS;       // m-tiles per panel
        constexpr int PAN_D = S::PANB / (Q8 ? 1 : 2);           // dims per panel
        const int d0 = (mt / PER_PANEL) * PAN_D + gid * (2 * PER_PANEL) + 2 * (mt % PER_PANEL);
        const int r0 = 2 * tig;
        float* base = s_acc + (size_t)warp * 8 * D;
        if (r0 < G) *reinterpret_cast<float2*>(base + r0 * D + d0) = make_float2(acc[mt][0] * fo[0], acc[mt][2] * fo[0]);
        if (r0 + 1 < G)
            *reinterpret_cast<float2*>(base + (r0 + 1) * D + d0) = make_float2(acc[mt][1] * fo[1], acc[mt][3] * fo[1]);
    }
    if (gid == 0) {
        const int r0 = 2 * tig;
        s_ml[(warp * 8 + r0) * 2] = m_run[0];
        s_ml[(warp * 8 + r0) * 2 + 1] = l_run[0];
        s_ml[(warp * 8 + r0 + 1) * 2] = m_run[1];
        s_ml[(warp * 8 + r0 + 1) * 2 + 1] = l_run[1];
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * D; idx += NW * 32) {
        const int r = idx / D;
        const int d = idx % D;
        float Mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) Mx = fmaxf(Mx, s_ml[(w * 8 + r) * 2]);
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            // a warp without a finite maximum adds its sum times zero: nothing, or the NaN of its logits
            const float mw = s_ml[(w * 8 + r) * 2];
            const float sc = mw == -INFINITY ? 0.f : exp2f(mw - Mx);
            L = fmaf(s_ml[(w * 8 + r) * 2 + 1], sc, L);
            O = fmaf(s_acc[((size_t)w * 8 + r) * D + d], sc, O);
        }
        const size_t row = (size_t)s * a.n_q + (size_t)g * G + r;
        if (single) reinterpret_cast<T*>(a.out)[row * D + d] = from_float<T>(L == 0.f ? 0.f : O / L);
        if (!single || fa.z) {
            const size_t prow = row * a.n_parts + p;
            if (!single) a.part_o[prow * D + d] = O;
            if (d == 0) {
                a.part_ml[prow * 2] = Mx;
                a.part_ml[prow * 2 + 1] = L;
            }
        }
    }
    if (!single)
        frag_merge_if_last<T, D, G, NW * 32>(a, s, g, (nb + a.bpp - 1) / a.bpp,
                                             reinterpret_cast<float*>(smem + S::MERGE));
}

template <typename T, bool Q8, int D, int G>
struct FragKernel {
    static constexpr int NW = 4;
    // 64 KiB of tiles per CTA: 3 CTAs per SM
    static constexpr int ST = 64 * 1024 / (NW * 2 * kBlock * D * (Q8 ? 1 : 2));
    static constexpr size_t smem = FragGeom<Q8, D, NW, ST>::ALLOC;
    static unsigned long long attr_done;
    static cudaError_t prepare() { return allow_dynamic_smem(frag_decode_kernel<T, Q8, D, G, NW, ST>, smem, &attr_done); }
    static cudaError_t ctas_per_sm(int* out) {
        cudaError_t err = prepare();
        if (err != cudaSuccess) return err;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, frag_decode_kernel<T, Q8, D, G, NW, ST>, NW * 32, smem);
    }
    static cudaError_t launch(const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
        cudaError_t err = prepare();
        if (err != cudaSuccess) return err;
        frag_decode_kernel<T, Q8, D, G, NW, ST>
            <<<dim3(a.d.n_parts, a.d.n_kv, a.d.n_seqs), NW * 32, smem, stream>>>(a, tk, tv);
        return cudaGetLastError();
    }
};
template <typename T, bool Q8, int D, int G>
unsigned long long FragKernel<T, Q8, D, G>::attr_done = 0;

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

}  // namespace pkv
