// linear_chunk.cuh -- linear attention of long chunks on the tensor cores (tcgen05), fp16 and bf16 (sm_103a).
//
// With G_i the sum of the log decays up to token i of a piece of 128 tokens and S the state before the piece,
//   o_i = scale ( exp(G_i) q_i S + sum_{j<=i} exp(G_i - G_j) (q_i . k_j) v_j )
//   S'  = exp(G_128) S + sum_j exp(G_128 - G_j) k_j^T v_j
// so a piece is four matrix products: P = Q K^T, OI = Q S, OA = (P * D) V and U = K^T V~, V~ the rows of V
// weighted by exp(G_128 - G_j).
//
// A CTA takes one sequence, one head and 64 columns of v (the columns of S do not depend on one another; a head of
// 128 has two CTAs, which both compute P), and walks its pieces with the roles below working on different
// ones: the state is the only thing that passes from piece to piece.
//   warps 0-3    P: tensor memory -> weights -> P' (16 bits, the A operand of OA, in tensor memory). Row i against 32
//                columns of an earlier block of 32: exp(G_i - R) times exp(R - G_j), R the sum up to the block's end:
//                both at most 1 for decays, and one exponential a row and block; only the block on the diagonal takes
//                one for each pair
//   warps 4-7    V~, in quarters of 32 rows through a ring: split into numbers of the type that add up to it (two of
//                fp16, three of bf16: 2^-22 is left), beside one another along N, so that one product of N = 128 or 192
//                gives their sums and the state keeps fp32's precision
//   warps 8-11   the state: S in fp32 registers, a thread a row (of dim_k; at dim_k = 64 half a row, the product's 128
//                rows being K's 64 twice), decays it, adds U and hands the tensor cores a rounded copy
//   warps 12-15  results: exp(G_i) OI + OA, through shared memory to whole rows
//   warp 16      tensor copies of Q, K and V, two pieces ahead
//   warp 17      issues the products
//   warp 18      sums of decays (in 64 bits: differences of far sums; held as two fp32 where pairs need them)
//
// Rounded to 16 bits are P' and the copy of S that Q meets, each term of a result once, as attention weights are.
// fp16 cannot hold their range: rows of P', the copy of S and V~ are then brought to 2^14 by a power of two each, which
// the sums undo in fp32.
//
// A piece past the sequence's end: rows of K and V behind it are zeroed in shared memory (another sequence's rows, or
// nobody's, NaN perhaps). A non-finite v would reach earlier tokens of its piece through 0 x NaN: it is taken
// out of V (not of V~), and the results get NaN from its token on.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "decode_mma.cuh"
#include "linear.h"
#include "umma.cuh"

namespace pkv {

constexpr int kPiece = 128;   // tokens of a piece: the M of a product
constexpr int kSlice = 64;    // columns of v of a CTA
constexpr int kChunkThreads = 19 * 32;

// Pieces of a piece's 128 gates, as the roles need them.
struct __align__(16) PieceGates {
    float hi[kPiece], lo[kPiece];  // sum of the log decays from the start of token's block of 32 to it, base 2
    float col[kPiece];             // 2^(sum to the block's end - sum to the token)
    float block[4];                // sum over each block
    float after[4];                // 2^(sum over the blocks behind it)
    float keep;                    // 2^(sum over all)
    float keep_less1;              // that - 1, exact where the sum is small
    int small;                     // whether it is
    float grow;                    // sum of the positive ones
};

template <typename T, int DK>
struct ChunkSmem {
    static constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NT = BF ? 3 : 2;                  // numbers a value of V~ is split into
    static constexpr int NR = BF ? 3 : 4;                  // quarters of V~ in the ring
    static constexpr uint32_t PANEL = kPiece * 128;        // 64 columns of 128 rows
    static constexpr uint32_t QK = PANEL * (DK / 64);
    static constexpr uint32_t QUARTER = 32 * 128 * NT;     // [NT][32 rows][128 B]
    static constexpr uint32_t Q = 0;
    static constexpr uint32_t K = Q + 2 * QK;
    static constexpr uint32_t V = K + 2 * QK;
    static constexpr uint32_t VT = V + 2 * PANEL;
    static constexpr uint32_t S = VT + NR * QUARTER;       // [DK rows][128 B]
    static constexpr uint32_t O = S + DK * 128;            // [4 warps][32 rows][64 B]
    static constexpr uint32_t GATES = O + 4 * 2048;        // [2]
    static constexpr uint32_t BAD = GATES + 2 * sizeof(PieceGates);  // int [4][64]: first non-finite v of a column
    static constexpr uint32_t ROW = BAD + 4 * 64 * 4;      // fp16: float [2][128], 2^-e of P's rows
    static constexpr uint32_t MISC = ROW + (BF ? 0 : 2 * 128 * 4);  // any_bad[4] s_unit[2] u_unit[2] part[2][4]
    static constexpr uint32_t BARS = MISC + 64;
    static constexpr int NBARS = 2 + 2 + 2 + 2 + 2 + 2 * NR + 7 + 4;
    static constexpr uint32_t TADDR = BARS + NBARS * 8;
    static constexpr uint32_t TOTAL = TADDR + 16;
    static constexpr uint32_t ALLOC = TOTAL + 1024;
    static_assert(ALLOC <= 232448, "shared memory");
    static_assert((VT % 1024) == 0 && (S % 1024) == 0 && (QUARTER % 1024) == 0 && (BARS % 8) == 0, "alignment");
};

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e, e clamped to what a normal number holds
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// e with 2^(14 - e) bringing x into [2^14, 2^15); 14 (no change) for 0
__device__ __forceinline__ int exponent14(float x) {
    const int e = (int)((__float_as_uint(x) >> 23) & 255u) - 127;
    return x == 0.f ? 14 : min(max(e, -100), 120);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// STATES: the first pass over a sequence's segments but the last, which keeps only what they add to the state.
template <typename T, int DK, bool STATES>
__global__ void __launch_bounds__(kChunkThreads, 1)
    linear_chunk_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using L = ChunkSmem<T, DK>;
    using M = MmaType<T>;
    constexpr bool BF = L::BF;
    constexpr int NT = L::NT, NR = L::NR;
    constexpr uint32_t PANEL = L::PANEL;
    constexpr uint32_t P_COL = 0, PW_COL = 128, OI_COL = 192, OA_COL = 256, U_COL = 320;
    static_assert(U_COL + 64 * NT <= 512, "tensor memory");
    constexpr uint32_t IDESC_P = umma_idesc_f16(BF, 128, kPiece, false);
    constexpr uint32_t IDESC_O = umma_idesc_f16(BF, 128, kSlice, true);
    constexpr uint32_t IDESC_U = umma_idesc_f16(BF, 128, kSlice * NT, true) | (1u << 15);  // A = K^T: M-major
    constexpr uint32_t GATE_READERS = STATES ? 8 : 16;  // warps

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    PieceGates* gates = reinterpret_cast<PieceGates*>(smem + L::GATES);
    int* bad = reinterpret_cast<int*>(smem + L::BAD);
    float* row_unit = reinterpret_cast<float*>(smem + L::ROW);
    int* any_bad = reinterpret_cast<int*>(smem + L::MISC);
    float* s_unit = reinterpret_cast<float*>(smem + L::MISC + 16);
    float* u_unit = reinterpret_cast<float*>(smem + L::MISC + 24);
    float* part = reinterpret_cast<float*>(smem + L::MISC + 32);  // [2 roles][4 warps]
    uint64_t* qk_full = reinterpret_cast<uint64_t*>(smem + L::BARS);  // [2] Q and K of a piece have landed
    uint64_t* v_full = qk_full + 2;                                   // [2]
    uint64_t* done = v_full + 2;       // [2] every product of a piece is done: its buffers and results
    uint64_t* g_full = done + 2;       // [2] gates
    uint64_t* g_free = g_full + 2;     // [2]
    uint64_t* vt_full = g_free + 2;    // [NR] a quarter of V~ is written
    uint64_t* vt_free = vt_full + NR;  // [NR] and read
    uint64_t* u_full = vt_free + NR;   // U is done
    uint64_t* u_free = u_full + 1;     // and read
    uint64_t* s_full = u_free + 1;     // the copy of S is written
    uint64_t* s_free = s_full + 1;     // and read
    uint64_t* p_full = s_free + 1;     // P is done
    uint64_t* w_full = p_full + 1;     // P' is written (and P read)
    uint64_t* o_free = w_full + 1;     // OI and OA are read
    uint64_t* role = o_free + 1;       // [3] the four warps of a role meet
    uint64_t* all_done = role + 3;     // every product issued is done
    uint32_t* taddr_s = reinterpret_cast<uint32_t*>(smem + L::TADDR);

    const LinearArgs& l = a.l;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = blockIdx.x % a.slices;
    long long unit = blockIdx.x / a.slices;
    const int h = (int)(unit % l.n_v);
    unit /= l.n_v;
    const int segs = STATES ? a.n_segs - 1 : a.n_segs;
    const int seg = (int)(unit % segs), s = (int)(unit / segs);
    const int hq = h / (l.n_v / l.n_qk);
    const int q0 = l.q_start[s], q1 = l.q_start[s + 1];
    const int src = l.src[s], dst = l.dst[s];
    const bool bad_range = q0 < 0 || q1 < q0 || q1 > l.n_tokens || q1 - q0 > l.max_query;
    const bool bad_slot = src >= l.n_slots || dst >= l.n_slots;
    if (bad_range || bad_slot) {
        if (!STATES && h == 0 && slice == 0 && seg == 0 && threadIdx.x == 0)
            atomicOr(l.status, (bad_range ? (unsigned)PKV_DEV_BAD_QUERY_RANGE : 0u) |
                                   (bad_slot ? (unsigned)PKV_DEV_BAD_STATE_SLOT : 0u));
        return;
    }
    const int whole = q1 - q0;
    // a sequence that fits fewer segments leaves the others nothing; its last keeps the state
    const int used_segs = whole > 0 ? (whole + a.seg_tokens - 1) / a.seg_tokens : 1;
    if (seg >= (STATES ? used_segs - 1 : used_segs)) return;
    const int t0 = q0 + seg * a.seg_tokens;
    const int tokens = min(a.seg_tokens, q1 - t0);
    const int pieces = (tokens + kPiece - 1) / kPiece;
    const size_t head = (size_t)DK * a.dv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&done[i], 1);
            mbar_init(&g_full[i], 1);
            mbar_init(&g_free[i], GATE_READERS);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&vt_full[i], 4);
            mbar_init(&vt_free[i], 1);
        }
        mbar_init(u_full, 1);
        mbar_init(u_free, 4);
        mbar_init(s_full, 4);
        mbar_init(s_free, 1);
        mbar_init(p_full, 1);
        mbar_init(w_full, 4);
        mbar_init(o_free, 4);
        for (int i = 0; i < 3; ++i) mbar_init(&role[i], 4);
        mbar_init(all_done, 1);
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 4 * 64; i += kChunkThreads) bad[i] = kPiece;
    if (threadIdx.x < 4) any_bad[threadIdx.x] = 0;
    if (warp == 17) tmem_alloc_cg<1>(taddr_s, 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *taddr_s;
    // The n-th phase of a barrier, for one thread, or for a whole warp, which goes on or gives up together.
    auto wait1 = [](uint64_t* bar, int n) -> bool { return mbar_wait_bounded(bar, (uint32_t)n & 1u); };
    auto wait = [](uint64_t* bar, int n) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, (uint32_t)n & 1u));
    };
    auto arrive_warp = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    int met = 0;
    auto meet = [&](int id) -> bool {  // the four warps of a role
        arrive_warp(&role[id]);
        return wait(&role[id], met++);
    };
    bool ok = true;

    if (warp < 4) {
        // ===================== weights of the pairs inside a piece: thread = row =====================
        if constexpr (!STATES) {
            const int row = threadIdx.x;
            const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
            for (int c = 0; c < pieces; ++c) {
                const PieceGates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1) || !wait(p_full, c)) { ok = false; break; }
                tcgen05_after_sync();
                const float mine = g.hi[row], mine_lo = g.lo[row];
                float shift = 0.f;  // log2 of what the row is multiplied by
                if constexpr (!BF) {
                    float m0 = 0.f, m1 = 0.f;
#pragma unroll 1
                    for (int b = 0; b <= warp; ++b) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float p[16];
                            tmem_ld16(lanes + P_COL + b * 32 + half * 16, p);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const bool in0 = b < warp || half * 16 + j <= lane, in1 = b < warp || half * 16 + j + 1 <= lane;
                                m0 = fmaxf(m0, in0 ? fabsf(p[j]) : 0.f);
                                m1 = fmaxf(m1, in1 ? fabsf(p[j + 1]) : 0.f);
                            }
                        }
                    }
                    const int e = exponent14(fmaxf(m0, m1)) + (int)ceilf(fminf(g.grow, 200.f));
                    shift = (float)(14 - e);
                    row_unit[(c & 1) * kPiece + row] = ex2(-shift);
                }
                // P' of the piece before has been read
                if (c > 0 && !wait(&done[(c - 1) & 1], (c - 1) >> 1)) { ok = false; break; }
                tcgen05_after_sync();
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float from = shift + mine;  // to the row from the end of block b
                    for (int i = b + 1; i < warp; ++i) from += g.block[i];
                    const float f = ex2(from);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int j0 = b * 32 + half * 16;
                        uint32_t w[8];
                        if (b > warp) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = 0u;
                        } else {
                            float p[16], x[16];
                            tmem_ld16(lanes + P_COL + j0, p);
                            if (b < warp) {
#pragma unroll
                                for (int j = 0; j < 16; j += 4) {
                                    const float4 y = *reinterpret_cast<const float4*>(&g.col[j0 + j]);
                                    x[j] = y.x * f, x[j + 1] = y.y * f, x[j + 2] = y.z * f, x[j + 3] = y.w * f;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; j += 4) {
                                    const float4 y = *reinterpret_cast<const float4*>(&g.hi[j0 + j]);
                                    const float4 z = *reinterpret_cast<const float4*>(&g.lo[j0 + j]);
                                    x[j] = ex2((mine - y.x) + (mine_lo - z.x) + shift);
                                    x[j + 1] = ex2((mine - y.y) + (mine_lo - z.y) + shift);
                                    x[j + 2] = ex2((mine - y.z) + (mine_lo - z.z) + shift);
                                    x[j + 3] = ex2((mine - y.w) + (mine_lo - z.w) + shift);
                                }
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                x[j] *= p[j];
                                if (b == warp && half * 16 + j > lane) x[j] = 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = M::pack(x[2 * j], x[2 * j + 1]);
                        }
                        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                                         lanes + PW_COL + j0 / 2),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                     : "memory");
                    }
                }
                tmem_wait_st();
                tcgen05_before_sync();
                arrive_warp(w_full);
                arrive_warp(&g_free[c & 1]);
            }
        }
    } else if (warp < 8) {
        // ===================== V~: 32 rows at a time, four threads a row =====================
        const int tid = threadIdx.x - 128;
        const int r = tid >> 2;
        // which four 16-byte units of its row: two threads' rows share the banks of half a row otherwise
        const int u0 = (tid & 3) + 4 * (r & 1), u1 = u0 ^ 4;
        for (int c = 0; c < pieces; ++c) {
            const int st = c & 1;
            const int n = min(kPiece, tokens - c * kPiece);
            unsigned char* v = smem + L::V + st * PANEL;
            const PieceGates& g = gates[st];
            if (!wait(&g_full[st], c >> 1) || !wait(&v_full[st], c >> 1)) { ok = false; break; }
            if (n < kPiece) {  // rows behind the sequence's end
                if (!wait(&qk_full[st], c >> 1)) { ok = false; break; }
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int i = n * 8 + tid; i < kPiece * 8; i += 128) {
                    *reinterpret_cast<uint4*>(v + i * 16) = zero;
#pragma unroll
                    for (int p = 0; p < DK / 64; ++p)
                        *reinterpret_cast<uint4*>(smem + L::K + st * L::QK + p * PANEL + i * 16) = zero;
                }
                fence_proxy_async_smem();
                if (!meet(0)) { ok = false; break; }
            }
            float unit = 1.f;
            if constexpr (!BF) {  // the largest of V~, to bring it to 2^14
                float most = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float f = g.col[q * 32 + r] * g.after[q];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 x = *reinterpret_cast<const uint4*>(v + (q * 32 + r) * 128 + (((k ? u1 : u0) ^ (r & 7)) << 4));
                        float y[8];
                        Vec16<T>::to_float(x, y);
#pragma unroll
                        for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(y[j]) <= 65504.f ? fabsf(y[j] * f) : 0.f);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (lane == 0) part[warp - 4] = most;
                if (!meet(0)) { ok = false; break; }
                const int e = exponent14(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
                unit = pow2i(14 - e);
                // (read for the piece before the last one: that piece's gates have been released by the state's warps)
                if (tid == 0) u_unit[st] = pow2i(e - 14);
                if (!meet(0)) { ok = false; break; }  // part may be written again
            }
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const int p = c * 4 + q, slot = p % NR;
                const int row = q * 32 + r;
                uint4 x[2];
                unsigned char* from[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    from[k] = v + row * 128 + (((k ? u1 : u0) ^ (r & 7)) << 4);
                    x[k] = *reinterpret_cast<const uint4*>(from[k]);
                }
                const float f = g.col[row] * g.after[q] * unit;
                if (p >= NR && !wait(&vt_free[slot], p / NR - 1)) { ok = false; break; }
                unsigned char* to = smem + L::VT + slot * L::QUARTER + r * 128;
                bool non_finite = false;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[8], probe = 0.f;
                    Vec16<T>::to_float(x[k], y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) probe = fmaf(y[j], 0.f, probe);
                    non_finite |= !(probe == 0.f);
                    const uint32_t at = (((k ? u1 : u0) ^ (r & 7)) << 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = row < n ? y[j] * f : 0.f;
#pragma unroll
                    for (int term = 0; term < NT; ++term) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            w[j] = M::pack(y[2 * j], y[2 * j + 1]);
                            if (term + 1 < NT) {
                                const float2 z = M::unpack(w[j]);
                                y[2 * j] -= z.x;
                                y[2 * j + 1] -= z.y;
                            }
                        }
                        *reinterpret_cast<uint4*>(to + term * 4096 + at) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (!STATES && non_finite) {  // out of V, and noted for the results
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float y[8];
                        Vec16<T>::to_float(x[k], y);
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!(fabsf(y[j]) <= 3.4028234e38f)) {
                                y[j] = 0.f;
                                atomicMin(&bad[(c & 3) * 64 + (k ? u1 : u0) * 8 + j], row);
                                any_bad[c & 3] = 1;
                            }
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = M::pack(y[2 * j], y[2 * j + 1]);
                        *reinterpret_cast<uint4*>(from[k]) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                fence_proxy_async_smem();
                arrive_warp(&vt_full[slot]);
            }
            if (!ok) break;
            arrive_warp(&g_free[st]);
        }
    } else if (warp < 12) {
        // ===================== the state: thread = row of dim_k (half a row at dim_k = 64) =====================
        constexpr int NC = DK == 128 ? 64 : 32;
        const int tid = threadIdx.x - 256;
        const int row = tid & (DK - 1);
        const int c0 = DK == 128 ? 0 : (tid >> 6) * 32;
        const uint32_t lanes = tmem + ((uint32_t)((warp - 8) * 32) << 16);
        const size_t at = (size_t)row * a.dv + slice * kSlice + c0;  // in a head's state
        float x[NC];
        auto load = [&](const float* from, bool add, float keep) {
#pragma unroll
            for (int i = 0; i < NC; i += 4) {
                const float4 y = *reinterpret_cast<const float4*>(from + at + i);
                x[i] = add ? fmaf(x[i], keep, y.x) : y.x;
                x[i + 1] = add ? fmaf(x[i + 1], keep, y.y) : y.y;
                x[i + 2] = add ? fmaf(x[i + 2], keep, y.z) : y.z;
                x[i + 3] = add ? fmaf(x[i + 3], keep, y.w) : y.w;
            }
        };
        auto save = [&](float* to) {
#pragma unroll
            for (int i = 0; i < NC; i += 4)
                *reinterpret_cast<float4*>(to + at + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        };
#pragma unroll
        for (int i = 0; i < NC; ++i) x[i] = 0.f;
        if (seg == 0) {
            // shared out, the second pass reads the start from where the first left it: its last segment writes dst
            if (!STATES && used_segs > 1)
                load(a.start + ((size_t)s * l.n_v + h) * head, false, 0.f);
            else if (src >= 0)
                load(l.state + ((size_t)src * l.n_v + h) * head, false, 0.f);
            if (STATES) save(a.start + ((size_t)s * l.n_v + h) * head);
        } else if (!STATES) {
            for (int i = 0; i < seg; ++i) {
                const size_t to = ((size_t)s * (a.n_segs - 1) + i) * l.n_v + h;
                load(a.added + to * head, i > 0, i > 0 ? exp2f(a.sums[to]) : 0.f);
            }
        }
        for (int c = 0; c < pieces; ++c) {
            if constexpr (!STATES) {  // the copy that Q meets
                float unit = 1.f, back_s = 1.f;
                if constexpr (!BF) {
                    float most = 0.f;
#pragma unroll
                    for (int i = 0; i < NC; ++i) most = fmaxf(most, fabsf(x[i]));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    if (lane == 0) part[4 + warp - 8] = most;
                    if (!meet(1)) { ok = false; break; }
                    const int e = exponent14(fmaxf(fmaxf(part[4], part[5]), fmaxf(part[6], part[7])));
                    unit = pow2i(14 - e);
                    back_s = pow2i(e - 14);
                    if (!meet(1)) { ok = false; break; }  // part may be written again
                }
                if (c > 0 && !wait(s_free, c - 1)) { ok = false; break; }
                // (Q S of the piece before is done: it began when the results of the one before that had been read)
                if (!BF && tid == 0) s_unit[c & 1] = back_s;
                unsigned char* to = smem + L::S + row * 128;
#pragma unroll
                for (int i = 0; i < NC; i += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = M::pack(x[i + 2 * j] * unit, x[i + 2 * j + 1] * unit);
                    *reinterpret_cast<uint4*>(to + ((((c0 + i) >> 3) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                arrive_warp(s_full);
            }
            const PieceGates& g = gates[c & 1];
            if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
            const float keep = g.keep, less1 = g.keep_less1;
            const bool small = g.small != 0;
            if (!wait(u_full, c)) { ok = false; break; }
            tcgen05_after_sync();
            const float back = BF ? 1.f : u_unit[c & 1];
#pragma unroll
            for (int i = 0; i < NC; i += 16) {
                float u[16];
                tmem_ld16(lanes + U_COL + c0 + i, u);
                tmem_wait_ld();
                if (!BF) {
                    float y[16];
                    tmem_ld16(lanes + U_COL + 64 + c0 + i, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) u[j] = (u[j] + y[j]) * back;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    x[i + j] = small ? fmaf(x[i + j], less1, x[i + j] + u[j]) : fmaf(x[i + j], keep, u[j]);
                if (BF) {
#pragma unroll
                    for (int term = 1; term < NT; ++term) {
                        tmem_ld16(lanes + U_COL + 64 * term + c0 + i, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[i + j] += u[j];
                    }
                }
            }
            tcgen05_before_sync();
            arrive_warp(u_free);
            arrive_warp(&g_free[c & 1]);
        }
        if (ok) {
            if (STATES)
                save(a.added + (((size_t)s * (a.n_segs - 1) + seg) * l.n_v + h) * head);
            else if (seg == used_segs - 1 && dst >= 0)
                save(l.state + ((size_t)dst * l.n_v + h) * head);
        }
    } else if (warp < 16) {
        // ===================== results: thread = row =====================
        if constexpr (!STATES) {
            const int w4 = warp - 12;
            const int row = w4 * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
            unsigned char* stage = smem + L::O + w4 * 2048;
            for (int c = 0; c < pieces; ++c) {
                const int n = min(kPiece, tokens - c * kPiece);
                const PieceGates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                float sum = g.hi[row];
                for (int i = 0; i < w4; ++i) sum += g.block[i];
                arrive_warp(&g_free[c & 1]);
                float fi = ex2(sum) * l.scale, fa = l.scale;
                if (!wait(&done[c & 1], c >> 1)) { ok = false; break; }
                tcgen05_after_sync();
                if constexpr (!BF) {
                    fi *= s_unit[c & 1];
                    fa *= row_unit[(c & 1) * kPiece + row];
                }
                const bool poisoned = any_bad[c & 3] != 0;
#pragma unroll
                for (int c0 = 0; c0 < kSlice; c0 += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int half = 0; half < 32; half += 16) {
                        float x[16], y[16];
                        tmem_ld16(lanes + OI_COL + c0 + half, x);
                        tmem_ld16(lanes + OA_COL + c0 + half, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = fmaf(x[j], fi, y[j] * fa);
                        if (poisoned) {
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (bad[(c & 3) * 64 + c0 + half + j] <= row) x[j] = __int_as_float(0x7fffffff);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[half / 2 + j] = M::pack(x[2 * j], x[2 * j + 1]);
                    }
                    if (c0 + 32 == kSlice) {
                        tcgen05_before_sync();
                        arrive_warp(o_free);
                    }
                    // 64 bytes of each of the warp's 32 rows: unit u of row r at u ^ (r / 2 & 3), so that eight
                    // rows' units lie in different banks
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int rr = k * 8 + (lane >> 2), u = lane & 3, in = w4 * 32 + rr;
                        if (in < n) {
                            const uint4 y = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((u ^ ((rr >> 1) & 3)) << 4));
                            T* out = static_cast<T*>(l.out) + ((size_t)(t0 + c * kPiece + in) * l.n_v + h) * a.dv +
                                     slice * kSlice + c0 + u * 8;
                            *reinterpret_cast<uint4*>(out) = y;
                        }
                    }
                    __syncwarp();
                }
                if (poisoned) {  // the columns' marks are used again four pieces on
                    if (!meet(2)) { ok = false; break; }
                    if (row < 64) bad[(c & 3) * 64 + row] = kPiece;
                    if (row == 0) any_bad[c & 3] = 0;
                }
            }
        }
    } else if (warp == 16) {
        // ===================== tensor copies =====================
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < pieces; ++c) {
                const int st = c & 1;
                if (c >= 2 && !wait1(&done[st], (c >> 1) - 1)) { ok = false; break; }
                const int y = t0 + c * kPiece;
                mbar_arrive_expect_tx(&qk_full[st], (STATES ? 1 : 2) * L::QK);
#pragma unroll
                for (int p = 0; p < DK / 64; ++p) {
                    if (!STATES) tma_rows(sbase + L::Q + st * L::QK + p * PANEL, &tm_q, hq * DK + p * 64, y, &qk_full[st]);
                    tma_rows(sbase + L::K + st * L::QK + p * PANEL, &tm_k, hq * DK + p * 64, y, &qk_full[st]);
                }
                mbar_arrive_expect_tx(&v_full[st], PANEL);
                tma_rows(sbase + L::V + st * PANEL, &tm_v, h * a.dv + slice * kSlice, y, &v_full[st]);
                issued = c + 1;
            }
            // no copy is in flight when the CTA leaves
            for (int c = max(issued - 2, 0); c < issued; ++c) {
                ok = wait1(&qk_full[c & 1], c >> 1) && ok;
                ok = wait1(&v_full[c & 1], c >> 1) && ok;
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ===================== products =====================
        if (lane == 0) {
            const uint64_t dq = umma_desc_sw128(sbase + L::Q, 16, 1024);
            const uint64_t dk = umma_desc_sw128(sbase + L::K, 16, 1024);
            // K^T: 64 rows of the product a panel; at dim_k = 64 the second 64 are the first again
            const uint64_t dkt = umma_desc_sw128(sbase + L::K, DK == 128 ? PANEL : 0, 1024);
            const uint64_t dv = umma_desc_sw128(sbase + L::V, PANEL, 1024);
            const uint64_t ds = umma_desc_sw128(sbase + L::S, DK * 128, 1024);
            const uint64_t dvt = umma_desc_sw128(sbase + L::VT, 4096, 1024);
            auto pairs = [&](int c) {  // P = Q K^T
                const uint32_t st = (uint32_t)(c & 1) * L::QK;
                tcgen05_after_sync();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t off = (st + (uint32_t)(k >> 2) * PANEL + (uint32_t)(k & 3) * 32) >> 4;
                    umma_f16_cg<1>(tmem + P_COL, dq + off, dk + off, IDESC_P, k > 0);
                }
                umma_commit_cg<1>(p_full);
            };
            if (!STATES && pieces > 0) {
                ok = wait1(&qk_full[0], 0);
                if (ok) pairs(0);
            }
            for (int c = 0; c < pieces && ok; ++c) {
                const uint32_t st = (uint32_t)(c & 1);
                // U = K^T V~
                if (!wait1(&qk_full[st], c >> 1) || (c > 0 && !wait1(u_free, c - 1))) { ok = false; break; }
                for (int q = 0; q < 4; ++q) {
                    const int p = c * 4 + q, slot = p % NR;
                    if (!wait1(&vt_full[slot], p / NR)) { ok = false; break; }
                    tcgen05_after_sync();
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        umma_f16_cg<1>(tmem + U_COL, dkt + (uint64_t)((st * L::QK + (uint32_t)(q * 2 + k) * 2048) >> 4),
                                       dvt + (uint64_t)(((uint32_t)slot * L::QUARTER + (uint32_t)k * 2048) >> 4), IDESC_U,
                                       q > 0 || k > 0);
                    umma_commit_cg<1>(&vt_free[slot]);
                }
                if (!ok) break;
                umma_commit_cg<1>(u_full);
                if constexpr (STATES) {
                    umma_commit_cg<1>(&done[st]);
                } else {
                    // OI = Q S
                    if (!wait1(s_full, c) || (c > 0 && !wait1(o_free, c - 1))) { ok = false; break; }
                    tcgen05_after_sync();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        umma_f16_cg<1>(tmem + OI_COL,
                                       dq + (uint64_t)((st * L::QK + (uint32_t)(k >> 2) * PANEL + (uint32_t)(k & 3) * 32) >> 4),
                                       ds + (uint64_t)(((uint32_t)k * 2048) >> 4), IDESC_O, k > 0);
                    umma_commit_cg<1>(s_free);
                    if (!wait1(w_full, c)) { ok = false; break; }
                    if (c + 1 < pieces) {
                        if (!wait1(&qk_full[st ^ 1], (c + 1) >> 1)) { ok = false; break; }
                        pairs(c + 1);
                    }
                    // OA = P' V
                    if (!wait1(&v_full[st], c >> 1)) { ok = false; break; }
                    tcgen05_after_sync();
#pragma unroll
                    for (int k = 0; k < kPiece / 16; ++k)
                        umma_f16_tmem_a_cg<1>(tmem + OA_COL, tmem + PW_COL + k * 8,
                                              dv + (uint64_t)((st * PANEL + (uint32_t)k * 2048) >> 4), IDESC_O, k > 0);
                    umma_commit_cg<1>(&done[st]);
                }
            }
            // every product is done before tensor memory is given back
            umma_commit_cg<1>(all_done);
            ok = wait1(all_done, 0) && ok;
        }
        __syncwarp();
    } else if (warp == 18) {
        // ===================== sums of the log decays: lane = 4 tokens =====================
        float raw[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = c * kPiece + lane * 4 + i;
                raw[i] = l.log_decay && t < tokens ? l.log_decay[(size_t)(t0 + t) * l.decay_stride + h] : 0.f;
            }
        };
        if (pieces > 0) fetch(0);
        double total = 0.0;
        for (int c = 0; c < pieces; ++c) {
            double x[4], grow = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // 2^-150 is 0 in fp32: a token that forgets (-infinity) then takes part in sums
                const float y = raw[i] < -104.f ? -104.f : raw[i];
                x[i] = (double)y * 1.4426950408889634;
                if (x[i] > 0.0) grow += x[i];
            }
            if (c + 1 < pieces) fetch(c + 1);
#pragma unroll
            for (int i = 1; i < 4; ++i) x[i] += x[i - 1];
            double before = x[3];  // over the lanes of a block of 32 tokens (eight)
#pragma unroll
            for (int o = 1; o < 8; o *= 2) {
                const double y = __shfl_up_sync(0xffffffffu, before, o);
                if ((lane & 7) >= o) before += y;
            }
            const double block = __shfl_sync(0xffffffffu, before, lane | 7);
            before -= x[3];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) grow += __shfl_xor_sync(0xffffffffu, grow, o);
            double blocks[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) blocks[b] = __shfl_sync(0xffffffffu, block, b * 8);
            if (c >= 2 && !wait(&g_free[c & 1], (c >> 1) - 1)) { ok = false; break; }
            PieceGates& g = gates[c & 1];
            float hi[4], lo[4], col[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const double y = before + x[i];
                hi[i] = (float)y;
                lo[i] = (float)(y - (double)hi[i]);
                col[i] = exp2f((float)(block - y));
            }
            *reinterpret_cast<float4*>(&g.hi[lane * 4]) = make_float4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<float4*>(&g.lo[lane * 4]) = make_float4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<float4*>(&g.col[lane * 4]) = make_float4(col[0], col[1], col[2], col[3]);
            const double all = (blocks[0] + blocks[1]) + (blocks[2] + blocks[3]);
            total += all;
            if (lane == 0) {
                double behind = 0.0;
#pragma unroll
                for (int b = 3; b >= 0; --b) {
                    g.block[b] = (float)blocks[b];
                    g.after[b] = exp2f((float)behind);
                    behind += blocks[b];
                }
                g.keep = exp2f((float)all);
                g.keep_less1 = expm1f((float)(all * 0.6931471805599453));
                g.small = all > -0.7 && all < 0.7;
                g.grow = (float)grow;
            }
            arrive_warp(&g_full[c & 1]);
        }
        if (STATES && ok && lane == 0 && slice == 0) a.sums[((size_t)s * (a.n_segs - 1) + seg) * l.n_v + h] = (float)total;
    }
    if (!ok && lane == 0) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 17) tmem_dealloc_cg<1>(tmem, 512);
}

template <typename T, int DK, bool STATES>
cudaError_t run_chunk(const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      cudaStream_t stream) {
    static unsigned long long attr_done = 0;  // one bit a device
    constexpr uint32_t smem = ChunkSmem<T, DK>::ALLOC;
    auto kern = linear_chunk_kernel<T, DK, STATES>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (!(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        __atomic_fetch_or(&attr_done, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    const unsigned segs = STATES ? a.n_segs - 1 : a.n_segs;
    kern<<<(unsigned)a.l.n_seqs * segs * a.l.n_v * a.slices, kChunkThreads, smem, stream>>>(a, q, k, v);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_linear_chunk_dtype(int dk, const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                      const CUtensorMap& v, cudaStream_t stream) {
    if (a.n_segs > 1) {
        const cudaError_t err = dk == 64 ? run_chunk<T, 64, true>(a, q, k, v, stream) : run_chunk<T, 128, true>(a, q, k, v, stream);
        if (err != cudaSuccess) return err;
    }
    return dk == 64 ? run_chunk<T, 64, false>(a, q, k, v, stream) : run_chunk<T, 128, false>(a, q, k, v, stream);
}

}  // namespace pkv
