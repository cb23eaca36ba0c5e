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
//   warps 0-7    P: tensor memory -> weights -> P' (16 bits, the A operand of OA, in tensor memory). Row i against
//                columns of an earlier block of 32: exp(G_i - R) times exp(R - G_j), R the sum up to the block's end:
//                both at most 1 for decays, and one exponential a row and block; only the block on the diagonal takes
//                one for each pair. A thread takes a row's even or odd halves of 32 columns
//   warps 8-15   V~, in quarters of 32 rows through a ring, four warps on every other one: split into numbers of the type that add up to it (two of
//                fp16: 2^-22 is left; three of bf16: exact), beside one another along N, so that one product of N = 128
//                or 192 gives their sums and the state keeps fp32's precision
//   warps 16-19  the state: S in fp32 registers, a thread a row (of dim_k; at dim_k = 64 half a row, the product's 128
//                rows being K's 64 twice), decays it, adds U and hands the tensor cores a rounded copy
//   warps 20-23  results: exp(G_i) OI + OA, through shared memory to whole rows
//   warp 24      tensor copies of Q, K and V, two pieces ahead
//   warp 25      issues the products
//   warps 26, 27 sums of decays (in 64 bits: differences of far sums; held as two fp32 where pairs need them)
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
#include "linear.h"
#include "umma.cuh"

namespace pkv {

constexpr int kPiece = 128;   // tokens of a piece: the M of a product
constexpr int kSlice = 64;    // columns of v of a CTA
constexpr int kChunkThreads = 7 * 128;

// Pairs of 16-bit numbers in a word.
template <typename T>
struct Pair16;
template <>
struct Pair16<__half> {
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
    __device__ __forceinline__ static uint32_t zero_times(uint32_t w, uint32_t sum) {
        const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.f), *reinterpret_cast<const __half2*>(&sum));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Pair16<__nv_bfloat16> {
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ static float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t zero_times(uint32_t w, uint32_t sum) {
        const __nv_bfloat162 h = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.f),
                                         *reinterpret_cast<const __nv_bfloat162*>(&sum));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// Pieces of a piece's 128 gates, as the roles need them.
struct __align__(16) PieceGates {
    float hi[kPiece], lo[kPiece];  // minus the sum of the log decays from the start of token's block of 32 to it, base 2
    float col[kPiece];             // 2^(sum to the block's end - sum to the token)
    float block[4];                // sum over each block
    float after[4];                // 2^(sum over the blocks behind it)
    float keep, once;              // S' = S + (U + S * keep) with 2^(sum over all) - 1 where that is small, once = 1,
    float grow;                    // else S * keep + U, once = 0; sum of the positive ones
    float sum;                     // over all
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
    static constexpr uint32_t MISC = ROW + (BF ? 0 : 2 * 128 * 4);  // any_bad[4] s_unit[2] u_unit[2] part[8 + 4]
    static constexpr uint32_t BARS = MISC + 96;
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

// Every thread of the four warps: registers a thread from here on. The kernel's 72 a thread are shared out anew, as
// 64 + 64 + 64 + 64 + 136 + 64 + 48 = 7 * 72.
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}

__device__ __forceinline__ float2 f2_get(uint64_t v) {
    float2 r;
    f2_unpack(v, r.x, r.y);
    return r;
}

// mbar_wait_bounded in few instructions: the roles' loops compete for the instruction caches.
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity) {
    uint64_t begin = 0;
    while (!mbar_try_wait(bar, parity)) {
        const uint64_t now = global_timer_ns();
        if (begin == 0) begin = now;
        if (now - begin > kWaitLimitNs) return false;
    }
    return true;
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
    using M = Pair16<T>;
    constexpr bool BF = L::BF;
    constexpr int NT = L::NT, NR = L::NR;
    constexpr uint32_t PANEL = L::PANEL;
    constexpr uint32_t P_COL = 0, PW_COL = 128, OI_COL = 192, OA_COL = 256, U_COL = 320;
    static_assert(U_COL + 64 * NT <= 512, "tensor memory");
    constexpr uint32_t IDESC_P = umma_idesc_f16(BF, 128, kPiece, false);
    constexpr uint32_t IDESC_O = umma_idesc_f16(BF, 128, kSlice, true);
    constexpr uint32_t IDESC_U = umma_idesc_f16(BF, 128, kSlice * NT, true) | (1u << 15);  // A = K^T: M-major
    constexpr uint32_t GATE_READERS = STATES ? 12 : 24;  // warps

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
    float* part = reinterpret_cast<float*>(smem + L::MISC + 32);  // of V~'s warps, then the state's
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
    uint64_t* role = o_free + 1;       // [3] the warps of a role meet
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
        mbar_init(w_full, 8);
        mbar_init(o_free, 4);
        for (int i = 0; i < 3; ++i) mbar_init(&role[i], i == 0 ? 8 : 4);
        mbar_init(all_done, 1);
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 4 * 64; i += kChunkThreads) bad[i] = kPiece;
    if (threadIdx.x < 4) any_bad[threadIdx.x] = 0;
    if (warp == 25) tmem_alloc_cg<1>(taddr_s, 512);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *taddr_s;
    // The n-th phase of a barrier, for one thread, or for a whole warp, which goes on or gives up together.
    auto wait1 = [](uint64_t* bar, int n) -> bool { return wait_short(bar, (uint32_t)n & 1u); };
    auto wait = [](uint64_t* bar, int n) -> bool { return __all_sync(0xffffffffu, wait_short(bar, (uint32_t)n & 1u)); };
    auto arrive_warp = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    int met = 0;
    auto meet = [&](int id) -> bool {  // the warps of a role
        arrive_warp(&role[id]);
        return wait(&role[id], met++);
    };
    bool ok = true;

    if (warp < 8) {
        // ===================== weights of the pairs inside a piece: thread = row, half of its columns =====================
        registers_down<64>();
        if constexpr (!STATES) {
            const int w4 = warp & 3, side = (warp >> 2) * 16;
            const int row = w4 * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
            const uint32_t from_col = lanes + P_COL + side, to_col = lanes + PW_COL + side / 2;
            uint32_t seen[8];  // of the block on the diagonal: the pairs of columns up to the row
#pragma unroll
            for (int j = 0; j < 8; ++j)
                seen[j] = (lane >= side + 2 * j ? 0xffffu : 0u) | (lane > side + 2 * j ? 0xffff0000u : 0u);
            auto put = [&](int b, const uint32_t (&w)[8]) {
                asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(to_col + b * 16),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                             : "memory");
            };
            {  // the blocks behind the row's own stay 0
                const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                for (int b = w4 + 1; b < 4; ++b) put(b, zero);
            }
            for (int c = 0; c < pieces; ++c) {
                const PieceGates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                const float mine = -g.hi[row];
                float mine_lo = -g.lo[row];
                if (!wait(p_full, c)) { ok = false; break; }
                tcgen05_after_sync();
                float shift = 0.f;  // log2 of what the row is multiplied by
                if constexpr (!BF) {
                    float m0 = 0.f, m1 = 0.f;
#pragma unroll 1
                    for (int h16 = 0; h16 < 2 * w4 + 2; ++h16) {
                        float p[16];
                        tmem_ld16(lanes + P_COL + h16 * 16, p);
                        tmem_wait_ld();
                        if (h16 < 2 * w4) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) m0 = fmaxf(m0, fabsf(p[j])), m1 = fmaxf(m1, fabsf(p[j + 1]));
                        } else {
                            const int last = lane - (h16 & 1) * 16;
#pragma unroll
                            for (int j = 0; j < 16; ++j) m0 = fmaxf(m0, j <= last ? fabsf(p[j]) : 0.f);
                        }
                    }
                    const int e = exponent14(fmaxf(m0, m1)) + (int)ceilf(fminf(g.grow, 200.f));
                    shift = (float)(14 - e);
                    if (side == 0) row_unit[(c & 1) * kPiece + row] = ex2_approx(-shift);
                    mine_lo += shift;
                }
                uint32_t p[16], w[8];
                float* pf = reinterpret_cast<float*>(p);
                tmem_ld16(from_col + w4 * 32, *reinterpret_cast<float(*)[16]>(pf));
                // P' of the piece before has been read
                if (c > 0 && !wait(&done[(c - 1) & 1], (c - 1) >> 1)) { ok = false; break; }
                tcgen05_after_sync();
                {  // the block on the diagonal: an exponential for each pair
                    const uint64_t hi2 = f2_pack(mine, mine), lo2 = f2_pack(mine_lo, mine_lo);
                    const ulonglong2* gh = reinterpret_cast<const ulonglong2*>(&g.hi[w4 * 32 + side]);
                    const ulonglong2* gl = reinterpret_cast<const ulonglong2*>(&g.lo[w4 * 32 + side]);
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 y = gh[j], z = gl[j];
                        const float2 d0 = f2_get(f2_add(f2_add(hi2, y.x), f2_add(lo2, z.x)));
                        const float2 d1 = f2_get(f2_add(f2_add(hi2, y.y), f2_add(lo2, z.y)));
                        x[4 * j] = ex2_approx(d0.x), x[4 * j + 1] = ex2_approx(d0.y);
                        x[4 * j + 2] = ex2_approx(d1.x), x[4 * j + 3] = ex2_approx(d1.y);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 y = f2_get(f2_mul(f2_pack(x[2 * j], x[2 * j + 1]), f2_pack(pf[2 * j], pf[2 * j + 1])));
                        w[j] = M::pack(y.x, y.y) & seen[j];
                    }
                }
                float from = mine + shift;  // the sum from the end of block b to the row
#pragma unroll 1
                for (int b = w4 - 1; b >= 0; --b) {
                    tmem_ld16(from_col + b * 32, *reinterpret_cast<float(*)[16]>(pf));
                    put(b + 1, w);
                    const float f = ex2_approx(from);
                    from += g.block[b];
                    const uint64_t f2 = f2_pack(f, f);
                    const ulonglong2* gc = reinterpret_cast<const ulonglong2*>(&g.col[b * 32 + side]);
                    uint64_t x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 y = gc[j];
                        x[2 * j] = f2_mul(y.x, f2), x[2 * j + 1] = f2_mul(y.y, f2);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 y = f2_get(f2_mul(x[j], f2_pack(pf[2 * j], pf[2 * j + 1])));
                        w[j] = M::pack(y.x, y.y);
                    }
                }
                put(0, w);
                tmem_wait_st();
                tcgen05_before_sync();
                arrive_warp(w_full);
                if (lane == 0) mbar_arrive(&g_free[c & 1]);
            }
        }
    } else if (warp < 16) {
        // ===================== V~: 32 rows at a time, four threads a row =====================
        registers_down<64>();
        const int tid = threadIdx.x - 256;
        const int half = tid >> 7;  // quarters 0 and 2, or 1 and 3
        const int r = (tid & 127) >> 2;
        // which four 16-byte units of its row: two threads' rows share the banks of half a row otherwise
        const int u0 = (tid & 3) + 4 * (r & 1);
        const uint32_t at[2] = {(uint32_t)((u0 ^ (r & 7)) << 4), (uint32_t)((u0 ^ 4 ^ (r & 7)) << 4)};
        for (int c = 0; c < pieces; ++c) {
            const int st = c & 1;
            const int n = min(kPiece, tokens - c * kPiece);
            unsigned char* v = smem + L::V + st * PANEL;
            const PieceGates& g = gates[st];
            if (!wait(&g_full[st], c >> 1) || !wait(&v_full[st], c >> 1)) { ok = false; break; }
            if (n < kPiece) {  // rows behind the sequence's end
                if (!wait(&qk_full[st], c >> 1)) { ok = false; break; }
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int i = n * 8 + tid; i < kPiece * 8; i += 256) {
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
#pragma unroll 1
                for (int q = half; q < 4; q += 2) {
                    __half2 m = __float2half2_rn(0.f);
                    uint4 x[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        x[k] = *reinterpret_cast<const uint4*>(v + (q * 32 + r) * 128 + at[k]);
                        const __half2* y = reinterpret_cast<const __half2*>(&x[k]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) m = __hmax2(m, __habs2(y[j]));
                    }
                    float top = fmaxf(__low2float(m), __high2float(m));
                    if (top > 65504.f) {  // an infinity: the largest of the others
                        top = 0.f;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float y[8];
                            Vec16<T>::to_float(x[k], y);
#pragma unroll
                            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(y[j]) <= 65504.f ? fabsf(y[j]) : 0.f);
                        }
                    }
                    most = fmaxf(most, top * (g.col[q * 32 + r] * g.after[q]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (lane == 0) part[warp - 8] = most;
                if (!meet(0)) { ok = false; break; }
                const float4 p0 = *reinterpret_cast<const float4*>(part), p1 = *reinterpret_cast<const float4*>(part + 4);
                const int e = exponent14(fmaxf(fmaxf(fmaxf(p0.x, p0.y), fmaxf(p0.z, p0.w)), fmaxf(fmaxf(p1.x, p1.y), fmaxf(p1.z, p1.w))));
                unit = pow2i(14 - e);
                // (read for the piece before the last one: that piece's gates have been released by the state's warps)
                if (tid == 0) u_unit[st] = pow2i(e - 14);
                if (!meet(0)) { ok = false; break; }  // part may be written again
            }
#pragma unroll 1
            for (int q = half; q < 4; q += 2) {
                const int turn = (c * 4 + q) / NR, slot = c * 4 + q - turn * NR;
                const int row = q * 32 + r;
                unsigned char* from = v + row * 128;
                uint4 x[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
                const float f = g.col[row] * g.after[q] * unit;
                const uint64_t f2 = f2_pack(f, f);
                if (turn > 0 && !wait(&vt_free[slot], turn - 1)) { ok = false; break; }
                unsigned char* to = smem + L::VT + slot * L::QUARTER + r * 128;
                uint32_t probe = 0;  // 0 x v, summed: not 0 if one is not finite
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t xw[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                    uint32_t w[NT][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (!STATES) probe = M::zero_times(xw[j], probe);
                        const float2 a2 = M::unpack(xw[j]);
                        uint64_t y2 = f2_mul(f2_pack(a2.x, a2.y), f2);
#pragma unroll
                        for (int term = 0; term < NT; ++term) {
                            const float2 y = f2_get(y2);
                            if constexpr (BF) {  // the 24 bits of a number cut into three of 8
                                const uint32_t b0 = __float_as_uint(y.x), b1 = __float_as_uint(y.y);
                                w[term][j] = __byte_perm(b0, b1, 0x7632);
                                if (term + 1 < NT)
                                    y2 = f2_add(y2, f2_pack(-__uint_as_float(b0 & 0xffff0000u), -__uint_as_float(b1 & 0xffff0000u)));
                            } else {
                                w[term][j] = M::pack(y.x, y.y);
                                const float2 z = M::unpack(w[term][j]);
                                if (term + 1 < NT) y2 = f2_add(y2, f2_pack(-z.x, -z.y));
                            }
                        }
                    }
#pragma unroll
                    for (int term = 0; term < NT; ++term)
                        *reinterpret_cast<uint4*>(to + term * 4096 + at[k]) =
                            make_uint4(w[term][0], w[term][1], w[term][2], w[term][3]);
                }
                if (!STATES && (probe & 0x7fff7fffu) != 0) {  // out of V, and noted for the results
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        T* y = reinterpret_cast<T*>(from + at[k]);
                        for (int j = 0; j < 8; ++j)
                            if (!(fabsf(static_cast<float>(y[j])) <= 3.4028234e38f)) {
                                y[j] = from_float<T>(0.f);
                                atomicMin(&bad[(c & 3) * 64 + (u0 ^ (k * 4)) * 8 + j], row);
                                any_bad[c & 3] = 1;
                            }
                    }
                }
                fence_proxy_async_smem();
                arrive_warp(&vt_full[slot]);
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&g_free[st]);
        }
    } else if (warp < 20) {
        // ===================== the state: thread = row of dim_k (half a row at dim_k = 64) =====================
        registers_up<136>();
        constexpr int NC = DK == 128 ? 64 : 32;
        const int tid = threadIdx.x - 512;
        const int row = tid & (DK - 1);
        const int c0 = DK == 128 ? 0 : (tid >> 6) * 32;
        const uint32_t lanes = tmem + ((uint32_t)((warp - 16) * 32) << 16);
        const size_t at = (size_t)row * a.dv + slice * kSlice + c0;  // in a head's state
        uint64_t x[NC / 2];  // pairs of columns
        auto load = [&](const float* from, bool add, float keep) {
            const uint64_t k2 = f2_pack(keep, keep);
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float4 y = *reinterpret_cast<const float4*>(from + at + 2 * i);
                const uint64_t y0 = f2_pack(y.x, y.y), y1 = f2_pack(y.z, y.w);
                x[i] = add ? f2_fma(x[i], k2, y0) : y0;
                x[i + 1] = add ? f2_fma(x[i + 1], k2, y1) : y1;
            }
        };
        auto save = [&](float* to) {
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float2 y = f2_get(x[i]), z = f2_get(x[i + 1]);
                *reinterpret_cast<float4*>(to + at + 2 * i) = make_float4(y.x, y.y, z.x, z.y);
            }
        };
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) x[i] = 0;
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
        float sum = 0.f;
        for (int c = 0; c < pieces; ++c) {
            if constexpr (!STATES) {  // the copy that Q meets
                uint64_t unit2 = 0;
                float back_s = 1.f;
                if constexpr (!BF) {
                    float most = 0.f, other = 0.f;
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) {
                        const float2 y = f2_get(x[i]);
                        most = fmaxf(most, fabsf(y.x)), other = fmaxf(other, fabsf(y.y));
                    }
                    most = fmaxf(most, other);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    if (lane == 0) part[8 + warp - 16] = most;
                    if (!meet(1)) { ok = false; break; }
                    const int e = exponent14(fmaxf(fmaxf(part[8], part[9]), fmaxf(part[10], part[11])));
                    unit2 = f2_pack(pow2i(14 - e), pow2i(14 - e));
                    back_s = pow2i(e - 14);
                    if (!meet(1)) { ok = false; break; }  // part may be written again
                }
                if (c > 0 && !wait(s_free, c - 1)) { ok = false; break; }
                // (Q S of the piece before is done: it began when the results of the one before that had been read)
                if (!BF && tid == 0) s_unit[c & 1] = back_s;
                unsigned char* to = smem + L::S + row * 128;
#pragma unroll
                for (int i = 0; i < NC / 2; i += 4) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = f2_get(BF ? x[i + j] : f2_mul(x[i + j], unit2));
                        w[j] = M::pack(y.x, y.y);
                    }
                    *reinterpret_cast<uint4*>(to + ((((c0 + 2 * i) >> 3) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                arrive_warp(s_full);
            }
            const PieceGates& g = gates[c & 1];
            if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
            const uint64_t keep = f2_pack(g.keep, g.keep), once = f2_pack(g.once, g.once);
            if (STATES) sum += g.sum;
            if (!wait(u_full, c)) { ok = false; break; }
            tcgen05_after_sync();
            const float back = BF ? 1.f : u_unit[c & 1];
#pragma unroll
            for (int i = 0; i < NC / 2; i += 8) {
                float u[NT][16];
#pragma unroll
                for (int term = 0; term < NT; ++term) tmem_ld16(lanes + U_COL + 64 * term + c0 + 2 * i, u[term]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint64_t y = f2_pack(u[NT - 1][2 * j], u[NT - 1][2 * j + 1]);
#pragma unroll
                    for (int term = NT - 2; term >= 0; --term) y = f2_add(y, f2_pack(u[term][2 * j], u[term][2 * j + 1]));
                    if (!BF) y = f2_mul(y, f2_pack(back, back));
                    x[i + j] = f2_fma(x[i + j], keep, f2_fma(x[i + j], once, y));
                }
            }
            tcgen05_before_sync();
            arrive_warp(u_free);
            if (lane == 0) mbar_arrive(&g_free[c & 1]);
        }
        if (ok) {
            if (STATES) {
                const size_t to = ((size_t)s * (a.n_segs - 1) + seg) * l.n_v + h;
                save(a.added + to * head);
                if (tid == 0 && slice == 0) a.sums[to] = sum;
            } else if (seg == used_segs - 1 && dst >= 0)
                save(l.state + ((size_t)dst * l.n_v + h) * head);
        }
    } else if (warp < 24) {
        // ===================== results: thread = row =====================
        registers_down<64>();
        if constexpr (!STATES) {
            const int w4 = warp - 20;
            const int row = w4 * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
            // 64 bytes of each of the warp's 32 rows are staged at a time: unit u of row r at u ^ (r / 2 & 3), so that
            // eight rows' units lie in different banks; a store then takes eight rows, four lanes a row
            unsigned char* stage = smem + L::O + w4 * 2048;
            const uint32_t swz = (lane >> 1) & 3;
            const int out_row = w4 * 32 + (lane >> 2);
            const uint32_t from = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
            const size_t pitch = (size_t)l.n_v * a.dv * sizeof(T);
            char* out = static_cast<char*>(l.out) + (size_t)(t0 + out_row) * pitch +
                        ((size_t)h * a.dv + slice * kSlice + (lane & 3) * 8) * sizeof(T);
            for (int c = 0; c < pieces; ++c) {
                const int n = min(kPiece, tokens - c * kPiece);
                const PieceGates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                float sum = -g.hi[row];
                for (int i = 0; i < w4; ++i) sum += g.block[i];
                arrive_warp(&g_free[c & 1]);
                float fi = ex2_approx(sum) * l.scale, fa = l.scale;
                if (!wait(&done[c & 1], c >> 1)) { ok = false; break; }
                tcgen05_after_sync();
                if constexpr (!BF) {
                    fi *= s_unit[c & 1];
                    fa *= row_unit[(c & 1) * kPiece + row];
                }
                const uint64_t fi2 = f2_pack(fi, fi), fa2 = f2_pack(fa, fa);
                const bool poisoned = any_bad[c & 3] != 0;
#pragma unroll 1
                for (int c0 = 0; c0 < kSlice; c0 += 16) {
                    float x[16], y[16];
                    tmem_ld16(lanes + OI_COL + c0, x);
                    tmem_ld16(lanes + OA_COL + c0, y);
                    tmem_wait_ld();
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float2 z = f2_get(f2_fma(f2_pack(x[j], x[j + 1]), fi2, f2_mul(f2_pack(y[j], y[j + 1]), fa2)));
                        w[j / 2] = M::pack(z.x, z.y);
                    }
                    if (poisoned) {
                        const int* mark = &bad[(c & 3) * 64 + c0];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (mark[j] <= row) w[j / 2] |= 0x7fffu << (16 * (j & 1));
                    }
                    const int u = (c0 >> 3) & 2;
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ swz) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(stage + lane * 64 + (((u + 1) ^ swz) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
                    if (c0 & 16) {
                        if (c0 + 16 == kSlice) {
                            tcgen05_before_sync();
                            arrive_warp(o_free);
                        } else {
                            __syncwarp();
                        }
                        char* to = out + (size_t)(c0 - 16) * sizeof(T);
#pragma unroll
                        for (int k = 0; k < 4; ++k, to += 8 * pitch)
                            if (out_row + k * 8 < n) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(stage + from + k * 512);
                        __syncwarp();
                    }
                }
                out += kPiece * pitch;
                if (poisoned) {  // the columns' marks are used again four pieces on
                    if (!meet(2)) { ok = false; break; }
                    if (row < 64) bad[(c & 3) * 64 + row] = kPiece;
                    if (row == 0) any_bad[c & 3] = 0;
                }
            }
        }
    } else {
        registers_down<48>();  // (one instruction for the four warps)
        if (warp == 24) {
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
        } else if (warp == 25) {
            // ===================== products: one thread =====================
            if (elect_one()) {
                const uint64_t dq = umma_desc_sw128(sbase + L::Q, 16, 1024);
                const uint64_t dk = umma_desc_sw128(sbase + L::K, 16, 1024);
                // K^T: 64 rows of the product a panel; at dim_k = 64 the second 64 are the first again
                const uint64_t dkt = umma_desc_sw128(sbase + L::K, DK == 128 ? PANEL : 0, 1024);
                const uint64_t dv = umma_desc_sw128(sbase + L::V, PANEL, 1024);
                const uint64_t ds = umma_desc_sw128(sbase + L::S, DK * 128, 1024);
                const uint64_t dvt = umma_desc_sw128(sbase + L::VT, 4096, 1024);
                auto pairs = [&](uint32_t st) {  // P = Q K^T
                    const uint64_t q = dq + ((st * L::QK) >> 4), k = dk + ((st * L::QK) >> 4);
                    tcgen05_after_sync();
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i) {
                        const uint32_t off = (((uint32_t)(i >> 2) * PANEL + (uint32_t)(i & 3) * 32) >> 4);
                        umma_f16_cg<1>(tmem + P_COL, q + off, k + off, IDESC_P, i > 0);
                    }
                    umma_commit_cg<1>(p_full);
                };
                if (!STATES && pieces > 0) {
                    ok = wait1(&qk_full[0], 0);
                    if (ok) pairs(0);
                }
                int slot = 0, turn = 0;  // of V~'s ring
                for (int c = 0; c < pieces && ok; ++c) {
                    const uint32_t st = (uint32_t)(c & 1);
                    // U = K^T V~ (V~'s warps have seen V land; K has landed where P was computed)
                    if ((STATES && !wait1(&qk_full[st], c >> 1)) || (c > 0 && !wait1(u_free, c - 1))) { ok = false; break; }
                    const uint64_t kt = dkt + ((st * L::QK) >> 4);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        if (!wait1(&vt_full[slot], turn)) { ok = false; break; }
                        tcgen05_after_sync();
                        const uint64_t vt = dvt + (((uint32_t)slot * L::QUARTER) >> 4), k0 = kt + (uint32_t)q * (4096 >> 4);
                        umma_f16_cg<1>(tmem + U_COL, k0, vt, IDESC_U, q > 0);
                        umma_f16_cg<1>(tmem + U_COL, k0 + (2048 >> 4), vt + (2048 >> 4), IDESC_U, true);
                        umma_commit_cg<1>(&vt_free[slot]);
                        if (++slot == NR) slot = 0, ++turn;
                    }
                    if (!ok) break;
                    umma_commit_cg<1>(u_full);
                    if constexpr (STATES) {
                        umma_commit_cg<1>(&done[st]);
                    } else {
                        // OI = Q S
                        if (!wait1(s_full, c) || (c > 0 && !wait1(o_free, c - 1))) { ok = false; break; }
                        tcgen05_after_sync();
                        const uint64_t q = dq + ((st * L::QK) >> 4);
#pragma unroll
                        for (int i = 0; i < DK / 16; ++i)
                            umma_f16_cg<1>(tmem + OI_COL, q + (((uint32_t)(i >> 2) * PANEL + (uint32_t)(i & 3) * 32) >> 4),
                                           ds + (uint32_t)i * (2048 >> 4), IDESC_O, i > 0);
                        umma_commit_cg<1>(s_free);
                        if (!wait1(w_full, c)) { ok = false; break; }
                        if (c + 1 < pieces) {
                            if (!wait1(&qk_full[st ^ 1], (c + 1) >> 1)) { ok = false; break; }
                            pairs(st ^ 1);
                        }
                        // OA = P' V
                        tcgen05_after_sync();
                        const uint64_t v = dv + ((st * PANEL) >> 4);
#pragma unroll
                        for (int i = 0; i < kPiece / 16; ++i)
                            umma_f16_tmem_a_cg<1>(tmem + OA_COL, tmem + PW_COL + i * 8, v + (uint32_t)i * (2048 >> 4), IDESC_O, i > 0);
                        umma_commit_cg<1>(&done[st]);
                    }
                }
                // every product is done before tensor memory is given back
                umma_commit_cg<1>(all_done);
                ok = wait1(all_done, 0) && ok;
                if (!ok) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
            }
            __syncwarp();
        } else {
            // ===================== sums of the log decays: lane = 4 tokens, a warp for every other piece =====================
            // Whole numbers of 2^-40 (in 64 bits): sums and differences are exact, and 64-bit floats too slow here.
            constexpr float UNIT = 1.0f / 1099511627776.0f;
            float raw[4];
            auto fetch = [&](int c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = c * kPiece + lane * 4 + i;
                    raw[i] = l.log_decay && t < tokens ? l.log_decay[(size_t)(t0 + t) * l.decay_stride + h] : 0.f;
                }
            };
            const int odd = warp - 26;
            if (odd < pieces) fetch(odd);
            for (int c = odd; c < pieces; c += 2) {
                long long x[4];
                float poison[4], grow = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // 2^-150 is 0 in fp32, 2^(10^4) infinite: a token that forgets (-infinity) takes part in sums
                    const float y = fminf(fmaxf(raw[i], -104.f), 1e4f);
                    const float hi = y * 1.44269504f;
                    const float lo = fmaf(y, 1.44269504f, -hi) + y * 1.92596299e-8f;
                    x[i] = __float2ll_rn(hi * 1099511627776.0f) + __float2ll_rn(lo * 1099511627776.0f);
                    grow += fmaxf(hi, 0.f);
                    poison[i] = raw[i] != raw[i] ? raw[i] : 0.f;  // a NaN is kept apart
                }
                const bool nan = __any_sync(0xffffffffu, (poison[0] + poison[1]) + (poison[2] + poison[3]) != 0.f);
                if (c + 2 < pieces) fetch(c + 2);
#pragma unroll
                for (int i = 1; i < 4; ++i) x[i] += x[i - 1];
                long long before = x[3];  // over the lanes of a block of 32 tokens (eight)
#pragma unroll
                for (int o = 1; o < 8; o *= 2) {
                    const long long y = __shfl_up_sync(0xffffffffu, before, o);
                    if ((lane & 7) >= o) before += y;
                }
                const long long block = __shfl_sync(0xffffffffu, before, lane | 7);
                before -= x[3];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) grow += __shfl_xor_sync(0xffffffffu, grow, o);
                long long blocks[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) blocks[b] = __shfl_sync(0xffffffffu, block, b * 8);
                float hi[4], lo[4], col[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long y = -(before + x[i]);
                    hi[i] = __ll2float_rn(y);
                    lo[i] = __ll2float_rn(y - __float2ll_rn(hi[i])) * UNIT;
                    hi[i] *= UNIT;
                    col[i] = exp2f(__ll2float_rn(block + y) * UNIT);
                }
                float block_nan = 0.f, any_nan = 0.f, blocks_nan[4] = {0.f, 0.f, 0.f, 0.f};
                if (nan) {  // from its token on, and wherever a sum has it
#pragma unroll
                    for (int i = 1; i < 4; ++i) poison[i] += poison[i - 1];
                    float p = poison[3];
#pragma unroll
                    for (int o = 1; o < 8; o *= 2) {
                        const float y = __shfl_up_sync(0xffffffffu, p, o);
                        if ((lane & 7) >= o) p += y;
                    }
                    block_nan = __shfl_sync(0xffffffffu, p, lane | 7);
                    p = __shfl_up_sync(0xffffffffu, p, 1);
                    if ((lane & 7) == 0) p = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) hi[i] += p + poison[i], col[i] += block_nan;
#pragma unroll
                    for (int b = 0; b < 4; ++b) any_nan += blocks_nan[b] = __shfl_sync(0xffffffffu, block_nan, b * 8);
                }
                if (c >= 2 && !wait(&g_free[c & 1], (c >> 1) - 1)) { ok = false; break; }
                PieceGates& g = gates[c & 1];
                *reinterpret_cast<float4*>(&g.hi[lane * 4]) = make_float4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<float4*>(&g.lo[lane * 4]) = make_float4(lo[0], lo[1], lo[2], lo[3]);
                *reinterpret_cast<float4*>(&g.col[lane * 4]) = make_float4(col[0], col[1], col[2], col[3]);
                const long long all = (blocks[0] + blocks[1]) + (blocks[2] + blocks[3]);
                if (lane < 4) {
                    const long long behind = (lane < 1 ? blocks[1] : 0) + (lane < 2 ? blocks[2] : 0) + (lane < 3 ? blocks[3] : 0);
                    const float behind_nan = (lane < 1 ? blocks_nan[1] : 0.f) + (lane < 2 ? blocks_nan[2] : 0.f) +
                                             (lane < 3 ? blocks_nan[3] : 0.f);
                    const long long mine = lane == 0 ? blocks[0] : lane == 1 ? blocks[1] : lane == 2 ? blocks[2] : blocks[3];
                    const float mine_nan = lane == 0   ? blocks_nan[0]
                                           : lane == 1 ? blocks_nan[1]
                                           : lane == 2 ? blocks_nan[2]
                                                       : blocks_nan[3];
                    g.block[lane] = __ll2float_rn(mine) * UNIT + mine_nan;
                    g.after[lane] = exp2f(__ll2float_rn(behind) * UNIT) + behind_nan;
                } else if (lane == 4) {
                    const float sum = __ll2float_rn(all) * UNIT;
                    const bool small = sum > -0.7f && sum < 0.7f;
                    g.keep = (small ? expm1f(sum * 0.693147181f) : exp2f(sum)) + any_nan;
                    g.once = small ? 1.f : 0.f;
                    g.grow = grow;
                    g.sum = sum;
                }
                arrive_warp(&g_full[c & 1]);
            }
        }
    }
    if (!ok && lane == 0) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 25) tmem_dealloc_cg<1>(tmem, 512);
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
