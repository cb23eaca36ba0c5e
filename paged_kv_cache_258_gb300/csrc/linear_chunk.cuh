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
//   warps 8-15   V~, in quarters of 32 rows one after the other, four warps on every other one: split into numbers of the type that add up to it (two of
//                fp16: 2^-22 is left; three of bf16: exact), beside one another along N, so that one product of N = 128
//                or 192 gives their sums and the state keeps fp32's precision
//   warps 16-19  the state: S in fp32 registers, a thread a row (of dim_k; at dim_k = 64 half a row, the product's 128
//                rows being K's 64 twice), decays it, adds U and hands the tensor cores a rounded copy
//   warps 20-23  results: exp(G_i) OI + OA, whole 32-byte sectors of a row from its thread
//   warp 24      tensor copies of Q, K and V, two pieces ahead
//   warp 25      issues the products
//   warps 26, 27 sums of decays (whole numbers of 64 bits: differences of far sums)
//
// Rounded to 16 bits are P' and the copy of S that Q meets, each term of a result once, as attention weights are.
// fp16 cannot hold their range: rows of P' and the copy of S are then brought to 2^14 by a power of two each, which the
// sums undo in fp32.
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
// fp16: the second number of a value of V~ is this times what the first lacks of it: at most the value, so it fits, and
// the two are within 2^-22 of a value, or within 2^-36 where that is more.
constexpr float kSecond = 2048.f;
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

// A piece's 128 log decays, as the roles need them.
template <bool LO>
struct __align__(16) PieceGates {
    float hi[kPiece];              // minus the sum from the start of a token's block of 32 to it, base 2
    float lo[LO ? kPiece : 4];     // what hi lacks of it (fp16; bf16 weights are coarser than what it changes: with every
                                   // token of a block forgetting all, 2^-12)
    float col[kPiece];             // 2^(sum from the token to its block's end)
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
    static constexpr uint32_t PANEL = kPiece * 128;        // 64 columns of 128 rows
    static constexpr uint32_t QK = PANEL * (DK / 64);
    static constexpr uint32_t QUARTER = 32 * 128 * NT;     // [NT][32 rows][128 B]
    static constexpr uint32_t Q = 0;
    static constexpr uint32_t K = Q + 2 * QK;
    static constexpr uint32_t V = K + 2 * QK;
    static constexpr uint32_t VT = V + 2 * PANEL;
    static constexpr uint32_t S = VT + 4 * QUARTER;        // [DK rows][128 B]
    using Gates = PieceGates<!BF>;
    static constexpr uint32_t GATES = S + DK * 128;        // [2]
    static constexpr uint32_t BAD = GATES + 2 * sizeof(Gates);  // bytes [4][64]: first token whose v is not finite
    static constexpr uint32_t ROW = BAD + 4 * 64;      // fp16: float [2][128], 2^-e of P's rows
    static constexpr uint32_t MISC = ROW + (BF ? 0 : 2 * 128 * 4);  // any_bad[4] s_unit[2] - part[2][4]
    static constexpr uint32_t BARS = MISC + 64;
    static constexpr int NBARS = 5 * 2 + 2 * 4 + 7 + 4;
    static constexpr uint32_t TADDR = BARS + NBARS * 8;
    static constexpr uint32_t TOTAL = TADDR + 16;
    static constexpr uint32_t ALLOC = TOTAL;               // (on a 1,024-byte boundary: the array is declared so)
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

// mbar_wait_bounded in few instructions (28 warps of seven roles share the instruction caches): a thread sleeps up to a
// microsecond in each try, and gives up after as many as make about a second.
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_addr(bar);
#pragma unroll 1
    for (int tries = 1 << 20; tries > 0; --tries) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// *p = min(*p, x), of bytes in shared memory
__device__ __forceinline__ void byte_min(uint8_t* p, int x) {
    uint32_t* word = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
    const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 3) * 8;
    uint32_t old = *word;
    while ((int)((old >> shift) & 255u) > x) {
        const uint32_t seen = atomicCAS(word, old, (old & ~(255u << shift)) | ((uint32_t)x << shift));
        if (seen == old) break;
        old = seen;
    }
}

// What keeps values of fp16 that gates with sums of positive parts `grow` weigh within fp16: a power of two.
__device__ __forceinline__ float down_by(float grow) { return ex2_approx(-ceilf(fminf(grow, 100.f))); }

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
    constexpr int NT = L::NT;
    constexpr uint32_t PANEL = L::PANEL;
    constexpr uint32_t P_COL = 0, PW_COL = 128, OI_COL = 192, OA_COL = 256, U_COL = 320;
    static_assert(U_COL + 64 * NT <= 512, "tensor memory");
    constexpr uint32_t IDESC_P = umma_idesc_f16(BF, 128, kPiece, false);
    constexpr uint32_t IDESC_O = umma_idesc_f16(BF, 128, kSlice, true);
    constexpr uint32_t IDESC_U = umma_idesc_f16(BF, 128, kSlice * NT, true) | (1u << 15);  // A = K^T: M-major
    constexpr uint32_t GATE_READERS = STATES ? 12 : 24;  // warps

    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    using Gates = typename L::Gates;
    Gates* gates = reinterpret_cast<Gates*>(smem + L::GATES);
    uint8_t* bad = smem + L::BAD;
    float* row_unit = reinterpret_cast<float*>(smem + L::ROW);
    int* any_bad = reinterpret_cast<int*>(smem + L::MISC);
    float* s_unit = reinterpret_cast<float*>(smem + L::MISC + 16);
    float* part = reinterpret_cast<float*>(smem + L::MISC + 32);
    uint64_t* qk_full = reinterpret_cast<uint64_t*>(smem + L::BARS);  // [2] Q and K of a piece have landed
    uint64_t* v_full = qk_full + 2;                                   // [2]
    uint64_t* done = v_full + 2;       // [2] every product of a piece is done: its buffers and results
    uint64_t* g_full = done + 2;       // [2] gates
    uint64_t* g_free = g_full + 2;     // [2]
    uint64_t* vt_full = g_free + 2;    // [4] a quarter of V~ is written
    uint64_t* vt_free = vt_full + 4;   // [4] and read
    uint64_t* u_full = vt_free + 4;    // U is done
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
    if ((sbase & 1023u) != 0) {  // (the swizzled tiles need it; never seen)
        if (threadIdx.x == 0) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
        return;
    }
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
        for (int i = 0; i < 4; ++i) {
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
    if (threadIdx.x < 4 * 64) bad[threadIdx.x] = kPiece;
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
#pragma unroll 1
                for (int b = w4 + 1; b < 4; ++b) put(b, zero);
            }
#pragma unroll 1
            for (int c = 0; c < pieces; ++c) {
                const Gates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                const float mine = -g.hi[row];
                float mine_lo = BF ? 0.f : -g.lo[row];
                if (!wait(p_full, c)) { ok = false; break; }
                tcgen05_after_sync();
                float shift = 0.f;  // log2 of what the row is multiplied by
                if constexpr (!BF) {
                    float m0 = 0.f, m1 = 0.f;
#pragma unroll 1
                    for (int b = 0; b <= w4; ++b) {
                        uint32_t x[32];
                        tmem_ld32(lanes + P_COL + b * 32, x);
                        tmem_wait_ld();
                        const int last = b < w4 ? 31 : lane;
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float y0 = __uint_as_float(x[j]), y1 = __uint_as_float(x[j + 1]), y2 = __uint_as_float(x[j + 2]),
                                        y3 = __uint_as_float(x[j + 3]);
                            m0 = fmax3(m0, j <= last ? fabsf(y0) : 0.f, j + 1 <= last ? fabsf(y1) : 0.f);
                            m1 = fmax3(m1, j + 2 <= last ? fabsf(y2) : 0.f, j + 3 <= last ? fabsf(y3) : 0.f);
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
                    const ulonglong2* gl = reinterpret_cast<const ulonglong2*>(BF ? g.lo : &g.lo[w4 * 32 + side]);
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 y = gh[j];
                        uint64_t e0 = f2_add(hi2, y.x), e1 = f2_add(hi2, y.y);
                        if constexpr (!BF) {
                            const ulonglong2 z = gl[j];
                            e0 = f2_add(e0, f2_add(lo2, z.x)), e1 = f2_add(e1, f2_add(lo2, z.y));
                        }
                        const float2 d0 = f2_get(e0), d1 = f2_get(e1);
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
#pragma unroll 1
        for (int c = 0; c < pieces; ++c) {
            const int st = c & 1;
            const int n = min(kPiece, tokens - c * kPiece);
            unsigned char* v = smem + L::V + st * PANEL;
            const Gates& g = gates[st];
            if (!wait(&g_full[st], c >> 1) || !wait(&v_full[st], c >> 1)) { ok = false; break; }
            if (n < kPiece) {  // rows behind the sequence's end
                if (!wait(&qk_full[st], c >> 1)) { ok = false; break; }
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                for (int i = n * 8 + tid; i < kPiece * 8; i += 256) {
                    *reinterpret_cast<uint4*>(v + i * 16) = zero;
#pragma unroll
                    for (int p = 0; p < DK / 64; ++p)
                        *reinterpret_cast<uint4*>(smem + L::K + st * L::QK + p * PANEL + i * 16) = zero;
                }
                fence_proxy_async_smem();
                if (!meet(0)) { ok = false; break; }
            }
            const float unit = BF ? 1.f : down_by(g.grow);
#pragma unroll 1
            for (int q = half; q < 4; q += 2) {
                const int row = q * 32 + r;
                unsigned char* from = v + row * 128;
                uint4 x[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
                const float f = g.col[row] * g.after[q] * unit;
                const uint64_t f2 = f2_pack(f, f);
                if (c > 0 && !wait(&vt_free[q], c - 1)) { ok = false; break; }
                unsigned char* to = smem + L::VT + q * L::QUARTER + r * 128;
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
                                if (term + 1 < NT) y2 = f2_mul(f2_add(y2, f2_pack(-z.x, -z.y)), f2_pack(kSecond, kSecond));
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
#pragma unroll 1
                        for (int j = 0; j < 8; ++j)
                            if (!(fabsf(static_cast<float>(y[j])) <= 3.4028234e38f)) {
                                y[j] = from_float<T>(0.f);
                                byte_min(&bad[(c & 3) * 64 + (u0 ^ (k * 4)) * 8 + j], row);
                                any_bad[c & 3] = 1;
                            }
                    }
                }
                fence_proxy_async_smem();
                arrive_warp(&vt_full[q]);
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
        auto load = [&](const float* from, float keep) {
            const uint64_t k2 = f2_pack(keep, keep);
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float4 y = *reinterpret_cast<const float4*>(from + at + 2 * i);
                x[i] = f2_fma(x[i], k2, f2_pack(y.x, y.y));
                x[i + 1] = f2_fma(x[i + 1], k2, f2_pack(y.z, y.w));
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
        {
            // shared out, the second pass reads the start from where the first left it (its last segment writes dst), or
            // adds up what the segments before leave
            const size_t mine = (size_t)s * l.n_v + h;
            const bool from_state = STATES || used_segs == 1;
            const int n = seg > 0 ? (STATES ? 0 : seg) : !from_state || src >= 0;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const size_t to = ((size_t)s * (a.n_segs - 1) + i) * l.n_v + h;
                load(seg > 0      ? a.added + to * head
                     : from_state ? l.state + ((size_t)src * l.n_v + h) * head
                                  : a.start + mine * head,
                     i > 0 ? exp2f(a.sums[to]) : 0.f);
            }
            if (STATES && seg == 0) save(a.start + mine * head);
        }
        float sum = 0.f;
#pragma unroll 1
        for (int c = 0; c < pieces; ++c) {
            if constexpr (!STATES) {  // the copy that Q meets
                uint64_t unit2 = 0;
                float back_s = 1.f;
                if constexpr (!BF) {
                    float most = 0.f;
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) {
                        const float2 y = f2_get(x[i]);
                        most = fmax3(most, fabsf(y.x), fabsf(y.y));
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    float* mine = part + (c & 1) * 4;  // (read for piece c by all before any of them meets for c + 1)
                    if (lane == 0) mine[warp - 16] = most;
                    if (!meet(1)) { ok = false; break; }
                    const int e = exponent14(fmaxf(fmaxf(mine[0], mine[1]), fmaxf(mine[2], mine[3])));
                    unit2 = f2_pack(pow2i(14 - e), pow2i(14 - e));
                    back_s = pow2i(e - 14);
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
            const Gates& g = gates[c & 1];
            if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
            const float unit_v = BF ? 1.f : down_by(g.grow);
            const uint64_t keep = f2_pack(g.keep, g.keep), once = f2_pack(g.once, g.once);
            if (STATES) sum += g.sum;
            arrive_warp(&g_free[c & 1]);
            if (!wait(u_full, c)) { ok = false; break; }
            tcgen05_after_sync();
            const float back = BF ? 1.f : 1.f / unit_v, back2 = back / kSecond;
#pragma unroll
            for (int i = 0; i < NC / 2; i += 8) {
                float u[NT][16];
#pragma unroll
                for (int term = 0; term < NT; ++term) tmem_ld16(lanes + U_COL + 64 * term + c0 + 2 * i, u[term]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint64_t y = f2_pack(u[NT - 1][2 * j], u[NT - 1][2 * j + 1]);
                    if constexpr (BF) {
#pragma unroll
                        for (int term = NT - 2; term >= 0; --term) y = f2_add(y, f2_pack(u[term][2 * j], u[term][2 * j + 1]));
                    } else {
                        y = f2_fma(f2_pack(u[0][2 * j], u[0][2 * j + 1]), f2_pack(back, back), f2_mul(y, f2_pack(back2, back2)));
                    }
                    x[i + j] = f2_fma(x[i + j], keep, f2_fma(x[i + j], once, y));
                }
            }
            tcgen05_before_sync();
            arrive_warp(u_free);
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
            const size_t pitch = (size_t)l.n_v * a.dv * sizeof(T);
            char* out = static_cast<char*>(l.out) + (size_t)(t0 + row) * pitch + ((size_t)h * a.dv + slice * kSlice) * sizeof(T);
            float sum = 0.f;  // of the log decays up to the row
            auto decays = [&](int c) -> bool {
                if (!wait(&g_full[c & 1], c >> 1)) return false;
                const Gates& g = gates[c & 1];
                sum = -g.hi[row];
#pragma unroll 1
                for (int i = 0; i < w4; ++i) sum += g.block[i];
                arrive_warp(&g_free[c & 1]);
                return true;
            };
            if (pieces > 0) ok = decays(0);
            const bool sectors = (reinterpret_cast<uintptr_t>(l.out) & 31) == 0;
#pragma unroll 1
            for (int c = 0; c < pieces && ok; ++c) {
                const int n = min(kPiece, tokens - c * kPiece);
                if (!wait(&done[c & 1], c >> 1)) { ok = false; break; }
                tcgen05_after_sync();
                float fi = ex2_approx(sum) * l.scale, fa = l.scale;
                if (c + 1 < pieces && !decays(c + 1)) { ok = false; break; }  // (early: their buffer is waited for)
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
                        const uint8_t* mark = &bad[(c & 3) * 64 + c0];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (mark[j] <= row) w[j / 2] |= 0x7fffu << (16 * (j & 1));
                    }
                    if (c0 + 16 == kSlice) {
                        tcgen05_before_sync();
                        arrive_warp(o_free);
                    }
                    if (row < n) {
                        char* to = out + c0 * sizeof(T);
                        if (sectors) {
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]),
                                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                         : "memory");
                        } else {
                            reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
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
#pragma unroll 1
                for (int c = 0; c < pieces; ++c) {
                    const int st = c & 1;
                    if (c >= 2 && !wait1(&done[st], (c >> 1) - 1)) { ok = false; break; }
                    const int y = t0 + c * kPiece;
                    // (V first: its warps are the furthest ahead)
                    mbar_arrive_expect_tx(&v_full[st], PANEL);
                    tma_rows(sbase + L::V + st * PANEL, &tm_v, h * a.dv + slice * kSlice, y, &v_full[st]);
                    mbar_arrive_expect_tx(&qk_full[st], (STATES ? 1 : 2) * L::QK);
#pragma unroll
                    for (int p = 0; p < DK / 64; ++p) {
                        if (!STATES) tma_rows(sbase + L::Q + st * L::QK + p * PANEL, &tm_q, hq * DK + p * 64, y, &qk_full[st]);
                        tma_rows(sbase + L::K + st * L::QK + p * PANEL, &tm_k, hq * DK + p * 64, y, &qk_full[st]);
                    }
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
            // ===================== products: one thread (an instruction takes the tensor core 50 to 100 cycles: short
            // code counts more than unrolled loops) =====================
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
#pragma unroll 1
                    for (int i = 0; i < DK / 16; ++i) {
                        const uint32_t off = ((uint32_t)(i >> 2) * PANEL + (uint32_t)(i & 3) * 32) >> 4;
                        umma_f16_cg<1>(tmem + P_COL, q + off, k + off, IDESC_P, i > 0);
                    }
                    umma_commit_cg<1>(p_full);
                };
                if (!STATES && pieces > 0) {
                    ok = wait1(&qk_full[0], 0);
                    if (ok) pairs(0);
                }
#pragma unroll 1
                for (int c = 0; c < pieces && ok; ++c) {
                    const uint32_t st = (uint32_t)(c & 1);
                    // U = K^T V~ (V~'s warps have seen V land; K has landed where P was computed)
                    if ((STATES && !wait1(&qk_full[st], c >> 1)) || (c > 0 && !wait1(u_free, c - 1))) { ok = false; break; }
                    const uint64_t kt = dkt + ((st * L::QK) >> 4);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        if (!wait1(&vt_full[q], c)) { ok = false; break; }
                        tcgen05_after_sync();
                        const uint64_t vt = dvt + (((uint32_t)q * L::QUARTER) >> 4), k0 = kt + (uint32_t)q * (4096 >> 4);
                        umma_f16_cg<1>(tmem + U_COL, k0, vt, IDESC_U, q > 0);
                        umma_f16_cg<1>(tmem + U_COL, k0 + (2048 >> 4), vt + (2048 >> 4), IDESC_U, true);
                        umma_commit_cg<1>(&vt_free[q]);
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
#pragma unroll 1
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
#pragma unroll 1
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
            // ===================== sums of the log decays: lane = token of a block, a warp for every other piece =====================
            // Whole numbers of 2^-40 (in 64 bits): sums and differences are exact, and 64-bit floats too slow here.
            constexpr float UNIT = 1.0f / 1099511627776.0f;
            const int odd = warp - 26;
            auto fetch = [&](int t) -> float {  // t: within the segment
                return l.log_decay && t < tokens ? l.log_decay[(size_t)(t0 + t) * l.decay_stride + h] : 0.f;
            };
            // a whole piece's loads are in flight, the warp's next piece's
            float n0 = fetch(odd * kPiece + lane), n1 = fetch(odd * kPiece + 32 + lane), n2 = fetch(odd * kPiece + 64 + lane),
                  n3 = fetch(odd * kPiece + 96 + lane);
#pragma unroll 1
            for (int c = odd; c < pieces; c += 2) {
                if (c >= 2 && !wait(&g_free[c & 1], (c >> 1) - 1)) { ok = false; break; }
                Gates& g = gates[c & 1];
                long long total = 0;      // lane b: of block b
                float grow = 0.f;
                unsigned nans = 0;        // bit b: a NaN in block b
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    const float raw = n0;
                    n0 = n1, n1 = n2, n2 = n3;
                    n3 = fetch((c + 2) * kPiece + b * 32 + lane);
                    const unsigned nan = __ballot_sync(0xffffffffu, raw != raw);
                    // 2^-150 is 0 in fp32, 2^(10^4) infinite: a token that forgets (-infinity) takes part in sums
                    const float y = fminf(fmaxf(raw, -104.f), 1e4f);
                    const float yh = y * 1.44269504f;
                    const float yl = fmaf(y, 1.44269504f, -yh) + y * 1.92596299e-8f;
                    long long x = __float2ll_rn(yh * 1099511627776.0f) + __float2ll_rn(yl * 1099511627776.0f);
                    grow += fmaxf(yh, 0.f);
#pragma unroll
                    for (int o = 1; o < 32; o *= 2) {
                        const long long z = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += z;
                    }
                    const long long all = __shfl_sync(0xffffffffu, x, 31);
                    if (lane == b) total = all;
                    const float hi = __ll2float_rn(-x);
                    float to_end = ex2_approx(__ll2float_rn(all - x) * UNIT);
                    float hi_out = hi * UNIT;
                    if (nan) {  // from its token on, and in every sum that has it
                        nans |= 1u << b;
                        to_end = __int_as_float(0x7fffffff);
                        if (nan & (0xffffffffu >> (31 - lane))) hi_out = to_end;
                    }
                    g.hi[b * 32 + lane] = hi_out;
                    if constexpr (!BF) g.lo[b * 32 + lane] = __ll2float_rn(-x - __float2ll_rn(hi)) * UNIT;
                    g.col[b * 32 + lane] = to_end;
                }
                if (__any_sync(0xffffffffu, grow != 0.f)) {
#pragma unroll 1
                    for (int o = 16; o > 0; o >>= 1) grow += __shfl_xor_sync(0xffffffffu, grow, o);
                }
                long long behind = total;  // lanes 0-3: over the lane's block and those behind it
                if (lane > 3) behind = 0;
#pragma unroll
                for (int o = 1; o < 4; o *= 2) behind += __shfl_down_sync(0xffffffffu, behind, o);
                const float nan_b = __int_as_float(0x7fffffff);
                if (lane < 4) {
                    g.block[lane] = nans >> lane & 1 ? nan_b : __ll2float_rn(total) * UNIT;
                    g.after[lane] = nans >> lane >> 1 ? nan_b : ex2_approx(__ll2float_rn(behind - total) * UNIT);
                }
                if (lane == 0) {
                    const float sum = __ll2float_rn(behind) * UNIT;
                    const bool small = sum > -0.7f && sum < 0.7f;
                    g.keep = nans ? nan_b : small ? expm1f(sum * 0.693147181f) : ex2_approx(sum);
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
