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
//   warps 8-15   V~, in quarters of 32 rows, four warps on every other one: split into numbers of the type that add up
//                to it (two of fp16: 2^-22 is left, or 2^-50 of the piece's largest; three of bf16: exact), two beside one
//                another along N, so that one product of N = 128 gives both sums (the third is added to the second's), and
//                the state is not rounded to the type
//   warps 16-19  the state: S in fp32 registers, a thread a row (of dim_k; at dim_k = 64 half a row, the product's 128
//                rows being K's 64 twice), decays it, adds U and hands the tensor cores a rounded copy
//   warps 20-23  results: exp(G_i) OI + OA, whole 32-byte sectors of a row from its thread
//   warp 24      tensor copies of Q, K and V, two pieces ahead
//   warps 25, 26 issue the products: P, OI and OA, and U: a thread's waits (some 150 cycles each here, met or not) then
//                leave the tensor cores to the other's products
//   warp 27      sums of the log decays, for all the others
//
// Rounded to 16 bits are P' and the copy of S that Q meets, each term of a result once, as attention weights are.
// fp16 cannot hold their range: the largest number of each row of P', of V~ and of the copy of S (of its columns, where they
// are far apart) is then brought to 2^14 by a power of two, which the sums undo in fp32. It is the largest as weighted by the
// decays: their own largest alone says little, growing ones may weigh what is 0, and what is large may be what they leave
// nothing of.
//
// Fewer units than the GPU holds: a long sequence is shared out along its length in segments, a first pass leaving what
// each adds to the state (STATES). More: a CTA goes on with others' work (MORE), its roles without a pause, so that a
// second unit of one piece takes 4.5 us instead of 8.1 (a CTA's start, first copies and end, with nothing beside them).
//
// What bounds it: the walk along a sequence. A piece takes 1.8 us of a CTA, twice what its products take alone: U, the
// state's sum and rounding, OI and the reading of results follow one another, and the roles' instructions share four
// schedulers. 48 heads x 128 x 128, bf16: 8,192 tokens of one sequence 115 us (2.3 TB/s of q, k, v and results, 0.78 PFLOP/s
// of products), 4 x 2,048 112 us, 8 x 64 tokens 32 us. fp16, whose largest numbers are looked for and whose longer loops wait
// for instructions: 172, 131 and 40 us.
//
// A piece past the sequence's end: rows of K and V behind it are zeroed in shared memory (another sequence's rows, or
// nobody's, NaN perhaps). A non-finite v would reach earlier tokens of its piece through 0 x NaN: it is taken
// out of V (not of V~), and the results get NaN from its token on.
#pragma once

#include <type_traits>

#include "arith.cuh"
#include "common.cuh"
#include "linear.h"
#include "umma.cuh"

namespace pkv {

constexpr int kPiece = 128;   // tokens of a piece: the M of a product
constexpr int kSlice = 64;    // columns of v of a CTA
// fp16: the second number of a value of V~ is this times what the first lacks of it: at most the value, so it fits, and
// the two are within 2^-22 of a value, or within 2^-50 of the piece's largest where that is more.
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
struct __align__(16) PieceGates {
    float hi[kPiece];              // minus the sum from the start of a token's block of 32 to it, base 2 (fp16: or from behind the
                                   // last token up to it that forgets; HalfScales::front is from the start)
    float col[kPiece];             // 2^(sum from behind the token to its block's end)
    float block[4];                // sum over each block
    float after[4];                // 2^(sum over the blocks behind it)
    float keep, once;              // S' = S + (U + S * keep) with 2^(sum over all) - 1 where that is small, once = 1,
    float sum;                     // else S * keep + U, once = 0; the sum over all
};

// fp16: what tokens forget, and the powers of two that bring what the products take into its range.
struct __align__(16) HalfScales {
    uint32_t forgotten[2][kPiece]; // of a token's block of 32: those that it, or one between, forgets
    float front[2][kPiece];        // sums from a token's block's start all the same
    float row_unit[4][kPiece];     // of the rows of P', undone: 2^-shift
    float row_most[2][2][kPiece];  // largest weighted pair of a row's even and odd halves
    float v_most[2][8];            // largest number of V~ that a warp has
    float v_back[4];               // of V~, undone
    float s_most[2][4][2];         // of a warp's part of S: the largest number, the largest of its rows' smallest
    float s_back[4];               // of the copy of S, undone, where its columns have one power of two,
    int s_columns[4];              // else, of each column:
    float col_most[4][kSlice];     // the largest number that a warp has
    float col_up[kSlice], col_back[4][kSlice];
};

// The work of one CTA of the grid: a sequence (or a segment of it), a head, 64 columns of v.
struct __align__(16) ChunkWork {
    int valid, slice, h, s, seg, used_segs, src, dst;
    int t0, tokens, pieces, pad;  // its first token and how many; pieces of 128
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
    using Gates = PieceGates;
    static constexpr uint32_t GATES = S + DK * 128;        // [2]
    static constexpr uint32_t BAD = GATES + 2 * sizeof(Gates);  // bytes [4][64]: first token whose v is not finite
    static constexpr uint32_t HALF = BAD + 4 * 64;     // fp16: HalfScales
    static constexpr uint32_t MISC = HALF + (BF ? 0 : sizeof(HalfScales));  // any_bad[4]
    static constexpr uint32_t NEXT = MISC + 16;            // 16 bytes: the answer to a request for another CTA's work
    static constexpr uint32_t WORK = NEXT + 16;            // [2]
    static constexpr uint32_t BARS = WORK + 2 * sizeof(ChunkWork);
    static constexpr int NBARS = 10 * 2 + 2 * 4 + 7 + 3 + 2 + 2 + (BF ? 0 : 4);
    static constexpr uint32_t TADDR = BARS + NBARS * 8;
    static constexpr uint32_t TOTAL = TADDR + 16;
    static constexpr uint32_t ALLOC = TOTAL;               // (on a 1,024-byte boundary: the array is declared so)
    static_assert(ALLOC <= 232448, "shared memory");
    static_assert(4 * QUARTER >= DK * kSlice * 4, "a segment's first state fits where V~ goes");
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
// 64 + 64 + 56 + 56 + 128 + 88 + 48 = 7 * 72, or where a CTA goes on with other work (results by 16 columns, which take
// fewer) 64 + 64 + 64 + 64 + 128 + 72 + 48.
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

// The largest of 16 fp16 numbers' absolute values, as bits: infinity and NaN are above the others.
__device__ __forceinline__ uint32_t largest_half(const uint4 (&x)[2]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        top = __vmaxu2(__vmaxu2(top, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu)),
                       __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
    return max(top & 0xffffu, top >> 16);
}

// max(|x|) over the warp; NaN counts only where nothing else is
__device__ __forceinline__ float warp_most(float x) {
    float y;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// min(a, b, c) in one instruction
__device__ __forceinline__ float fmin3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^e, e clamped to what a normal number holds
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// e with 2^(14 - e) bringing x into [2^14, 2^15), if x >= 2^-100; 14 (no change) for 0
__device__ __forceinline__ int exponent14(float x) {
    const int e = (int)((__float_as_uint(x) >> 23) & 255u) - 127;
    return x == 0.f ? 14 : min(max(e, -100), 127);
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// STATES: the first pass over a sequence's segments but the last, which keeps only what they add to the state.
// MORE: the grid has more CTAs than the GPU holds, and a CTA goes on with others' work.
template <typename T, int DK, bool STATES, bool MORE>
__global__ void __launch_bounds__(kChunkThreads, 1)
    linear_chunk_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using L = ChunkSmem<T, DK>;
    using M = Pair16<T>;
    constexpr bool BF = L::BF;
    constexpr int NT = L::NT;
    constexpr uint32_t PANEL = L::PANEL;
    constexpr uint32_t P_COL = 0, PW_COL = 128, OI_COL = 256, OA_COL = 320, U_COL = 384;  // (all 512 columns)
    constexpr uint32_t IDESC_P = umma_idesc_f16(BF, 128, kPiece, false);
    constexpr uint32_t IDESC_O = umma_idesc_f16(BF, 128, kSlice, true);
    constexpr uint32_t IDESC_U = umma_idesc_f16(BF, 128, kSlice * 2, true) | (1u << 15);  // A = K^T: M-major
    constexpr uint32_t IDESC_U3 = umma_idesc_f16(BF, 128, kSlice, true) | (1u << 15);     // bf16's third numbers
    constexpr uint32_t GATE_READERS = STATES ? 12 : 24;  // warps

    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    using Gates = typename L::Gates;
    Gates* gates = reinterpret_cast<Gates*>(smem + L::GATES);
    uint8_t* bad = smem + L::BAD;
    HalfScales& half = *reinterpret_cast<HalfScales*>(smem + L::HALF);  // (fp16 alone)
    int* any_bad = reinterpret_cast<int*>(smem + L::MISC);
    uint64_t* qk_full = reinterpret_cast<uint64_t*>(smem + L::BARS);  // [2] Q and K of a piece have landed
    uint64_t* v_full = qk_full + 2;                                   // [2]
    uint64_t* done = v_full + 2;       // [2] P, OI and OA of a piece are done: V, P' and results
    uint64_t* q_free = done + 2;       // [2] P and OI are
    uint64_t* k_free = q_free + 2;     // [2] U is
    uint64_t* v_clean = k_free + 2;    // [2] V's warps are through with a piece of V
    uint64_t* g_full = v_clean + 2;       // [2] gates
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
    uint64_t* all_done = role + 3;     // [2] every product a thread issued is done
    uint64_t* begun = all_done + 2;    // a segment's first state has been taken from V~'s place
    uint64_t* next_full = begun + 1;   // an answer has come
    uint64_t* work_full = next_full + 1;  // [2] work is written
    uint64_t* work_free = work_full + 2;  // [2] and read
    uint64_t* halves = work_free + 2;     // [4] fp16: the two warps of 32 rows of P have their largest
    uint32_t* taddr_s = reinterpret_cast<uint32_t*>(smem + L::TADDR);

    if (STATES) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the second pass may set itself up
    const LinearArgs& l = a.l;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t head = (size_t)DK * a.dv;
    if ((sbase & 1023u) != 0) {  // (the swizzled tiles need it; never seen)
        if (threadIdx.x == 0) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
        return;
    }
    ChunkWork* work = reinterpret_cast<ChunkWork*>(smem + L::WORK);
    // What CTA `block` of the grid has to do; valid: anything at all.
    auto work_of = [&](int block, bool report) -> ChunkWork {
        ChunkWork w;
        w.slice = block % a.slices;
        int unit = block / a.slices;
        w.h = unit % l.n_v;
        unit /= l.n_v;
        const int segs = STATES ? a.n_segs - 1 : a.n_segs;
        w.seg = unit % segs, w.s = unit / segs;
        const int q0 = l.q_start[w.s], q1 = l.q_start[w.s + 1];
        w.src = l.src[w.s], w.dst = l.dst[w.s];
        const bool bad_range = q0 < 0 || q1 < q0 || q1 > l.n_tokens || q1 - q0 > l.max_query;
        const bool bad_slot = w.src >= l.n_slots || w.dst >= l.n_slots;
        const bool bad_any = bad_range || bad_slot;
        if (bad_any && report && !STATES && w.h == 0 && w.slice == 0 && w.seg == 0)
            atomicOr(l.status, (bad_range ? (unsigned)PKV_DEV_BAD_QUERY_RANGE : 0u) |
                                   (bad_slot ? (unsigned)PKV_DEV_BAD_STATE_SLOT : 0u));
        // a sequence that fits fewer segments leaves the others nothing; its last keeps the state
        const int whole = bad_any ? 0 : q1 - q0;
        w.used_segs = whole > 0 ? (whole + a.seg_tokens - 1) / a.seg_tokens : 1;
        w.valid = !bad_any && w.seg < (STATES ? w.used_segs - 1 : w.used_segs);
        w.t0 = q0 + w.seg * a.seg_tokens;
        w.tokens = w.valid ? min(a.seg_tokens, q1 - w.t0) : 0;
        w.pieces = (w.tokens + kPiece - 1) / kPiece;
        if (!w.valid) w.src = w.dst = -1;  // (nothing read, nothing kept)
        return w;
    };
    const ChunkWork first = work_of(blockIdx.x, threadIdx.x == 0);
    if (!first.valid && !MORE) return;  // (otherwise the CTA may still take other work)
    if (threadIdx.x == 0) work[0] = first;
    const int seg = MORE ? 0 : first.seg;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&done[i], 1);
            mbar_init(&q_free[i], 1);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_clean[i], 8);
            mbar_init(&all_done[i], 1);
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
        mbar_init(begun, 4);
        mbar_init(next_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&work_full[i], 1);
            mbar_init(&work_free[i], 8 + 8 + 4 + 4 + 3);  // warps, or the one thread of a warp
        }
        for (int i = 0; i < 3; ++i) mbar_init(&role[i], i == 0 ? 8 : 4);
        if (!BF)
            for (int i = 0; i < 4; ++i) mbar_init(&halves[i], 2);
        fence_mbar_init();
    }
    if (threadIdx.x < 4 * 64) bad[threadIdx.x] = kPiece;
    if (threadIdx.x < 4) any_bad[threadIdx.x] = 0;
    if (warp == 25) tmem_alloc_cg<1>(taddr_s, 512);
    if (!STATES && a.n_segs > 1) grid_dependency_wait();  // the first pass is done
    if (!STATES && seg > 0) {
        // The state before a later segment: what those before leave, each decayed over the ones behind it. All threads
        // add it up, a thread's two or three places at once, a dozen loads in flight (9,005 tokens of 8 heads in 18 segments,
        // calls behind one another in a graph, 28.6 us; place after place 31.4; with a launch of its own for the sums 30).
        float4* to = reinterpret_cast<float4*>(smem + L::VT);
        const size_t step = (size_t)l.n_v * head, at0 = ((size_t)first.s * (a.n_segs - 1) * l.n_v + first.h);
        constexpr int QUADS = DK * kSlice / 4, E = (QUADS + kChunkThreads - 1) / kChunkThreads;
        const float* from[E];
        float4 sum[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int e = threadIdx.x + k * kChunkThreads;
            from[k] = a.added + at0 * head + (size_t)(e / (kSlice / 4)) * a.dv + first.slice * kSlice + e % (kSlice / 4) * 4;
            sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float since = 0.f;
#pragma unroll 4
        for (int i = seg - 1; i >= 0; --i) {
            const float w = ex2_approx(since);
            since += a.sums[at0 + (size_t)i * l.n_v];
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (threadIdx.x + k * kChunkThreads < QUADS) {
                    const float4 y = *reinterpret_cast<const float4*>(from[k] + i * step);
                    sum[k].x = fmaf(y.x, w, sum[k].x), sum[k].y = fmaf(y.y, w, sum[k].y);
                    sum[k].z = fmaf(y.z, w, sum[k].z), sum[k].w = fmaf(y.w, w, sum[k].w);
                }
        }
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (threadIdx.x + k * kChunkThreads < QUADS) to[threadIdx.x + k * kChunkThreads] = sum[k];
    }
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
    // The roles run on from work to work without a pause: behind the CTA's own that of CTAs of the grid that have not
    // started, whose launch the thread that issues the copies cancels for it. (Not where the GPU holds the whole grid at
    // once, as it does where sequences are shared out.)
    constexpr bool steal = MORE;
    int slice, h, s, used_segs, src, dst, t0, tokens, pieces;
    int base = 0;   // pieces of the work before: the phases go on
    int taken = 0;  // works before
    auto read = [&]() -> bool {
        const ChunkWork& w = work[taken & 1];
        slice = w.slice, h = w.h, s = w.s, used_segs = w.used_segs, src = w.src, dst = w.dst;
        t0 = w.t0, tokens = w.tokens, pieces = w.pieces;
        return w.valid || taken == 0;
    };
    auto begin = [&]() {
        read();
        if (steal) arrive_warp(&work_free[0]);
    };
    auto begin1 = [&]() {
        read();
        if (steal) mbar_arrive(&work_free[0]);
    };
    auto more = [&]() -> bool {  // whole warp
        base += pieces;
        if (!steal || !ok) return false;
        ++taken;
        if (!wait(&work_full[taken & 1], (taken - 1) >> 1)) { ok = false; return false; }
        const bool yes = read();
        arrive_warp(&work_free[taken & 1]);
        return yes;
    };
    auto more1 = [&]() -> bool {  // one thread
        base += pieces;
        if (!steal || !ok) return false;
        ++taken;
        if (!wait1(&work_full[taken & 1], (taken - 1) >> 1)) { ok = false; return false; }
        const bool yes = read();
        mbar_arrive(&work_free[taken & 1]);
        return yes;
    };

    if (warp < 8) {
        // ===================== weights of the pairs inside a piece: thread = row, half of its columns =====================
        registers_down<64>();
        if constexpr (!STATES) {
            begin();
            const int w4 = warp & 3, side = (warp >> 2) * 16;
            const int row = w4 * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
            const uint32_t from_col = lanes + P_COL + side;
            uint32_t to_col = lanes + PW_COL + side / 2;  // of two buffers
            uint32_t seen[8];  // bf16, of the block on the diagonal: the pairs of columns up to the row
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
                for (int b = w4 + 1; b < 4; ++b) put(b, zero), put(b + 4, zero);
            }
            do {
#pragma unroll 1
                for (int c = base; c < base + pieces; ++c) {
                    const Gates& g = gates[c & 1];
                    if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                    const float mine = BF ? -g.hi[row] : half.front[c & 1][row];
                    if (!wait(p_full, c)) { ok = false; break; }
                    tcgen05_after_sync();
                    float shift = 0.f;  // log2 of what the row is multiplied by
                    uint32_t p[16], w[8];
                    float* pf = reinterpret_cast<float*>(p);
                    // what the pairs of block b, at [.][side ..], are weighted by: 2^(the sum from the block's end to the row) = f
                    // times 2^(that from a token to the block's end)
                    auto weights = [&](int b, float f, uint64_t (&x)[8]) {
                        const uint64_t f2 = f2_pack(f, f);
                        const ulonglong2* gc = reinterpret_cast<const ulonglong2*>(&g.col[b * 32 + side]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const ulonglong2 y = gc[j];
                            x[2 * j] = f2_mul(y.x, f2), x[2 * j + 1] = f2_mul(y.y, f2);
                        }
                    };
                    float most = 0.f;  // fp16: the largest of the row, as weighted
                    if constexpr (!BF) {
                        float from = mine;
#pragma unroll 1
                        for (int b = w4 - 1; b >= 0; --b) {
                            tmem_ld16(from_col + b * 32, *reinterpret_cast<float(*)[16]>(pf));
                            uint64_t x[8];
                            weights(b, ex2_approx(from), x);
                            from += g.block[b];
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 y = f2_get(f2_mul(x[j], f2_pack(pf[2 * j], pf[2 * j + 1])));
                                most = fmax3(most, fabsf(y.x), fabsf(y.y));
                            }
                        }
                    }
                    tmem_ld16(from_col + w4 * 32, *reinterpret_cast<float(*)[16]>(pf));
                    // P' of the piece before the last has been read
                    if (c > 1 && !wait(&done[c & 1], (c >> 1) - 1)) { ok = false; break; }
                    to_col = lanes + PW_COL + (c & 1) * 64 + side / 2;
                    tcgen05_after_sync();
                    {  // the block on the diagonal: an exponential for each pair
                        const float hi = BF ? mine : -g.hi[row];
                        const uint64_t hi2 = f2_pack(hi, hi);
                        const ulonglong2* gh = reinterpret_cast<const ulonglong2*>(&g.hi[w4 * 32 + side]);
                        float x[16];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const ulonglong2 y = gh[j];
                            const float2 d0 = f2_get(f2_add(hi2, y.x)), d1 = f2_get(f2_add(hi2, y.y));
                            x[4 * j] = ex2_approx(d0.x), x[4 * j + 1] = ex2_approx(d0.y);
                            x[4 * j + 2] = ex2_approx(d1.x), x[4 * j + 3] = ex2_approx(d1.y);
                        }
                        if constexpr (!BF) {
                            const uint32_t forgotten = half.forgotten[c & 1][row] >> side;
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = forgotten & (1u << j) ? 0.f : x[j];
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 y = f2_get(f2_mul(f2_pack(x[2 * j], x[2 * j + 1]), f2_pack(pf[2 * j], pf[2 * j + 1])));
                            if constexpr (BF)
                                w[j] = M::pack(y.x, y.y) & seen[j];
                            else
                                pf[2 * j] = y.x, pf[2 * j + 1] = y.y;
                        }
                    }
                    if constexpr (!BF) {  // the row's largest, of both halves, goes to 2^14
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            pf[j] = j <= lane - side ? pf[j] : 0.f;
                            most = fmaxf(most, fabsf(pf[j]));
                        }
                        // (the other warp has read that of two pieces ago: it met since)
                        half.row_most[c & 1][side >> 4][row] = most;
                        arrive_warp(&halves[w4]);
                        if (!wait(&halves[w4], c)) { ok = false; break; }
                        const int e = exponent14(fmaxf(most, half.row_most[c & 1][(side >> 4) ^ 1][row]));
                        shift = (float)(14 - e);
                        if (side == 0) half.row_unit[c & 3][row] = pow2i(e - 14);
                        const uint64_t up = f2_pack(pow2i(14 - e), pow2i(14 - e));
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 y = f2_get(f2_mul(f2_pack(pf[2 * j], pf[2 * j + 1]), up));
                            w[j] = M::pack(y.x, y.y);
                        }
                    }
                    float from = mine + shift;  // the sum from the end of block b to the row
#pragma unroll 1
                    for (int b = w4 - 1; b >= 0; --b) {
                        tmem_ld16(from_col + b * 32, *reinterpret_cast<float(*)[16]>(pf));
                        put(b + 1, w);
                        uint64_t x[8];
                        weights(b, ex2_approx(from), x);
                        from += g.block[b];
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
            } while (more());
        }
    } else if (warp < 16) {
        // ===================== V~: 32 rows at a time, four threads a row =====================
        registers_down<MORE ? 64 : 56>();
        begin();
        const int tid = threadIdx.x - 256;
        const int odd = tid >> 7;  // quarters 0 and 2, or 1 and 3
        const int r = (tid & 127) >> 2;
        // which four 16-byte units of its row: two threads' rows share the banks of half a row otherwise
        const int u0 = (tid & 3) + 4 * (r & 1);
        const uint32_t at[2] = {(uint32_t)((u0 ^ (r & 7)) << 4), (uint32_t)((u0 ^ 4 ^ (r & 7)) << 4)};
        do {
#pragma unroll 1
            for (int c = base; c < base + pieces; ++c) {
                const int st = c & 1;
                const int n = min(kPiece, tokens - (c - base) * kPiece);
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
                float unit = 1.f;
                if constexpr (!BF) {  // the largest number of V~ goes to 2^14
                    float most = 0.f;
#pragma unroll 1
                    for (int q = odd; q < 4; q += 2) {
                        const unsigned char* from = v + (q * 32 + r) * 128;
                        uint4 x[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
                        uint32_t top = largest_half(x);
                        if (top >= 0x7c00u) {  // one is not finite
                            top = 0;
#pragma unroll 1
                            for (int j = 0; j < 16; ++j) {
                                const uint32_t y = reinterpret_cast<const uint16_t*>(from + (j < 8 ? at[0] : at[1]))[j & 7] & 0x7fffu;
                                top = max(top, y < 0x7c00u ? y : 0u);
                            }
                        }
                        most = fmaxf(most, g.col[q * 32 + r] * g.after[q] * __half2float(__ushort_as_half((unsigned short)top)));
                    }
                    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));  // (not negative)
                    if (lane == 0) half.v_most[c & 1][warp - 8] = most;
                    if (!meet(0)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = fmaxf(most, half.v_most[c & 1][i]);
                    const int e = exponent14(most);
                    unit = pow2i(14 - e);
                    if (tid == 0) half.v_back[c & 3] = pow2i(e - 14);  // (the state's warps have read that of four pieces ago)
                }
#pragma unroll 1
                for (int q = odd; q < 4; q += 2) {
                    const int row = q * 32 + r;
                    unsigned char* from = v + row * 128;
                    uint4 x[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
                    const float f = g.col[row] * g.after[q] * unit;
                    const uint64_t f2 = f2_pack(f, f);
                    if (c > 0 ? !wait(&vt_free[q], c - 1) : !STATES && seg > 0 && !wait(begun, 0)) { ok = false; break; }
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
                if (lane == 0) {
                    mbar_arrive(&v_clean[st]);
                    mbar_arrive(&g_free[st]);
                }
            }
        } while (more());
    } else if (warp < 20) {
        // ===================== the state: thread = row of dim_k (half a row at dim_k = 64) =====================
        registers_up<128>();
        begin();
        constexpr int NC = DK == 128 ? 64 : 32;
        const int tid = threadIdx.x - 512;
        const int row = tid & (DK - 1);
        const int c0 = DK == 128 ? 0 : (tid >> 6) * 32;
        const uint32_t lanes = tmem + ((uint32_t)((warp - 16) * 32) << 16);
        size_t at;  // in a head's state
        uint64_t x[NC / 2];  // pairs of columns
        auto load = [&](const float* from) {
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float4 y = *reinterpret_cast<const float4*>(from + 2 * i);
                x[i] = f2_pack(y.x, y.y);
                x[i + 1] = f2_pack(y.z, y.w);
            }
        };
        auto save = [&](float* to) {
#pragma unroll
            for (int i = 0; i < NC / 2; i += 2) {
                const float2 y = f2_get(x[i]), z = f2_get(x[i + 1]);
                *reinterpret_cast<float4*>(to + at + 2 * i) = make_float4(y.x, y.y, z.x, z.y);
            }
        };
        do {
            at = (size_t)row * a.dv + slice * kSlice + c0;
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) x[i] = 0;
            if (seg == 0) {
                // shared out, the second pass reads the start from where the first left it: its last segment writes dst
                const size_t mine = (size_t)s * l.n_v + h;
                const bool from_state = STATES || used_segs == 1;
                if (!from_state || src >= 0)
                    load((from_state ? l.state + ((size_t)src * l.n_v + h) * head : a.start + mine * head) + at);
                if (STATES) save(a.start + mine * head);
            } else if (!STATES) {
                load(reinterpret_cast<const float*>(smem + L::VT) + row * kSlice + c0);
                arrive_warp(begun);
            }
            float sum = 0.f;
            // fp16: the largest and the smallest of the row, kept up to date as the row is written (two of each, as such chains are
            // long)
            float row_most[2], row_least[2];
            auto none_yet = [&]() { row_most[0] = row_most[1] = 0.f, row_least[0] = row_least[1] = 3.4028234e38f; };
            auto count = [&](int i) {
                const float2 y = f2_get(x[i]);
                row_most[i & 1] = fmax3(row_most[i & 1], fabsf(y.x), fabsf(y.y));
                row_least[i & 1] = fmin3(row_least[i & 1], fabsf(y.x), fabsf(y.y));
            };
            if (!BF && !STATES) {
                none_yet();
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) count(i);
            }
#pragma unroll 1
            for (int c = base; c < base + pieces; ++c) {
                if constexpr (!STATES) {  // the copy that Q meets
                    unsigned char* to = smem + L::S + row * 128;
                    auto copy = [&](auto up) {  // up(i): what pair i of columns is multiplied by
#pragma unroll
                        for (int i = 0; i < NC / 2; i += 4) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 y = f2_get(BF ? x[i + j] : f2_mul(x[i + j], up(i + j)));
                                w[j] = M::pack(y.x, y.y);
                            }
                            *reinterpret_cast<uint4*>(to + ((((c0 + 2 * i) >> 3) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    };
                    if constexpr (BF) {
                        if (c > 0 && !wait(s_free, c - 1)) { ok = false; break; }
                        copy([](int) { return uint64_t(0); });
                    } else {
                        // One power of two for all columns serves where each has a number of 2^-16 of the largest: what is lost
                        // below fp16's normal numbers is then 2^-23 of a column's largest. That is so where a row has no
                        // smaller ones, which costs a comparison a number. (A column's own largest, always: packed prompts
                        // 234 us for 193.)
                        float most = warp_most(fmaxf(row_most[0], row_most[1]));
                        const float least = warp_most(fminf(row_least[0], row_least[1]));
                        float(*part)[2] = half.s_most[c & 1];  // (read for piece c by all before any of them meets for c + 1)
                        if (lane == 0) part[warp - 16][0] = most, part[warp - 16][1] = least;
                        if (!meet(1)) { ok = false; break; }
                        most = fmaxf(fmaxf(part[0][0], part[1][0]), fmaxf(part[2][0], part[3][0]));
                        const float l0 = fmaxf(part[0][1], part[1][1]), l1 = fmaxf(part[2][1], part[3][1]);
                        // (at dim_k = 64 two warps have one half of the columns, two the other)
                        const bool one = (DK == 128 ? fmaxf(l0, l1) : fminf(l0, l1)) >= most * 0x1p-16f;
                        // (of four buffers each: the results of four pieces ago have been read)
                        if (tid == 0) half.s_columns[c & 3] = !one;
                        if (one) {
                            const int e = exponent14(most);
                            if (tid == 0) half.s_back[c & 3] = pow2i(e - 14);
                            if (c > 0 && !wait(s_free, c - 1)) { ok = false; break; }
                            const uint64_t unit2 = f2_pack(pow2i(14 - e), pow2i(14 - e));
                            copy([&](int) { return unit2; });
                        } else {  // nothing of an infinite or far larger column may reach another
#pragma unroll
                            for (int i = 0; i < NC / 2; i += 2) {
                                const float2 y = f2_get(x[i]), z = f2_get(x[i + 1]);
                                const float4 m = make_float4(warp_most(y.x), warp_most(y.y), warp_most(z.x), warp_most(z.y));
                                if (lane == 0) *reinterpret_cast<float4*>(&half.col_most[warp - 16][c0 + 2 * i]) = m;
                            }
                            if (!meet(1)) { ok = false; break; }
                            if (tid < kSlice) {
                                const float(*m)[kSlice] = &half.col_most[DK == 128 ? 0 : tid >> 5 << 1];
                                most = fmaxf(m[0][tid], m[1][tid]);
                                if (DK == 128) most = fmaxf(most, fmaxf(m[2][tid], m[3][tid]));
                                const int e = exponent14(most);
                                half.col_up[tid] = pow2i(14 - e);
                                half.col_back[c & 3][tid] = pow2i(e - 14);
                            }
                            if (!meet(1)) { ok = false; break; }
                            if (c > 0 && !wait(s_free, c - 1)) { ok = false; break; }
                            const uint64_t* up = reinterpret_cast<const uint64_t*>(&half.col_up[c0]);
                            copy([&](int i) { return up[i]; });
                        }
                    }
                    fence_proxy_async_smem();
                    arrive_warp(s_full);
                }
                const Gates& g = gates[c & 1];
                if (!wait(&g_full[c & 1], c >> 1)) { ok = false; break; }
                const uint64_t keep = f2_pack(g.keep, g.keep), once = f2_pack(g.once, g.once);
                if (STATES) sum += g.sum;
                arrive_warp(&g_free[c & 1]);
                if (!wait(u_full, c)) { ok = false; break; }
                tcgen05_after_sync();
                const float back = BF ? 1.f : half.v_back[c & 3], back2 = back / kSecond;
                if (!BF && !STATES) none_yet();
#pragma unroll
                for (int i = 0; i < NC / 2; i += 8) {
                    float u[2][16];  // the first numbers' product, and the others'
#pragma unroll
                    for (int term = 0; term < 2; ++term) tmem_ld16(lanes + U_COL + 64 * term + c0 + 2 * i, u[term]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint64_t first = f2_pack(u[0][2 * j], u[0][2 * j + 1]), other = f2_pack(u[1][2 * j], u[1][2 * j + 1]);
                        const uint64_t y = BF ? f2_add(first, other)
                                              : f2_fma(first, f2_pack(back, back), f2_mul(other, f2_pack(back2, back2)));
                        x[i + j] = f2_fma(x[i + j], keep, f2_fma(x[i + j], once, y));
                        if (!BF && !STATES) count(i + j);
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
        } while (more());
    } else if (warp < 24) {
        // ===================== results: thread = row =====================
        if constexpr (!MORE) registers_up<88>();
        if constexpr (!STATES) {
            begin();
            const int w4 = warp - 20;
            const int row = w4 * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
            const size_t pitch = (size_t)l.n_v * a.dv * sizeof(T);
            float sum = 0.f;  // of the log decays up to the row
            auto decays = [&](int c) -> bool {
                if (!wait(&g_full[c & 1], c >> 1)) return false;
                const Gates& g = gates[c & 1];
                sum = BF ? -g.hi[row] : half.front[c & 1][row];
#pragma unroll 1
                for (int i = 0; i < w4; ++i) sum += g.block[i];
                arrive_warp(&g_free[c & 1]);
                return true;
            };
            const bool sectors = (reinterpret_cast<uintptr_t>(l.out) & 31) == 0;
            do {
                char* out = static_cast<char*>(l.out) + (size_t)(t0 + row) * pitch + ((size_t)h * a.dv + slice * kSlice) * sizeof(T);
                if (pieces > 0) ok = decays(base);
#pragma unroll 1
                for (int c = base; c < base + pieces && ok; ++c) {
                    const int n = min(kPiece, tokens - (c - base) * kPiece);
                    if (!wait(&done[c & 1], c >> 1)) { ok = false; break; }
                    tcgen05_after_sync();
                    float fi = ex2_approx(sum) * l.scale, fa = l.scale;
                    if (c + 1 < base + pieces && !decays(c + 1)) { ok = false; break; }  // (early: their buffer is waited for)
                    bool columns = false;
                    if constexpr (!BF) {
                        columns = half.s_columns[c & 3];
                        if (!columns) fi *= half.s_back[c & 3];
                        fa *= half.row_unit[c & 3][row];
                    }
                    const uint64_t fi2 = f2_pack(fi, fi), fa2 = f2_pack(fa, fa);
                    const bool poisoned = any_bad[c & 3] != 0;
                    // All of a row is read before any of it is stored, for the next product waits for that (117 us for 64 pieces,
                    // in slices 142); where a CTA goes on with other work, whose loop wants registers too, in slices (packed
                    // prompts 277 us, whole 317).
                    // A slice of 16 columns, words at w0 .. of w; factor(j): what pair j of OI's columns is multiplied by.
                    auto slice_of = [&](int c0, auto& w, int w0, auto factor) {
                        float x[16], y[16];
                        tmem_ld16(lanes + OI_COL + c0, x);
                        tmem_ld16(lanes + OA_COL + c0, y);
                        tmem_wait_ld();
                        if (c0 + 16 == kSlice) {
                            tcgen05_before_sync();
                            arrive_warp(o_free);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 z = f2_get(f2_fma(f2_pack(x[j], x[j + 1]), factor(c0 + j), f2_mul(f2_pack(y[j], y[j + 1]), fa2)));
                            w[w0 + j / 2] = M::pack(z.x, z.y);
                        }
                        if (poisoned) {
                            const uint8_t* mark = &bad[(c & 3) * 64 + c0];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (mark[j] <= row) w[w0 + j / 2] |= 0x7fffu << (16 * (j & 1));
                        }
                    };
                    auto out_words = [&](char* to, auto& w) {
                        constexpr int WORDS = sizeof(w) / 4;
                        if (row < n) {
                            if (sectors) {
#pragma unroll
                                for (int j = 0; j < WORDS; j += 8)
                                    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + j * 4), "r"(w[j]),
                                                 "r"(w[j + 1]), "r"(w[j + 2]), "r"(w[j + 3]), "r"(w[j + 4]), "r"(w[j + 5]),
                                                 "r"(w[j + 6]), "r"(w[j + 7])
                                                 : "memory");
                            } else {
#pragma unroll
                                for (int j = 0; j < WORDS; j += 4)
                                    *reinterpret_cast<uint4*>(to + j * 4) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                            }
                        }
                    };
                    if (!BF && columns) {
#pragma unroll 1
                        for (int c0 = 0; c0 < kSlice; c0 += 16) {
                            uint32_t w[8];
                            const float* back = half.col_back[c & 3];
                            slice_of(c0, w, 0, [&](int j) { return f2_mul(fi2, *reinterpret_cast<const uint64_t*>(back + j)); });
                            out_words(out + c0 * sizeof(T), w);
                        }
                    } else if constexpr (MORE) {
#pragma unroll 1
                        for (int c0 = 0; c0 < kSlice; c0 += 16) {
                            uint32_t w[8];
                            slice_of(c0, w, 0, [&](int) { return fi2; });
                            out_words(out + c0 * sizeof(T), w);
                        }
                    } else {
                        uint32_t w[kSlice / 2];
#pragma unroll
                        for (int c0 = 0; c0 < kSlice; c0 += 16) slice_of(c0, w, c0 / 2, [&](int) { return fi2; });
                        out_words(out, w);
                    }
                    out += kPiece * pitch;
                    if (poisoned) {  // the columns' marks are used again four pieces on
                        if (!meet(2)) { ok = false; break; }
                        if (row < 64) bad[(c & 3) * 64 + row] = kPiece;
                        if (row == 0) any_bad[c & 3] = 0;
                    }
                }
            } while (more());
        }
    } else {
        registers_down<48>();  // (one instruction for the four warps)
        if (warp == 24) {
            // ===================== tensor copies =====================
            if (lane == 0) {
                int issued_qk = 0, issued = 0;
                read();
                while (true) {
                    const int hq = h / (l.n_v / l.n_qk);
#pragma unroll 1
                    for (int c = base; c < base + pieces; ++c) {
                        const int st = c & 1;
                        const int y = t0 + (c - base) * kPiece;
                        if (c >= 2 && ((!STATES && !wait1(&q_free[st], (c >> 1) - 1)) || !wait1(&k_free[st], (c >> 1) - 1))) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&qk_full[st], (STATES ? 1 : 2) * L::QK);
#pragma unroll 1
                        for (int p = 0; p < DK / 64; ++p) {
                            tma_rows(sbase + L::K + st * L::QK + p * PANEL, &tm_k, hq * DK + p * 64, y, &qk_full[st]);
                            if (!STATES) tma_rows(sbase + L::Q + st * L::QK + p * PANEL, &tm_q, hq * DK + p * 64, y, &qk_full[st]);
                        }
                        issued_qk = c + 1;
                        if (!STATES && c >= 2 && !wait1(&done[st], (c >> 1) - 1)) { ok = false; break; }
                        mbar_arrive_expect_tx(&v_full[st], PANEL);
                        tma_rows(sbase + L::V + st * PANEL, &tm_v, h * a.dv + slice * kSlice, y, &v_full[st]);
                        issued = c + 1;
                    }
                    base += pieces;
                    if (!steal || !ok) break;
                    // Ask for the work behind this one now that its last copies are issued, two pieces before it ends. (Asked at
                    // the front of the work, the first CTAs took work from some that were about to start.)
                    mbar_arrive_expect_tx(next_full, 16);
                    asm volatile(
                        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                            sbase + L::NEXT),
                        "r"(smem_addr(next_full))
                        : "memory");
                    if (!wait1(next_full, taken)) { ok = false; break; }
                    uint32_t yes, block;
                    asm volatile(
                        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
                        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                        : "=r"(yes), "=r"(block)
                        : "r"(sbase + L::NEXT)
                        : "memory");
                    fence_proxy_async_smem();  // (the next answer is written there)
                    ++taken;
                    if (taken >= 2 && !wait1(&work_free[taken & 1], (taken >> 1) - 1)) { ok = false; break; }
                    ChunkWork w;
                    w.valid = 0;
                    if (yes) {
                        w = work_of((int)block, true);
                        w.valid = 1;  // (work, if only to be skipped)
                    }
                    work[taken & 1] = w;
                    mbar_arrive(&work_full[taken & 1]);
                    if (!yes) break;
                    read();
                }
                // no copy is in flight when the CTA leaves
                for (int c = max(issued - 2, 0); c < issued_qk; ++c) {
                    ok = wait1(&qk_full[c & 1], c >> 1) && ok;
                    if (c < issued) ok = wait1(&v_full[c & 1], c >> 1) && ok;
                }
            }
            __syncwarp();
        } else if (warp == 25) {
            // ===================== products P, OI and OA: one thread =====================
            if (!STATES && elect_one()) {
                const uint64_t dq = umma_desc_sw128(sbase + L::Q, 16, 1024);
                const uint64_t dk = umma_desc_sw128(sbase + L::K, 16, 1024);
                const uint64_t dv = umma_desc_sw128(sbase + L::V, PANEL, 1024);
                const uint64_t ds = umma_desc_sw128(sbase + L::S, DK * 128, 1024);
                begin1();
                do {
                    for (int c = base - 1; c < base + pieces; ++c) {
                        const uint32_t st = (uint32_t)(c & 1);
                        if (c >= base) {  // OI = Q S
                            if (!wait1(s_full, c) || (c > 0 && !wait1(o_free, c - 1))) { ok = false; break; }
                            tcgen05_after_sync();
                            const uint64_t q = dq + ((st * L::QK) >> 4);
#pragma unroll
                            for (int i = 0; i < DK / 16; ++i)
                                umma_f16_cg<1>(tmem + OI_COL, q + (((uint32_t)(i >> 2) * PANEL + (uint32_t)(i & 3) * 32) >> 4),
                                               ds + (uint32_t)i * (2048 >> 4), IDESC_O, i > 0);
                            umma_commit_cg<1>(s_free);
                            umma_commit_cg<1>(&q_free[st]);
                            if (!wait1(w_full, c)) { ok = false; break; }
                        }
                        if (c + 1 < base + pieces) {  // P = Q K^T of the next piece
                            if (!wait1(&qk_full[st ^ 1], (c + 1) >> 1)) { ok = false; break; }
                            const uint64_t q = dq + (((st ^ 1) * L::QK) >> 4), k = dk + (((st ^ 1) * L::QK) >> 4);
                            tcgen05_after_sync();
#pragma unroll
                            for (int i = 0; i < DK / 16; ++i) {
                                const uint32_t off = ((uint32_t)(i >> 2) * PANEL + (uint32_t)(i & 3) * 32) >> 4;
                                umma_f16_cg<1>(tmem + P_COL, q + off, k + off, IDESC_P, i > 0);
                            }
                            umma_commit_cg<1>(p_full);
                        }
                        if (c >= base) {  // OA = P' V
                            if (!wait1(&v_clean[st], c >> 1)) { ok = false; break; }
                            tcgen05_after_sync();
                            const uint64_t v = dv + ((st * PANEL) >> 4);
#pragma unroll
                            for (int i = 0; i < kPiece / 16; ++i)
                                umma_f16_tmem_a_cg<1>(tmem + OA_COL, tmem + PW_COL + st * 64 + i * 8, v + (uint32_t)i * (2048 >> 4),
                                                      IDESC_O, i > 0);
                            umma_commit_cg<1>(&done[st]);
                        }
                    }
                } while (more1());
                // every product is done before tensor memory is given back
                umma_commit_cg<1>(&all_done[0]);
                ok = wait1(&all_done[0], 0) && ok;
                if (!ok) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
            }
            __syncwarp();
        } else if (warp == 26) {
            // ===================== product U = K^T V~: one thread =====================
            if (elect_one()) {
                // K^T: 64 rows of the product a panel; at dim_k = 64 the second 64 are the first again
                const uint64_t dkt = umma_desc_sw128(sbase + L::K, DK == 128 ? PANEL : 0, 1024);
                const uint64_t dvt = umma_desc_sw128(sbase + L::VT, 4096, 1024);
                begin1();
                do {
                    for (int c = base; c < base + pieces && ok; ++c) {
                        const uint32_t st = (uint32_t)(c & 1);
                        if (!wait1(&qk_full[st], c >> 1) || (c > 0 && !wait1(u_free, c - 1))) { ok = false; break; }
                        uint64_t kt = dkt + ((st * L::QK) >> 4), vt = dvt;
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            if (!wait1(&vt_full[q], c)) { ok = false; break; }
                            tcgen05_after_sync();
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint64_t ka = kt + k * (2048 >> 4), vb = vt + k * (2048 >> 4);
                                umma_f16_cg<1>(tmem + U_COL, ka, vb, IDESC_U, q > 0 || k > 0);
                                if (NT == 3) umma_f16_cg<1>(tmem + U_COL + 64, ka, vb + (2 * 4096 >> 4), IDESC_U3, true);
                            }
                            umma_commit_cg<1>(&vt_free[q]);
                            kt += 4096 >> 4, vt += L::QUARTER >> 4;
                        }
                        if (!ok) break;
                        umma_commit_cg<1>(u_full);
                        umma_commit_cg<1>(&k_free[st]);
                    }
                } while (more1());
                umma_commit_cg<1>(&all_done[1]);
                ok = wait1(&all_done[1], 0) && ok;
                if (!ok) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
            }
            __syncwarp();
        } else {
            // ===================== sums of the log decays: lane = four tokens, eight lanes a block of 32 =====================
            // Sums from a block's front and from its back are added up apart: a difference of two front sums would lose
            // what comes behind a token that forgets. The pairs inside a block do take a difference of two front sums. For fp16
            // those begin anew behind a token that forgets, and what it makes forgotten is masked. bf16, which has no room
            // left for that, bears it: 32 that forget make sums of -4,800, whose last bit is 2^-11, and so its weights are
            // off by up to 2^-10 where they are rounded by 2^-9 (as are fp16's in a block of 32 decays of 2^-140 each).
            const int sub = lane & 7;
            float raw[4];
            auto fetch = [&](int c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = c * kPiece + lane * 4 + i;
                    raw[i] = l.log_decay && t < tokens ? l.log_decay[(size_t)(t0 + t) * l.decay_stride + h] : 0.f;
                }
            };
            begin();
            do {
                fetch(0);
#pragma unroll 1
                for (int c = base; c < base + pieces; ++c) {
                    float y[4], front[4], back[4], all[4];
                    uint32_t forgets = 0;  // fp16: of the lane's four
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // 2^-150 is 0 in fp32, 2^(10^4) infinite: a token that forgets (-infinity) takes part in sums; NaN stays
                        if (!BF && raw[i] < -104.f) forgets |= 1u << i;
                        y[i] = raw[i] < -104.f ? -104.f : raw[i];
                        y[i] = (y[i] > 1e4f ? 1e4f : y[i]) * 1.44269504f;
                    }
                    if (c + 1 < base + pieces) fetch(c + 1 - base);
                    // sums over the block's lanes up to this one and from it on, then those before and behind it
                    float up = (y[0] + y[1]) + (y[2] + y[3]), down = up;
#pragma unroll
                    for (int o = 1; o < 8; o *= 2) {
                        const float f = __shfl_up_sync(0xffffffffu, up, o, 8), k = __shfl_down_sync(0xffffffffu, down, o, 8);
                        if (sub >= o) up += f;
                        if (sub + o < 8) down += k;
                    }
                    up = __shfl_up_sync(0xffffffffu, up, 1, 8), down = __shfl_down_sync(0xffffffffu, down, 1, 8);
                    front[0] = (sub > 0 ? up : 0.f) + y[0];
                    back[3] = sub < 7 ? down : 0.f;
#pragma unroll
                    for (int i = 1; i < 4; ++i) front[i] = front[i - 1] + y[i], back[3 - i] = back[4 - i] + y[4 - i];
#pragma unroll
                    for (int b = 0; b < 4; ++b) all[b] = __shfl_sync(0xffffffffu, front[3], b * 8 + 7);
                    if (c >= 2 && !wait(&g_free[c & 1], (c >> 1) - 1)) { ok = false; break; }
                    Gates& g = gates[c & 1];
                    if constexpr (!BF) {
                        *reinterpret_cast<float4*>(&half.front[c & 1][lane * 4]) = make_float4(front[0], front[1], front[2], front[3]);
                        uint32_t gone[4] = {0u, 0u, 0u, 0u};
                        if (__any_sync(0xffffffffu, forgets != 0)) {
                            uint32_t block = forgets << sub * 4;  // of the block's 32
#pragma unroll
                            for (int o = 1; o < 8; o *= 2) block |= __shfl_xor_sync(0xffffffffu, block, o);
                            const uint32_t before = block & ((1u << sub * 4) - 1);  // in lanes before this one
                            const int last = forgets ? sub : before ? (31 - __clz(before)) / 4 : 0;  // the lane of the last
                            // sums from behind the last one: over the lane, then from lane to lane
                            float since = 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) since = forgets & (1u << i) ? 0.f : since + y[i];
#pragma unroll
                            for (int o = 1; o < 8; o *= 2) {
                                const float f = __shfl_up_sync(0xffffffffu, since, o, 8);
                                if (sub - last >= o) since += f;
                            }
                            since = __shfl_up_sync(0xffffffffu, since, 1, 8);
                            if (sub == 0) since = 0.f;
                            uint32_t mask = before ? (1u << (31 - __clz(before))) - 1 : 0u;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                since += y[i];
                                if (forgets & (1u << i)) since = 0.f, mask = (1u << (sub * 4 + i)) - 1;
                                front[i] = since;
                                gone[i] = mask;
                            }
                        }
                        *reinterpret_cast<uint4*>(&half.forgotten[c & 1][lane * 4]) = make_uint4(gone[0], gone[1], gone[2], gone[3]);
                    }
                    *reinterpret_cast<float4*>(&g.hi[lane * 4]) = make_float4(-front[0], -front[1], -front[2], -front[3]);
                    *reinterpret_cast<float4*>(&g.col[lane * 4]) =
                        make_float4(ex2_approx(back[0]), ex2_approx(back[1]), ex2_approx(back[2]), ex2_approx(back[3]));
                    const float sum = (all[0] + all[1]) + (all[2] + all[3]);
                    if (lane < 4) {
                        g.block[lane] = lane == 0 ? all[0] : lane == 1 ? all[1] : lane == 2 ? all[2] : all[3];
                        g.after[lane] = ex2_approx(lane == 0 ? all[1] + (all[2] + all[3]) : lane == 1 ? all[2] + all[3] : lane == 2 ? all[3] : 0.f);
                    } else if (lane == 4) {
                        const bool small = sum > -0.7f && sum < 0.7f;
                        g.keep = small ? expm1f(sum * 0.693147181f) : ex2_approx(sum);
                        g.once = small ? 1.f : 0.f;
                        g.sum = sum;
                    }
                    arrive_warp(&g_full[c & 1]);
                }
            } while (more());
        }
    }
    if (!ok && lane == 0) atomicOr(l.status, (unsigned)PKV_DEV_WAIT_TIMEOUT);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 25) tmem_dealloc_cg<1>(tmem, 512);
}

template <typename T, int DK, bool STATES, bool MORE>
cudaError_t run_chunk(const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      cudaStream_t stream) {
    static unsigned long long attr_done = 0;  // one bit a device
    constexpr uint32_t smem = ChunkSmem<T, DK>::ALLOC;
    auto kern = linear_chunk_kernel<T, DK, STATES, MORE>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (!(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        __atomic_fetch_or(&attr_done, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    const unsigned segs = STATES ? a.n_segs - 1 : a.n_segs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.l.n_seqs * segs * a.l.n_v * a.slices);
    cfg.blockDim = dim3(kChunkThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = !STATES && a.n_segs > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, q, k, v);
}

template <typename T, int DK>
cudaError_t launch_linear_chunk_dim(const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    cudaStream_t stream) {
    if (a.take_more) return run_chunk<T, DK, false, true>(a, q, k, v, stream);
    if (a.n_segs > 1) {
        const cudaError_t err = run_chunk<T, DK, true, false>(a, q, k, v, stream);
        if (err != cudaSuccess) return err;
    }
    return run_chunk<T, DK, false, false>(a, q, k, v, stream);
}

template <typename T>
cudaError_t launch_linear_chunk_dtype(int dk, const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                      const CUtensorMap& v, cudaStream_t stream) {
    return dk == 64 ? launch_linear_chunk_dim<T, 64>(a, q, k, v, stream) : launch_linear_chunk_dim<T, 128>(a, q, k, v, stream);
}

}  // namespace pkv
