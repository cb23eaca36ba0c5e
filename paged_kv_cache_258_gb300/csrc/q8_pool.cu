// q8_pool.cu -- 8-bit pools: quantising append, block copies, widening of rows for prefill (sm_103a).
//
// A code is an e4m3 number (1 sign, 4 exponent, 3 mantissa bits; largest 448), a value is code * S with
// one power of two S for each (block, KV head) of each of K and V. Why a power of two: e4m3 rounds
// relative to the value, so within its 15 binades any other scale rounds no better, and with a power of
// two x / S is exact, widening is exact, and raising a block's scale only moves the exponents of its
// codes -- codes are rounded again only where they fall below 2^-6. The scale is the least that lets the
// largest finite element of the block in.
//
// Append: a block's scale is raised once for all the call's rows in it, so somebody has to see these rows
// together. A CTA takes a window of 16 tokens, one KV head and K or V, and the runs that start there: a
// token whose block none of the 31 before it lies in starts a run, the tokens of that block up to 31
// later belong to it. Each warp reads whole rows (all of a CTA's rows are in flight at once), the
// largest elements meet in shared memory, and the warps write their rows as codes of the run's scale.
// A block is started when a row at offset 0 arrives: its old scale, the previous owner's, is forgotten.
// Otherwise S' = max(S, what the new rows need) and, if that grew, the other rows are brought to S'.
// Bound by latency in a decode step (three dependent trips to memory; 64 rows of 32 heads x 128 5.1 us), by issue and
// barriers in a long chunk (2,432 rows of 4 x 256 8 us, 15 MB: 2.4 instructions a cycle and SM, DRAM at 9 %).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "shrink.h"

namespace pkv {
namespace {

constexpr float kMaxFinite = 3.4028234e38f;

// Two floats -> two e4m3 codes (lo in the low byte), round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes -> two floats (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
    uint32_t h;
    const uint16_t c = (uint16_t)w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// The least power of two S >= 2^min_exp with amax <= 448 S (448 = 1.75 * 2^8), as its exponent.
__device__ __forceinline__ int scale_exp(float amax, int min_exp) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, min_exp);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

constexpr int kWindow = 16;                  // tokens whose runs a CTA looks for
constexpr int kReach = 31;                   // how far behind its first token a run may end
constexpr int kSeen = kWindow + kReach;      // tokens that may belong to a CTA's runs
constexpr int kAppendWarps = 8;

// EPL elements of a lane, as loaded.
template <int EPL>
struct Piece;
template <>
struct Piece<2> {
    using raw = uint32_t;
    using codes = uint16_t;
};
template <>
struct Piece<4> {
    using raw = uint2;
    using codes = uint32_t;
};
template <>
struct Piece<8> {
    using raw = uint4;
    using codes = uint2;
};

template <typename T>
__device__ __forceinline__ void widen_word(uint32_t w, float* f) {
    Vec16<T>::word(w, f);
}

// grid: (window, KV head, K or V)
template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) q8_append_kernel(const Q8AppendArgs a) {
    constexpr int EPL = D / 32;
    constexpr int WORDS = EPL / 2;
    constexpr int ROWS = (kSeen + kAppendWarps - 1) / kAppendWarps;  // rows of a warp
    using Raw = typename Piece<EPL>::raw;
    using Codes = typename Piece<EPL>::codes;
    __shared__ long long s_slot[kReach + kSeen];  // of tokens first - 31 .. first + 46; -1: none, padding or bad
    __shared__ int s_run[kSeen];                  // the window's token that starts this token's run, or -1
    __shared__ int s_leader[kWindow];
    __shared__ unsigned s_rows[kWindow];          // offsets a run writes
    __shared__ unsigned s_amax[kWindow];
    __shared__ float s_inv[kWindow], s_ratio[kWindow];  // 1 / S', and S / S' where the other rows need it (else 0)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = 2 * a.n_kv;
    const long long window = blockIdx.x / parts;
    const int part = (int)(blockIdx.x % parts);
    const bool is_v = part >= a.n_kv;
    const int g = is_v ? part - a.n_kv : part;
    const long long first = window * kWindow;
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x < kReach + kSeen) {
        const long long t = first - kReach + threadIdx.x;
        long long slot = t >= 0 && t < a.n_tok ? a.slots[t] : -1;
        if (slot >= (long long)a.num_blocks * kBlock) {
            if (part == 0 && threadIdx.x >= kReach) atomicOr(a.status, (unsigned)PKV_DEV_BAD_SLOT);
            slot = -1;
        }
        s_slot[threadIdx.x] = slot < 0 ? -1 : slot;
    }
    if (threadIdx.x < kSeen) s_run[threadIdx.x] = -1;
    if (threadIdx.x < kWindow) s_rows[threadIdx.x] = s_amax[threadIdx.x] = 0u;
    __syncthreads();
    {  // half a warp per token of the window: does its block lie among the 31 before?
        const int u = threadIdx.x >> 4, l = threadIdx.x & 15;
        const long long slot = s_slot[kReach + u];
        bool seen = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int back = 1 + l + 16 * i;
            if (back <= kReach && slot >= 0) {
                const long long other = s_slot[kReach + u - back];
                seen = seen || (other >= 0 && other / kBlock == slot / kBlock);
            }
        }
        const unsigned b = __ballot_sync(0xffffffffu, seen);
        if (l == 0) s_leader[u] = slot >= 0 && ((b >> (lane & 16)) & 0xffffu) == 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kSeen * kWindow; i += kAppendWarps * 32) {
        const int u = i / kWindow, l = i % kWindow;
        const long long slot = s_slot[kReach + u];
        if (u >= l && u - l <= kReach && slot >= 0 && s_leader[l] && s_slot[kReach + l] / kBlock == slot / kBlock) {
            s_run[u] = l;
            atomicOr(&s_rows[l], 1u << (slot % kBlock));
        }
    }
    __syncthreads();

    float* scales = is_v ? a.v_scales : a.k_scales;
    uint8_t* codes = is_v ? a.v_codes : a.k_codes;
    auto cell_of = [&](int l) -> size_t { return (size_t)(s_slot[kReach + l] / kBlock) * a.n_kv + g; };
    const bool starts = threadIdx.x < kWindow && s_leader[threadIdx.x];
    const float old = starts ? scales[cell_of(threadIdx.x)] : 0.f;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v : a.k);
    Raw x[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int u = i * kAppendWarps + warp;
        if (u < kSeen && s_run[u] >= 0) x[i] = reinterpret_cast<const Raw*>(src + ((size_t)(first + u) * a.n_kv + g) * D)[lane];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int u = i * kAppendWarps + warp;
        if (u < kSeen && s_run[u] >= 0) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < WORDS; ++e) {
                float f[2];
                widen_word<T>(w[e], f);
                if (fabsf(f[0]) <= kMaxFinite) amax = fmaxf(amax, fabsf(f[0]));
                if (fabsf(f[1]) <= kMaxFinite) amax = fmaxf(amax, fabsf(f[1]));
            }
            // non-negative floats are ordered like their bits
            const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
            if (lane == 0) atomicMax(&s_amax[s_run[u]], m);
        }
    }
    __syncthreads();
    if (starts) {
        const float need = pow2(scale_exp(__uint_as_float(s_amax[threadIdx.x]), a.min_exp));
        const bool started = s_rows[threadIdx.x] & 1u;
        const float now = started ? need : fmaxf(old, need);
        s_inv[threadIdx.x] = 1.f / now;  // exact: a power of two (or a caller's own scale that was the larger)
        s_ratio[threadIdx.x] = !started && now != old ? old / now : 0.f;
        s_leader[threadIdx.x] = !started && now != old ? 2 : 1;
        scales[cell_of(threadIdx.x)] = now;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int u = i * kAppendWarps + warp;
        if (u < kSeen && s_run[u] >= 0) {
            const int l = s_run[u];
            const float inv = s_inv[l];
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
            Codes c;
            uint16_t* h = reinterpret_cast<uint16_t*>(&c);
#pragma unroll
            for (int e = 0; e < WORDS; ++e) {
                float f[2];
                widen_word<T>(w[e], f);
#pragma unroll
                for (int v = 0; v < 2; ++v) f[v] = fabsf(f[v]) <= kMaxFinite ? f[v] * inv : __int_as_float(0x7fc00000);
                h[e] = (uint16_t)to_e4m3x2(f[0], f[1]);
            }
            reinterpret_cast<Codes*>(codes + (cell_of(l) * kBlock + s_slot[kReach + u] % kBlock) * D)[lane] = c;
        }
    }
    for (int l = 0; l < kWindow; ++l) {  // rare: a block continued with a larger scale
        if (s_leader[l] != 2) continue;
        for (int r = warp; r < kBlock; r += kAppendWarps) {
            if ((s_rows[l] >> r) & 1u) continue;
            Codes* p = reinterpret_cast<Codes*>(codes + (cell_of(l) * kBlock + r) * D) + lane;
            Codes c = *p;
            uint16_t* h = reinterpret_cast<uint16_t*>(&c);
#pragma unroll
            for (int e = 0; e < WORDS; ++e) {
                const float2 f = from_e4m3x2(h[e]);
                h[e] = (uint16_t)to_e4m3x2(f.x * s_ratio[l], f.y * s_ratio[l]);
            }
            *p = c;
        }
    }
}

// grid (pair, layer, K/V): each CTA copies one block of one layer, codes and scales.
__global__ void __launch_bounds__(256) q8_copy_kernel(const Q8CopyArgs a) {
    const int layer = blockIdx.y;
    grid_dependency_wait();
    grid_launch_dependents();
    const int src = a.pairs[2 * blockIdx.x];
    const int dst = a.pairs[2 * blockIdx.x + 1];
    if ((unsigned)src >= (unsigned)a.num_blocks || (unsigned)dst >= (unsigned)a.num_blocks) {
        if (threadIdx.x == 0 && layer == 0 && blockIdx.z == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_PAIR);
        return;
    }
    uint8_t* pool = (blockIdx.z == 0 ? a.k_codes : a.v_codes) + (size_t)layer * a.num_blocks * a.block_bytes;
    const uint4* s = reinterpret_cast<const uint4*>(pool + (size_t)src * a.block_bytes);
    uint4* d = reinterpret_cast<uint4*>(pool + (size_t)dst * a.block_bytes);
    const size_t n = a.block_bytes / 16;
    constexpr int U = 8;  // loads in flight per thread before their stores
    for (size_t i0 = threadIdx.x; i0 < n; i0 += (size_t)U * blockDim.x) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + (size_t)u * blockDim.x < n) r[u] = s[i0 + (size_t)u * blockDim.x];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + (size_t)u * blockDim.x < n) d[i0 + (size_t)u * blockDim.x] = r[u];
    }
    float* scales = (blockIdx.z == 0 ? a.k_scales : a.v_scales) + (size_t)layer * a.num_blocks * a.n_kv;
    for (int h = threadIdx.x; h < a.n_kv; h += blockDim.x)
        scales[(size_t)dst * a.n_kv + h] = scales[(size_t)src * a.n_kv + h];
}

// x in the activations' type, beyond its largest number as that number. Codes that the append wrote reach the
// next power of two at most: fp16 rows near 65,504 round to 65,536 (bf16 ones above 3.35e38 to 2^128).
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float x, float y);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float x, float y) {
    constexpr float kMax = 3.38953139e38f;
    const __nv_bfloat162 h = __floats2bfloat162_rn(fabsf(x) > kMax ? copysignf(kMax, x) : x,
                                                   fabsf(y) > kMax ? copysignf(kMax, y) : y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float x, float y) {
    const __half2 h = __floats2half2_rn(fabsf(x) > 65504.f ? copysignf(65504.f, x) : x,
                                        fabsf(y) > 65504.f ? copysignf(65504.f, y) : y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two codes * S. `over` is raised for what lies beyond that power of two.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, float s, bool& over) {
    constexpr float kHalf = std::is_same<T, __half>::value ? 32768.f : 1.70141183e38f;  // of it, to stay finite
    const float2 f = from_e4m3x2(codes);
    over = over || fmaxf(fabsf(f.x), fabsf(f.y)) * (0.5f * s) > kHalf;
    return narrow2<T>(f.x * s, f.y * s);
}

constexpr int kWidenWarps = 8;

// One warp per (sequence, logical block, KV head): K and V chunk, 16 codes a lane and step. Sequences
// that share blocks write the same values to the same places. NaN codes of V become 0 and are reported: the
// attention kernel multiplies every row of a tile with weights, 0 for tokens that do not see it, and 0 x NaN
// would reach those too.
template <typename T, int D>
__global__ void __launch_bounds__(kWidenWarps * 32) q8_widen_kernel(const Q8WidenArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.z;
    const int cap = a.max_blocks * kBlock;
    const int ctx = a.lens[s];
    if (ctx <= 0 || ctx > cap) return;  // the attention launch flags such a sequence
    const int nb = (ctx + kBlock - 1) / kBlock;
    const long long item = (long long)blockIdx.x * kWidenWarps + warp;
    const int b = (int)(item / a.n_kv), g = (int)(item % a.n_kv);
    if (b >= nb) return;
    const int phys = a.tables[(size_t)s * a.max_blocks + b];
    if ((unsigned)phys >= (unsigned)a.num_blocks) return;  // flagged by the attention launch
    const size_t cell = (size_t)phys * a.n_kv + g;
    constexpr int STEPS = kBlock * D / (32 * 16);
    uint4 x[2][STEPS];
    float sc[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const uint4* src = reinterpret_cast<const uint4*>((v ? a.v_codes : a.k_codes) + cell * kBlock * D);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) x[v][i] = __ldcs(src + i * 32 + lane);
        sc[v] = __ldg((v ? a.v_scales : a.k_scales) + cell);
    }
    bool over = false, nan = false;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<T*>(v ? a.v_out : a.k_out) + cell * kBlock * D);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
            uint32_t o[8];
            const bool inside = b * kBlock + (i * 32 + lane) * 16 / D < ctx;  // rows past the context may hold anything
            if (v == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t m = __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    nan = nan || (m != 0u && inside);
                    w[e] &= ~m;
                }
            }
            bool past = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = widen2<T>(w[e], sc[v], past);
                o[2 * e + 1] = widen2<T>(w[e] >> 16, sc[v], past);
            }
            over = over || (past && inside);
            out[2 * (i * 32 + lane)] = make_uint4(o[0], o[1], o[2], o[3]);
            out[2 * (i * 32 + lane) + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
    if (__any_sync(0xffffffffu, over) && lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_SCALE);
    if (__any_sync(0xffffffffu, nan) && lane == 0) *a.v_nan = 1u;
}

template <typename T>
cudaError_t append_of(int head_dim, const Q8AppendArgs& a, cudaStream_t stream) {
    const long long ctas = ((long long)a.n_tok + kWindow - 1) / kWindow * 2 * a.n_kv;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas);
    switch (head_dim) {
    case 64: return launch_dependent(q8_append_kernel<T, 64>, grid, kAppendWarps * 32, 0, stream, 1, a);
    case 128: return launch_dependent(q8_append_kernel<T, 128>, grid, kAppendWarps * 32, 0, stream, 1, a);
    case 256: return launch_dependent(q8_append_kernel<T, 256>, grid, kAppendWarps * 32, 0, stream, 1, a);
    default: return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t widen_of(int head_dim, const Q8WidenArgs& a, cudaStream_t stream) {
    const long long ctas = ((long long)a.max_blocks * a.n_kv + kWidenWarps - 1) / kWidenWarps;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, 1, a.n_seqs);
    switch (head_dim) {
    case 64: q8_widen_kernel<T, 64><<<grid, kWidenWarps * 32, 0, stream>>>(a); break;
    case 128: q8_widen_kernel<T, 128><<<grid, kWidenWarps * 32, 0, stream>>>(a); break;
    case 256: q8_widen_kernel<T, 256><<<grid, kWidenWarps * 32, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_append(int dtype, int head_dim, const Q8AppendArgs& a, cudaStream_t stream) {
    return dtype == PKV_F16 ? append_of<__half>(head_dim, a, stream) : append_of<__nv_bfloat16>(head_dim, a, stream);
}

cudaError_t launch_q8_copy(const Q8CopyArgs& a, cudaStream_t stream) {
    return launch_dependent(q8_copy_kernel, dim3(a.n_pairs, a.n_layers, 2), 256, 0, stream, 1, a);
}

cudaError_t launch_q8_widen(int dtype, int head_dim, const Q8WidenArgs& a, cudaStream_t stream) {
    return dtype == PKV_F16 ? widen_of<__half>(head_dim, a, stream) : widen_of<__nv_bfloat16>(head_dim, a, stream);
}

}  // namespace pkv
