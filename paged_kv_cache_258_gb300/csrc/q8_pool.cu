// q8_pool.cu -- 8-bit pools: quantising append, block copies, widening of rows for prefill (sm_103a).
//
// A code is an e4m3 number (1 sign, 4 exponent, 3 mantissa bits; largest 448), a value is code * S with
// one power of two S for each (block, KV head) of each of K and V. Why a power of two: e4m3 rounds
// relative to the value, so within its 15 binades any other scale rounds no better, and with a power of
// two x / S is exact, widening is exact, and raising a block's scale only moves the exponents of its
// codes -- codes are rounded again only where they fall below 2^-6. The scale is the least that lets the
// largest finite element of the block in.
//
// Append (one launch, a few bytes of arithmetic a byte): a block's scale is raised once for all the
// call's rows in it, so one warp handles a (block, KV head, K or V): the warp of the block's first token
// in the call. It reads slots[t-31 .. t+31], leaves if an earlier one lies in its block, and gathers the
// later ones by ballot. A block is started when a row at offset 0 arrives: its old scale, the previous
// owner's, is forgotten. Otherwise S' = max(S, what the new rows need) and, if that grew, the other rows
// are brought to S'.
#include <math.h>

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

// codes * f for the eight codes of two words, back to codes.
__device__ __forceinline__ uint2 rescale8(uint2 c, float f) {
    uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = from_e4m3x2(w[i]), b = from_e4m3x2(w[i] >> 16);
        w[i] = to_e4m3x2(a.x * f, a.y * f) | (to_e4m3x2(b.x * f, b.y * f) << 16);
    }
    return make_uint2(w[0], w[1]);
}

constexpr int kAppendWarps = 8;

// One warp per (token, KV head, K or V); warps of tokens that are not their block's first leave.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) q8_append_kernel(const Q8AppendArgs a) {
    constexpr int NCH = D / 8;          // 8-element pieces of a row
    constexpr int RPP = 32 / NCH;       // rows a warp covers at once (1, 2, 4)
    constexpr int PASSES = kBlock / RPP;
    __shared__ int s_tok[kAppendWarps][kBlock];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kAppendWarps + warp;
    const long long per_tok = 2LL * a.n_kv;
    if (item >= a.n_tok * per_tok) return;
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = (int)(item / per_tok);
    const int rest = (int)(item % per_tok);
    const bool is_v = rest >= a.n_kv;
    const int g = is_v ? rest - a.n_kv : rest;
    const long long slot = a.slots[t];
    if (slot < 0) return;  // padding token
    if (slot >= (long long)a.num_blocks * kBlock) {
        if (lane == 0) atomicOr(a.status, (unsigned)PKV_DEV_BAD_SLOT);
        return;
    }
    const long long block = slot / kBlock;
    const long long before = lane > 0 && t - lane >= 0 ? a.slots[t - lane] : -1;
    if (__any_sync(0xffffffffu, before >= 0 && before / kBlock == block)) return;
    const long long after = (long long)t + lane < a.n_tok ? a.slots[t + lane] : -1;
    const bool member = after >= 0 && after / kBlock == block;
    if (lane < kBlock) s_tok[warp][lane] = -1;
    __syncwarp();
    if (member) s_tok[warp][after % kBlock] = t + lane;
    __syncwarp();

    const int c = lane % NCH, sub = lane / NCH;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v : a.k);
    uint4 x[PASSES];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int tok = s_tok[warp][i * RPP + sub];
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tok >= 0) x[i] = __ldg(reinterpret_cast<const uint4*>(src + ((size_t)tok * a.n_kv + g) * D) + c);
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        float f[8];
        Vec16<T>::to_float(x[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = fabsf(f[e]);
            if (v <= kMaxFinite) amax = fmaxf(amax, v);
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));

    const size_t cell = (size_t)block * a.n_kv + g;
    float* scale = (is_v ? a.v_scales : a.k_scales) + cell;
    const float need = pow2(scale_exp(amax, a.min_exp));
    const bool started = s_tok[warp][0] >= 0;
    const float old = *scale;
    const float now = started ? need : fmaxf(old, need);
    const float inv = 1.f / now;  // exact: a power of two (or a caller's own scale that was the larger)
    uint8_t* dst = (is_v ? a.v_codes : a.k_codes) + cell * kBlock * D;
    const bool grew = !started && now != old;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = i * RPP + sub;
        uint2* out = reinterpret_cast<uint2*>(dst + r * D) + c;
        if (s_tok[warp][r] >= 0) {
            float f[8];
            Vec16<T>::to_float(x[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fabsf(f[e]) <= kMaxFinite ? f[e] * inv : __int_as_float(0x7fc00000);
            *out = make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16),
                              to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
        } else if (grew) {
            *out = rescale8(*out, old * inv);
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = now;
}

// grid (pair, layer, K/V): each CTA copies one block of one layer, codes and scales.
__global__ void __launch_bounds__(256) q8_copy_kernel(const Q8CopyArgs a) {
    const int layer = blockIdx.y;
    grid_launch_dependents();
    grid_dependency_wait();
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

// code * S in the activations' type. fp16 has no room for the 65,536 that rows near 65,504 round to:
// it is read as the largest half.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, float s);
template <>
__device__ __forceinline__ uint32_t widen2<__nv_bfloat16>(uint32_t codes, float s) {
    const float2 f = from_e4m3x2(codes);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * s, f.y * s);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t widen2<__half>(uint32_t codes, float s) {
    const float2 f = from_e4m3x2(codes);
    float x = f.x * s, y = f.y * s;
    if (fabsf(x) == 65536.f) x = copysignf(65504.f, x);
    if (fabsf(y) == 65536.f) y = copysignf(65504.f, y);
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kWidenWarps = 8;

// One warp per (sequence, logical block, KV head): K and V chunk, 16 codes a lane and step. Sequences
// that share blocks write the same values to the same places.
template <typename T, int D>
__global__ void __launch_bounds__(kWidenWarps * 32) q8_widen_kernel(const Q8WidenArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.z;
    const int cap = a.max_blocks * kBlock;
    grid_dependency_wait();
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
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<T*>(v ? a.v_out : a.k_out) + cell * kBlock * D);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = widen2<T>(w[e], sc[v]);
                o[2 * e + 1] = widen2<T>(w[e] >> 16, sc[v]);
            }
            out[2 * (i * 32 + lane)] = make_uint4(o[0], o[1], o[2], o[3]);
            out[2 * (i * 32 + lane) + 1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

template <typename T>
cudaError_t append_of(int head_dim, const Q8AppendArgs& a, cudaStream_t stream) {
    const long long items = 2LL * a.n_tok * a.n_kv;
    const long long ctas = (items + kAppendWarps - 1) / kAppendWarps;
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
    case 64: return launch_dependent(q8_widen_kernel<T, 64>, grid, kWidenWarps * 32, 0, stream, 1, a);
    case 128: return launch_dependent(q8_widen_kernel<T, 128>, grid, kWidenWarps * 32, 0, stream, 1, a);
    case 256: return launch_dependent(q8_widen_kernel<T, 256>, grid, kWidenWarps * 32, 0, stream, 1, a);
    default: return cudaErrorInvalidValue;
    }
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
