// scores.cu -- attention weights from the logits a decode launch left behind, added to each sequence's
// running sums (sm_103a).
//
//   scores[s][g][j] += sum_{h in group g} 2^(z_hj - m_h) / l_h,   j < len_s,
// m_h and l_h the row's maximum and sum. A position's weight needs them, and they exist only when the whole row has been read, so this is a launch of its
// own, a programmatic dependent of the attention: its CTAs are resident and wait when the last
// attention CTA ends. It reads 4 G bytes and reads and writes 4 bytes a token and head (the logits of
// moderate batches still lie in L2). Sums are fp32; every score is written by one thread and heads are
// added in order, so results do not depend on timing.
#include <math.h>

#include "common.cuh"
#include "shrink.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;  // positions of a thread, kThreads apart

// 2^x within 2 ulp; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int G>
__device__ __forceinline__ void load_logits(const float* p, float* z) {
    if constexpr (G == 1) {
        z[0] = __ldcs(p);
    } else if constexpr (G == 2) {
        const float2 u = __ldcs(reinterpret_cast<const float2*>(p));
        z[0] = u.x;
        z[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) {
            const float4 u = __ldcs(reinterpret_cast<const float4*>(p) + i);
            z[4 * i] = u.x;
            z[4 * i + 1] = u.y;
            z[4 * i + 2] = u.z;
            z[4 * i + 3] = u.w;
        }
    }
}

template <int G>
__global__ void __launch_bounds__(kThreads) add_scores_kernel(const ScoreArgs a) {
    __shared__ float s_m[8], s_inv[8];
    const int s = blockIdx.z, g = blockIdx.y;
    const int cap = a.max_blocks * kBlock;
    grid_dependency_wait();
    grid_launch_dependents();
    const int ctx = min(max(a.lens[s], 0), cap);
    const int j0 = blockIdx.x * kThreads * kPerThread;
    if (j0 >= ctx) return;
    const size_t base = ((size_t)s * a.n_kv + g);
    float z[kPerThread][G], was[kPerThread];  // all of a thread's loads in flight with the statistics'
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int j = j0 + i * kThreads + threadIdx.x;
        if (j < ctx) {
            load_logits<G>(a.z + (base * cap + j) * G, z[i]);
            was[i] = a.scores[base * a.stride + j];
        }
    }
    if (threadIdx.x < G) {
        const float2 u = __ldcg(a.row_ml + base * G + threadIdx.x);
        s_m[threadIdx.x] = u.x == -INFINITY ? 0.f : u.x;
        s_inv[threadIdx.x] = u.y == 0.f ? 0.f : 1.f / u.y;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int j = j0 + i * kThreads + threadIdx.x;
        if (j < ctx) {
            float w = 0.f;
#pragma unroll
            for (int r = 0; r < G; ++r) w += ex2(z[i][r] - s_m[r]) * s_inv[r];
            a.scores[base * a.stride + j] = was[i] + w;
        }
    }
}

}  // namespace

cudaError_t launch_scores(const ScoreArgs& a, cudaStream_t stream) {
    constexpr int kChunk = kThreads * kPerThread;
    const dim3 grid((unsigned)(((long long)a.max_blocks * kBlock + kChunk - 1) / kChunk), a.n_kv, a.n_seqs);
    switch (a.group) {
    case 1: return launch_dependent(add_scores_kernel<1>, grid, kThreads, 0, stream, 1, a);
    case 2: return launch_dependent(add_scores_kernel<2>, grid, kThreads, 0, stream, 1, a);
    case 4: return launch_dependent(add_scores_kernel<4>, grid, kThreads, 0, stream, 1, a);
    case 8: return launch_dependent(add_scores_kernel<8>, grid, kThreads, 0, stream, 1, a);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkv
