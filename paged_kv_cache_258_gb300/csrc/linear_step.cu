// linear_step.cu -- linear attention token after token, the state in registers (sm_103a): decode steps, short
// chunks, and every length in fp32.
//
//   S_t = exp(g_t) S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t
//
// The columns of S (dim_v) do not depend on one another, so a CTA takes NC of them for one sequence and head: 128
// threads, each with 4 adjacent columns and DK * NC / 512 rows in registers, all loads of the state in flight at once.
// A token costs two fused multiply-adds an element for the state and one for o, and o is summed over the rows by
// shuffles in a warp and through shared memory between the four warps, once for every kStep tokens.
//
// exp(g) S is taken as S + S expm1(g) while exp(g) > 0.6: exp(g) itself, rounded to 24 bits, is off by up to 2^-25
// whatever g, the same way at every token, which a slow decay (g = -1e-4) would make 2^-11 of what it keeps; expm1
// is as exact as g is.
#include <type_traits>

#include "common.cuh"
#include "linear.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
// Tokens staged in shared memory at a time. 16 where a token's latency counts (columns of 32, 500 tokens of 8 heads x 64 x
// 64 in fp32: 73 us, in steps of 8 83, of 4 106) and where a whole short chunk fits; 8 for many long fp32 rows (256 tokens of
// 8 x 32 heads x 128 x 128: 172 us against 189).
template <typename T, int NC>
constexpr int kStep = sizeof(T) == 2 || NC == 32 ? 16 : 8;

template <typename T, int DK, int DV, int NC, bool ONE>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearArgs a) {
    constexpr int TB = ONE ? 1 : kStep<T, NC>;
    constexpr int SLICES = DV / NC;
    constexpr int LPR = NC / 4;                   // lanes of a row of S
    constexpr int GROUPS = kThreads / LPR;        // row groups of the CTA
    constexpr int R = DK / GROUPS;                // rows of a thread
    constexpr int N = Vec16<T>::N;
    constexpr int QV = TB * DK / N, VV = TB * NC / N;  // 16-byte vectors of a step's q (or k) and v
    __shared__ __align__(16) float s_q[TB][DK];
    __shared__ __align__(16) float s_k[TB][DK];
    __shared__ __align__(16) float s_v[TB][NC];
    __shared__ float s_d[TB];       // what a token's decay multiplies the state by (exp(g)), or that less 1
    __shared__ float s_once[TB];    // 0 for the first, 1 for the second
    __shared__ __align__(16) float s_o[TB][kThreads / 32][NC];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = blockIdx.x % SLICES;
    const long long unit = blockIdx.x / SLICES;
    const int h = (int)(unit % a.n_v), s = (int)(unit / a.n_v);
    const int hq = h / (a.n_v / a.n_qk);
    int q0 = s, q1 = s + 1;
    if (!ONE) {
        q0 = a.q_start[s];
        q1 = a.q_start[s + 1];
    }
    const int src = a.src[s], dst = a.dst[s];
    const bool bad_range = !ONE && (q0 < 0 || q1 < q0 || q1 > a.n_tokens || q1 - q0 > a.max_query);
    const bool bad_slot = src >= a.n_slots || dst >= a.n_slots;
    if (bad_range || bad_slot) {
        if (h == 0 && slice == 0 && tid == 0)
            atomicOr(a.status, (bad_range ? (unsigned)PKV_DEV_BAD_QUERY_RANGE : 0u) |
                                   (bad_slot ? (unsigned)PKV_DEV_BAD_STATE_SLOT : 0u));
        return;
    }
    const int col = (tid % LPR) * 4, row0 = (tid / LPR) * R;
    const size_t head = (size_t)DK * DV;
    const size_t at = (size_t)row0 * DV + slice * NC + col;
    float4 x[R];
    if (src >= 0) {
        const float4* p = reinterpret_cast<const float4*>(a.state + ((size_t)src * a.n_v + h) * head + at);
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = __ldcs(p + (size_t)i * (DV / 4));
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const T* q = static_cast<const T*>(a.q);
    const T* k = static_cast<const T*>(a.k);
    const T* v = static_cast<const T*>(a.v);
    constexpr int QN = (QV + kThreads - 1) / kThreads, VN = (VV + kThreads - 1) / kThreads;
    uint4 rq[QN], rk[QN], rv[VN];
    float rg = 0.f;
    auto widen = [](const uint4& u, float* to) {
        float f[N];
        Vec16<T>::to_float(u, f);
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    };
    // the next step's rows, into registers (tokens past the last are not read)
    auto fetch = [&](int t0) {
        const int n = min(TB, q1 - t0);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = (i * kThreads + tid) * N, t = e / DK;
            if (t < n) {
                const size_t from = ((size_t)(t0 + t) * a.n_qk + hq) * DK + e % DK;
                rq[i] = *reinterpret_cast<const uint4*>(q + from);
                rk[i] = *reinterpret_cast<const uint4*>(k + from);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int e = (i * kThreads + tid) * N, t = e / NC;
            if (t < n) rv[i] = *reinterpret_cast<const uint4*>(v + ((size_t)(t0 + t) * a.n_v + h) * DV + slice * NC + e % NC);
        }
        if (tid < n) rg = a.log_decay ? a.log_decay[(size_t)(t0 + tid) * a.decay_stride + h] : 0.f;
    };
    if (q0 < q1) fetch(q0);
    for (int t0 = q0; t0 < q1; t0 += TB) {
        const int n = min(TB, q1 - t0);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = (i * kThreads + tid) * N;
            if (e / DK < n) {
                widen(rq[i], &s_q[0][0] + e);
                widen(rk[i], &s_k[0][0] + e);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int e = (i * kThreads + tid) * N;
            if (e / NC < n) widen(rv[i], &s_v[0][0] + e);
        }
        if (tid < n) {
            const bool slow = rg > -0.5f && rg < 0.5f;
            s_d[tid] = slow ? expm1f(rg) : expf(rg);
            s_once[tid] = slow ? 1.f : 0.f;
        }
        __syncthreads();
        if (t0 + TB < q1) fetch(t0 + TB);
        auto token = [&](auto slow, int t) {
            const float d = s_d[t], once = s_once[t];
            const float4 vt = *reinterpret_cast<const float4*>(&s_v[t][col]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&s_k[t][row0 + i]);
                const float4 q4 = *reinterpret_cast<const float4*>(&s_q[t][row0 + i]);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4& y = x[i + j];
                    if constexpr (decltype(slow)::value) {  // d = expm1(g)
                        y.x = fmaf(y.x, d, fmaf(kk[j], vt.x, y.x));
                        y.y = fmaf(y.y, d, fmaf(kk[j], vt.y, y.y));
                        y.z = fmaf(y.z, d, fmaf(kk[j], vt.z, y.z));
                        y.w = fmaf(y.w, d, fmaf(kk[j], vt.w, y.w));
                    } else {                                // either
                        y.x = fmaf(y.x, d, fmaf(kk[j], vt.x, y.x * once));
                        y.y = fmaf(y.y, d, fmaf(kk[j], vt.y, y.y * once));
                        y.z = fmaf(y.z, d, fmaf(kk[j], vt.z, y.z * once));
                        y.w = fmaf(y.w, d, fmaf(kk[j], vt.w, y.w * once));
                    }
                    o.x = fmaf(qq[j], y.x, o.x);
                    o.y = fmaf(qq[j], y.y, o.y);
                    o.z = fmaf(qq[j], y.z, o.z);
                    o.w = fmaf(qq[j], y.w, o.w);
                }
            }
#pragma unroll
            for (int m = LPR; m < 32; m *= 2) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
            }
            if (lane < LPR) *reinterpret_cast<float4*>(&s_o[t][warp][col]) = o;
        };
        // tokens follow one another without a branch: the loads, products and shuffles of one overlap those of the next,
        // whose state needs only the products
        bool any = false;
#pragma unroll
        for (int t = 0; t < TB; ++t) any |= t < n && s_once[t] == 0.f;
        constexpr int AT_ONCE = !ONE && R <= 8 ? 4 : 1;
        if (!any) {
#pragma unroll AT_ONCE
            for (int t = 0; t < n; ++t) token(std::true_type{}, t);
        } else {
#pragma unroll AT_ONCE
            for (int t = 0; t < n; ++t) token(std::false_type{}, t);
        }
        __syncthreads();
        for (int e = tid; e < n * NC; e += kThreads) {
            const int t = e / NC, c = e % NC;
            const float sum = (s_o[t][0][c] + s_o[t][1][c]) + (s_o[t][2][c] + s_o[t][3][c]);
            static_cast<T*>(a.out)[((size_t)(t0 + t) * a.n_v + h) * DV + slice * NC + c] = from_float<T>(sum * a.scale);
        }
        // (the next step's values go to s_q .. s_g, which nobody reads any more; s_o is written behind its barrier)
    }
    if (dst >= 0) {
        float4* p = reinterpret_cast<float4*>(a.state + ((size_t)dst * a.n_v + h) * head + at);
#pragma unroll
        for (int i = 0; i < R; ++i) __stcs(p + (size_t)i * (DV / 4), x[i]);
    }
}

template <typename T, int DK, int DV, int NC>
cudaError_t run(const LinearArgs& a, cudaStream_t stream) {
    const unsigned ctas = (unsigned)a.n_seqs * a.n_v * (DV / NC);
    if (a.q_start)
        linear_step_kernel<T, DK, DV, NC, false><<<ctas, kThreads, 0, stream>>>(a);
    else
        linear_step_kernel<T, DK, DV, NC, true><<<ctas, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int DK, int DV>
cudaError_t pick(int sms, const LinearArgs& a, cudaStream_t stream) {
    // columns of 64 while there are enough of them to fill the GPU, else of 32
    return (long long)a.n_seqs * a.n_v * (DV / 64) >= 2LL * sms ? run<T, DK, DV, 64>(a, stream) : run<T, DK, DV, 32>(a, stream);
}

template <typename T>
cudaError_t dims(int dk, int dv, int sms, const LinearArgs& a, cudaStream_t stream) {
    if (dk == 64) return dv == 64 ? pick<T, 64, 64>(sms, a, stream) : pick<T, 64, 128>(sms, a, stream);
    return dv == 64 ? pick<T, 128, 64>(sms, a, stream) : pick<T, 128, 128>(sms, a, stream);
}

}  // namespace

cudaError_t launch_linear_step(int dtype, int dk, int dv, int sms, const LinearArgs& a, cudaStream_t stream) {
    switch (dtype) {
    case PKV_F32: return dims<float>(dk, dv, sms, a, stream);
    case PKV_F16: return dims<__half>(dk, dv, sms, a, stream);
    default: return dims<__nv_bfloat16>(dk, dv, sms, a, stream);
    }
}

}  // namespace pkv
