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
//
// What bounds it: decode, the states' bytes (bf16, 250 sequences of 32 heads x 128 x 64: 80 us, 6.6 TB/s; fp16, 64 of 32 x
// 128 x 128: 43.3 us, 6.25 TB/s; one of 48 x 128 x 128: 3 us on the device, a trip to memory and back). Chunks of many
// sequences, the products' instructions (32 sequences of 16 tokens, 48 x 128 x 128: 68 us, 5.9e12 updates of a state element
// a second); chunks of few heads, one warp's latency (60 ns a token).
#include <type_traits>

#include "arith.cuh"
#include "common.cuh"
#include "linear.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
// Tokens staged in shared memory at a time: 16 where a whole short chunk fits, 8 for many long fp32 rows (256 tokens of
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

// The same for chunks of few heads, where what counts is how long a token takes one warp: NC is 32 or 16, 16 threads take
// a row, each with NC / 16 adjacent columns and an eighth of the rows as pairs of rows, which packed arithmetic takes at
// once (k and q come from shared memory as pairs already, v and decays twice each), four tokens at a time. Tokens are
// staged in two buffers, one barrier a step: behind it the results of the step before are summed up and the next step's
// rows are asked for. HELPERS more threads do both for the four warps that walk, where there is room: a step of 16 tokens
// takes those 0.7 us and everything else 0.65.
constexpr int kRowLanes = 16;
constexpr int kGroups = kThreads / kRowLanes;  // row groups

// n adjacent floats
template <int n>
struct Floats;
template <>
struct Floats<1> {
    using type = float;
    __device__ __forceinline__ static void get(float v, float (&x)[1]) { x[0] = v; }
    __device__ __forceinline__ static float put(const float (&x)[1]) { return x[0]; }
};
template <>
struct Floats<2> {
    using type = float2;
    __device__ __forceinline__ static void get(float2 v, float (&x)[2]) { x[0] = v.x, x[1] = v.y; }
    __device__ __forceinline__ static float2 put(const float (&x)[2]) { return make_float2(x[0], x[1]); }
};
template <>
struct Floats<4> {
    using type = float4;
    __device__ __forceinline__ static void get(float4 v, float (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
    __device__ __forceinline__ static float4 put(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};

template <typename T, int DK, int DV, int NC, int HELPERS>
__global__ void __launch_bounds__(kThreads + HELPERS, HELPERS ? 2 : 0) linear_walk_kernel(const LinearArgs a) {
    constexpr int TB = DK * NC <= 2048 ? 16 : 8;  // tokens staged at a time
    constexpr int SLICES = DV / NC;
    constexpr int C = NC / kRowLanes;             // columns of a thread
    constexpr int R = DK / kGroups;               // and rows
    constexpr int N = Vec16<T>::N;
    constexpr int QV = TB * DK / N, VV = TB * NC / N;  // 16-byte vectors of a step's q (or k) and v
    __shared__ __align__(16) float s_q[2][TB][DK];
    __shared__ __align__(16) float s_k[2][TB][DK];
    __shared__ __align__(16) float2 s_v[2][TB][NC];  // twice each, as packed products take it
    // What a token's decay multiplies the state by, and how often the state itself is added: exp(g) and 0, or
    // exp(g) - 1 and 1.
    __shared__ __align__(16) float4 s_d[2][TB];  // (twice each)
    __shared__ __align__(16) float s_o[2][TB][kThreads / 32][NC];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int STAGERS = HELPERS ? HELPERS : kThreads;  // threads that stage and sum up
    const int help = HELPERS ? tid - kThreads : tid;
    const bool walker = !HELPERS || help < 0;
    const int slice = blockIdx.x % SLICES;
    const long long unit = blockIdx.x / SLICES;
    const int h = (int)(unit % a.n_v), s = (int)(unit / a.n_v);
    const int hq = h / (a.n_v / a.n_qk);
    const int q0 = a.q_start[s], q1 = a.q_start[s + 1];
    const int src = a.src[s], dst = a.dst[s];
    const bool bad_range = q0 < 0 || q1 < q0 || q1 > a.n_tokens || q1 - q0 > a.max_query;
    const bool bad_slot = src >= a.n_slots || dst >= a.n_slots;
    if (bad_range || bad_slot) {
        if (h == 0 && slice == 0 && tid == 0)
            atomicOr(a.status, (bad_range ? (unsigned)PKV_DEV_BAD_QUERY_RANGE : 0u) |
                                   (bad_slot ? (unsigned)PKV_DEV_BAD_STATE_SLOT : 0u));
        return;
    }
    const int col = (tid % kRowLanes) * C, row0 = (tid / kRowLanes) * R;
    const size_t head = (size_t)DK * DV;
    const size_t at = (size_t)row0 * DV + slice * NC + col;
    using Cols = typename Floats<C>::type;
    uint64_t x[C][R / 2];  // pairs of rows
    {
        float y[R][C];
        if (src >= 0 && walker) {
            const float* p = a.state + ((size_t)src * a.n_v + h) * head + at;
#pragma unroll
            for (int i = 0; i < R; ++i) Floats<C>::get(__ldcs(reinterpret_cast<const Cols*>(p + (size_t)i * DV)), y[i]);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c) y[i][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < R / 2; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) x[c][i] = f2_pack(y[2 * i][c], y[2 * i + 1][c]);
    }
    const T* q = static_cast<const T*>(a.q);
    const T* k = static_cast<const T*>(a.k);
    const T* v = static_cast<const T*>(a.v);
    constexpr int QN = (QV + STAGERS - 1) / STAGERS, VN = (VV + STAGERS - 1) / STAGERS;
    uint4 rq[QN], rk[QN], rv[VN];
    float rg = 0.f;
    auto widen = [](const uint4& u, float* to) {
        float f[N];
        Vec16<T>::to_float(u, f);
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    };
    // a step's rows, into registers (tokens past the last are not read) and from there to shared memory
    auto fetch = [&](int t0) {
        const int n = min(TB, q1 - t0);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = (i * STAGERS + help) * N, t = e / DK;
            if (t < n) {
                const size_t from = ((size_t)(t0 + t) * a.n_qk + hq) * DK + e % DK;
                rq[i] = *reinterpret_cast<const uint4*>(q + from);
                rk[i] = *reinterpret_cast<const uint4*>(k + from);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int e = (i * STAGERS + help) * N, t = e / NC;
            if (t < n) rv[i] = *reinterpret_cast<const uint4*>(v + ((size_t)(t0 + t) * a.n_v + h) * DV + slice * NC + e % NC);
        }
        if (help < n) rg = a.log_decay ? a.log_decay[(size_t)(t0 + help) * a.decay_stride + h] : 0.f;
    };
    auto stage = [&](int t0, int b) -> bool {  // whether any token's decay is not a slow one
        const int n = min(TB, q1 - t0);
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = (i * STAGERS + help) * N;
            if (e / DK < n) {
                widen(rq[i], &s_q[b][0][0] + e);
                widen(rk[i], &s_k[b][0][0] + e);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int e = (i * STAGERS + help) * N;
            if (e / NC < n) {
                float f[N];
                Vec16<T>::to_float(rv[i], f);
                float4* to = reinterpret_cast<float4*>(&s_v[b][0][0] + e);
#pragma unroll
                for (int j = 0; j < N; j += 2) to[j / 2] = make_float4(f[j], f[j], f[j + 1], f[j + 1]);
            }
        }
        if (help >= n) return false;
        const bool slow = rg > -0.5f && rg < 0.5f;
        const float d = slow ? expm1f(rg) : expf(rg), once = slow ? 1.f : 0.f;
        s_d[b][help] = make_float4(d, d, once, once);
        return !slow;
    };
    auto results = [&](int t0, int b) {
        const int n = min(TB, q1 - t0);
#pragma unroll(HELPERS ? 4 : 1)
        for (int e = help; e < n * NC; e += STAGERS) {
            const int t = e / NC, c = e % NC;
            const float sum = (s_o[b][t][0][c] + s_o[b][t][1][c]) + (s_o[b][t][2][c] + s_o[b][t][3][c]);
            static_cast<T*>(a.out)[((size_t)(t0 + t) * a.n_v + h) * DV + slice * NC + c] = from_float<T>(sum * a.scale);
        }
    };
    int b = 0;
    if (q0 < q1) {
        bool fast = false;
        if (!HELPERS || help >= 0) {
            fetch(q0);
            fast = stage(q0, 0);
            if (HELPERS && q0 + TB < q1) fetch(q0 + TB);
        }
        for (int t0 = q0; t0 < q1; t0 += TB, b ^= 1) {
            const int n = min(TB, q1 - t0);
            const bool any = __syncthreads_or(fast);
            if (!HELPERS) {
                if (t0 + TB < q1) fetch(t0 + TB);
                if (t0 > q0) results(t0 - TB, b ^ 1);
            } else if (help >= 0) {
                if (t0 + TB < q1) fast = stage(t0 + TB, b ^ 1);
                if (t0 + 2 * TB < q1) fetch(t0 + 2 * TB);
                if (t0 > q0) results(t0 - TB, b ^ 1);
                continue;
            }
            // G tokens at once: what they read is on its way before the first is worked out, and a token's products need
            // only the state that the one before left
            auto tokens = [&](auto slow, auto count, int t) {
                constexpr bool SLOW = decltype(slow)::value;
                constexpr int G = decltype(count)::value;
                uint64_t d2[G], once2[G], v2[G][C], o2[G][C];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s_d[b][t + g]);
                    d2[g] = d.x, once2[g] = d.y;
#pragma unroll
                    for (int c = 0; c < C; ++c) v2[g][c] = reinterpret_cast<const uint64_t*>(&s_v[b][t + g][col])[c];
                }
#pragma unroll
                for (int i = 0; i < R; i += 4) {
                    ulonglong2 k4[G], q4[G];
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        k4[g] = *reinterpret_cast<const ulonglong2*>(&s_k[b][t + g][row0 + i]);
                        q4[g] = *reinterpret_cast<const ulonglong2*>(&s_q[b][t + g][row0 + i]);
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint64_t kk = j == 0 ? k4[g].x : k4[g].y, qq = j == 0 ? q4[g].x : q4[g].y;
#pragma unroll
                            for (int c = 0; c < C; ++c) {
                                uint64_t& y = x[c][i / 2 + j];
                                y = f2_fma(y, d2[g], f2_fma(kk, v2[g][c], SLOW ? y : f2_mul(y, once2[g])));
                                o2[g][c] = i + j == 0 ? f2_mul(qq, y) : f2_fma(qq, y, o2[g][c]);
                            }
                        }
                }
                float o[G][C];
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float2 y = f2_get(o2[g][c]);
                        o[g][c] = y.x + y.y;
                    }
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int c = 0; c < C; ++c) o[g][c] += __shfl_xor_sync(0xffffffffu, o[g][c], kRowLanes);
                if (lane < kRowLanes) {
#pragma unroll
                    for (int g = 0; g < G; ++g) *reinterpret_cast<Cols*>(&s_o[b][t + g][warp][col]) = Floats<C>::put(o[g]);
                }
            };
            auto all = [&](auto slow) {
                int t = 0;
#pragma unroll 1
                for (; t + 4 <= n; t += 4) tokens(slow, std::integral_constant<int, 4>{}, t);
#pragma unroll 1
                for (; t < n; ++t) tokens(slow, std::integral_constant<int, 1>{}, t);
            };
            if (!any)
                all(std::true_type{});
            else
                all(std::false_type{});
            if (!HELPERS && t0 + TB < q1) fast = stage(t0 + TB, b ^ 1);
        }
        __syncthreads();
        if (!HELPERS || help >= 0) results(q0 + (q1 - 1 - q0) / TB * TB, b ^ 1);
    }
    if (dst >= 0 && walker) {
        float* p = a.state + ((size_t)dst * a.n_v + h) * head + at;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float2 z = f2_get(x[c][i / 2]);
                y[c] = i % 2 ? z.y : z.x;
            }
            __stcs(reinterpret_cast<Cols*>(p + (size_t)i * DV), Floats<C>::put(y));
        }
    }
}

template <typename T, int DK, int DV, int NC>
cudaError_t run(const LinearArgs& a, cudaStream_t stream) {
    const unsigned ctas = (unsigned)a.n_seqs * a.n_v * (DV / NC);
    if (!a.q_start) {
        linear_step_kernel<T, DK, DV, NC, true><<<ctas, kThreads, 0, stream>>>(a);
    } else if constexpr (DK == 128 || NC == 64) {  // (others walk)
        linear_step_kernel<T, DK, DV, NC, false><<<ctas, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename T, int DK, int DV, int NC, int HELPERS>
cudaError_t walk(const LinearArgs& a, cudaStream_t stream) {
    linear_walk_kernel<T, DK, DV, NC, HELPERS><<<(unsigned)a.n_seqs * a.n_v * (DV / NC), kThreads + HELPERS, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int DK, int DV>
cudaError_t pick(int sms, const LinearArgs& a, cudaStream_t stream) {
    // In units of 64 columns: columns of 64 from two units an SM on, else of 32. Chunks of up to two units for three SMs
    // take columns of 16 and packed pairs of rows (256 tokens of 96 units of 128 x 64 in fp32: 52 us, against 65 in columns
    // of 32; of 128 units 73 and 65), with helpers up to a unit for two SMs (500 tokens of 24 units of 64 x 64: 32 us, 43
    // without, 73 in columns of 32; with two CTAs of 192 threads an SM: 96 units 72 and 66), and at dim_k = 64 the others
    // pairs in columns of 32 (500 tokens of 128 units 70 us against 91; at 128 rows nothing is gained).
    const long long units = (long long)a.n_seqs * a.n_v * (DV / 64);
    if (a.q_start && units * 2 <= sms) return walk<T, DK, DV, 16, 64>(a, stream);
    if (a.q_start && units * 3 <= 2LL * sms) return walk<T, DK, DV, 16, 0>(a, stream);
    if (units >= 2LL * sms) return run<T, DK, DV, 64>(a, stream);
    if constexpr (DK == 64)
        if (a.q_start) return walk<T, DK, DV, 32, 0>(a, stream);
    return run<T, DK, DV, 32>(a, stream);
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
