// shrink.h -- declarations of the cache-shrinking calls: 8-bit pools, decode that sums its attention
// weights, eviction (not installed).
#pragma once

#include "internal.h"

namespace pkv {

// Tensor-map element code of an 8-bit pool (beside the pkv_dtype values kv_tensor_map takes).
constexpr int kCodesE4M3 = 3;

#ifdef __CUDACC__
// Lets the next launch on the stream, if it is a programmatic dependent, be placed from here on. Called behind
// the wait for the launch before: a next launch with an OVERLAP_PREVIOUS flag reads its inputs at once, trusting
// this kernel not to write them, and must not do so while the launch before this one still may. Ahead of
// the wait it was no faster either: a step's append and decode over 24 layers, 4 x 300 tokens in 8 bits, 206.6 us
// against 203.4.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// Least exponent of a block's scale: below it the scale of all-tiny rows stops shrinking, so that
// code * scale (codes go down to 2^-9) stays a normal number of the rows' type (bf16: 2^-126) or a
// multiple of its least step (fp16: 2^-24).
inline int q8_min_exp(int dtype) { return dtype == PKV_F16 ? -15 : -117; }

// Least blocks of a partition (one iteration of each of a CTA's warps), and arrival counters of a workspace
// (one for each CTA of the widest launch).
constexpr int kMinPartition = 8;
constexpr int kMaxRuns = 2048;
// Runs of a prompt chunk's launch, whose workspace is sized without asking a device.
constexpr int kChunkRuns = 640;
// Most partitions of a context in a grid of partitions: they are one cluster, and 8 is the portable limit.
constexpr int kMaxCluster = 8;
// Most blocks of a partition in a grid of partitions (its logits stay in shared memory).
constexpr int kMaxPartition = 32;

// One decode launch over an 8-bit pool, or over a 16-bit pool with its weights summed. Inside `d`:
// k_layer / v_layer are codes for an 8-bit pool; n_parts = CTAs along x; part_o [n_parts][2][G][D] and
// part_ml [n_parts][2][G] (max, sum) are the runs' partials; dense, counters, call_tag and bpp are unused.
struct FragArgs {
    DecodeArgs d;
    const float* k_scales = nullptr;  // [num_blocks][n_kv] of this layer (8-bit pools)
    const float* v_scales = nullptr;
    unsigned int* arrivals = nullptr; // [n_parts], zero between calls
    float2* row_ml = nullptr;         // [n_seqs][n_q] each row's (max, sum), or null: weights not summed
    float* z = nullptr;               // [n_seqs][n_kv][max_blocks*16][G] base-2 logits, or null
    float* scores = nullptr;          // partitions: [n_seqs][n_kv][score_stride], or null
    long long score_stride = 0;
    // Prompt chunks (C columns of C / G tokens x G heads): d.n_seqs = sequences x groups of tokens.
    const int32_t* q_start = nullptr; // [sequences + 1]
    int n_tokens = 0, max_query = 0;
    int groups = 0;                   // groups of a sequence: ceil(max_query / (C / G))
    int shift = 0;                    // log2 G
    int partition = 0;                // > 0: a grid of partitions of so many blocks, n_parts a cluster; 0: runs
};

// scores[s][g][j] += sum over the group's heads of 2^(z - max) / sum, j < the sequence's length.
struct ScoreArgs {
    const float* z;
    const float2* row_ml;  // [n_seqs][n_q]
    const int32_t* lens;
    float* scores;         // [n_seqs][n_kv][stride]
    long long stride;
    int n_seqs, n_kv, group, max_blocks;
};

struct Q8AppendArgs {
    const void* k;         // [n_tok][n_kv][D] fp16 or bf16
    const void* v;
    const int64_t* slots;
    uint8_t* k_codes;      // [num_blocks][n_kv][16][D] of this layer
    uint8_t* v_codes;
    float* k_scales;       // [num_blocks][n_kv] of this layer
    float* v_scales;
    unsigned int* status;
    int n_tok, n_kv, num_blocks, min_exp;
};

struct Q8CopyArgs {
    uint8_t* k_codes;      // whole pools
    uint8_t* v_codes;
    float* k_scales;
    float* v_scales;
    const int32_t* pairs;
    unsigned int* status;
    int n_pairs, n_layers, n_kv, num_blocks;
    size_t block_bytes;    // codes of one block of one layer
};

// Rows of the listed sequences' blocks widened to the activations' type in a scratch layer that is
// indexed by physical block like the pool.
struct Q8WidenArgs {
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scales;
    const float* v_scales;
    const int32_t* tables;
    const int32_t* lens;
    void* k_out;
    void* v_out;
    unsigned int* status;
    unsigned int* v_nan;   // set to 1 if a row of V in a context holds a NaN code
    int n_seqs, n_kv, num_blocks, max_blocks;
};

struct EvictArgs {
    void* k_pool;          // whole pools (codes for 8-bit pools)
    void* v_pool;
    float* k_scales;       // whole scale arrays, or null (pools of another type)
    float* v_scales;
    const int32_t* src;    // [n_seqs][max_blocks]
    const int32_t* dst;
    const int32_t* lens;
    const int32_t* keep;
    const float* scores;   // [L][n_seqs][n_kv][stride]
    float* new_scores;
    int32_t* kept;         // [L][n_seqs][n_kv][max_keep]
    float* old_scales;     // workspace [2][L][n_seqs][n_kv][max_blocks] (8-bit pools)
    unsigned int* status;
    long long stride;
    int n_layers, n_seqs, n_kv, num_blocks, max_blocks, max_keep, recent;
    int row_bytes;         // one row of one head
    int parts;             // CTAs that share the rows of one (layer, sequence, head) of K or V
    int slices;            // most column slices of a row, where rows move in place
};

// Launches `kernel` as a programmatic dependent of the kernel before it on the stream: its CTAs may be
// placed while that one drains, and wait (griddepcontrol.wait) for its end before they touch anything
// in global memory. So the order is that of an ordinary launch, without its start-up.
// cluster > 1: thread-block clusters of that many CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                             const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t frag_ctas_per_sm(int dtype, bool q8, int head_dim, int group, int* out);
cudaError_t launch_frag_decode(int dtype, bool q8, int head_dim, int group, const FragArgs& a, cudaStream_t stream);
cudaError_t frag_multi_ctas_per_sm(int dtype, int head_dim, int columns, int* out);
cudaError_t launch_frag_multi(int dtype, int head_dim, int columns, const FragArgs& a, cudaStream_t stream);
cudaError_t launch_scores(const ScoreArgs& a, cudaStream_t stream);
cudaError_t launch_q8_append(int dtype, int head_dim, const Q8AppendArgs& a, cudaStream_t stream);
cudaError_t launch_q8_copy(const Q8CopyArgs& a, cudaStream_t stream);
// Prefill attention over the layer that launch_q8_widen filled, and before either its tensor maps: they refuse
// (cudaErrorInvalidDevicePointer) codes or a workspace that are not memory of the current device.
cudaError_t widened_maps(int dtype, int head_dim, const Q8WidenArgs& w, CUtensorMap* tk, CUtensorMap* tv);
cudaError_t launch_prefill_widened(int dtype, int head_dim, int group, const PrefillArgs& a, const CUtensorMap& tk,
                                   const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_q8_widen(int dtype, int head_dim, const Q8WidenArgs& a, cudaStream_t stream);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace pkv
