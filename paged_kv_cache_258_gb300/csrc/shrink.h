// shrink.h -- declarations of the cache-shrinking calls: 8-bit pools, decode that sums its attention
// weights, eviction (not installed).
#pragma once

#include "internal.h"

namespace pkv {

// Tensor-map element code of an 8-bit pool (beside the pkv_dtype values kv_tensor_map takes).
constexpr int kCodesE4M3 = 3;

// Least exponent of a block's scale: below it the scale of all-tiny rows stops shrinking, so that
// code * scale (codes go down to 2^-9) stays a normal number of the rows' type (bf16: 2^-126) or a
// multiple of its least step (fp16: 2^-24).
inline int q8_min_exp(int dtype) { return dtype == PKV_F16 ? -15 : -117; }

// One decode launch over an 8-bit pool, or over a 16-bit pool with its weights summed. Inside `d`
// k_layer / v_layer are codes for an 8-bit pool.
struct FragArgs {
    DecodeArgs d;
    const float* k_scales = nullptr;  // [num_blocks][n_kv] of this layer (8-bit pools)
    const float* v_scales = nullptr;
    float* z = nullptr;               // [n_seqs][n_kv][max_blocks*16][G] base-2 logits, or null: weights not summed
};

// scores[s][g][j] += sum over the group's heads of 2^(z - lse), j < the sequence's length.
struct ScoreArgs {
    const float* z;
    const float* part_ml;  // [n_seqs][n_q][n_parts][2]
    const int32_t* lens;
    float* scores;         // [n_seqs][n_kv][stride]
    long long stride;
    int n_seqs, n_kv, group, max_blocks, n_parts, bpp;
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
    int slices;            // CTAs that share the columns of one (sequence, head)
};

cudaError_t frag_ctas_per_sm(int dtype, bool q8, int head_dim, int group, int* out);
cudaError_t launch_frag_decode(int dtype, bool q8, int head_dim, int group, const FragArgs& a, cudaStream_t stream);
cudaError_t launch_scores(const ScoreArgs& a, cudaStream_t stream);
cudaError_t launch_q8_append(int dtype, int head_dim, const Q8AppendArgs& a, cudaStream_t stream);
cudaError_t launch_q8_copy(const Q8CopyArgs& a, cudaStream_t stream);
cudaError_t launch_q8_widen(int dtype, int head_dim, const Q8WidenArgs& a, cudaStream_t stream);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace pkv
