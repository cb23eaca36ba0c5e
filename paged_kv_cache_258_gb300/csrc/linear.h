// linear.h -- arguments and launchers of linear attention and of tables built on the GPU (not installed).
#pragma once

#include "internal.h"

namespace pkv {

struct ExtendArgs {
    const int32_t* free_blocks;  // [n_free]
    const int32_t* used;
    int32_t* tables;             // [n_seqs][max_blocks]
    const int32_t* lens;         // [n_seqs]
    const int32_t* new_tokens;   // [n_seqs], or nullptr: one each
    int64_t* slots;              // [max_tokens]
    int32_t* query_start;        // [n_seqs + 1]
    int32_t* new_lens;           // [n_seqs], lens itself or apart
    int32_t* totals;             // [3], its first may be used
    unsigned int* status;
    int num_blocks, n_free, max_blocks, n_seqs, max_tokens;
};

// One layer of linear attention. Sequence s owns rows q_start[s] .. q_start[s+1]-1 of the packed tokens, or row s
// where q_start is nullptr.
struct LinearArgs {
    const void* q;               // [n_tokens][n_qk][DK]
    const void* k;
    const void* v;               // [n_tokens][n_v][DV]
    void* out;                   // [n_tokens][n_v][DV]
    const float* log_decay;      // nullptr: none
    long long decay_stride;      // floats from token to token, 0: one for each head
    float* state;                // this layer: [n_slots][n_v][DK][DV]
    const int32_t* src;          // [n_seqs], negative: zeros
    const int32_t* dst;          // [n_seqs], negative: not kept
    const int32_t* q_start;
    unsigned int* status;
    int n_seqs, n_qk, n_v, n_slots, n_tokens, max_query;
    float scale;
};

cudaError_t launch_extend_tables(const ExtendArgs& a, cudaStream_t stream, int sms, int* n_launches);
// Token after token with the state in registers (linear_step.cu).
cudaError_t launch_linear_step(int dtype, int dk, int dv, int sms, const LinearArgs& a, cudaStream_t stream);

// Long chunks of 16-bit types on the tensor cores (linear_chunk.cuh). A sequence may be shared out in segments along
// its length: a first launch leaves what each segment but the last adds to the state, the second starts each from
// the sum of those before.
struct ChunkArgs {
    LinearArgs l;
    int dv, slices;         // dim_v, and its slices of 64
    int n_segs, seg_tokens; // segments of a sequence (1: whole), tokens of each: a multiple of 128
    bool take_more = false; // a CTA goes on with other CTAs' work (n_segs == 1, and more CTAs than the GPU holds)
    float* start = nullptr; // [n_seqs][n_v][DK][DV]: the states the sequences start from
    float* added = nullptr; // [n_seqs][n_segs - 1][n_v][DK][DV]: what a segment leaves (the first: with the start)
    float* sums = nullptr;  // [n_seqs][n_segs - 1][n_v]: log2 of the decay over a segment
};
cudaError_t launch_linear_chunk_f16(int dk, const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                    const CUtensorMap& v, cudaStream_t stream);
cudaError_t launch_linear_chunk_bf16(int dk, const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, cudaStream_t stream);

// Tensor map of packed rows of `width` 16-bit elements, in boxes of 64 columns x box_rows rows (tmap.cu).
cudaError_t rows_tensor_map(const void* base, long long rows, int width, int dtype, int box_rows, CUtensorMap* out);

}  // namespace pkv
