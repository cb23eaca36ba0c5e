// decode_scored_bf16.cu -- decode attention of decode_frag.cuh: 16-bit pools, weights summed, __nv_bfloat16 activations.
#include "decode_frag.cuh"

namespace pkv {

cudaError_t launch_frag_scored_bf16(int head_dim, int group, const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t stream) {
    return launch_frag_of<__nv_bfloat16, false>(head_dim, group, a, tk, tv, stream);
}

cudaError_t frag_ctas_per_sm_scored_bf16(int head_dim, int group, int* out) {
    return frag_ctas_per_sm_of<__nv_bfloat16, false>(head_dim, group, out);
}

}  // namespace pkv
