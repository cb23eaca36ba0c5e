// decode_q8_bf16.cu -- decode attention of decode_frag.cuh: 8-bit pools, __nv_bfloat16 activations.
#include "decode_frag.cuh"

namespace pkv {

cudaError_t launch_frag_q8_bf16(int head_dim, int group, const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t stream) {
    return launch_frag_of<__nv_bfloat16, true>(head_dim, group, a, tk, tv, stream);
}

cudaError_t frag_ctas_per_sm_q8_bf16(int head_dim, int group, int* out) {
    return frag_ctas_per_sm_of<__nv_bfloat16, true>(head_dim, group, out);
}

cudaError_t launch_frag_multi_bf16(int head_dim, int columns, const FragArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t stream) {
    return launch_frag_multi_of<__nv_bfloat16>(head_dim, columns, a, tk, tv, stream);
}

cudaError_t frag_multi_ctas_per_sm_bf16(int head_dim, int columns, int* out) {
    return frag_multi_ctas_per_sm_of<__nv_bfloat16>(head_dim, columns, out);
}

}  // namespace pkv
