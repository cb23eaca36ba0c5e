// prefill_widened_bf16.cu -- prefill attention over rows widened from 8-bit codes to __nv_bfloat16.
#include "prefill_umma.cuh"
#include "shrink.h"

namespace pkv {

cudaError_t launch_prefill_widened_bf16(int head_dim, int group, const PrefillArgs& a, const CUtensorMap& tk,
                                       const CUtensorMap& tv, cudaStream_t stream) {
    return launch_prefill_umma_dtype<__nv_bfloat16, true>(head_dim, group, a, tk, tv, stream);
}

}  // namespace pkv
