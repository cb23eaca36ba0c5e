// prefill_widened_f16.cu -- prefill attention over rows widened from 8-bit codes to __half.
#include "prefill_umma.cuh"
#include "shrink.h"

namespace pkv {

cudaError_t launch_prefill_widened_f16(int head_dim, int group, const PrefillArgs& a, const CUtensorMap& tk,
                                       const CUtensorMap& tv, cudaStream_t stream) {
    return launch_prefill_umma_dtype<__half, true>(head_dim, group, a, tk, tv, stream);
}

}  // namespace pkv
