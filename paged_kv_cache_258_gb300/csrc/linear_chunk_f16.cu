// linear_chunk_f16.cu -- the tensor-core kernel of linear attention for fp16.
#include "linear_chunk.cuh"

namespace pkv {
cudaError_t launch_linear_chunk_f16(int dk, const ChunkArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, cudaStream_t stream) {
    return launch_linear_chunk_dtype<__half>(dk, a, q, k, v, stream);
}
}  // namespace pkv
