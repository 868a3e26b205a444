// bf16 instances of the CUDA-core decode that keeps its scores (pa_decode_weights).
#include "pa_decode.cuh"

namespace pa {
int launch_decode_scores_bf16(int head_dim, int block_size, int group, const DecodeParams &p, cudaStream_t stream) {
    return launch_decode_dtype<__nv_bfloat16, true>(head_dim, block_size, group, p, stream);
}
}  // namespace pa
