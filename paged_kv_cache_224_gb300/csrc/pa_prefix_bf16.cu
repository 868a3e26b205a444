// bf16 instances of the shared-prefix step.
#include "pa_prefix.cuh"

namespace pa {
int launch_prefix_bf16(int block_size, int group, const PrefixLaunch &pl, unsigned grid, cudaStream_t stream) {
    return pfx::launch_prefix_dtype<__nv_bfloat16>(block_size, group, pl, grid, stream);
}
}  // namespace pa
