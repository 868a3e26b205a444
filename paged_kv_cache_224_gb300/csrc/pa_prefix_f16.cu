// f16 instances of the shared-prefix pass.
#include "pa_prefix.cuh"

namespace pa {
int launch_prefix_f16(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    return pfx::launch_prefix_dtype<__half>(block_size, group, p, grid, stream);
}
}  // namespace pa
