// f16 instances of the kernel for several query positions over one cache.
#include "pa_window.cuh"

namespace pa {
int launch_window_f16(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    return wnd::launch_window_dtype<__half>(block_size, group, p, grid, stream);
}
}  // namespace pa
