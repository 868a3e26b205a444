// bf16 instances of the decode over an 8-bit cache.
#include "pa_fp8_decode.cuh"

namespace pa {
int launch_decode_fp8_bf16(int head_dim, int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return d8::launch_dtype<__nv_bfloat16>(head_dim, group, p, stream);
}
}  // namespace pa
