// The chunked-prefill kernel with softmax weights as two 16-bit values, for the prompt
// chunks over an 8-bit cache, whose values it attends laid out in blocks of kExpandRows
// rows.  One 16-bit value a weight, as pa_prefill_batch has, would add half as much again
// to the outputs' own rounding (root mean square 2.06e-3 where that alone is 1.66e-3 in
// bf16).
#include "pa_prefill.cuh"

namespace pa {
namespace {
using namespace pf;

template <typename T>
int launch_group(int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    return group == 1   ? launch_tc_t<T, kExpandRows, 1, true>(p, grid, stream)
           : group == 2 ? launch_tc_t<T, kExpandRows, 2, true>(p, grid, stream)
           : group == 4 ? launch_tc_t<T, kExpandRows, 4, true>(p, grid, stream)
           : group == 8 ? launch_tc_t<T, kExpandRows, 8, true>(p, grid, stream)
                        : PA_ERR_UNSUPPORTED;
}
}  // namespace

int launch_prefill_two(pa_dtype dt, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    return dt == PA_BF16 ? launch_group<__nv_bfloat16>(group, p, grid, stream) : launch_group<__half>(group, p, grid, stream);
}
}  // namespace pa
