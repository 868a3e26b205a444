// The chunked-prefill kernel for prompt chunks over an 8-bit cache, whose values it attends
// laid out in blocks of kExpandRows rows.  One 16-bit value of the model's type a weight, as
// pa_prefill_batch has, would add a quarter to the outputs' own rounding (root mean square
// 2.06e-3 where that alone is 1.66e-3 in bf16).  So
//   bf16: V and weights in fp16, eight times as fine, V over the greatest scale of a tile
//         (kScaled).  512 queries after 8192 tokens, 64/8 heads, with the layout in front:
//         126 us, where one bf16 value takes 115 and two 185.  (V's codes as they are, and a
//         block's scale added to its keys' scores: exact for all scales, 145.)
//   fp16: each weight as two values (kTwoP).
#include "pa_prefill.cuh"

namespace pa {
namespace {
using namespace pf;

template <typename T>
int launch_group(int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    constexpr bool kScaled = std::is_same<T, __nv_bfloat16>::value;
    return group == 1   ? launch_tc_t<T, kExpandRows, 1, !kScaled, kScaled>(p, grid, stream)
           : group == 2 ? launch_tc_t<T, kExpandRows, 2, !kScaled, kScaled>(p, grid, stream)
           : group == 4 ? launch_tc_t<T, kExpandRows, 4, !kScaled, kScaled>(p, grid, stream)
           : group == 8 ? launch_tc_t<T, kExpandRows, 8, !kScaled, kScaled>(p, grid, stream)
                        : PA_ERR_UNSUPPORTED;
}
}  // namespace

int launch_prefill_fp8(pa_dtype dt, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    return dt == PA_BF16 ? launch_group<__nv_bfloat16>(group, p, grid, stream) : launch_group<__half>(group, p, grid, stream);
}
}  // namespace pa
