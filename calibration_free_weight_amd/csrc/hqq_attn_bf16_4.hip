// hqq_attn_bf16_4.hip -- attention over a cache of 4-bit codes, bfloat16 rows.
#include "hqq_attn_kernel.h"

namespace hqq {

hipError_t launch_attn_bf16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    return by_dim<Bf16, 4, false>(a, x, stream);
}

}  // namespace hqq
