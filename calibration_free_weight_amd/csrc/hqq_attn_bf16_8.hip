// hqq_attn_bf16_8.hip -- attention over a cache of 8-bit codes, bfloat16 rows.
#include "hqq_attn_kernel.h"

namespace hqq {

hipError_t launch_attn_bf16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    return by_dim<Bf16, 8>(a, x, stream);
}

}  // namespace hqq
