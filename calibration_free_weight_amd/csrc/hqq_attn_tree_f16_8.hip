// hqq_attn_tree_f16_8.hip -- attention over a cache of 8-bit codes, binary16 rows.
#include "hqq_attn_kernel.h"

namespace hqq {

hipError_t launch_attn_tree_f16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    return by_dim<F16, 8, true>(a, x, stream);
}

}  // namespace hqq
