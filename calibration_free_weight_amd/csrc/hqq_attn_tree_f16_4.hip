// hqq_attn_tree_f16_4.hip -- attention over a cache of 4-bit codes, binary16 rows.
#include "hqq_attn_kernel.h"

namespace hqq {

hipError_t launch_attn_tree_f16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    return by_dim<F16, 4, true>(a, x, stream);
}

}  // namespace hqq
