// ops_moe_b2_g128.hip -- expert products, 2-bit codes in groups of 128
#include "ops_moe_kernel.hpp"

namespace ops {
int expert_launch_b2_g128(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st)
{
    return sbf ? expert_pick<2, 128, true>(which, p, xf32, st) : expert_pick<2, 128, false>(which, p, xf32, st);
}
}  // namespace ops
