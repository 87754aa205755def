// ops_moe_b4_g64.hip -- expert products, 4-bit codes in groups of 64
#include "ops_moe_kernel.hpp"

namespace ops {
int expert_launch_b4_g64(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st)
{
    return sbf ? expert_pick<4, 64, true>(which, p, xf32, st) : expert_pick<4, 64, false>(which, p, xf32, st);
}
}  // namespace ops
