// ops_lora_b2_g64.hip -- adapted projection, 2-bit codes in groups of 64
#include "ops_lora_kernel.hpp"

namespace ops {
int lora_launch_b2_g64(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st)
{
    return lora_pick<2, 64>(p, rt, ct, xf32, sbf, st);
}
}  // namespace ops
