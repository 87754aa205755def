// ops_lora_b4_g64.hip -- adapted projection, 4-bit codes in groups of 64
#include "ops_lora_kernel.hpp"

namespace ops {
int lora_launch_b4_g64(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st)
{
    return lora_pick<4, 64>(p, rt, ct, xf32, sbf, st);
}
}  // namespace ops
