// ops_lora_b4_g128.hip -- adapted projection, 4-bit codes in groups of 128
#include "ops_lora_kernel.hpp"

namespace ops {
int lora_launch_b4_g128(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st)
{
    return lora_pick<4, 128>(p, rt, ct, xf32, sbf, st);
}
}  // namespace ops
