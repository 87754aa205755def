// ops_attend_block_256.hip -- blocks of new tokens, heads of up to 256 values.
#include "ops_attend_block.hpp"

namespace ops {

const void* block_kernel_256(bool f16, bool f32_out, bool share, int row_tiles, int* lds) { return block_kernel_types<256>(f16, f32_out, share, row_tiles, lds); }

}  // namespace ops
