// ops_attend_block_64.hip -- blocks of new tokens, heads of up to 64 values.
#include "ops_attend_block.hpp"

namespace ops {

const void* block_kernel_64(bool f16, bool f32_out, bool share, int row_tiles, int* lds) { return block_kernel_types<64>(f16, f32_out, share, row_tiles, lds); }

}  // namespace ops
