// ops_attend_block_128.hip -- blocks of new tokens, heads of up to 128 values.
#include "ops_attend_block.hpp"

namespace ops {

const void* block_kernel_128(bool f16, bool f32_out, bool share, int row_tiles, int* lds) { return block_kernel_types<128>(f16, f32_out, share, row_tiles, lds); }

}  // namespace ops
