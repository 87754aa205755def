// ops_attend_chunk_128.hip -- chunks of new tokens, heads of up to 128 values.
#include "ops_attend_chunk.hpp"

namespace ops {

const void* chunk_kernel_128(bool f16, bool f32_out, int row_tiles, ChunkShape* shape) { return chunk_kernel_types<128>(f16, f32_out, row_tiles, shape); }

}  // namespace ops
