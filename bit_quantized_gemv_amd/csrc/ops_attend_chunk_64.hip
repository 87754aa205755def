// ops_attend_chunk_64.hip -- chunks of new tokens, heads of up to 64 values.
#include "ops_attend_chunk.hpp"

namespace ops {

const void* chunk_kernel_64(bool f16, bool f32_out, int row_tiles, ChunkShape* shape) { return chunk_kernel_types<64>(f16, f32_out, row_tiles, shape); }

}  // namespace ops
