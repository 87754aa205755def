// ops_attend_chunk_96.hip -- chunks of new tokens, heads of up to 96 values.
#include "ops_attend_chunk.hpp"

namespace ops {

const void* chunk_kernel_96(bool f16, bool f32_out, int row_tiles, ChunkShape* shape) { return chunk_kernel_types<96>(f16, f32_out, row_tiles, shape); }

}  // namespace ops
