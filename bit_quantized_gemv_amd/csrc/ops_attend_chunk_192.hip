// ops_attend_chunk_192.hip -- chunks of new tokens, heads of up to 192 values.
#include "ops_attend_chunk.hpp"

namespace ops {

const void* chunk_kernel_192(bool f16, bool f32_out, int row_tiles, ChunkShape* shape) { return chunk_kernel_types<192>(f16, f32_out, row_tiles, shape); }

}  // namespace ops
