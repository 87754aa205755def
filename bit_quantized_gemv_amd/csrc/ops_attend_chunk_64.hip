// ops_attend_chunk_64.hip -- chunks of new tokens, heads of up to 64 values.
#include "ops_attend_chunk.hpp"

namespace ops {

const void* chunk_kernel_64(bool f16, bool f32_out, int* rows, int* threads, int* lds) { return chunk_kernel_types<64>(f16, f32_out, rows, threads, lds); }

}  // namespace ops
