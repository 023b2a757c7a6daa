// Attention of new tokens over a int8 cache (a file a format, so that they compile side by side).
#include "fq_attn_chunk.h"

namespace fq {

hipError_t launch_attn_chunk_int8(const ChunkArgs& a, void* ws, hipStream_t s) { return chunk_mode<kKvInt8>(a, ws, s); }

}  // namespace fq
