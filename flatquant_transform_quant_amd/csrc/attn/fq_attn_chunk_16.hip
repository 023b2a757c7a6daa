// Attention of new tokens over a 16-bit cache (a file a format, so that they compile side by side).
#include "fq_attn_chunk.h"

namespace fq {

hipError_t launch_attn_chunk_16(const ChunkArgs& a, void* ws, hipStream_t s) { return chunk_mode<kKv16>(a, ws, s); }

}  // namespace fq
