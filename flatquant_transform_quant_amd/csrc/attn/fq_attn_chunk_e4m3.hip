// Attention of new tokens over a E4M3 cache (a file a format, so that they compile side by side).
#include "fq_attn_chunk.h"

namespace fq {

hipError_t launch_attn_chunk_e4m3(const ChunkArgs& a, void* ws, hipStream_t s) { return chunk_mode<kKvE4M3>(a, ws, s); }

}  // namespace fq
