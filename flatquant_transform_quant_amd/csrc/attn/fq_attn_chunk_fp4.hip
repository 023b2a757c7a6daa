// Attention of new tokens over a E2M1 cache (a file a format, so that they compile side by side).
#include "fq_attn_chunk.h"

namespace fq {

hipError_t launch_attn_chunk_fp4(const ChunkArgs& a, void* ws, hipStream_t s) { return chunk_mode<kKvFp4>(a, ws, s); }

}  // namespace fq
