// The attention kernels for rows of up to 256 values (cache_attention_few.cuh, cache_attention_many.cuh).
#include "cache_attention_launch.cuh"

namespace db {
int launch_attention_256(const AttnParams& p, uint32_t type, uint32_t blocks, cudaStream_t s) {
  return launch_attention<256>(p, type, blocks, s);
}
}  // namespace db
