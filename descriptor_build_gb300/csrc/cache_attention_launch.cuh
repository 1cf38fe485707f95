// The choice among the attention kernels of one padded width.
#pragma once

#include "cache_attention_few.cuh"
#include "cache_attention_many.cuh"

namespace db {

template <typename T, uint32_t kPad, bool kCodes>
int launch_blocks(const AttnParams& p, uint32_t blocks, cudaStream_t s) {
  switch (blocks) {
    case 1:
      return launch_few<T, kPad, kCodes, 1, 1>(p, s);
    case 2:
      // 16 rows of 256 16-bit values are more than a warp's registers hold: two
      // warps share them, and two CTAs an SM (113 sequences of 4,223 tokens, 8 key
      // heads: 687 us, 928 with a warp for all; int8 697 and 661, E4M3 475 and 544).
      if constexpr (kPad == 256 && !kCodes)
        return launch_few<T, kPad, kCodes, 1, 2>(p, s);
      else
        return launch_few<T, kPad, kCodes, 2, 1>(p, s);
    case 4:
      if constexpr (kCodes) return launch_few<T, kPad, kCodes, 2, 2>(p, s);
      return -EINVAL;
    case kManyBlocks:
      return launch_many<T, kPad, kCodes, 1>(p, s);
    default:
      if constexpr (kPad <= 128) return launch_many<T, kPad, kCodes, 2>(p, s);
      return -EINVAL;
  }
}

template <uint32_t kPad>
int launch_attention(const AttnParams& p, uint32_t type, uint32_t blocks, cudaStream_t s) {
  const bool codes = item_bytes(p.c.type) == 1;
  if (type == DB_BF16)
    return codes ? launch_blocks<__nv_bfloat16, kPad, true>(p, blocks, s)
                 : launch_blocks<__nv_bfloat16, kPad, false>(p, blocks, s);
  return codes ? launch_blocks<__half, kPad, true>(p, blocks, s)
               : launch_blocks<__half, kPad, false>(p, blocks, s);
}

}  // namespace db
