// db_cache_attention: arguments, workspace and the choice of a kernel
// (cache_attention.cuh).
#include <cmath>

#include <algorithm>

#include "cache_attention.cuh"

namespace db {
namespace {

constexpr size_t kHeader = 4 * kMaxAttnCtas;  // arrival counters

uint32_t padded_width(uint32_t width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }

// Blocks of 8 query rows of an item. Up to 16 rows memory is the bound of the
// kernel for few; with 32, warps that share a ring two by two are faster for
// most codes (64 sequences of 20,000 tokens, 2 key heads: int8 380 us, the kernel for
// many 412, E4M3 290 and 255; 48 of 3,000, 8 key heads, E4M3 148 and 161) and slower for
// 16-bit values (334, 270).
// Above 128 rows two tiles of 128 share a CTA's loads (wide trees of 488 rows
// 396 us one by one, 312 so) where TMEM holds the sums of both.
// The rows are those of max_tokens, for all requests of a call: 100 single tokens of 8
// query heads to a key head over 3,000 E4M3 tokens take 41 us with max_tokens 1, 124 with
// 61 (bf16 58 and 89).
uint32_t blocks_for(uint64_t rows, uint32_t pad, bool codes) {
  if (rows > 128 && pad <= 128) return 2 * kManyBlocks;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 && codes ? 4 : kManyBlocks;
}

bool shape_ok(uint32_t n, uint32_t q_heads, uint32_t heads, uint32_t width, uint32_t max_tokens) {
  if (n > 65536 || !heads || !q_heads || q_heads % heads || q_heads / heads > kMaxGroup) return false;
  return width && width % 16 == 0 && width <= 256 && max_tokens && max_tokens < 1u << 24;
}

size_t workspace_bytes(uint32_t group, uint32_t width, uint32_t max_tokens) {
  const uint32_t pad = padded_width(width);
  size_t floats = 0;  // the larger need of 16-bit values and codes
  for (const bool codes : {false, true}) {
    const uint32_t blocks = blocks_for((uint64_t)max_tokens * group, pad, codes);
    floats = std::max(floats, (size_t)2 * attn_grid(attn_ctas_per_sm(pad, codes, blocks)) * partial_floats(8 * blocks, pad));
  }
  return (kHeader + floats * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_cache_attention_workspace_size(uint32_t n, uint32_t q_heads, uint32_t heads,
                                                 uint32_t width, uint32_t max_tokens, size_t* bytes) {
  if (!bytes || !shape_ok(n, q_heads, heads, width, max_tokens)) return -EINVAL;
  *bytes = workspace_bytes(q_heads / heads, width, max_tokens);
  return 0;
}

extern "C" int db_cache_attention(const db_page_tables* t, const db_cache_batch* b,
                                  const db_cache_layer* c, const db_cache_rows* q,
                                  const db_cache_rows* out, uint32_t type, uint32_t q_heads,
                                  uint32_t max_tokens, float scale, const uint32_t* mask,
                                  uint32_t mask_words, float* lse, uint8_t* status, db_counters* ctr,
                                  void* ws, size_t ws_bytes, void* stream) {
  CacheView view;
  if (check_cache(t, b, status, ctr, &view) || check_layer(t, c)) return -EINVAL;
  if (type != DB_BF16 && type != DB_F16) return -EINVAL;
  if (item_bytes(c->type) == 2 && c->type != type) return -EINVAL;
  if (!shape_ok(b->n, q_heads, c->heads, c->width, max_tokens)) return -EINVAL;
  if (check_rows(q, b->rows, q_heads, c->width, type, false) ||
      check_rows(out, b->rows, q_heads, c->width, type, true))
    return -EINVAL;
  if (!std::isfinite(scale * 1.4426950408889634f)) return -EINVAL;
  if (!aligned(mask, 4) || !aligned(lse, 4) || (mask && (!mask_words || max_tokens > 32ull * mask_words)))
    return -EINVAL;
  if (!ws || !aligned(ws, 256)) return -EINVAL;
  if (ws_bytes < workspace_bytes(q_heads / c->heads, c->width, max_tokens)) return -ENOSPC;
  const cudaStream_t s = (cudaStream_t)stream;
  if (const int e = zero_counters(ctr, s)) return e;
  if (!b->n) return 0;
  AttnParams p = {};
  p.view = view;
  p.c = *c;
  p.q = *q;
  p.out = *out;
  p.group = q_heads / c->heads;
  p.max_tokens = max_tokens;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.mask = mask;
  p.mask_words = mask_words;
  p.lse = lse;
  const uint64_t row = (uint64_t)c->width * item_bytes(c->type);
  p.token_step = c->heads_first ? row : c->heads * row;
  p.head_step = c->heads_first ? t->page_tokens * row : row;
  p.scale_token_step = c->heads_first ? 1 : c->heads;
  p.scale_head_step = c->heads_first ? t->page_tokens : 1;
  p.narrow = std::max(c->k_stride, c->v_stride) <= ((1ull << 36) - 16) / t->n_pages;
  p.arrived = (unsigned int*)ws;
  p.partial = (float*)((char*)ws + kHeader);
  const uint32_t blocks = blocks_for((uint64_t)max_tokens * p.group, padded_width(c->width), item_bytes(c->type) == 1);
  switch (padded_width(c->width)) {
    case 64:
      return launch_attention_64(p, type, blocks, s);
    case 128:
      return launch_attention_128(p, type, blocks, s);
    default:
      return launch_attention_256(p, type, blocks, s);
  }
}
