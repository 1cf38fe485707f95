// Attention over a paged cache for up to 16 query rows of a key head, with codes
// 32 (cache_attention.cuh: the mathematics and the way work is cut): single
// tokens, mostly, of which memory is the bound.
//
// A CTA's four warps work for themselves (with 17 to 32 rows two by two, 16 rows
// each): of every tile of 64 tokens each has 16, which it fetches from their pages by 16-byte asynchronous copies into a
// ring of its own, several tiles ahead, and no barrier is passed until the item
// is done and their results are joined. Products are turned so that few rows
// do not leave the matrix instructions empty: S^T = K Q^T with 16 tokens by 8
// rows, O^T += V^T P^T with 16 values by 8 rows (mma.sync; at 16 rows a tile of
// tcgen05 would be an eighth full, and its hand-overs take longer than the
// loads). The weights turn over between the two by movmatrix.
//
// 8-bit codes go from the ring straight into the matrix instructions'
// registers, in an order of the values that makes a thread's codes neighbours:
// keys as they lie, values with those of two tokens interleaved bytewise. They
// are multiplied as f16, exactly; queries are f16 too, each row times the power
// of two that takes its largest value to 2^14, so that what a bf16 query loses
// is 2^-38 of that.
//
// 64 sequences of 80,003 tokens, E4M3, 2 key heads of 128 values by 8 query heads:
// 406 to 419 us, 6.4 to 6.6 TB/s of 2.67 GB (the copy rate is 6.8); bf16 caches of 64
// sequences of 20,000 tokens come at 6.6 to 6.9.
// With two CTAs an SM the codes took 494 us; with the type of codes tested at each
// product, which kept them from overlapping, 712.
#pragma once

#include <type_traits>

#include "cache_attention.cuh"

namespace db {

constexpr uint32_t kJoined = 256;  // quads of values that are joined at a time

template <uint32_t kPad, bool kCodes, uint32_t kN, uint32_t kShare>
struct Few {
  static constexpr uint32_t kRows = 8 * kN * kShare;
  static constexpr uint32_t kGroups = 4 / kShare;                          // of kShare warps with a ring
  static constexpr uint32_t kTokens = 16;                                  // of a stage
  static constexpr uint32_t kRaw = kTokens * kPad * (kCodes ? 1 : 2);      // keys or values
  static constexpr uint32_t kStage = 2 * kRaw + (kCodes ? 2 * kTokens * 4 : 0);
  static constexpr uint32_t kCtas = attn_ctas_per_sm(kPad, kCodes, kN * kShare);
  static constexpr uint32_t kStages =
      kPad == 256 && !kCodes ? 3 : kShare * (kCodes ? (kPad == 64 ? 5 : kPad == 128 ? 4 : 3) : kPad == 128 && kN == 1 ? 2 : 3);
  static constexpr uint32_t kBytes = kGroups * kStages * kStage;
  static_assert(kBytes >= kGroups * kRows * kPad * 4 && kBytes >= 4 * kJoined * 16, "joins reuse the rings");
};

constexpr int kFewSlack = 6;

// Transposes an 8 x 8 matrix of 16-bit values, a row in four lanes.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The parts of an item whose rows are few, joined by a whole CTA: long
// sequences leave it tens of parts, so the warps share them out (one after
// another they took 20 us of 110 for 23 parts) and are summed in their order.
template <typename T, uint32_t kRows, uint32_t kPad>
static __device__ __noinline__ void join_few(const AttnParams& p, const JoinedItem item, float* const room) {
  constexpr uint32_t kPart = kRows * (kPad + 2), kQuads = kPad / 4, kSlices = kAttnThreads / kRows, kMany = kJoined / 32;
  __shared__ float s_top[kSlices][kRows], s_sum[kSlices][kRows];
  __shared__ float4 s_note[kRows];
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const float* const parts = p.partial + (uint64_t)2 * item.c0 * kPart;  // the first is its CTA's second
  const auto part_at = [&](uint32_t k) { return parts + (k == item.c0 ? kPart : (uint64_t)2 * (k - item.c0) * kPart); };
  {
    const uint32_t row = tid % kRows, slice = tid / kRows;
    float m = -INFINITY, l = 0.f;
#pragma unroll 2
    for (uint32_t k = item.c0 + slice; k <= item.c1; k += kSlices) {
      const float mk = __ldcg(part_at(k) + kRows * kPad + row), lk = __ldcg(part_at(k) + kRows * kPad + kRows + row);
      const float now = fmaxf(m, mk), by = now == -INFINITY ? 0.f : now;
      l = times_exp2(l, m - by) + times_exp2(lk, mk - by);
      m = now;
    }
    s_top[slice][row] = m;
    s_sum[slice][row] = l;
  }
  __syncthreads();
  if (tid < item.rows) {
    const uint32_t row = tid;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (uint32_t k = 0; k < kSlices; ++k) m = fmaxf(m, s_top[k][row]);
    const float by = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (uint32_t k = 0; k < kSlices; ++k) l += times_exp2(s_sum[k][row], s_top[k][row] - by);
    const uint32_t all = item.row0 + row, node = all / p.group, qh = item.head * p.group + (all - node * p.group);
    const uint64_t to = (uint64_t)(item.first + node) * p.out.row_stride + qh * p.out.head_stride;
    s_note[row] = make_float4(by, l == 0.f ? 0.f : 1.f / l, __uint_as_float((uint32_t)to),
                              __uint_as_float((uint32_t)(to >> 32)));
    if (p.lse)
      p.lse[(uint64_t)(item.first + node) * (p.c.heads * p.group) + qh] =
          l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
  }
  __syncthreads();
  const uint32_t all = item.rows * kQuads;
  float4* const sums = (float4*)room;  // [4][32 * kMany]
#pragma unroll 1
  for (uint32_t c = 0; c < all; c += 32 * kMany) {
    float4 v[kMany];
#pragma unroll
    for (uint32_t j = 0; j < kMany; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t k = item.c0 + warp; k <= item.c1; k += 4) {
      const float* const at = part_at(k);
      float m[kMany];
      float4 y[kMany];
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        const uint32_t of = min(c + lane + j * 32, all - 1), row = of / kQuads, quad = min(of % kQuads, p.c.width / 4 - 1);
        m[j] = __ldcg(at + kRows * kPad + row);
        y[j] = __ldcg((const float4*)(at + row * kPad) + quad);
      }
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        const float b = exp2_of(m[j] - s_note[min(c + lane + j * 32, all - 1) / kQuads].x);
        v[j].x += y[j].x * b, v[j].y += y[j].y * b, v[j].z += y[j].z * b, v[j].w += y[j].w * b;
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < kMany; ++j) sums[warp * 32 * kMany + lane + j * 32] = v[j];
    __syncthreads();
#pragma unroll
    for (uint32_t at = tid; at < 32 * kMany; at += kAttnThreads) {
      const uint32_t of = c + at;
      if (of < all && of % kQuads * 4 < p.c.width) {
        const float4 w0 = sums[at], w1 = sums[32 * kMany + at], w2 = sums[64 * kMany + at], w3 = sums[96 * kMany + at];
        const float4 n = s_note[of / kQuads];
        const uint64_t to = (uint64_t)__float_as_uint(n.w) << 32 | __float_as_uint(n.z);
        *(uint2*)((char*)p.out.base + to + of % kQuads * 8) = four_answers<T>(
            make_float4(w0.x + w1.x + w2.x + w3.x, w0.y + w1.y + w2.y + w3.y, w0.z + w1.z + w2.z + w3.z, w0.w + w1.w + w2.w + w3.w), n.y);
      }
    }
    __syncthreads();
  }
}

template <typename T, uint32_t kPad, bool kCodes, uint32_t kN, uint32_t kShare>
__global__ void __launch_bounds__(kAttnThreads, (Few<kPad, kCodes, kN, kShare>::kCtas)) attention_few_kernel(const AttnParams p) {
  typedef Few<kPad, kCodes, kN, kShare> F;
  typedef typename std::conditional<kCodes, __half, T>::type H;  // what is multiplied
  constexpr uint32_t kChunks = kCodes ? kPad / 16 : kPad / 8;    // 16-byte chunks of a row
  constexpr uint32_t kStep = 32 / kChunks, kEach = F::kTokens / kStep;  // tokens between a lane's chunks, and how many
  constexpr uint32_t kSteps = kPad / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr uint32_t kCopies = (kEach + kShare - 1) / kShare;    // of a lane in a stage
  constexpr uint32_t kStride = F::kTokens * F::kGroups;
  __shared__ float s_ref[F::kGroups][F::kRows], s_sum[F::kGroups][F::kRows];
  __shared__ uint32_t s_there[4][F::kStages];  // the tokens that are there, of each warp's stages
  __shared__ uint32_t s_last;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, c = lane & 3;
  const uint32_t team = warp / kShare, member = warp % kShare, row0 = member * 8 * kN;  // its rows of the item
  unsigned char* const ring = smem + team * F::kStages * F::kStage;
  const uint32_t steps = p.c.width / 16;
  const bool e4m3 = p.c.type == DB_E4M3, one_stride = p.c.k_stride == p.c.v_stride;
  // the values whose sums this lane has: value_of(d) and kOther on
  const auto value_of = [g](uint32_t d) __attribute__((always_inline)) {
    return !kCodes ? 16 * d + g : kPad == 64 ? 8 * g + 2 * d : 128 * (d / 8) + 16 * g + 2 * (d % 8);
  };
  constexpr uint32_t kOther = kCodes ? 1 : 8;
  constexpr float kLift = (float)attn_lift<H>(kFewSlack);
  // Weights are rounded to the type that is multiplied. Where that is as coarse as the
  // answers' type, which made their error 1.4 times that of rounding them, more where
  // few weights count, what the rounding left is multiplied too, if that costs little:
  // bf16 values of 128 198 -> 200 us (64 sequences of 20,000, 2 key heads by 8), of 256
  // 237 -> 257 (32); f16 answers from E4M3 codes of 128 120 -> 124, 158 -> 177 with 16
  // rows, 291 -> 328 with 32.
  constexpr uint32_t kParts = std::is_same<H, T>::value && (kCodes ? F::kRows == 8 : kPad <= 128) ? 2 : 1;
  // a lane copies the same chunk of every kStep-th token
  const uint32_t chunk = lane % kChunks, token0 = lane / kChunks;
  const bool has = chunk < (kCodes ? p.c.width / 16 : p.c.width / 8);
  // Place of a chunk in a stage's keys or values: the lanes of one access differ in banks, in eight
  // tokens' same chunk (16 bits), two tokens' four keys and four tokens' two values (codes).
  const auto place = [](uint32_t token, uint32_t ch) __attribute__((always_inline)) {
    const uint32_t turn = !kCodes ? token & 7 : kPad == 64 ? token >> 1 & 3 : (token & 1) << 2 ^ (token >> 1 & 3) << 1;
    return (token * kChunks + (ch ^ turn)) * 16;
  };

  const Share share = plan_share<F::kRows, kAttnThreads>(p);
  uint64_t at = share.lo, before = share.before;
  uint32_t i = share.request;
  while (at < share.hi) {
    const Request r = near_request(p, share, i);
    const Extent e = extent_of<F::kRows>(p, r);
    if (at - before >= e.units) {
      before += e.units;
      ++i;
      continue;
    }
    const uint64_t x = at - before;
    const uint32_t item0 = (uint32_t)quotient(x, e.tiles);
    const uint32_t t0 = (uint32_t)(x - (uint64_t)item0 * e.tiles);
    const uint32_t t1 = (uint32_t)min((uint64_t)e.tiles, t0 + (share.hi - at));
    // Where as many whole items as teams follow one another in a request, each
    // team takes one: what an item waits for beside its loads is then waited for
    // once for all of them (1,024 sequences of 200 tokens, 8 key heads by 4: 198
    // us one by one, 170 so; with half of the teams idle it took longer).
    const bool alone = t0 == 0 && e.blocks * p.c.heads - item0 >= F::kGroups && share.hi - at >= (uint64_t)F::kGroups * e.tiles;
    const uint32_t item = item0 + (alone ? team : 0), head = item / e.blocks, rb = item - head * e.blocks;
    const uint32_t rows = min(F::kRows, r.rows * p.group - rb * F::kRows);
    const uint32_t base = r.length - r.rows;  // tokens before the request's own

    const uint32_t stride = alone ? F::kTokens : kStride;  // tokens from one stage to the next
    const uint32_t stages = alone ? (r.length + F::kTokens - 1) / F::kTokens : (t1 - t0) * kShare;

    // Lanes 0 to 15 look up a token each, of the next stage to be fetched.
    const int32_t* const table = p.view.table + (uint64_t)r.seq * p.view.columns;
    uint32_t position = t0 * kTile + (alone ? 0 : team * F::kTokens) + (lane & 15);
    uint32_t column = position / p.view.page_tokens, in_page = position - column * p.view.page_tokens;
    const uint32_t columns_on = stride / p.view.page_tokens, tokens_on = stride - columns_on * p.view.page_tokens;
    int2 w;  // page and slot, or -1 and -1
    const auto look = [&]() __attribute__((always_inline)) {
      w = make_int2(-1, -1);
      if (position < r.length) w = make_int2(__ldg(table + column), (int)in_page);
      position += stride;
      column += columns_on;
      in_page += tokens_on;
      if (in_page >= p.view.page_tokens) in_page -= p.view.page_tokens, ++column;
    };
    const char* const keys = (const char*)p.c.k + head * p.head_step + chunk * 16;
    const char* const values = (const char*)p.c.v + head * p.head_step + chunk * 16;
    const auto fetch = [&](uint32_t slot, bool any) __attribute__((always_inline)) {
      uint32_t there = 0;
      if (any) {
        if ((uint32_t)w.x >= p.view.n_pages) {
          if (w.y >= 0 && lane < 16) report_table(p.view.ctr);
          w = make_int2(-1, -1);
        }
        there = __ballot_sync(kFull, w.x >= 0) & 0xFFFFu;
        if (lane == 0) s_there[warp][slot] = there;
        const uint64_t page = (uint32_t)max(w.x, 0), in = (uint64_t)(uint32_t)max(w.y, 0) * p.token_step;
        const uint64_t off = page * p.c.k_stride + in, off_v = one_stride ? off : page * p.c.v_stride + in;
        const uint32_t to = smem_at(ring + slot * F::kStage);
        const uint32_t token1 = token0 + member * kCopies * kStep;  // this warp's share of the copies
        const bool mine = has && token1 < F::kTokens;
        uint64_t from_k[kCopies], from_v[kCopies];
#pragma unroll
        for (uint32_t k = 0; k < kCopies; ++k) from_v[k] = from_k[k] = __shfl_sync(kFull, off, token1 + k * kStep);
        if (!one_stride) {
#pragma unroll
          for (uint32_t k = 0; k < kCopies; ++k) from_v[k] = __shfl_sync(kFull, off_v, token1 + k * kStep);
        }
        if (there == 0xFFFFu) {
          if (mine) {
#pragma unroll
            for (uint32_t k = 0; k < kCopies; ++k) {
              const uint32_t at_chunk = to + place(token1 + k * kStep, chunk);
              copy16(at_chunk, keys + from_k[k], true);
              copy16(at_chunk + F::kRaw, values + from_v[k], true);
            }
          }
        } else {
#pragma unroll
          for (uint32_t k = 0; k < kCopies; ++k) {
            const uint32_t token = token1 + k * kStep, at_chunk = to + place(token, chunk);
            if (!mine) continue;
            copy16(at_chunk, keys + from_k[k], there >> token & 1);
            copy16(at_chunk + F::kRaw, values + from_v[k], there >> token & 1);
          }
        }
        if (kCodes && member == 0) {  // lanes 0 to 15 the keys' scales, the others the values'
          const uint32_t of = (uint32_t)__shfl_sync(kFull, max(w.y, 0), lane & 15) * p.scale_token_step + head * p.scale_head_step;
          const uint64_t pg = (uint64_t)__shfl_sync(kFull, (uint32_t)page, lane & 15);
          const char* const scales = lane < 16 ? (const char*)p.c.k_scale + pg * p.c.k_scale_stride : (const char*)p.c.v_scale + pg * p.c.v_scale_stride;
          const bool real = there >> (lane & 15) & 1;
          copy4(to + 2 * F::kRaw + lane * 4, real ? (const float*)scales + of : (const float*)p.c.k_scale, real);
        }
      }
      copies_commit();
    };

    __syncthreads();  // the item before is done with the rings
    if (kCodes && !has) {  // keys behind the width's end are zeros, as queries are there
#pragma unroll 1
      for (uint32_t k = 0; k < F::kStages; ++k)
        for (uint32_t j = 0; j < kEach; ++j)
          *(uint4*)(ring + k * F::kStage + place(token0 + j * kStep, chunk)) = make_uint4(0, 0, 0, 0);
    }
    look();
#pragma unroll 1
    for (uint32_t k = 0; k + 1 < F::kStages; ++k) {
      fetch(k, k < stages);
      look();
    }

    // Queries as the second operand: this lane's are of row g of each block.
    uint32_t q[kSteps][2 * kN];
    float factor[kN][2];  // of scores of rows 2c and 2c + 1
    uint32_t node[kN][2];
#pragma unroll
    for (uint32_t n = 0; n < kN; ++n) {
      const uint32_t row = row0 + n * 8 + g, all = rb * F::kRows + (row < rows ? row : 0), nd = all / p.group;
      const char* const from = (const char*)p.q.base + (uint64_t)(r.first + nd) * p.q.row_stride +
                               (head * p.group + (all - nd * p.group)) * p.q.head_stride;
      if constexpr (kCodes) {
        uint32_t top = 0;
#pragma unroll
        for (uint32_t st = 0; st < kSteps; ++st) {  // values 64 (st / 4) + 16 c + 4 (st % 4) and three more
          const uint32_t d = 64 * (st / 4) + 16 * c + 4 * (st % 4);
          uint2 v = make_uint2(0, 0);
          if (row < rows && d < p.c.width) v = __ldg((const uint2*)(from + d * 2));
          q[st][2 * n] = v.x;
          q[st][2 * n + 1] = v.y;
          const float2 a = unpack2<T>(v.x & 0x7FFF7FFFu), b = unpack2<T>(v.y & 0x7FFF7FFFu);
          const float y[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
          for (int k = 0; k < 4; ++k)  // (infinities and NaN left out)
            if (__float_as_uint(y[k]) < 0x7F800000u) top = max(top, __float_as_uint(y[k]));
        }
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int exponent = top == 0 ? 14 : max((int)(top >> 23) - 127, 14 - 126);
        const float up = __uint_as_float((uint32_t)(14 - exponent + 127) << 23);
#pragma unroll
        for (uint32_t st = 0; st < kSteps; ++st)
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            const float2 a = unpack2<T>(q[st][2 * n + h]);
            q[st][2 * n + h] = pack2<__half>(a.x * up, a.y * up);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ex = __shfl_sync(kFull, exponent, (2 * c + h) * 4);
          factor[n][h] = p.scale_log2 * __uint_as_float((uint32_t)(max(ex - 14, -126) + 127) << 23);
        }
      } else {
#pragma unroll
        for (uint32_t st = 0; st < kSteps; ++st)
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h)
            q[st][2 * n + h] = row < rows && st < steps ? __ldg((const uint32_t*)(from + (st * 16 + 2 * c + 8 * h) * 2)) : 0u;
        factor[n][0] = factor[n][1] = p.scale_log2;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t row = row0 + n * 8 + 2 * c + h;
        node[n][h] = row < rows ? (rb * F::kRows + row) / p.group : 0;
      }
    }

    float o[kSteps][kN][4];
    float top[kN][2], sum[kN][2];
#pragma unroll
    for (uint32_t d = 0; d < kSteps; ++d)
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[d][n][k] = 0.f;
#pragma unroll
    for (uint32_t n = 0; n < kN; ++n) top[n][0] = top[n][1] = -INFINITY, sum[n][0] = sum[n][1] = 0.f;

    uint32_t slot = 0;
    uint32_t first = t0 * kTile + (alone ? 0 : team * F::kTokens);  // position of the stage's first token
    for (uint32_t t = 0; t < stages; ++t, first += stride) {
      copies_wait<F::kStages - 2>();
      if (kShare > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kShare) : "memory");
      else
        __syncwarp();
      // the stage is here for all, and the one before is done with
      const uint32_t there = s_there[warp][slot];
      fetch(slot == 0 ? F::kStages - 1 : slot - 1, t + F::kStages - 1 < stages);
      look();
      unsigned char* const kt = ring + slot * F::kStage;
      unsigned char* const vt = kt + F::kRaw;
      const float* const scales = (const float*)(kt + 2 * F::kRaw);
      slot = slot + 1 == F::kStages ? 0 : slot + 1;

      // scores of tokens g and g + 8, rows 2c and 2c + 1 of each block
      float s[kN][4];
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[n][k] = 0.f;
      if constexpr (kCodes) {
        const auto scores = [&](auto is_float) __attribute__((always_inline)) {
          constexpr bool kFloat = decltype(is_float)::value;
#pragma unroll
          for (uint32_t j = 0; j < kPad / 64; ++j) {
            const uint4 lo = *(const uint4*)(kt + place(g, 4 * j + c)), hi = *(const uint4*)(kt + place(g + 8, 4 * j + c));
            const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint2 u = widen4(a[m], kFloat), v = widen4(b[m], kFloat);
              const uint32_t f[4] = {u.x, v.x, u.y, v.y};
#pragma unroll
              for (uint32_t n = 0; n < kN; ++n) multiply<H>(s[n], f, q[4 * j + m][2 * n], q[4 * j + m][2 * n + 1]);
            }
          }
        };
        if (e4m3)
          scores(std::true_type());
        else
          scores(std::false_type());
        const float k0 = scales[g], k1 = scales[g + 8];
        // (an infinite scale stands for values of both signs, whose products have no sum)
        const float f0 = __fmaf_rn(k0, 0.f, k0), f1 = __fmaf_rn(k1, 0.f, k1);
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n)
          s[n][0] *= f0, s[n][1] *= f0, s[n][2] *= f1, s[n][3] *= f1;
      } else {
#pragma unroll
        for (uint32_t st = 0; st < kSteps; ++st) {
          if (st >= steps) break;
          uint32_t f[4];
          load_matrices(f, smem_at(kt) + place((lane & 7) + (lane >> 3 & 1) * 8, 2 * st + (lane >> 4)));
#pragma unroll
          for (uint32_t n = 0; n < kN; ++n) multiply<H>(s[n], f, q[st][2 * n], q[st][2 * n + 1]);
        }
      }
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[n][k] *= factor[n][k & 1];
      // what is not seen: only the last tiles, or those of broken tables, have any
      const bool masked = first + F::kTokens > base || there != 0xFFFFu;
      uint32_t sees = 0xFFFFFFFFu;
      if (masked) {
        sees = 0;
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t token = g + (k >> 1) * 8, nd = node[n][k & 1];
            bool yes = there >> token & 1;
            if (yes && first + token >= base) {
              const uint32_t own = first + token - base;
              yes = p.mask ? __ldg(p.mask + (uint64_t)(r.first + nd) * p.mask_words + own / 32) >> (own & 31) & 1 : own <= nd;
            }
            if (yes)
              sees |= 1u << (n * 4 + k);
            else
              s[n][k] = -INFINITY;
          }
      }
      // Weights are exp2(score - ref). ref is kLift below what was a row's largest score,
      // followed when one is 2^kFewSlack above it; with codes the largest score times
      // its values' scale, of the tokens that the row sees, so that weights times scales
      // stay in the middle of f16's range. (Of all tokens of a tile, or without the
      // scores, one large scale would take the others' products out of that range,
      // though no row sees it or it hardly counts.)
      float v0 = 1.f, v1 = 1.f, e0 = 0.f, e1 = 0.f;
      if (kCodes) {
        v0 = scales[16 + g], v1 = scales[24 + g];
        e0 = scale_size(v0), e1 = scale_size(v1);
      }
      float most[kN][2];
      bool rises = false;
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          most[n][h] = kCodes ? fmaxf(s[n][h] + e0, s[n][2 + h] + e1) : fmaxf(s[n][h], s[n][2 + h]);
          rises |= most[n][h] > top[n][h] + (float)kFewSlack || (top[n][h] == -INFINITY && most[n][h] > -INFINITY);
        }
      if (__any_sync(kFull, rises)) {
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float m = most[n][h];
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            const float was = top[n][h];
            if (m > was + (float)kFewSlack || was == -INFINITY) top[n][h] = m;
            const float fall = was - (top[n][h] == -INFINITY ? 0.f : top[n][h]), down = exp2_of(fall);
            sum[n][h] = times_exp2(sum[n][h], fall);
#pragma unroll
            for (uint32_t d = 0; d < kSteps; ++d) {
              o[d][n][h] *= down;
              o[d][n][2 + h] *= down;
            }
          }
      }
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float ref = top[n][k & 1] == -INFINITY ? 0.f : top[n][k & 1] - kLift;
          s[n][k] = exp2_of(s[n][k] - ref);
          sum[n][k & 1] += s[n][k];
        }
      if (kCodes) {
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n)
          s[n][0] *= v0, s[n][1] *= v0, s[n][2] *= v1, s[n][3] *= v1;
      }
      // Values that not every row sees and that are not finite: rare, by hand.
      if (masked) {
        bool bad = false;
#pragma unroll 2
        for (uint32_t k = 0; k < kEach; ++k) {
          const uint4 v = *(const uint4*)(vt + place(token0 + k * kStep, chunk));
          bool here;
          if (kCodes) {
            const auto nan4 = [](uint32_t a) { return ((a & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
            here = e4m3 && (nan4(v.x) | nan4(v.y) | nan4(v.z) | nan4(v.w));
          } else {
            here = not_finite2<H>(v.x) || not_finite2<H>(v.y) || not_finite2<H>(v.z) || not_finite2<H>(v.w);
          }
          bad |= has && here;
        }
        const auto odd_scale = [](float a) { return (__float_as_uint(a) & 0x7F800000u) == 0x7F800000u; };
        if (kCodes) bad |= odd_scale(v0) || odd_scale(v1);
        if (__any_sync(kFull, bad)) {
#pragma unroll 1
          for (uint32_t token = 0; token < F::kTokens; ++token) {
            // the weights of rows 2c and 2c + 1 with the token, by the lane that has them
            const uint32_t from = (token & 7) * 4 + c;
            float weight[kN][2];
            bool yes[kN][2];
            const uint32_t bits = __shfl_sync(kFull, sees, from);
#pragma unroll
            for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float a = __shfl_sync(kFull, s[n][h], from), b = __shfl_sync(kFull, s[n][2 + h], from);
                weight[n][h] = token < 8 ? a : b;
                yes[n][h] = bits >> (n * 4 + (token < 8 ? 0 : 2) + h) & 1;
              }
#pragma unroll
            for (uint32_t d = 0; d < kSteps; ++d)
#pragma unroll
              for (uint32_t half = 0; half < 2; ++half) {
                float v;
                if (kCodes) {
                  const uint32_t of = value_of(d) + half;
                  const unsigned char code = vt[place(token, of / 16) + of % 16];
                  v = e4m3 ? unpack2<__half>(e4m3x2_to_f16x2(code)).x : (float)(int8_t)code;
                } else {
                  const uint32_t of = value_of(d) + 8 * half;
                  v = d < steps ? to_float(*(const H*)(vt + place(token, of / 8) + of % 8 * 2)) : 0.f;
                }
#pragma unroll
                for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (yes[n][h]) o[d][n][2 * half + h] += weight[n][h] * v;
              }
          }
          continue;
        }
        if (kCodes) {  // an unseen token's scale may be anything finite: its weights are 0
#pragma unroll
          for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(sees >> (n * 4 + k) & 1)) s[n][k] = 0.f;
        }
      }
      uint32_t b[kParts][kN][2];
#pragma unroll
      for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const float x = s[n][2 * h], y = s[n][2 * h + 1];
          const uint32_t w = pack2<H>(x, y);
          b[0][n][h] = turned(w);
          if constexpr (kParts == 2) {  // what the rounding left (of infinities and NaN nothing)
            const float2 r = unpack2<H>(w);
            const float u = x - r.x, v = y - r.y;
            b[1][n][h] = turned(pack2<H>(fabsf(u) < 64.f ? u : 0.f, fabsf(v) < 64.f ? v : 0.f));
          }
        }
      if constexpr (kCodes) {
        const auto outputs = [&](auto is_float) __attribute__((always_inline)) {
          constexpr bool kFloat = decltype(is_float)::value;
          // words of this lane's values of tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (uint32_t j = 0; j < (kPad == 64 ? 1 : kPad / 128); ++j) {
            constexpr uint32_t kWords = kPad == 64 ? 2 : 4;
            uint32_t u[4][kWords];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
              const uint32_t token = 2 * c + (k & 1) + (k >> 1) * 8;
              if constexpr (kPad == 64) {
                const uint2 y = *(const uint2*)(vt + place(token, g / 2) + (g & 1) * 8);
                u[k][0] = y.x, u[k][1] = y.y;
              } else {
                const uint4 y = *(const uint4*)(vt + place(token, 8 * j + g));
                u[k][0] = y.x, u[k][1] = y.y, u[k][kWords - 2] = y.z, u[k][kWords - 1] = y.w;
              }
            }
#pragma unroll
            for (uint32_t m = 0; m < kWords; ++m)
#pragma unroll
              for (uint32_t half = 0; half < 2; ++half) {
                const uint2 lo = widen4(__byte_perm(u[0][m], u[1][m], half ? 0x7362 : 0x5140), kFloat);
                const uint2 hi = widen4(__byte_perm(u[2][m], u[3][m], half ? 0x7362 : 0x5140), kFloat);
                const uint32_t f[4] = {lo.x, lo.y, hi.x, hi.y};
                const uint32_t d = j * 8 + 2 * m + half;
#pragma unroll
                for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
                  for (uint32_t k = 0; k < kParts; ++k) multiply<H>(o[d][n], f, b[k][n][0], b[k][n][1]);
              }
          }
        };
        if (e4m3)
          outputs(std::true_type());
        else
          outputs(std::false_type());
      } else {
#pragma unroll
        for (uint32_t d = 0; d < kSteps; ++d) {
          if (d >= steps) break;
          uint32_t f[4];
          load_matrices_t(f, smem_at(vt) + place((lane & 7) + (lane >> 4) * 8, 2 * d + (lane >> 3 & 1)));
#pragma unroll
          for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
            for (uint32_t k = 0; k < kParts; ++k) multiply<H>(o[d][n], f, b[k][n][0], b[k][n][1]);
        }
      }
    }

    // The warps' results joined, through shared memory.
#pragma unroll
    for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = sum[n][h];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        sum[n][h] = l;
        top[n][h] -= kLift;  // the reference of what was summed
        if (g == 0) s_ref[team][row0 + n * 8 + 2 * c + h] = top[n][h];
      }
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (uint32_t n = 0; n < kN; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t row = row0 + n * 8 + 2 * c + h;
        float m = top[n][h];
        if (!alone) {
#pragma unroll
          for (uint32_t k = 0; k < F::kGroups; ++k) m = fmaxf(m, s_ref[k][row]);
        }
        const float fall = top[n][h] - (m == -INFINITY ? 0.f : m), a = exp2_of(fall);
        if (g == 0) s_sum[team][row] = times_exp2(sum[n][h], fall);
        float* const to = (float*)smem + (team * F::kRows + row) * kPad;
#pragma unroll
        for (uint32_t d = 0; d < kSteps; ++d) {
          to[value_of(d)] = o[d][n][h] * a;
          to[value_of(d) + kOther] = o[d][n][2 + h] * a;
        }
      }
    __syncthreads();
    const bool whole = alone || (t0 == 0 && t1 == e.tiles);
    float* const mine = p.partial + (uint64_t)(2 * blockIdx.x + (t0 == 0)) * partial_floats(F::kRows, kPad);
    constexpr uint32_t kQuads = kPad / 4;
#pragma unroll 1
    for (uint32_t k0 = 0; k0 < (alone ? F::kGroups : 1); ++k0) {
      const uint32_t of_head = (item0 + k0) / e.blocks, of_rb = item0 + k0 - of_head * e.blocks;
      const uint32_t of_rows = min(F::kRows, r.rows * p.group - of_rb * F::kRows);
#pragma unroll 1
      for (uint32_t of = tid; of < of_rows * kQuads; of += kAttnThreads) {
        const uint32_t row = of / kQuads, quad = of % kQuads;
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (uint32_t k = 0; k < F::kGroups; ++k) {
          if (alone && k != k0) continue;
          m = fmaxf(m, s_ref[k][row]);
          l += s_sum[k][row];
          const float4 y = *((const float4*)((const float*)smem + (k * F::kRows + row) * kPad) + quad);
          v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        if (whole) {
          const uint32_t all = of_rb * F::kRows + row, nd = all / p.group, qh = of_head * p.group + (all - nd * p.group);
          const float by = l == 0.f ? 0.f : 1.f / l;
          if (quad * 4 < p.c.width)
            *(uint2*)((char*)p.out.base + (uint64_t)(r.first + nd) * p.out.row_stride + qh * p.out.head_stride + quad * 8) =
                four_answers<T>(v, by);
          if (quad == 0 && p.lse)
            p.lse[(uint64_t)(r.first + nd) * (p.c.heads * p.group) + qh] =
                l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
        } else {
          __stcg((float4*)(mine + row * kPad) + quad, v);
          if (quad == 0) {
            __stcg(mine + F::kRows * kPad + row, m);
            __stcg(mine + F::kRows * kPad + F::kRows + row, l);
          }
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      const uint64_t first = at - t0;
      const uint32_t c0 = owner_of(share, first), c1 = owner_of(share, first + e.tiles - 1);
      if (tid == 0) {
        const unsigned int seen = atomicAdd(p.arrived + c0, 1u);
        s_last = seen == c1 - c0;
        if (s_last) p.arrived[c0] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const JoinedItem item_of = {r.first, rb * F::kRows, rows, head, c0, c1};
        join_few<T, F::kRows, kPad>(p, item_of, (float*)smem);
      }
    }
    at += alone ? (uint64_t)F::kGroups * e.tiles : t1 - t0;
  }
}

template <typename T, uint32_t kPad, bool kCodes, uint32_t kN, uint32_t kShare>
int launch_few(const AttnParams& p, cudaStream_t s) {
  typedef Few<kPad, kCodes, kN, kShare> F;
  const cudaError_t e = cudaFuncSetAttribute(attention_few_kernel<T, kPad, kCodes, kN, kShare>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, F::kBytes);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_dependent(attention_few_kernel<T, kPad, kCodes, kN, kShare>, attn_grid(F::kCtas), kAttnThreads, F::kBytes, s, p);
}

}  // namespace db
