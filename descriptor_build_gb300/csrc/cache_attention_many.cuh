// Attention over a paged cache for many query rows (cache_attention.cuh: the
// mathematics and the way work is cut): 128 rows of an item at a time, with
// tcgen05 products.
//
// A CTA has three kinds of warps that hand tiles of 64 tokens on by mbarriers:
//   loaders (3 or 6)    keys and values from their pages into a ring of tiles, by
//                       16-byte asynchronous copies; 8-bit codes come into a
//                       ring of their own, from which they are widened
//   one issuing thread  S = Q K^T into TMEM (two buffers), O += P V from TMEM
//   weights (4 warps)   a thread for each query row: S -> maxima, weights P
//                       (over S in TMEM) and their sum
// so that the product of one tile runs while weights of the one before are
// made, and two CTAs share an SM. Items of more than 128 rows have a CTA of two
// such tiles of rows, each with its issuing thread and weights' warps, which
// share what is loaded and widened (wide trees of 488 rows 396 us with CTAs of
// 128 rows, 374 with two tiles and one issuing thread, 312 with two).
//
// A row's maximum is followed only when it has risen by 2^kSlack (weights of
// 2^kSlack are held as exactly as 1), so O is hardly ever rescaled.
//
// A row of a page is 128 or 256 bytes, the next token's some kilobytes on. Such
// rows of 16 tokens a page come at 6.6 TB/s (1 CTA an SM, 4 tiles ahead) by
// 16-byte copies of 128 threads and at 3.6 by TMA boxes of 64 values x 16 tokens,
// which a CTA starts every 150 cycles; in this kernel boxes took 225 us where
// the copies are done in less than 141 (48 trees of 25 nodes over 3,000 tokens).
//
// 48 trees of 25 nodes over 3,000 tokens (100 rows, bf16): 141 us, 4.6 TB/s: the
// loaders' and issuing thread's instructions, and at each item's ends latency (a
// third of the time before they were cut). 16 trees of 61 over 8,192 (488 rows,
// I8): 241 us, 0.45 PFLOP/s: the weights' warps, of which a scheduler has two,
// and instructions not yet fetched.
//
// Tiles lie as the tensor cores' 128-byte swizzle wants them: panels of 64
// values, a row of 128 bytes for each token, 16-byte chunks exchanged by the
// row's number; keys are read along their rows (K-major), values across
// (MN-major).
#pragma once

#include <type_traits>

#include "cache_attention.cuh"

namespace db {

template <uint32_t kPad, bool kCodes, uint32_t kTiles>
struct Many {
  static constexpr uint32_t kRows = 128 * kTiles;
  static constexpr uint32_t kWeights = 128 * kTiles;
  // Loaders that have units in turn. As they divide the ring, a place of it is
  // always the same warp's, which so sees every phase of its barrier (a wait by
  // parity is true too early when another phase lies between). (48 trees, 16 bits:
  // 144 us with two and a ring of four, 141 with three and a ring of three; four
  // would leave 96 registers a thread, 145.)
  static constexpr uint32_t kLoaderWarps = 3 * kTiles;
  static constexpr uint32_t kWarps = kWeights / 32 + kLoaderWarps + kTiles;
  static constexpr uint32_t kThreads = 32 * kWarps;
  static constexpr uint32_t kUnit = kTile * kPad * 2;  // keys or values of a tile
  static constexpr uint32_t kUnits = !kCodes && kPad == 64 ? 6 : 3 * kTiles;
  static_assert(kUnits % kLoaderWarps == 0, "see kLoaderWarps");
  static constexpr uint32_t kQuery = kRows * kPad * 2;
  static constexpr uint32_t kRaw = kTile * kPad;       // codes of a unit
  static constexpr uint32_t kRaws = kCodes ? kLoaderWarps : 0;
  static constexpr uint32_t kMeta = kUnits / 2 + 3;    // tiles that notes are kept of
  static constexpr uint32_t kColumns = kPad <= 128 && kTiles == 1 ? 256 : 512;  // of TMEM
  static_assert(kTiles * (2 * kTile + kPad) <= kColumns, "scores of two tiles of tokens, and sums");
  static constexpr uint32_t kCtas = kPad <= 128 && kTiles == 1 ? 2 : 1;   // of an SM
  static constexpr uint32_t kBytes = kUnits * kUnit + kQuery + kRaws * kRaw + 1024;
  // Shared memory for no more CTAs an SM than TMEM holds: another would wait for TMEM
  // until one of them is done, while a different SM has room.
  static constexpr uint32_t kLeast = (kCtas == 2 ? 80 : 200) * 1024;
  static constexpr uint32_t kAsk = kBytes < kLeast ? kLeast : kBytes;
};

// What the weights' warps need to know of a tile, by the loaders.
struct alignas(16) TileNotes {    // scales are read by fours
  int2 place[kTile];              // page (or -1) and slot of a token
  float k_scale[kTile], v_scale[kTile];
  uint32_t real[2], odd[2];       // bits of tokens: that are there; whose values are not all finite
  uint32_t exponent[2];           // of the largest scale of values (scale_exponent)
};

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Whether it is over now (try_wait may sleep for microseconds before it says no).
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for a phase; gives up after a second, or when another thread has. (The
// clock is read only when a wait is long: reading it takes longer than most.)
static __device__ __noinline__ bool barrier_wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* failed) {
  uint64_t began = 0;
  for (;;) {
    for (int k = 0; k < 256; ++k)
      if (barrier_try(bar, parity)) return true;
    if (*failed) return false;
    const uint64_t now = globaltimer_ns();
    if (!began) began = now;
    if (now - began > kWaitLimitNs) {
      *failed = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile uint32_t* failed) {
  for (int k = 0; k < 8; ++k)
    if (barrier_try(bar, parity)) return true;
  return barrier_wait_long(bar, parity, failed);
}
__device__ __forceinline__ void group_sync(uint32_t id, uint32_t threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, and whether `yes` held in all of them.
__device__ __forceinline__ bool group_all(uint32_t id, uint32_t threads, bool yes) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)yes)
      : "memory");
  return r;
}
__device__ __forceinline__ void writes_to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (TMEM) += A B: A from shared memory or from TMEM.
__device__ __forceinline__ void tensor_multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tensor_multiply_t(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
// A tile in shared memory: 128-byte swizzle, groups of 8 rows 1024 bytes
// apart; `panel`: bytes between panels where they lie along the rows' number.
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at, uint32_t panel) {
  return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)((panel >> 4) & 0x3FFF) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// The product's kind: 32-bit sums of 16-bit values (f16 0, bf16 1), M = 128.
__device__ __forceinline__ uint32_t product_kind(uint32_t type, uint32_t n, bool across) {
  return 1u << 4 | type << 7 | type << 10 | (across ? 1u << 16 : 0) | (n / 8) << 17 | (128u / 16) << 24;
}

#define DB_OUT8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define DB_IN8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : DB_OUT8(r, 0), DB_OUT8(r, 8), DB_OUT8(r, 16), DB_OUT8(r, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      DB_IN8(r, 0), DB_IN8(r, 8), DB_IN8(r, 16), DB_IN8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : DB_OUT8(r, 0), DB_OUT8(r, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      DB_IN8(r, 0), DB_IN8(r, 8)
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_load1(uint32_t at) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two 32-bit floats at a time.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t multiply2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t multiply_add2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float largest3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// What few tiles need is kept out of the loops' code, which is as long as the
// instruction caches bear: a kernel of 138 KB that had all of it inline took 324
// us for 48 trees of 25, a smaller one 270 then.

// Scores of a tile that a row does not see become -infinity, in TMEM. Codes:
// the others are multiplied by their keys' scales.
static __device__ __noinline__ void hide_scores(uint32_t here, uint32_t sees0, uint32_t sees1, const float* k_scale) {
#pragma unroll 1
  for (uint32_t h = 0; h < 4; ++h) {
    uint32_t s[16];
    tmem_load16(here + 16 * h, s);
    tmem_loaded();
    const uint32_t sees = (h & 2 ? sees1 : sees0) >> (16 * (h & 1));
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float x = __uint_as_float(s[j]);
      if (k_scale) x *= k_scale[16 * h + j];
      s[j] = __float_as_uint((sees >> j) & 1 ? x : -INFINITY);
    }
    tmem_store16(here + 16 * h, s);
  }
  tmem_stored();
}

// The largest score times its values' scale of a row: codes' reference (log2). (Of an
// item's first tile, and hardly another. As a function that is called it took 20 us more
// of 16 wide trees.)
__device__ __forceinline__ float largest_product(uint32_t here, float factor, const float* v_scale) {
  float most = -INFINITY;
#pragma unroll 1
  for (uint32_t h = 0; h < 4; ++h) {
    uint32_t s[16];
    __syncwarp();
    tmem_load16(here + 16 * h, s);
    tmem_loaded();
#pragma unroll
    for (int j = 0; j < 16; ++j) most = fmaxf(most, __fmaf_rn(__uint_as_float(s[j]), factor, scale_size(v_scale[16 * h + j])));
  }
  return most;
}

// Values that are not finite, which the product is not given, added to O for
// the rows that see them. `v`, `scale`: of the head.
template <typename T, bool kCodes>
static __device__ __noinline__ void add_odd(const TileNotes& m, uint32_t output, uint32_t here, uint64_t odd, uint64_t sees,
                                            float factor, float ref, const char* v, uint64_t v_stride, uint64_t token_step,
                                            const char* scale, uint64_t scale_stride, uint32_t scale_step, bool i8,
                                            uint32_t width) {
#pragma unroll 1
  for (uint64_t left = odd; left; left &= left - 1) {
    const uint32_t token = __ffsll((long long)left) - 1;
    __syncwarp();
    const float score = __uint_as_float(tmem_load1(here + token));
    tmem_loaded();
    const int2 place = m.place[token];
    const char* const from = v + (uint64_t)place.x * v_stride + (uint64_t)place.y * token_step;
    float weight = exp2_of(__fmaf_rn(score, factor, -ref));
    if (kCodes) weight *= ((const float*)(scale + (uint64_t)place.x * scale_stride))[(uint32_t)place.y * scale_step];
    const bool yes = (sees >> token) & 1;
#pragma unroll 1
    for (uint32_t c = 0; c < width; c += 16) {
      uint32_t o[16];
      __syncwarp();
      tmem_load16(output + c, o);
      tmem_loaded();
      if (yes) {
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float2 x;
          if (kCodes) {
            const uint16_t two = *(const uint16_t*)(from + c + j);
            // I8 has no values that are not finite, its scales have
            x = i8 ? make_float2((float)(int8_t)two, (float)(int8_t)(two >> 8)) : unpack2<__half>(e4m3x2_to_f16x2(two));
          } else {
            x = unpack2<T>(*(const uint32_t*)(from + 2 * (c + j)));
          }
          o[j] = __float_as_uint(__uint_as_float(o[j]) + weight * x.x);
          o[j + 1] = __float_as_uint(__uint_as_float(o[j + 1]) + weight * x.y);
        }
      }
      __syncwarp();
      tmem_store16(output + c, o);
    }
    tmem_stored();
  }
}

// The parts of an item, joined by kThreads threads (the named barrier is
// theirs). A part lies by fours of values, of all rows: a warp's rows are
// neighbours when it stores its sums, a row to a thread, and when it reads them
// here. A thread joins 32 values of a row (16 where rows are few), two parts' loads under way together.
template <typename T, uint32_t kRows, uint32_t kPad, uint32_t kThreads>
static __device__ __noinline__ void join_item(const AttnParams& p, const JoinedItem item, float4* row_notes, uint32_t barrier) {
  constexpr uint32_t kMany = 8, kPart = kRows * (kPad + 2);
  const float* const parts = p.partial + (uint64_t)2 * item.c0 * kPart;  // the first is its CTA's second
  const auto part_at = [&](uint32_t k) { return parts + (k == item.c0 ? kPart : (uint64_t)2 * (k - item.c0) * kPart); };
  if (threadIdx.x < item.rows) {
    const uint32_t row = threadIdx.x;
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (uint32_t k = item.c0; k <= item.c1; ++k) {
      const float mk = __ldcg(part_at(k) + kRows * kPad + row), lk = __ldcg(part_at(k) + kRows * kPad + kRows + row);
      const float now = fmaxf(m, mk), by = now == -INFINITY ? 0.f : now;
      l = times_exp2(l, m - by) + times_exp2(lk, mk - by);
      m = now;
    }
    const uint32_t all = item.row0 + row, node = all / p.group, qh = item.head * p.group + (all - node * p.group);
    const uint64_t to = (uint64_t)(item.first + node) * p.out.row_stride + qh * p.out.head_stride;
    row_notes[row] = make_float4(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l, __uint_as_float((uint32_t)to),
                                 __uint_as_float((uint32_t)(to >> 32)));
    if (p.lse)
      p.lse[(uint64_t)(item.first + node) * (p.c.heads * p.group) + qh] =
          l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
  }
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(kThreads) : "memory");
  const uint32_t bits = item.rows > 32 ? 32 - __clz(item.rows - 1) : 5;  // 2^bits rows side by side
  const uint32_t each = (p.c.width / 32) << bits >= kThreads ? kMany : 4;  // by fours, of a thread
#pragma unroll 1
  for (uint32_t c = threadIdx.x; c < (p.c.width / 4 + each - 1) / each << bits; c += kThreads) {
    const uint32_t row = c & ((1u << bits) - 1), quad0 = (c >> bits) * each;
    if (row >= item.rows) continue;
    const uint32_t quads = min(each, p.c.width / 4 - quad0);
    const float4 n = row_notes[row];
    float4 v[kMany];
#pragma unroll
    for (uint32_t j = 0; j < kMany; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t k = item.c0; k <= item.c1; k += 2) {
      const bool two = k < item.c1;
      const float* const a = part_at(k);
      const float* const b = part_at(two ? k + 1 : k);
      const float ma = __ldcg(a + kRows * kPad + row), mb = __ldcg(b + kRows * kPad + row);
      float4 x[kMany], y[kMany];
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        x[j] = __ldcg((const float4*)a + (quad0 + min(j, quads - 1)) * kRows + row);
        y[j] = __ldcg((const float4*)b + (quad0 + min(j, quads - 1)) * kRows + row);
      }
      const float fa = exp2_of(ma - n.x), fb = two ? exp2_of(mb - n.x) : 0.f;
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        v[j].x += x[j].x * fa, v[j].y += x[j].y * fa, v[j].z += x[j].z * fa, v[j].w += x[j].w * fa;
        if (two) v[j].x += y[j].x * fb, v[j].y += y[j].y * fb, v[j].z += y[j].z * fb, v[j].w += y[j].w * fb;
      }
    }
    char* const to = (char*)p.out.base + ((uint64_t)__float_as_uint(n.w) << 32 | __float_as_uint(n.z)) + quad0 * 8;
#pragma unroll
    for (uint32_t j = 0; j < kMany; j += 2)  // (width is a multiple of 16 values)
      if (j < quads) {
        const uint2 a = four_answers<T>(v[j], n.y), b = four_answers<T>(v[j + 1], n.y);
        *(uint4*)(to + j * 8) = make_uint4(a.x, a.y, b.x, b.y);
      }
  }
}

// Sums are rescaled seldom (16 wide trees: 297 us with a slack of 6, 279 with 8, 274 with 10).
constexpr int kSlack = 10;

template <typename T, uint32_t kPad, bool kCodes, uint32_t kTiles>
__global__ void __launch_bounds__((Many<kPad, kCodes, kTiles>::kThreads), (Many<kPad, kCodes, kTiles>::kCtas))
    attention_many_kernel(const AttnParams p) {
  typedef Many<kPad, kCodes, kTiles> F;
  typedef typename std::conditional<kCodes, __half, T>::type W;  // what is multiplied
  constexpr uint32_t kTypeW = std::is_same<W, __half>::value ? 0 : 1, kIssuer = F::kWarps - kTiles;  // the first warp with an issuing thread
  constexpr uint32_t kPanel = kTile * 128, kQueryPanel = 128 * 128, kQueryTile = 128 * kPad * 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ TileNotes s_notes[F::kMeta];
  __shared__ uint64_t s_full[F::kUnits], s_empty[F::kUnits], s_scores[kTiles][2], s_weights[kTiles][2], s_output[kTiles][2], s_odd[F::kMeta], s_asked, s_drained;
  __shared__ uint32_t s_tmem, s_last;
  __shared__ __align__(16) float s_ones[kCodes ? kTile : 4];  // keys' scales of scores that have theirs
  __shared__ volatile uint32_t s_failed;
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  unsigned char* const smem = smem_raw + ((1024 - (smem_at(smem_raw) & 1023)) & 1023);
  const uint32_t ring = smem_at(smem), query = ring + F::kUnits * F::kUnit;

  if (kCodes && tid < kTile) s_ones[tid] = 1.f;
  if (tid == 0) {
    for (uint32_t k = 0; k < F::kUnits; ++k) {
      barrier_init(smem_at(&s_full[k]), 32);  // a warp's lanes
      barrier_init(smem_at(&s_empty[k]), kTiles);
    }
    for (uint32_t k = 0; k < 2 * kTiles; ++k) {
      barrier_init(smem_at(&s_scores[k / 2][k & 1]), 2);  // the products, and the notes that came with the keys
      barrier_init(smem_at(&s_weights[k / 2][k & 1]), 128);
      // one for even and one for odd tiles: a wait by parity must not be two
      // phases behind, and not every product is waited for (those of two tiles
      // before are over when a tile's scores come)
      barrier_init(smem_at(&s_output[k / 2][k & 1]), 1);
    }
    for (uint32_t k = 0; k < F::kMeta; ++k) barrier_init(smem_at(&s_odd[k]), 32);
    barrier_init(smem_at(&s_asked), F::kWeights);  // an item's queries are there
    barrier_init(smem_at(&s_drained), kTiles);
    s_failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Keys behind the width's end are zeros, which nothing writes over, so that
  // the number of products is known to the code.
  if (p.c.width < kPad) {
    constexpr uint32_t kChunks = kPad / 8;
    for (uint32_t i = tid; i < F::kUnits * kTile * kChunks; i += F::kThreads) {
      const uint32_t chunk = i % kChunks, token = i / kChunks % kTile, unit = i / (kChunks * kTile);
      if (chunk * 8 >= p.c.width)
        *(uint4*)(smem + unit * F::kUnit + chunk / 8 * kPanel + token * 128 + ((chunk & 7) ^ (token & 7)) * 16) = make_uint4(0, 0, 0, 0);
    }
    writes_to_async_proxy();
  }
  wait_for_prerequisites();
  dependents_may_launch();
  // TMEM only now: a CTA that had it while it waits would keep it from the CTAs, of any
  // library, of the kernels that it waits for.
  if (warp == F::kWarps - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&s_tmem)), "n"(F::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tensor_fence_before();
  __shared__ Share share;  // not in every thread's registers
  {
    const Share mine = plan_share<F::kRows, F::kThreads>(p);
    if (tid == 0) share = mine;
  }
  __syncthreads();
  tensor_fence_after();
  const uint32_t tmem = s_tmem, scores = tmem, output = tmem + 2 * kTiles * kTile;  // of the first 128 rows
  const bool e4m3 = p.c.type == DB_E4M3;

  // All kinds of warps go through the same items and tiles.
  uint64_t at = share.lo, before = share.before;
  uint32_t request = share.request;
  uint32_t items = 0, tiles = 0, units = 0;  // behind this CTA
  uint32_t odd_phases = 0;
  bool go = true;
  while (go && at < share.hi) {
    const Request r = near_request(p, share, request);
    const Extent e = extent_of<F::kRows>(p, r);
    if (at - before >= e.units) {
      before += e.units;
      ++request;
      continue;
    }
    const uint64_t x = at - before;
    const uint32_t item = (uint32_t)quotient(x, e.tiles), head = item / e.blocks, rb = item - head * e.blocks;
    const uint32_t t0 = (uint32_t)(x - (uint64_t)item * e.tiles);
    const uint32_t t1 = (uint32_t)min((uint64_t)e.tiles, t0 + (share.hi - at)), n = t1 - t0;
    const uint32_t rows = min(F::kRows, r.rows * p.group - rb * F::kRows);
    const uint32_t base = r.length - r.rows;  // tokens before the request's own

    if (warp >= F::kWeights / 32 && warp < F::kWeights / 32 + F::kLoaderWarps) {
      // ------------------------------------------------------------- loaders
      // A warp has every third unit to itself (every sixth with two tiles of rows), and waits for no other.
      const uint32_t mine = warp - F::kWeights / 32, own = (mine + F::kLoaderWarps - units % F::kLoaderWarps) % F::kLoaderWarps;
      const int32_t* const table = p.view.table + (uint64_t)r.seq * p.view.columns;
      constexpr uint32_t kChunks = kPad / 8, kRawChunks = kCodes ? kPad / 16 : kChunks;  // 16-byte chunks of a row
      constexpr uint32_t kStep = 32 / kRawChunks, kEach = kTile / kStep;  // a lane has the same chunk of every kStep-th token
      const uint32_t chunk = lane % kRawChunks, token0 = lane / kRawChunks;
      const bool has = chunk < (kCodes ? p.c.width / 16 : p.c.width / 8);

      // unit u of the item: its tile, and whether it is of keys
      const auto unit_of = [&](uint32_t u, uint32_t& t, bool& key) __attribute__((always_inline)) {
        key = u == 0 || ((u & 1) && u != 2 * n - 1);
        t = t0 + (u == 0 ? 0 : u == 2 * n - 1 ? n - 1 : key ? (u + 1) / 2 : u / 2 - 1);
      };
      const auto slot_of = [&](uint32_t u) __attribute__((always_inline)) { return (units + u) % F::kUnits; };
      const auto phase_of = [&](uint32_t u) __attribute__((always_inline)) { return ((units + u) / F::kUnits + 1) & 1; };
      // What this lane has written of a unit is there for the tensor cores.
      const auto hand_on = [&](uint32_t u) __attribute__((always_inline)) {
        writes_to_async_proxy();
        barrier_arrive(smem_at(&s_full[slot_of(u)]));
      };
      // The places of a unit's tokens: a lane looks up tokens lane and lane + 32.
      struct Places {
        int2 at[2];  // page and slot, or -1 and -1
      };
      const auto look = [&](uint32_t u) __attribute__((always_inline)) {
        Places w;
        uint32_t t;
        bool key;
        unit_of(u, t, key);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w.at[h] = make_int2(-1, -1);
          const uint32_t position = t * kTile + 32 * h + lane;
          if (u < 2 * n && position < r.length) {
            const uint32_t column = position / p.view.page_tokens;
            w.at[h] = make_int2(__ldg(table + column), (int)(position - column * p.view.page_tokens));
          }
        }
        return w;
      };
      const auto settle = [&](Places& w) __attribute__((always_inline)) {  // entries that are no page
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((uint32_t)w.at[h].x >= p.view.n_pages) {
            if (w.at[h].y >= 0) report_table(p.view.ctr);
            w.at[h] = make_int2(-1, -1);
          }
      };
      // Notes of a tile for the weights, by the warp that has its keys.
      const auto note = [&](uint32_t t, const Places& w) __attribute__((always_inline)) {
        TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m.place[32 * h + lane] = w.at[h];
          const uint32_t real = __ballot_sync(kFull, w.at[h].x >= 0);
          if (lane == 0) m.real[h] = real;
        }
      };
      const auto all_seen = [&](uint32_t t, const Places& w) __attribute__((always_inline)) {
        return __all_sync(kFull, w.at[0].x >= 0 && w.at[1].x >= 0) && (t + 1) * kTile <= base;
      };
      // Offsets of a lane's two tokens in the pool, of all heads and chunks.
      const auto offset = [&](const int2& w, bool key) __attribute__((always_inline)) {
        return (uint64_t)(uint32_t)w.x * (key ? p.c.k_stride : p.c.v_stride) + (uint64_t)(uint32_t)w.y * p.token_step;
      };
      // Starts the copies of a unit; a token's chunk goes to place(token, k).
      const auto start = [&](bool key, bool whole, const Places& w, auto place) __attribute__((always_inline)) {
        const char* const from = (const char*)(key ? p.c.k : p.c.v) + head * p.head_step + chunk * 16;
        // Offsets of 32 bits, by 16 bytes, take half the shuffles (pools up to 64
        // GiB; 48 trees 152 us with those of 64, 144 so).
        if (whole && p.narrow) {
          const uint32_t page_step = (uint32_t)((key ? p.c.k_stride : p.c.v_stride) / 16), step = (uint32_t)p.token_step / 16;
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t off = (uint32_t)w.at[h].x * page_step + (uint32_t)w.at[h].y * step;
            constexpr uint32_t kBatch = kEach / 2 < 8 ? kEach / 2 : 8;
#pragma unroll 1
            for (uint32_t k0 = h * kEach / 2; k0 < (h + 1) * kEach / 2; k0 += kBatch) {
              uint32_t at[kBatch];
#pragma unroll
              for (uint32_t k = 0; k < kBatch; ++k) at[k] = __shfl_sync(kFull, off, (token0 + (k0 + k) * kStep) & 31);
              if (!has) continue;
#pragma unroll
              for (uint32_t k = 0; k < kBatch; ++k)
                copy16(place(token0 + (k0 + k) * kStep, k0 + k), from + (uint64_t)at[k] * 16, true);
            }
          }
          copies_commit();
          return;
        }
        const uint64_t off[2] = {offset(w.at[0], key), offset(w.at[1], key)};
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const uint32_t there = __ballot_sync(kFull, w.at[h].x >= 0);
          constexpr uint32_t kBatch = kEach / 2 < 8 ? kEach / 2 : 8;  // addresses first, then their copies
#pragma unroll 1
          for (uint32_t k0 = h * kEach / 2; k0 < (h + 1) * kEach / 2; k0 += kBatch) {
            uint64_t at[kBatch];
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) at[k] = __shfl_sync(kFull, off[h], (token0 + (k0 + k) * kStep) & 31);
            if (!has) continue;
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) {
              const uint32_t token = token0 + (k0 + k) * kStep;
              const bool real = (there >> (token & 31)) & 1;
              copy16(place(token, k0 + k), from + (real ? at[k] : 0), real);
            }
          }
        }
        copies_commit();
      };
      // Values of a tile that not every row sees, when they have come: tokens
      // with some that are not finite become zeros, and are noted for the
      // weights. at(token, k): where this lane's chunk is.
      const auto check = [&](uint32_t t, const Places& w, auto at) {
        uint32_t odd[2] = {0, 0};
        const auto bad_at = [&](uint32_t k) __attribute__((always_inline)) {
          const uint4 v = *(const uint4*)(smem + at(token0 + k * kStep, k));
          if (kCodes) {
            const auto nan4 = [](uint32_t c) { return ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
            return e4m3 && (nan4(v.x) | nan4(v.y) | nan4(v.z) | nan4(v.w));
          }
          return not_finite2<W>(v.x) || not_finite2<W>(v.y) || not_finite2<W>(v.z) || not_finite2<W>(v.w);
        };
        // (tokens before the request's own are seen by all rows, missing ones are zeros)
        const uint32_t k1 = t * kTile < base ? (base - t * kTile) / kStep : 0;
        bool any = false;
#pragma unroll 4
        for (uint32_t k = k1; k < kEach; ++k) any |= has && bad_at(k);
        if (__any_sync(kFull, any)) {
#pragma unroll 1
          for (uint32_t k = k1; k < kEach; ++k) {
            const uint32_t token = token0 + k * kStep;
            const uint32_t votes = __ballot_sync(kFull, has && bad_at(k)) >> token0 * kRawChunks % 32;
            if (votes & (kRawChunks == 32 ? 0xFFFFFFFFu : (1u << kRawChunks % 32) - 1)) {
              if (has) *(uint4*)(smem + at(token, k)) = make_uint4(0, 0, 0, 0);
              odd[0] |= token < 32 ? 1u << (token & 31) : 0u;
              odd[1] |= token < 32 ? 0u : 1u << (token & 31);
            }
          }
        }
        TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          odd[h] = __reduce_or_sync(kFull, odd[h]);
          if (kCodes) {  // a scale that is not finite: the token's values are not
            float sc = 0.f;
            if (w.at[h].x >= 0)
              sc = __ldg((const float*)((const char*)p.c.v_scale + (uint64_t)w.at[h].x * p.c.v_scale_stride) +
                         (uint32_t)w.at[h].y * p.scale_token_step + head * p.scale_head_step);
            odd[h] |= __ballot_sync(kFull, (__float_as_uint(sc) & 0x7F800000u) == 0x7F800000u);
          }
          if (lane == 0) m.odd[h] = odd[h];
        }
        barrier_arrive(smem_at(&s_odd[(tiles + t - t0) % F::kMeta]));
      };

      Places w = look(own);  // its first unit of the item
      if constexpr (kCodes) {
        // A lane widens the codes that it has copied itself.
        const uint32_t raw = query + F::kQuery + mine * F::kRaw + lane * 16;
        const unsigned char* const from = smem + (raw - ring);
        float k_sc[2], v_sc[2];
        bool whole = false;
        const auto ask = [&](uint32_t u) __attribute__((always_inline)) {
          uint32_t t;
          bool key;
          unit_of(u, t, key);
          settle(w);
          whole = all_seen(t, w);
          start(key, whole, w, [&](uint32_t, uint32_t k) __attribute__((always_inline)) { return raw + k * 512; });
          if (key) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              k_sc[h] = v_sc[h] = 0.f;
              if (w.at[h].x >= 0) {
                const uint32_t of = (uint32_t)w.at[h].y * p.scale_token_step + head * p.scale_head_step;
                k_sc[h] = __ldg((const float*)((const char*)p.c.k_scale + (uint64_t)w.at[h].x * p.c.k_scale_stride) + of);
                v_sc[h] = __ldg((const float*)((const char*)p.c.v_scale + (uint64_t)w.at[h].x * p.c.v_scale_stride) + of);
              }
            }
          }
        };
        if (own < 2 * n) ask(own);
        for (uint32_t u = own; u < 2 * n; u += F::kLoaderWarps) {
          uint32_t t;
          bool key;
          unit_of(u, t, key);
          Places next = look(u + F::kLoaderWarps);
          barrier_wait(smem_at(&s_empty[slot_of(u)]), phase_of(u), &s_failed);
          __syncwarp();
          if (key) {
            note(t, w);
            TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // an infinite scale stands for values of both signs, whose
              // products have no sum
              m.k_scale[32 * h + lane] = __fmaf_rn(k_sc[h], 0.f, k_sc[h]) * fabsf(p.scale_log2);
              const bool finite = (__float_as_uint(v_sc[h]) & 0x7F800000u) != 0x7F800000u;
              m.v_scale[32 * h + lane] = !whole && !finite ? 0.f : v_sc[h];  // odd tokens are added by themselves
              const uint32_t most = __reduce_max_sync(kFull, scale_exponent(v_sc[h]));
              if (lane == 0) m.exponent[h] = most;
            }
          }
          copies_wait<0>();
          if (!key && !whole) check(t, w, [&](uint32_t, uint32_t k) __attribute__((always_inline)) { return raw - ring + k * 512; });
          unsigned char* const to = smem + slot_of(u) * F::kUnit + chunk / 4 * kPanel;
          const auto widen_all = [&](auto four) __attribute__((always_inline)) {
            constexpr bool kFour = decltype(four)::value;
            constexpr uint32_t kBatch = kEach < 4 ? kEach : 4;  // (wide trees: 2 268 us, 4 236, 8 284)
#pragma unroll 1
            for (uint32_t k0 = 0; k0 < kEach; k0 += kBatch) {
              uint4 c[kBatch];
#pragma unroll
              for (uint32_t k = 0; k < kBatch; ++k) c[k] = *(const uint4*)(from + (k0 + k) * 512);
#pragma unroll
              for (uint32_t k = 0; k < kBatch; ++k) {
                const uint32_t token = token0 + (k0 + k) * kStep;
                const uint2 y[4] = {widen4(c[k].x, kFour), widen4(c[k].y, kFour), widen4(c[k].z, kFour), widen4(c[k].w, kFour)};
                *(uint4*)(to + token * 128 + (((2 * chunk) & 7) ^ (token & 7)) * 16) = make_uint4(y[0].x, y[0].y, y[1].x, y[1].y);
                *(uint4*)(to + token * 128 + (((2 * chunk + 1) & 7) ^ (token & 7)) * 16) = make_uint4(y[2].x, y[2].y, y[3].x, y[3].y);
              }
            }
          };
          if (has) {
            if (e4m3)
              widen_all(std::true_type{});
            else
              widen_all(std::false_type{});
          }
          hand_on(u);
          __syncwarp();
          w = next;
          if (u + F::kLoaderWarps < 2 * n) ask(u + F::kLoaderWarps);
        }
      } else {
        uint32_t waiting = 0xFFFFFFFFu;  // a unit whose copies are under way
        for (uint32_t u = own; u < 2 * n; u += F::kLoaderWarps) {
          uint32_t t;
          bool key;
          unit_of(u, t, key);
          const Places next = look(u + F::kLoaderWarps);
          settle(w);
          const bool whole = all_seen(t, w);
          const uint32_t bar = smem_at(&s_empty[slot_of(u)]);
          if (!__all_sync(kFull, barrier_test(bar, phase_of(u)))) {
            if (waiting != 0xFFFFFFFFu) {  // meanwhile what has come is handed on
              copies_wait<0>();
              hand_on(waiting);
              waiting = 0xFFFFFFFFu;
            }
            barrier_wait(bar, phase_of(u), &s_failed);
            __syncwarp();
          }
          if (key) note(t, w);
          const uint32_t to = slot_of(u) * F::kUnit + chunk / 8 * kPanel;
          const auto place = [&](uint32_t token, uint32_t) __attribute__((always_inline)) {
            return to + token * 128 + ((chunk & 7) ^ (token & 7)) * 16;
          };
          start(key, whole, w, [&](uint32_t token, uint32_t k) __attribute__((always_inline)) { return ring + place(token, k); });
          if (waiting != 0xFFFFFFFFu) {
            copies_wait<1>();
            hand_on(waiting);
          }
          waiting = u;
          if (!key && !whole) {
            copies_wait<0>();
            check(t, w, place);
          }
          w = next;
        }
        if (waiting != 0xFFFFFFFFu) {
          copies_wait<0>();
          hand_on(waiting);
        }
      }
      go = __all_sync(kFull, !s_failed);
    } else if (warp >= kIssuer) {
      // ------------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t kind_s = product_kind(kTypeW, kTile, false), kind_o = product_kind(kTypeW, p.c.width, true);
        // A thread makes all products of 128 rows, and is short of time.
        const uint32_t i = warp - kIssuer;
        const uint64_t queries = tile_descriptor(query + i * kQueryTile, 16), keys = tile_descriptor(ring, 16), values = tile_descriptor(ring, kPanel);
        const auto moved = [](uint64_t d, uint32_t bytes) __attribute__((always_inline)) {
          return d & 0xFFFFFFFF00000000ull | (uint32_t)((uint32_t)d + bytes / 16);
        };
        const auto unit_at = [&](uint32_t u, uint32_t& slot) __attribute__((always_inline)) {  // waits until a unit is there
          slot = (units + u) % F::kUnits;
          return barrier_wait(smem_at(&s_full[slot]), ((units + u) / F::kUnits) & 1, &s_failed);
        };
        const auto score = [&](uint32_t k) {
          uint32_t slot;
          if (!unit_at(k ? 2 * k - 1 : 0, slot)) return false;
          tensor_fence_after();
          const uint32_t buffer = (tiles + k) & 1, to = scores + (2 * i + buffer) * kTile;
          const uint64_t key = moved(keys, slot * F::kUnit);
#pragma unroll
          for (uint32_t st = 0; st < kPad / 16; ++st)
            tensor_multiply(to, moved(queries, st / 4 * kQueryPanel + st % 4 * 32), moved(key, st / 4 * kPanel + st % 4 * 32), kind_s, st > 0);
          tensor_commit(smem_at(&s_scores[i][buffer]));
          tensor_commit(smem_at(&s_empty[slot]));
          barrier_arrive(smem_at(&s_scores[i][buffer]));
          return true;
        };
        bool ok = barrier_wait(smem_at(&s_asked), items & 1, &s_failed) && score(0);
        for (uint32_t k = 0; ok && k < n; ++k) {
          if (k + 1 < n) ok = score(k + 1);
          if (!ok) break;
          const uint32_t buffer = (tiles + k) & 1;
          uint32_t slot;
          ok = unit_at(k + 1 < n ? 2 * k + 2 : 2 * n - 1, slot) &&
               barrier_wait(smem_at(&s_weights[i][buffer]), ((tiles + k) >> 1) & 1, &s_failed);
          if (!ok) break;
          tensor_fence_after();
          const uint64_t value = moved(values, slot * F::kUnit);
#pragma unroll
          for (uint32_t st = 0; st < kTile / 16; ++st)
            tensor_multiply_t(output + i * kPad, scores + (2 * i + buffer) * kTile + st * 8, moved(value, st * 2048), kind_o, true);
          tensor_commit(smem_at(&s_output[i][buffer]));
          tensor_commit(smem_at(&s_empty[slot]));
        }
        go = ok;
      }
      go = __shfl_sync(kFull, go, 0);
    } else if (warp < F::kWeights / 32) {
      // -------------------------------------------------------------- weights
      const uint32_t row = tid, lanes = (warp & 3) << 21, half = warp / 4;  // of 128 rows
      const uint32_t sums_at = output + half * kPad + lanes;
      const bool row_real = row < rows;
      const uint32_t all = rb * F::kRows + (row_real ? row : 0), node = all / p.group;
      const uint32_t* const mask = p.mask ? p.mask + (uint64_t)(r.first + node) * p.mask_words : nullptr;
      float factor = kCodes || p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);  // of the row's scores
      {
        // The row's query; the products with the one before were over when its
        // last scores came. For codes a bf16 one becomes f16, times the power of
        // two that takes its largest value to 2^14.
        constexpr uint32_t kFetch = kPad == 64 ? 8 : 16;
        constexpr bool kTurns = kCodes && !std::is_same<T, __half>::value;
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.f ? 0u : 0xFFFFFFFFu;
        const char* const from = (const char*)p.q.base + (uint64_t)(r.first + node) * p.q.row_stride +
                                 (head * p.group + (all - node * p.group)) * p.q.head_stride;
        uint32_t largest = 0;
#pragma unroll 1
        for (uint32_t pass = kTurns && kPad > 128 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
          for (uint32_t c0 = 0; c0 < p.c.width / 8; c0 += kFetch) {
            uint4 v[kFetch];
#pragma unroll
            for (uint32_t c = 0; c < kFetch; ++c) {
              v[c] = row_real && c0 + c < p.c.width / 8 ? __ldg((const uint4*)from + c0 + c) : make_uint4(0, 0, 0, 0);
              v[c].x = (v[c].x ^ flip) & keep, v[c].y = (v[c].y ^ flip) & keep, v[c].z = (v[c].z ^ flip) & keep, v[c].w = (v[c].w ^ flip) & keep;
            }
            float up = 1.f;
            if constexpr (kTurns) {
              if (kPad <= 128 || pass == 0) {
#pragma unroll
                for (uint32_t c = 0; c < kFetch; ++c) {
                  const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {  // bits of magnitudes, those of infinities and NaN left out
                    const uint32_t lo = w[k] & 0x7FFFu, hi = w[k] >> 16 & 0x7FFFu;
                    largest = max(largest, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                  }
                }
              }
              const int exponent = largest == 0 ? 14 : max((int)(largest >> 7) - 127, 14 - 126);
              up = __uint_as_float((uint32_t)(14 - exponent + 127) << 23);
              factor = __uint_as_float((uint32_t)(max(exponent - 14, -126) + 127) << 23);
            }
            if (pass == 0) continue;
#pragma unroll
            for (uint32_t c = 0; c < kFetch; ++c) {
              if constexpr (kTurns) {
                uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 a = unpack2<T>(w[k]);
                  w[k] = pack2<W>(a.x * up, a.y * up);
                }
                v[c] = make_uint4(w[0], w[1], w[2], w[3]);
              }
              *(uint4*)(smem + F::kUnits * F::kUnit + half * kQueryTile + (c0 + c) / 8 * kQueryPanel + (row & 127) * 128 +
                        ((c & 7) ^ (row & 7)) * 16) = v[c];
            }
          }
        }
        writes_to_async_proxy();
        barrier_arrive(smem_at(&s_asked));
      }
      // Weights are exp2(score - ref). ref is kLift below what was the largest score, for
      // codes the largest score times its values' scale of the tokens that the row sees:
      // P has the scales as a factor, and so stays in the middle of f16's range.
      constexpr float kLift = (float)attn_lift<W>(kSlack);
      float top = -INFINITY, sum = 0.f;
      {
        uint32_t zero[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) zero[j] = 0;
#pragma unroll 1
        for (uint32_t c = 0; c < p.c.width; c += 16) tmem_store16(sums_at + c, zero);
        tmem_stored();
      }
      bool ok = true;
      for (uint32_t k = 0; k < n; ++k) {
        const uint32_t tile = tiles + k, buffer = tile & 1, t = t0 + k;
        const uint32_t here = scores + (2 * half + buffer) * kTile + lanes;
        ok = barrier_wait(smem_at(&s_scores[half][buffer]), (tile >> 1) & 1, &s_failed);
        if (!__all_sync(kFull, ok)) break;
        tensor_fence_after();
        const TileNotes& m = s_notes[tile % F::kMeta];
        // which tokens this row sees
        const bool masked = (t + 1) * kTile > base || (m.real[0] & m.real[1]) != 0xFFFFFFFFu;
        uint32_t sees[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (masked) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int32_t own = (int32_t)(t * kTile + 32 * h - base);  // the node of the word's first token
            uint32_t bits;
            if (own <= -32) {
              bits = 0xFFFFFFFFu;
            } else if (!mask) {
              const int32_t upto = (int32_t)node - own + 1;
              bits = upto <= 0 ? 0u : upto >= 32 ? 0xFFFFFFFFu : (1u << upto) - 1;
            } else {
              const int32_t word = own >> 5;  // -1: tokens before the request's
              const uint32_t a = word < 0 ? 0xFFFFFFFFu : (uint32_t)word < p.mask_words ? __ldg(mask + word) : 0u;
              const uint32_t b = (uint32_t)(word + 1) < p.mask_words ? __ldg(mask + word + 1) : 0u;
              bits = __funnelshift_r(a, b, (uint32_t)own & 31);
            }
            sees[h] = bits & m.real[h];
          }
          hide_scores(here, sees[0], sees[1], kCodes ? m.k_scale : nullptr);
        }
        // Both passes over the scores read them from TMEM, by halves, in loops whose
        // code is short enough for the instruction caches (48 trees 185 us with all
        // of it unrolled, 156 so). Codes' scores go back times their keys' scales in
        // between (16 wide trees 249 us with them held in registers, 236 so).
        const ulonglong2* const scales = (const ulonglong2*)(masked ? s_ones : m.k_scale);
        const auto half_of = [&](uint32_t h, uint64_t (&x)[16]) __attribute__((always_inline)) {
          uint32_t w[32];
          __syncwarp();
          tmem_load32(here + 32 * h, w);
          tmem_loaded();
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = pair(w[2 * j], w[2 * j + 1]);
        };
        float most = -INFINITY, other = -INFINITY;
#pragma unroll 1
        for (uint32_t h = 0; h < 2; ++h) {
          uint64_t x[16];
          half_of(h, x);
          if constexpr (kCodes) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 y = scales[8 * h + j];
              x[2 * j] = multiply2(x[2 * j], y.x);
              x[2 * j + 1] = multiply2(x[2 * j + 1], y.y);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) w[2 * j] = __float_as_uint(low(x[j])), w[2 * j + 1] = __float_as_uint(high(x[j]));
            __syncwarp();
            tmem_store32(here + 32 * h, w);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2) most = largest3(most, low(x[j]), high(x[j])), other = largest3(other, low(x[j + 1]), high(x[j + 1]));
        }
        if (kCodes) tmem_stored();
        most = fmaxf(most, other);
        most *= factor;
        // With codes no product is larger than the largest score times the tile's largest
        // scale, hidden tokens' among them; only where that would move the reference is
        // the row's own largest looked for, so what is hidden has no part in it. (16 wide
        // trees 241 us; 253 with all scores times their scales in the loop above.)
        const auto rises = [&](float x) __attribute__((always_inline)) {
          return x > top + (float)kSlack || (top == -INFINITY && x > -INFINITY);
        };
        bool move = rises(kCodes ? most + (float)((int)max(m.exponent[0], m.exponent[1]) - 127) : most);
        uint64_t odd = 0;
        if (masked) {
          const uint32_t at_odd = tile % F::kMeta;
          ok = barrier_wait(smem_at(&s_odd[at_odd]), (odd_phases >> at_odd) & 1, &s_failed);
          if (!__all_sync(kFull, ok)) break;
          odd_phases ^= 1u << at_odd;
          odd = (uint64_t)m.odd[0] | (uint64_t)m.odd[1] << 32;
        }
        if (__any_sync(kFull, move) || odd) {
          if (kCodes) {
            most = largest_product(here, factor, m.v_scale);
            move = rises(most);
          }
          const float fall = move ? top - most : 0.f;
          if (move) top = most;
          // O belongs to this warp while no product adds to it
          if (k && (odd || __any_sync(kFull, move))) {
            ok = barrier_wait(smem_at(&s_output[half][buffer ^ 1]), ((tile - 1) >> 1) & 1, &s_failed);
            if (!__all_sync(kFull, ok)) break;
            tensor_fence_after();
            const float down = exp2_of(fall);
            sum = times_exp2(sum, fall);
#pragma unroll 1
            for (uint32_t c = 0; c < p.c.width; c += 16) {
              uint32_t o[16];
              tmem_load16(sums_at + c, o);
              tmem_loaded();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * down);
              tmem_store16(sums_at + c, o);
            }
            tmem_stored();
          }
          if (odd)
            add_odd<T, kCodes>(m, sums_at, here, odd, (uint64_t)sees[1] << 32 | sees[0], factor, top == -INFINITY ? 0.f : top - kLift,
                               (const char*)p.c.v + head * p.head_step, p.c.v_stride, p.token_step,
                               (const char*)(p.c.v_scale + (kCodes ? head * p.scale_head_step : 0)), p.c.v_scale_stride,
                               p.scale_token_step, !e4m3, p.c.width);
        }
        const float ref = top == -INFINITY ? 0.f : top - kLift;
        uint64_t sums = pair(__float_as_uint(sum), 0), more = pair(0, 0);
        const uint64_t by = pair(__float_as_uint(factor), __float_as_uint(factor));
        const uint64_t less = pair(__float_as_uint(-ref), __float_as_uint(-ref));
#pragma unroll 1
        for (uint32_t h = 0; h < 2; ++h) {
          uint64_t x[16];
          uint32_t w[16];
          half_of(h, x);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            uint64_t y[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint64_t z = multiply_add2(x[j + g], by, less);
              y[g] = pair(__float_as_uint(exp2_of(low(z))), __float_as_uint(exp2_of(high(z))));
            }
            sums = add2(sums, y[0]);
            more = add2(more, y[1]);
            if (kCodes) {
              const ulonglong2 z = ((const ulonglong2*)m.v_scale)[8 * h + j / 2];
              y[0] = multiply2(y[0], z.x);
              y[1] = multiply2(y[1], z.y);
            }
            w[j] = pack2<W>(low(y[0]), high(y[0]));
            w[j + 1] = pack2<W>(low(y[1]), high(y[1]));
          }
          __syncwarp();
          tmem_store16(here + 16 * h, w);  // over the scores that have been read
        }
        sums = add2(sums, more);
        sum = low(sums) + high(sums);
        tmem_stored();
        tensor_fence_before();
        barrier_arrive(smem_at(&s_weights[half][buffer]));
      }
      if (ok) ok = barrier_wait(smem_at(&s_output[half][(tiles + n - 1) & 1]), ((tiles + n - 1) >> 1) & 1, &s_failed);
      go = group_all(1, F::kWeights, ok);
      if (go) {
        tensor_fence_after();
        const float ref = top - kLift;
        const bool whole = t0 == 0 && t1 == e.tiles;
        const auto query_head = [&](uint32_t row_, uint32_t& nd) {
          const uint32_t a = rb * F::kRows + row_;
          nd = a / p.group;
          return head * p.group + (a - nd * p.group);
        };
        float* const mine = p.partial + (uint64_t)(2 * blockIdx.x + (t0 == 0)) * partial_floats(F::kRows, kPad);
        uint32_t nd;
        const uint32_t qh = query_head(row_real ? row : 0, nd);
        char* const to = (char*)p.out.base + (uint64_t)(r.first + nd) * p.out.row_stride + qh * p.out.head_stride;
        const float by = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 2
        for (uint32_t c = 0; c < p.c.width; c += 16) {
          uint32_t o[16];
          __syncwarp();
          tmem_load16(sums_at + c, o);
          tmem_loaded();
          if (!row_real) continue;
          const float* const f = (const float*)o;
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
              const uint2 a = four_answers<T>(make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]), by);
              const uint2 b = four_answers<T>(make_float4(f[j + 4], f[j + 5], f[j + 6], f[j + 7]), by);
              *(uint4*)(to + (c + j) * 2) = make_uint4(a.x, a.y, b.x, b.y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              __stcg((float4*)mine + (c + j) / 4 * F::kRows + row, make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]));
          }
        }
        const auto statistics = [&](uint32_t nd_, uint32_t qh_, float m_, float l_) {
          if (p.lse)
            p.lse[(uint64_t)(r.first + nd_) * (p.c.heads * p.group) + qh_] =
                l_ == 0.f ? -INFINITY : m_ * 0.6931471805599453f + logf(l_);
        };
        if (whole) {
          if (row_real) statistics(nd, qh, ref, sum);
        } else {
          if (row_real) {
            __stcg(mine + F::kRows * kPad + row, ref);
            __stcg(mine + F::kRows * kPad + F::kRows + row, sum);
          }
          __threadfence();
          group_sync(1, F::kWeights);
          const uint64_t first = at - t0;
          const uint32_t c0 = owner_of(share, first), c1 = owner_of(share, first + e.tiles - 1);
          if (tid == 0) {
            const unsigned int seen = atomicAdd(p.arrived + c0, 1u);
            s_last = seen == c1 - c0;
            if (s_last) p.arrived[c0] = 0;
          }
          group_sync(1, F::kWeights);
          if (s_last) {
            __threadfence();
            const JoinedItem item_of = {r.first, rb * F::kRows, rows, head, c0, c1};
            // the queries' place is free: all products with them are made
            join_item<T, F::kRows, kPad, F::kWeights>(p, item_of, (float4*)(smem + F::kUnits * F::kUnit), 1);
          }
          group_sync(1, F::kWeights);  // s_last has been read
        }
      }
    }
    at += n;
    ++items;
    tiles += n;
    units += 2 * n;
  }
  // nothing is under way when the shared memory and TMEM are given back
  if (warp >= F::kWeights / 32 && warp < kIssuer) copies_wait<0>();
  if (warp >= kIssuer && lane == 0) {
    tensor_commit(smem_at(&s_drained));
    const uint64_t began = globaltimer_ns();
    while (!barrier_try(smem_at(&s_drained), 0) && globaltimer_ns() - began < kWaitLimitNs) {
    }
  }
  tensor_fence_before();
  __syncthreads();
  if (warp == F::kWarps - 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(F::kColumns));
  if (s_failed) {  // (CTA 0 wrote the status when it began, the length of a wait's limit ago)
    if (tid == 0 && p.view.ctr) atomicOr((unsigned int*)&p.view.ctr->err, DB_ERR_TIMEOUT);
    if (p.view.status)
#pragma unroll 1
      for (uint32_t i = tid; i < p.view.n; i += F::kThreads) p.view.status[i] = DB_PAGE_INVALID;
  }
}

template <typename T, uint32_t kPad, bool kCodes, uint32_t kTiles>
int launch_many(const AttnParams& p, cudaStream_t s) {
  typedef Many<kPad, kCodes, kTiles> F;
  const cudaError_t e = cudaFuncSetAttribute(attention_many_kernel<T, kPad, kCodes, kTiles>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, F::kAsk);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_dependent(attention_many_kernel<T, kPad, kCodes, kTiles>, attn_grid(attn_ctas_per_sm(kPad, kCodes, F::kRows / 8)), F::kThreads, F::kAsk, s, p);
}

}  // namespace db
