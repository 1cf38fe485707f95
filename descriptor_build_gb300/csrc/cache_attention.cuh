// Attention of drafted tokens over a paged cache (include/cachedata.h:
// db_cache_attention): what its kernels share.
//
// With s = scale * <q, k> the output of a query row is sum exp(s) v / sum
// exp(s) over the tokens it sees; maximum, sum and the weighted values are
// carried through tiles of 64 tokens and rescaled when the maximum rises
// (log2 units, so that a weight is one exp2). Work is cut evenly over the
// CTAs whatever the lengths: a unit is one tile of one item, an item one
// request, key head and group of query rows; CTA c takes units [U*c/G,
// U*(c+1)/G) of all in order. An item that is cut leaves partial results in
// the workspace, and the last of its CTAs to finish joins them, in the order
// of the tokens: results do not depend on which one that is, and no CTA waits.
#pragma once

#include "cachedata.cuh"

namespace db {

constexpr uint32_t kTile = 64;             // tokens of a unit
constexpr uint32_t kAttnThreads = 128;
constexpr uint32_t kAttnCtasPerSm = 2;     // most CTAs an SM of the grid
constexpr uint32_t kMaxGroup = 64;
constexpr uint32_t kScaleSlack = 4;        // a larger exponent of scales is followed from here on
constexpr uint32_t kManyBlocks = 8;       // blocks of 16 query rows of the tcgen05 kernel's items

struct AttnParams {
  CacheView view;
  db_cache_layer c;
  db_cache_rows q, out;
  uint32_t group;       // query heads of a key head
  uint32_t max_tokens;
  float scale_log2;     // scale * log2(e)
  const uint32_t* mask;
  uint32_t mask_words;
  float* lse;
  uint64_t token_step, head_step;
  uint32_t scale_token_step, scale_head_step;
  float* partial;          // [2 * grid][rows of an item][width + 2 rounded]
  unsigned int* arrived;   // [grid], zero between calls
};

// Host: one instance of the kernels for a padded width.
int launch_attention_64(const AttnParams& p, uint32_t type, uint32_t blocks, unsigned grid, cudaStream_t s);
int launch_attention_128(const AttnParams& p, uint32_t type, uint32_t blocks, unsigned grid, cudaStream_t s);
int launch_attention_256(const AttnParams& p, uint32_t type, uint32_t blocks, unsigned grid, cudaStream_t s);

// Floats of a partial result of `rows` query rows: the weighted values, then
// maxima and sums.
__host__ __device__ inline uint32_t partial_floats(uint32_t rows, uint32_t padded) {
  return rows * (padded + 2);
}

// ---------------------------------------------------------------- the plan
__device__ __forceinline__ Request attention_request(const AttnParams& p, uint32_t i) {
  Request r = read_request(p.view, i, true);
  if (r.rows > p.max_tokens) {
    r.ok = false;
    r.rows = 0;
  }
  return r;
}

struct Extent {
  uint32_t blocks, tiles;  // groups of query rows of one key head, tiles of tokens
  uint64_t units;
};

template <uint32_t kRows>
__device__ __forceinline__ Extent extent_of(const AttnParams& p, const Request& r) {
  Extent e;
  e.blocks = (uint32_t)(((uint64_t)r.rows * p.group + kRows - 1) / kRows);
  e.tiles = r.rows ? (r.length + kTile - 1) / kTile : 0;
  e.units = (uint64_t)e.blocks * e.tiles * p.c.heads;
  return e;
}

struct Share {
  uint64_t all, lo, hi;  // units in all, of this CTA
  uint32_t ctas;         // that have any
  uint32_t request;      // the one that unit lo is of
  uint64_t before;       // units of the requests before it
  const Request* near;   // that one and the next few, in shared memory
};
constexpr uint32_t kNear = 8;

// A request that the CTA comes to: mostly one of the few that its plan looked
// up together, since its length is three loads one after the other.
__device__ __forceinline__ Request near_request(const AttnParams& p, const Share& s, uint32_t i) {
  return i - s.request < kNear ? s.near[i - s.request] : attention_request(p, i);
}

// This CTA's units. Every thread calls it.
template <uint32_t kRows, uint32_t kThreads>
__device__ __forceinline__ Share plan_share(const AttnParams& p) {
  __shared__ uint64_t s_scan[kThreads / 32];
  __shared__ uint64_t s_before;
  __shared__ uint32_t s_request;
  __shared__ Request s_near[kNear];
  const uint32_t tid = threadIdx.x, n = p.view.n;
  Share s;
  uint64_t units = 0, excl, all;
  uint32_t bad = 0;
  uint64_t rows = 0;
  for (uint32_t i = tid; i < n; i += kThreads) {
    const Request r = attention_request(p, i);
    units += extent_of<kRows>(p, r).units;
    rows += r.rows;
    bad += !r.ok;
    if (blockIdx.x == 0 && p.view.status) p.view.status[i] = r.ok ? DB_PAGE_OK : DB_PAGE_INVALID;
  }
  if (blockIdx.x == 0 && p.view.ctr) {
    if (rows) atomicAdd((unsigned long long*)&p.view.ctr->total, (unsigned long long)rows);
    if (bad) atomicAdd((unsigned long long*)&p.view.ctr->n_invalid, (unsigned long long)bad);
  }
  block_excl_scan64<kThreads / 32>(units, excl, all, s_scan);
  s.all = all;
  s.ctas = (uint32_t)min((uint64_t)gridDim.x, all);
  s.lo = s.hi = 0;
  s.request = 0;
  s.before = 0;
  if (blockIdx.x >= s.ctas) return s;
  s.lo = all * blockIdx.x / s.ctas;
  s.hi = all * (blockIdx.x + 1) / s.ctas;
  uint64_t base = 0;
  for (uint32_t i0 = 0;; i0 += kThreads) {
    const uint32_t i = i0 + tid;
    if (n > kThreads) {  // otherwise the scan above is the one that is needed
      __syncthreads();
      units = i < n ? extent_of<kRows>(p, attention_request(p, i)).units : 0;
      block_excl_scan64<kThreads / 32>(units, excl, all, s_scan);
    }
    if (s.lo >= base + excl && s.lo - (base + excl) < units) {
      s_request = i;
      s_before = base + excl;
    }
    base += all;
    if (s.lo < base) break;
  }
  __syncthreads();
  s.request = s_request;
  s.before = s_before;
  s.near = s_near;
  if (tid < kNear && s.request + tid < n) s_near[tid] = attention_request(p, s.request + tid);
  __syncthreads();
  return s;
}

// The CTA that has unit x.
static __device__ __noinline__ uint32_t owner_of(const Share& s, uint64_t x) {
  return (uint32_t)(((x + 1) * s.ctas - 1) / s.all);
}

// ------------------------------------------------------------ small operations
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes (or zeros) into shared memory, without a register. (The form with a
// size in a register is several times slower to start.)
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  if (real)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void multiply<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void multiply<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8-bit codes as four 16-bit values, exactly. I8 to bf16: a code's low
// seven bits c fit bf16's seven, 128 + c, from which 128 or, for a negative
// code, 256 goes. I8 to f16: 1024 + (code + 128), less 1152.
template <typename T>
__device__ __forceinline__ uint2 widen4(uint32_t w, bool e4m3);
template <>
__device__ __forceinline__ uint2 widen4<__half>(uint32_t w, bool e4m3) {
  if (e4m3) return make_uint2(e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
  uint2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = (__byte_perm(w, 0, h ? 0x4342 : 0x4140) ^ 0x00800080u) | 0x64006400u;
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&a), __half2half2(__ushort_as_half(0x6480)));
    (h ? r.y : r.x) = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}
template <>
__device__ __forceinline__ uint2 widen4<__nv_bfloat16>(uint32_t w, bool e4m3) {
  uint2 r;
  if (e4m3) {
    const float2 a = unpack2<__half>(e4m3x2_to_f16x2(w)), b = unpack2<__half>(e4m3x2_to_f16x2(w >> 16));
    return make_uint2(pack2<__nv_bfloat16>(a.x, a.y), pack2<__nv_bfloat16>(b.x, b.y));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __byte_perm(w, 0, h ? 0x4342 : 0x4140);
    const uint32_t x = (a & 0x007F007Fu) | 0x43004300u, y = (a & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    (h ? r.y : r.x) = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}

// Whether one of two 16-bit values is an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t w);
template <>
__device__ __forceinline__ bool not_finite2<__half>(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}
template <>
__device__ __forceinline__ bool not_finite2<__nv_bfloat16>(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// An item that several CTAs have parts of: rows [row0, row0 + rows) of a key
// head's queries of the request whose first row is `first`.
struct JoinedItem {
  uint32_t first, row0, rows, head, c0, c1;
};

// Joins the parts of CTAs c0 to c1, in their order, and writes the answer. A
// thread for each row finds the rows' maxima and sums, which go to `row_notes`
// (16 bytes a row of shared memory); then kMany times four values a thread are
// summed at a time, so that their loads are under way together. `group` is a
// named barrier of the kThreads threads.
template <typename T, uint32_t kRows, uint32_t kPad, uint32_t kThreads>
static __device__ __noinline__ void join_item(const AttnParams& p, const JoinedItem item, float4* row_notes, uint32_t barrier) {
  constexpr uint32_t kQuads = kPad / 4, kMany = 8, kPart = kRows * (kPad + 2);
  const float* const parts = p.partial + (uint64_t)2 * item.c0 * kPart;  // the first is its CTA's second
  const auto part_at = [&](uint32_t k) { return parts + (k == item.c0 ? kPart : (uint64_t)2 * (k - item.c0) * kPart); };
  if (threadIdx.x < item.rows) {
    const uint32_t row = threadIdx.x;
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (uint32_t k = item.c0; k <= item.c1; ++k) {
      const float mk = __ldcg(part_at(k) + kRows * kPad + row), lk = __ldcg(part_at(k) + kRows * kPad + kRows + row);
      const float now = fmaxf(m, mk), by = now == -INFINITY ? 0.f : now;
      l = l * exp2_of(m - by) + lk * exp2_of(mk - by);
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
  const uint32_t all = item.rows * kQuads;
#pragma unroll 1
  for (uint32_t c = threadIdx.x; c < all; c += kThreads * kMany) {
    float4 v[kMany];
#pragma unroll
    for (uint32_t j = 0; j < kMany; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t k = item.c0; k <= item.c1; ++k) {
      const float* const at = part_at(k);
      float m[kMany];
      float4 y[kMany];
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        const uint32_t of = min(c + j * kThreads, all - 1), row = of / kQuads, quad = min(of % kQuads, p.c.width / 4 - 1);
        m[j] = __ldcg(at + kRows * kPad + row);
        y[j] = __ldcg((const float4*)(at + row * kPad) + quad);
      }
#pragma unroll
      for (uint32_t j = 0; j < kMany; ++j) {
        const float b = exp2_of(m[j] - row_notes[min(c + j * kThreads, all - 1) / kQuads].x);
        v[j].x += y[j].x * b, v[j].y += y[j].y * b, v[j].z += y[j].z * b, v[j].w += y[j].w * b;
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < kMany; ++j) {
      const uint32_t of = c + j * kThreads;
      if (of < all && of % kQuads * 4 < p.c.width) {
        const float4 n = row_notes[of / kQuads];
        const uint64_t to = (uint64_t)__float_as_uint(n.w) << 32 | __float_as_uint(n.z);
        *(uint2*)((char*)p.out.base + to + of % kQuads * 8) =
            make_uint2(pack2<T>(v[j].x * n.y, v[j].y * n.y), pack2<T>(v[j].z * n.y, v[j].w * n.y));
      }
    }
  }
}

// --------------------------------------------------------- few rows: mma.sync
// A CTA of four warps. kBlocks blocks of 16 query rows; warp w works on block
// w % kBlocks and every (4 / kBlocks)-th part of a tile's tokens, so that few
// rows still feed all warps. Tiles come by 16-byte asynchronous copies, token
// by token from their pages, into a ring; 8-bit codes are widened from there
// into one tile of 16-bit values.
template <typename T, uint32_t kPad, bool kCodes, uint32_t kBlocks>
struct Few {
  static constexpr uint32_t kRows = 16 * kBlocks;
  static constexpr uint32_t kStages = kCodes ? (kPad > 128 ? 3 : 4) : (kPad > 128 ? 2 : 3);
  static constexpr uint32_t kRaw = kTile * kPad * (kCodes ? 1 : 2);        // keys or values of a stage
  static constexpr uint32_t kStage = 2 * kRaw + (kCodes ? 2 * kTile * 4 : 0);
  static constexpr uint32_t kWide = kCodes ? kTile * kPad * 2 : 0;         // widened keys or values
  static constexpr uint32_t kQuery = kPad > 128 ? kRows * kPad * 2 : 0;    // wide rows stay in shared memory
  static constexpr uint32_t kRing = kStages + 1;                           // of page lists
  static constexpr uint32_t kBytes = kStages * kStage + 2 * kWide + kQuery;
  static constexpr uint32_t kTokens = kTile * kBlocks / 4;                 // of a warp in a tile
  static_assert(kStages * kStage + 2 * kWide >= 4 * 16 * kPad * 4, "the join of the warps reuses the ring");
};

template <typename T, uint32_t kPad, bool kCodes, uint32_t kBlocks>
__global__ void __launch_bounds__(kAttnThreads, kPad > 128 ? 1 : 2) attention_few_kernel(const AttnParams p) {
  typedef Few<T, kPad, kCodes, kBlocks> F;
  typedef typename std::conditional<kCodes, __half, T>::type W;  // of weights and values
  constexpr uint32_t kChunks = kPad / 8;                 // 16-byte chunks of a 16-bit row
  constexpr uint32_t kRawChunks = kCodes ? kPad / 16 : kPad / 8;
  constexpr uint32_t kTokens = F::kTokens, kN = kTokens / 8, kSteps = kPad / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int2 s_place[F::kRing][kTile];  // page (or -1) and byte offset in it of a tile's tokens
  __shared__ float s_max[4][16], s_sum[4][16];
  __shared__ uint32_t s_broken, s_last, s_exponent[2];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const uint32_t block = warp % kBlocks, part = warp / kBlocks;
  const uint32_t ring = smem_at(smem), wide = ring + F::kStages * F::kStage, query = wide + 2 * F::kWide;
  const uint32_t chunks = p.c.width / 8, raw_chunks = kCodes ? p.c.width / 16 : chunks, steps = p.c.width / 16;
  const bool e4m3 = p.c.type == DB_E4M3;

  const Share share = plan_share<F::kRows, kAttnThreads>(p);
  uint64_t at = share.lo, before = share.before;
  uint32_t i = share.request;
  if (tid == 0) s_broken = 0;
  while (at < share.hi) {
    const Request r = near_request(p, share, i);
    const Extent e = extent_of<F::kRows>(p, r);
    if (at - before >= e.units) {
      before += e.units;
      ++i;
      continue;
    }
    const uint64_t x = at - before;
    const uint32_t t0 = (uint32_t)(x % e.tiles);
    const uint32_t item = (uint32_t)(x / e.tiles), head = item / e.blocks, rb = item - head * e.blocks;
    const uint32_t t1 = (uint32_t)min((uint64_t)e.tiles, t0 + (share.hi - at));
    const uint32_t rows = min(F::kRows, r.rows * p.group - rb * F::kRows);
    const uint32_t base = r.length - r.rows;  // tokens before the request's own
    const int32_t* const table = p.view.table + (uint64_t)r.seq * p.view.columns;

    // places of a tile's tokens: threads 0 to 63 look one up each
    const auto look = [&](uint32_t t) {
      int2 w = make_int2(-1, 0);
      const uint32_t position = t * kTile + tid;
      if (tid < kTile && t < t1 && position < r.length) {
        const uint32_t column = position / p.view.page_tokens;
        const uint32_t page = (uint32_t)__ldg(table + column);
        if (page < p.view.n_pages)
          w = make_int2((int)page, (int)(position - column * p.view.page_tokens));
        else
          w.y = -1;
      }
      return w;
    };
    const auto keep_places = [&](uint32_t t, int2 w) {
      if (tid < kTile) {
        s_place[t % F::kRing][tid] = w;
        if (w.y < 0) {
          s_broken = 1;
          report_table(p.view.ctr);
        }
      }
    };
    const char* const keys = (const char*)p.c.k + head * p.head_step;
    const char* const values = (const char*)p.c.v + head * p.head_step;
    const auto fetch = [&](uint32_t t) {  // starts the copies of a tile
      if (t < t1) {
        const uint32_t slot = ring + (t % F::kStages) * F::kStage;
        const uint32_t chunk = tid % kRawChunks;
#pragma unroll 4
        for (uint32_t k = 0; k < kTile * kRawChunks / kAttnThreads; ++k) {
          const uint32_t token = tid / kRawChunks + k * (kAttnThreads / kRawChunks);
          const int2 w = s_place[t % F::kRing][token];
          const bool real = w.x >= 0 && chunk < raw_chunks;
          const uint64_t page = real ? w.x : 0, off = (real ? w.y : 0) * p.token_step + (real ? chunk * 16 : 0);
          const uint32_t to = slot + (kCodes ? (token * kRawChunks + chunk) * 16
                                             : (token * kRawChunks + (chunk ^ (token & 7))) * 16);
          copy16(to, keys + page * p.c.k_stride + off, real);
          copy16(to + F::kRaw, values + page * p.c.v_stride + off, real);
        }
        if (kCodes) {
          const uint32_t token = tid % kTile;
          const bool val = tid >= kTile;
          const int2 w = s_place[t % F::kRing][token];
          const bool real = w.x >= 0;
          const uint64_t page = real ? w.x : 0;
          const char* const from = (const char*)(val ? p.c.v_scale : p.c.k_scale) +
                                   page * (val ? p.c.v_scale_stride : p.c.k_scale_stride);
          copy4(slot + 2 * F::kRaw + tid * 4,
                (const float*)from + (real ? w.y : 0) * p.scale_token_step + head * p.scale_head_step, real);
        }
      }
      copies_commit();
    };

    __syncthreads();  // the item before is done with the shared memory
#pragma unroll
    for (uint32_t k = 0; k < F::kStages; ++k) keep_places(t0 + k, look(t0 + k));

    // query rows of this thread: lane / 4 and 8 more
    uint32_t node[2];
    bool row_real[2];
    const char* q_at[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t row = block * 16 + lane / 4 + 8 * k, all = rb * F::kRows + row;
      row_real[k] = row < rows;
      node[k] = row_real[k] ? all / p.group : 0;
      const uint32_t qh = head * p.group + (row_real[k] ? all - node[k] * p.group : 0);
      q_at[k] = (const char*)p.q.base + (uint64_t)(r.first + node[k]) * p.q.row_stride + qh * p.q.head_stride;
    }
    uint32_t qa[kPad > 128 ? 1 : kSteps][4];
    if (kPad <= 128) {
#pragma unroll
      for (uint32_t s = 0; s < kSteps; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          qa[kPad > 128 ? 0 : s][k] = row_real[k & 1] && s < steps
                         ? __ldg((const uint32_t*)(q_at[k & 1] + (s * 16 + (lane & 3) * 2 + (k >> 1) * 8) * 2))
                         : 0u;
    } else {
      for (uint32_t c = tid; c < F::kRows * kChunks; c += kAttnThreads) {
        const uint32_t row = c / kChunks, chunk = c - row * kChunks, all = rb * F::kRows + row;
        const bool real = row < rows && chunk < chunks;
        const uint32_t nd = real ? all / p.group : 0, qh = head * p.group + (real ? all - nd * p.group : 0);
        const uint4 v = real ? __ldg((const uint4*)((const char*)p.q.base + (uint64_t)(r.first + nd) * p.q.row_stride +
                                                    qh * p.q.head_stride + chunk * 16))
                             : make_uint4(0, 0, 0, 0);
        *(uint4*)(smem + (query - ring) + (row * kChunks + (chunk ^ (row & 7))) * 16) = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k + 1 < F::kStages; ++k) fetch(t0 + k);

    float o[kPad / 8][4];
#pragma unroll
    for (uint32_t d = 0; d < kPad / 8; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[d][k] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    uint32_t exponent = 127;  // of the values' scales so far, which the weights of codes have as a factor

    for (uint32_t t = t0; t < t1; ++t) {
      copies_wait<F::kStages - 2>();
      __syncthreads();  // tile t is here, and tile t - 1 is done with
      fetch(t + F::kStages - 1);
      const int2 ahead = look(t + F::kStages);
      const uint32_t slot = ring + (t % F::kStages) * F::kStage;
      uint32_t kt = slot, vt = slot + F::kRaw;
      const float* scales = nullptr;
      if (kCodes) {
        float* const all = (float*)(smem + (t % F::kStages) * F::kStage + 2 * F::kRaw);
        scales = all;
        // keys' scales take the call's own factor along; an infinite one
        // stands for values of both signs, whose products have no sum
        if (tid < kTile) {
          all[tid] = __fmaf_rn(all[tid], 0.f, all[tid]) * p.scale_log2;
        } else {
          const uint32_t ex = (__float_as_uint(all[tid]) >> 23) & 0xFFu;
          const uint32_t largest = __reduce_max_sync(kFull, ex == 0xFFu ? 0u : ex);
          if (lane == 0) s_exponent[warp & 1] = largest;
        }
#pragma unroll
        for (uint32_t k = 0; k < 2 * kTile * kRawChunks / kAttnThreads; ++k) {
          const uint32_t c = tid + k * kAttnThreads;  // first the keys, then the values
          const bool val = k >= kTile * kRawChunks / kAttnThreads;
          const uint32_t cc = val ? c - kTile * kRawChunks : c, token = cc / kRawChunks, chunk = cc % kRawChunks;
          const uint4 w = *(const uint4*)(smem + (t % F::kStages) * F::kStage + c * 16);
          uint2 a, b, d, f;
          if (val) {
            a = widen4<W>(w.x, e4m3), b = widen4<W>(w.y, e4m3), d = widen4<W>(w.z, e4m3), f = widen4<W>(w.w, e4m3);
          } else {
            a = widen4<T>(w.x, e4m3), b = widen4<T>(w.y, e4m3), d = widen4<T>(w.z, e4m3), f = widen4<T>(w.w, e4m3);
          }
          unsigned char* const to = smem + F::kStages * F::kStage + (val ? F::kWide : 0) + token * kChunks * 16;
          *(uint4*)(to + ((2 * chunk) ^ (token & 7)) * 16) = make_uint4(a.x, a.y, b.x, b.y);
          *(uint4*)(to + ((2 * chunk + 1) ^ (token & 7)) * 16) = make_uint4(d.x, d.y, f.x, f.y);
        }
        kt = wide;
        vt = wide + F::kWide;
        __syncthreads();
      }
      const uint32_t tok0 = part * kTokens;
      // scores
      float s[kN][4];
#pragma unroll
      for (uint32_t b = 0; b < kN; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[b][k] = 0.f;
#pragma unroll
      for (uint32_t st = 0; st < kSteps; ++st) {
        if (st >= steps) break;
        uint32_t a[4];
        if (kPad <= 128) {
#pragma unroll
          for (int k = 0; k < 4; ++k) a[k] = qa[kPad > 128 ? 0 : st][k];
        } else {
          const uint32_t row = block * 16 + (lane & 15), chunk = 2 * st + (lane >> 4);
          load_matrices(a, query + (row * kChunks + (chunk ^ (row & 7))) * 16);
        }
#pragma unroll
        for (uint32_t b = 0; b < kN / 2; ++b) {
          const uint32_t token = tok0 + b * 16 + (lane & 7) + (lane >> 4) * 8, chunk = 2 * st + ((lane >> 3) & 1);
          uint32_t m[4];
          load_matrices(m, kt + (token * kChunks + (chunk ^ (token & 7))) * 16);
          multiply<T>(s[2 * b], a, m[0], m[1]);
          multiply<T>(s[2 * b + 1], a, m[2], m[3]);
        }
      }
#pragma unroll
      for (uint32_t b = 0; b < kN; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[b][k] *= kCodes ? scales[tok0 + b * 8 + (lane & 3) * 2 + (k & 1)] : p.scale_log2;
        }
      // what is not seen: only tiles with the request's own tokens (the last
      // ones), or of a table with broken entries, have any
      const bool masked = (t + 1) * kTile > base || s_broken;
      uint32_t sees = 0xFFFFFFFFu;
      if (masked) {
        sees = 0;
#pragma unroll
        for (uint32_t b = 0; b < kN; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t token = tok0 + b * 8 + (lane & 3) * 2 + (k & 1), position = t * kTile + token;
            const uint32_t nd = node[k >> 1];
            bool yes = position < r.length && s_place[t % F::kRing][token].x >= 0;
            if (yes && position >= base) {
              const uint32_t own = position - base;
              yes = p.mask ? (__ldg(p.mask + (uint64_t)(r.first + nd) * p.mask_words + own / 32) >> (own & 31)) & 1
                           : own <= nd;
            }
            if (yes)
              sees |= 1u << (b * 4 + k);
            else
              s[b][k] = -INFINITY;
          }
      }
      // running maxima
      float m[2] = {top[0], top[1]};
#pragma unroll
      for (uint32_t b = 0; b < kN; ++b) {
        m[0] = fmaxf(m[0], fmaxf(s[b][0], s[b][1]));
        m[1] = fmaxf(m[1], fmaxf(s[b][2], s[b][3]));
      }
      // Weights are exp2(score - ref): ref is the maximum, and for codes also
      // takes in the size of the values' scales, so that weights times scales
      // stay in the middle of f16's range.
      float less[2];
      uint32_t ex = 127;
      if (kCodes) {
        ex = min(max(max(s_exponent[0], s_exponent[1]), 31u), 227u);
        ex = t == t0 || ex > exponent + kScaleSlack ? ex : exponent;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[k] = fmaxf(m[k], __shfl_xor_sync(kFull, m[k], 1));
        m[k] = fmaxf(m[k], __shfl_xor_sync(kFull, m[k], 2));
        less[k] = m[k] == -INFINITY ? 0.f : m[k] + (float)((int)ex - 127);
      }
      if (__any_sync(kFull, m[0] != top[0] || m[1] != top[1]) || ex != exponent) {
        const float before = (float)((int)exponent - 127);
        const float a0 = exp2_of(top[0] + before - less[0]), a1 = exp2_of(top[1] + before - less[1]);
        sum[0] *= a0;
        sum[1] *= a1;
#pragma unroll
        for (uint32_t d = 0; d < kPad / 8; ++d) {
          o[d][0] *= a0;
          o[d][1] *= a0;
          o[d][2] *= a1;
          o[d][3] *= a1;
        }
        top[0] = m[0];
        top[1] = m[1];
        exponent = ex;
      }
#pragma unroll
      for (uint32_t b = 0; b < kN; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float w = exp2_of(s[b][k] - less[k >> 1]);
          sum[k >> 1] += w;
          s[b][k] = w;
          if (kCodes) {
            s[b][k] *= scales[kTile + tok0 + b * 8 + (lane & 3) * 2 + (k & 1)];
            if (!((sees >> (b * 4 + k)) & 1)) s[b][k] = 0.f;  // its scale may be NaN
          }
        }
      bool odd = false;  // infinities or NaN among values that not every row sees
      if (masked) {
        for (uint32_t c = lane; c < kTokens * kChunks; c += 32) {
          const uint32_t token = tok0 + c / kChunks, chunk = c % kChunks;
          const uint4 v = *(const uint4*)(smem + (vt - ring) + (token * kChunks + (chunk ^ (token & 7))) * 16);
          odd |= not_finite2<W>(v.x) || not_finite2<W>(v.y) || not_finite2<W>(v.z) || not_finite2<W>(v.w);
        }
        odd = __any_sync(kFull, odd);
      }
      if (!odd) {
#pragma unroll
        for (uint32_t b = 0; b < kN / 2; ++b) {
          const uint32_t a[4] = {pack2<W>(s[2 * b][0], s[2 * b][1]), pack2<W>(s[2 * b][2], s[2 * b][3]),
                                 pack2<W>(s[2 * b + 1][0], s[2 * b + 1][1]), pack2<W>(s[2 * b + 1][2], s[2 * b + 1][3])};
#pragma unroll
          for (uint32_t d = 0; d < kSteps; ++d) {
            if (d >= steps) break;
            const uint32_t token = tok0 + b * 16 + (lane & 15), chunk = 2 * d + (lane >> 4);
            uint32_t v[4];
            load_matrices_t(v, vt + (token * kChunks + (chunk ^ (token & 7))) * 16);
            multiply<W>(o[2 * d], a, v[0], v[1]);
            multiply<W>(o[2 * d + 1], a, v[2], v[3]);
          }
        }
      } else {
        // Rare: products one by one, of what a row sees alone (0 times an
        // infinity or NaN would reach the other rows of the matrix product).
#pragma unroll
        for (uint32_t b = 0; b < kN; ++b)
          for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t from = (lane & ~3u) | j / 2, token = tok0 + b * 8 + j;
            float w[2];
            bool yes[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w0 = __shfl_sync(kFull, s[b][2 * k], from), w1 = __shfl_sync(kFull, s[b][2 * k + 1], from);
              const uint32_t bits = __shfl_sync(kFull, sees, from);
              w[k] = j & 1 ? w1 : w0;
              yes[k] = (bits >> (b * 4 + 2 * k + (j & 1))) & 1;
            }
#pragma unroll
            for (uint32_t d = 0; d < kPad / 8; ++d) {
              const uint32_t v = *(const uint32_t*)(smem + (vt - ring) + (token * kChunks + (d ^ (token & 7))) * 16 + (lane & 3) * 4);
              const float2 f = unpack2<W>(v);
              if (yes[0]) o[d][0] += w[0] * f.x, o[d][1] += w[0] * f.y;
              if (yes[1]) o[d][2] += w[1] * f.x, o[d][3] += w[1] * f.y;
            }
          }
      }
      keep_places(t + F::kStages, ahead);
    }

    // The parts of a tile's tokens joined, through shared memory.
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sum[k] += __shfl_xor_sync(kFull, sum[k], 1);
      sum[k] += __shfl_xor_sync(kFull, sum[k], 2);
      top[k] += (float)((int)exponent - 127);  // the reference of what was summed
      if ((lane & 3) == 0) s_max[warp][lane / 4 + 8 * k] = top[k];
    }
    copies_wait<0>();
    __syncthreads();
    constexpr uint32_t kParts = 4 / kBlocks;
    float most[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      most[k] = -INFINITY;
#pragma unroll
      for (uint32_t w = 0; w < kParts; ++w) most[k] = fmaxf(most[k], s_max[block + w * kBlocks][lane / 4 + 8 * k]);
      const float a = exp2_of(top[k] - (most[k] == -INFINITY ? 0.f : most[k]));
      if ((lane & 3) == 0) s_sum[warp][lane / 4 + 8 * k] = sum[k] * a;
      float* const to = (float*)smem + (warp * 16 + lane / 4 + 8 * k) * kPad + (lane & 3) * 2;
#pragma unroll
      for (uint32_t d = 0; d < kPad / 8; ++d)
        *(float2*)(to + d * 8) = make_float2(o[d][2 * k] * a, o[d][2 * k + 1] * a);
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == e.tiles;
    float* const mine = p.partial + (uint64_t)(2 * blockIdx.x + (t0 == 0)) * partial_floats(F::kRows, kPad);
    constexpr uint32_t kQuads = kPad / 4;
    const auto joined = [&](uint32_t row, uint32_t quad, float& m, float& l) {
      const uint32_t b = row / 16, rr = row % 16;
      m = -INFINITY;
      l = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (uint32_t w = 0; w < kParts; ++w) {
        const uint32_t of = b + w * kBlocks;
        m = fmaxf(m, s_max[of][rr]);
        l += s_sum[of][rr];
        const float4 y = *((const float4*)((const float*)smem + (of * 16 + rr) * kPad) + quad);
        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      }
      return v;
    };
    const auto answer = [&](uint32_t row, uint32_t quad, float m, float l, float4 v) {
      const uint32_t all = rb * F::kRows + row, nd = all / p.group, qh = head * p.group + (all - nd * p.group);
      const float by = l == 0.f ? 0.f : 1.f / l;
      if (quad * 4 < p.c.width) {
        char* const to = (char*)p.out.base + (uint64_t)(r.first + nd) * p.out.row_stride + qh * p.out.head_stride + quad * 8;
        *(uint2*)to = make_uint2(pack2<T>(v.x * by, v.y * by), pack2<T>(v.z * by, v.w * by));
      }
      if (quad == 0 && p.lse)
        p.lse[(uint64_t)(r.first + nd) * (p.c.heads * p.group) + qh] =
            l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    };
    if (whole) {
      for (uint32_t c = tid; c < rows * kQuads; c += kAttnThreads) {
        float m, l;
        const float4 v = joined(c / kQuads, c % kQuads, m, l);
        answer(c / kQuads, c % kQuads, m, l, v);
      }
    } else {
      for (uint32_t c = tid; c < rows * kQuads; c += kAttnThreads) {
        const uint32_t row = c / kQuads, quad = c % kQuads;
        float m, l;
        const float4 v = joined(row, quad, m, l);
        __stcg((float4*)(mine + row * kPad) + quad, v);
        if (quad == 0) {
          __stcg(mine + F::kRows * kPad + row, m);
          __stcg(mine + F::kRows * kPad + F::kRows + row, l);
        }
      }
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
        join_item<T, F::kRows, kPad, kAttnThreads>(p, item_of, (float4*)smem, 0);
      }
    }
    at += t1 - t0;
  }
}

template <typename T, uint32_t kPad, bool kCodes, uint32_t kBlocks>
int launch_few(const AttnParams& p, unsigned grid, cudaStream_t s) {
  typedef Few<T, kPad, kCodes, kBlocks> F;
  const cudaError_t e = cudaFuncSetAttribute(attention_few_kernel<T, kPad, kCodes, kBlocks>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, F::kBytes);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_dependent(attention_few_kernel<T, kPad, kCodes, kBlocks>, grid, kAttnThreads, F::kBytes, s, p);
}

template <typename T, uint32_t kPad, bool kCodes>
int launch_blocks(const AttnParams& p, uint32_t blocks, unsigned grid, cudaStream_t s) {
  switch (blocks) {
    case 1:
      return launch_few<T, kPad, kCodes, 1>(p, grid, s);
    default:
      return launch_few<T, kPad, kCodes, 2>(p, grid, s);
  }
}

}  // namespace db
