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

#include <type_traits>

#include "cachedata.cuh"

namespace db {

constexpr uint32_t kTile = 64;             // tokens of a unit
constexpr uint32_t kAttnThreads = 128;
constexpr uint32_t kMaxGroup = 64;
// A row's reference is the largest score, for codes the largest score times its
// values' scale (as a power of two), of the tokens that the row sees, and is followed
// when one is more than 2^slack above it. f16 weights times scales are then below
// 2^(lift + slack + 1), those without scales below 2^(lift + slack). They start as far
// above 1 as f16 (below 2^16) allows, so that small ones are normal numbers still: the
// kernel for few rows follows sooner and starts higher, for which the error of long
// answers in f16 is 1.4 times their rounding's (1.5 with the other's).
template <typename W>
__host__ __device__ constexpr int attn_lift(int slack) {
  return std::is_same<W, __half>::value ? 14 - slack : 0;
}
constexpr uint32_t kManyBlocks = 16;      // blocks of 8 query rows of the tcgen05 kernel's items, or twice as many

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
  uint32_t narrow;         // offsets in the pools, by 16 bytes, fit 32 bits
};

// CTAs of an SM of a kernel for so many blocks of 8 query rows: as many as
// registers and shared memory hold.
constexpr uint32_t attn_ctas_per_sm(uint32_t pad, bool codes, uint32_t blocks) {
  if (blocks >= kManyBlocks) return pad <= 128 && blocks == kManyBlocks ? 2 : 1;
  return pad == 64 ? 4 : pad == 128 ? (codes || blocks == 1 ? 3 : 2) : codes || blocks == 2 ? 2 : 1;
}
constexpr unsigned kMaxAttnCtas = 1024;
inline unsigned attn_grid(uint32_t ctas_per_sm) {
  const unsigned g = ctas_per_sm * (unsigned)num_sms();
  return g < kMaxAttnCtas ? g : kMaxAttnCtas;
}

// Host: one instance of the kernels for a padded width.
int launch_attention_64(const AttnParams& p, uint32_t type, uint32_t blocks, cudaStream_t s);
int launch_attention_128(const AttnParams& p, uint32_t type, uint32_t blocks, cudaStream_t s);
int launch_attention_256(const AttnParams& p, uint32_t type, uint32_t blocks, cudaStream_t s);

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

// (most are of 32 bits, which take a tenth of the instructions)
static __device__ __noinline__ uint64_t quotient(uint64_t a, uint64_t b) {
  return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
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
  Request r = {};
  for (uint32_t i = tid; i < n; i += kThreads) {
    r = attention_request(p, i);
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
  s.lo = quotient(all * blockIdx.x, s.ctas);
  s.hi = quotient(all * (blockIdx.x + 1), s.ctas);
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
  if (n <= kThreads) {  // a thread has read each
    if (tid - s.request < kNear && tid < n) s_near[tid - s.request] = r;
  } else if (tid < kNear && s.request + tid < n) {
    s_near[tid] = attention_request(p, s.request + tid);
  }
  __syncthreads();
  return s;
}

// The CTA that has unit x.
static __device__ __noinline__ uint32_t owner_of(const Share& s, uint64_t x) {
  return (uint32_t)quotient((x + 1) * s.ctas - 1, s.all);
}

// ------------------------------------------------------------ small operations
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// l times 2^d, d <= 0, also where 2^d alone is below the range of the numbers.
__device__ __forceinline__ float times_exp2(float l, float d) {
  const float h = exp2_of(0.5f * d);
  return l * h * h;
}
// The exponent of a scale, for references. A row's weights are the larger the smaller its
// values' scales are, and 2^31 of them must not leave the numbers' range, nor those beside
// large scales fall out of it: scales below 2^-80 (zeros too) are taken as that, those from
// 2^101 on as 2^100. One that is not finite makes the answer so whatever the reference.
constexpr uint32_t kLeastExponent = 127 - 80, kMostExponent = 127 + 100;
__device__ __forceinline__ uint32_t scale_exponent(float scale) {
  const uint32_t e = __float_as_uint(scale) >> 23 & 0xFFu;
  return e == 0xFFu ? kLeastExponent : min(max(e, kLeastExponent), kMostExponent);
}
__device__ __forceinline__ float scale_size(float scale) { return (float)((int)scale_exponent(scale) - 127); }
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes (or zeros) into shared memory, without a register. (The form with a
// size in a register is several times slower to start.)
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  if (real)
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
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

// Four 8-bit codes as four f16, exactly. I8: 1024 + (code + 128), less 1152.
__device__ __forceinline__ uint2 widen4(uint32_t w, bool e4m3) {
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

// Four sums of weights times values as answers; `by`: 1 over the sum of weights, or 0 for a
// row that has none. Its answers are 0, also where values are not finite (0 times them is NaN).
template <typename T>
__device__ __forceinline__ uint2 four_answers(const float4& v, float by) {
  return by == 0.f ? make_uint2(0, 0) : make_uint2(pack2<T>(v.x * by, v.y * by), pack2<T>(v.z * by, v.w * by));
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

}  // namespace db
