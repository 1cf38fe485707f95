// Keys and values into a cache's pages and out of them, and tokens moved
// within (include/cachedata.h: db_cache_write, db_cache_read, db_cache_keep).
//
// All three are bound by memory: a value is read once and written once. A
// warp takes neighbouring rows (tokens) of the batch, finds its request once,
// and handles a row's keys and values of all heads, 8 values a lane, so that
// the 4 to 32 lanes that hold a head's row can reduce its largest magnitude.
// 192,000 tokens of 8 heads of 128 from bf16 to E4M3: 197 us, 6.0 TB/s (issue: 67 %
// of the schedulers' cycles), to bf16 235, 6.6; 384,000 tokens of 5 heads of 112 from I8
// to f16: 256 us, 4.6 TB/s of what is asked for, 5.6 of DRAM (rows of 112 bytes share
// their sectors; 14 of 16 lanes and 5 of 6 heads' places are in use).
#include "cachedata.cuh"

namespace db {

int check_cache(const db_page_tables* t, const db_cache_batch* b, uint8_t* status, db_counters* ctr,
                CacheView* v) {
  if (!t || !b || !t->table || !t->length || !aligned(t->table, 4) || !aligned(t->length, 4))
    return -EINVAL;
  if (!t->n_seqs || t->n_seqs >= 1u << 31 || !t->columns || !t->n_pages || t->n_pages >= 1u << 31 ||
      !t->page_tokens)
    return -EINVAL;
  if (b->n >= 1u << 31 || b->rows >= 1u << 31 || !aligned(ctr, 8)) return -EINVAL;
  if (b->n && (!b->seq || !b->start || !aligned(b->seq, 4) || !aligned(b->start, 4))) return -EINVAL;
  *v = CacheView{t->table, t->length, t->n_seqs, t->columns, t->n_pages, t->page_tokens,
                 b->seq,   b->start,  b->n,      b->rows,    status,     ctr};
  return 0;
}

int check_layer(const db_page_tables* t, const db_cache_layer* c) {
  if (!c || !c->k || !c->v || !c->heads || !c->width || c->width % 16 || c->width > 256)
    return -EINVAL;
  if (c->type != DB_BF16 && c->type != DB_F16 && c->type != DB_E4M3 && c->type != DB_I8) return -EINVAL;
  const uint64_t limit = 1ull << 31, rows = (uint64_t)c->heads * t->page_tokens;
  if (rows >= limit || rows * c->width >= limit) return -EINVAL;
  const uint64_t bytes = rows * c->width * item_bytes(c->type);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->k_stride % 16 || c->v_stride % 16) return -EINVAL;
  if (t->n_pages > 1 && (c->k_stride < bytes || c->v_stride < bytes)) return -EINVAL;
  if (item_bytes(c->type) == 1) {
    if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        c->k_scale_stride % 4 || c->v_scale_stride % 4)
      return -EINVAL;
    if (t->n_pages > 1 && (c->k_scale_stride < rows * 4 || c->v_scale_stride < rows * 4)) return -EINVAL;
  } else if (c->k_scale || c->v_scale) {
    return -EINVAL;
  }
  return 0;
}

int check_rows(const db_cache_rows* r, uint32_t rows, uint32_t heads, uint32_t width, uint32_t type,
               bool written) {
  if (!r || type > DB_F32) return -EINVAL;
  if (!rows) return 0;
  if (!r->base || !aligned(r->base, 16) || r->row_stride % 16 || r->head_stride % 16) return -EINVAL;
  if (written && heads > 1 && r->head_stride < (uint64_t)width * item_bytes(type)) return -EINVAL;
  return 0;
}

int zero_counters(db_counters* ctr, cudaStream_t s) {
  if (!ctr) return 0;
  const cudaError_t e = cudaMemsetAsync(ctr, 0, sizeof(*ctr), s);
  return e == cudaSuccess ? 0 : cuda_failure(e);
}

namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;

struct MoveParams {
  CacheView view;
  db_cache_layer c;
  db_cache_rows k, v;
  const int32_t* first;  // read: first positions or NULL
  uint32_t chunk;        // rows of a warp
  uint32_t lanes;        // of a head's row: a power of two, 8 values each
  uint64_t token_step, head_step;              // bytes within a page
  uint32_t scale_token_step, scale_head_step;  // floats
};

// Eight values of a row, as they lie in memory.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const char* p) {
  Eight<T> e;
#pragma unroll
  for (uint32_t j = 0; j < sizeof(T) / 2; ++j) e.w[j] = __ldcs((const uint4*)p + j);
  return e;
}

template <typename T>
__device__ __forceinline__ void floats8(const Eight<T>& e, float* x) {
  if (sizeof(T) == 4) {
#pragma unroll
    for (uint32_t j = 0; j < sizeof(T) / 2; ++j) {
      x[4 * j] = __uint_as_float(e.w[j].x), x[4 * j + 1] = __uint_as_float(e.w[j].y);
      x[4 * j + 2] = __uint_as_float(e.w[j].z), x[4 * j + 3] = __uint_as_float(e.w[j].w);
    }
  } else {
    const uint32_t w[4] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<typename std::conditional<sizeof(T) == 4, __half, T>::type>(w[j]);
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(char* p, const float* x) {
  if (sizeof(T) == 4) {
    ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    typedef typename std::conditional<sizeof(T) == 4, __half, T>::type H;
    *(uint4*)p = make_uint4(pack2<H>(x[0], x[1]), pack2<H>(x[2], x[3]), pack2<H>(x[4], x[5]),
                            pack2<H>(x[6], x[7]));
  }
}

// The largest magnitude of a lane's values as a float's bits (two 16-bit ones
// side by side for 16-bit values): of values without their sign, larger bits are
// larger values, infinities above every number and NaN above those.
template <typename T>
__device__ __forceinline__ uint32_t largest_bits(const Eight<T>& e) {
  uint32_t m = 0;
  if (sizeof(T) == 4) {
#pragma unroll
    for (uint32_t j = 0; j < sizeof(T) / 2; ++j)
      m = max(max(max(m, e.w[j].x & 0x7FFFFFFFu), max(e.w[j].y & 0x7FFFFFFFu, e.w[j].z & 0x7FFFFFFFu)), e.w[j].w & 0x7FFFFFFFu);
    return m;
  }
  return __vmaxu2(__vmaxu2(e.w[0].x & 0x7FFF7FFFu, e.w[0].y & 0x7FFF7FFFu), __vmaxu2(e.w[0].z & 0x7FFF7FFFu, e.w[0].w & 0x7FFF7FFFu));
}
template <typename T>
__device__ __forceinline__ uint32_t larger_bits(uint32_t a, uint32_t b) {
  return sizeof(T) == 4 ? max(a, b) : __vmaxu2(a, b);
}
template <typename T>
__device__ __forceinline__ uint32_t one_of(uint32_t m) {
  if (sizeof(T) == 4) return m;
  m = max(m & 0xFFFFu, m >> 16);
  return __float_as_uint(unpack2<typename std::conditional<sizeof(T) == 4, __half, T>::type>(m).x);
}

// The largest of kMany rows' values over the `lanes` lanes that share them: a
// lane ends with that of row (lane % lanes) / (lanes / kMany). Lanes hand half of
// their rows on at each step, so that 8 rows of 16 lanes take 8 shuffles, not 32.
template <typename T, int kMany>
__device__ __forceinline__ uint32_t largest_of_rows(uint32_t (&m)[kMany], uint32_t lanes) {
  uint32_t bit = lanes / 2;
#pragma unroll
  for (int n = kMany / 2; n; n /= 2) {
    const bool upper = threadIdx.x & bit;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const uint32_t sent = upper ? m[j] : m[j + n], kept = upper ? m[j + n] : m[j];
      m[j] = larger_bits<T>(kept, __shfl_xor_sync(kFull, sent, bit));
    }
    bit /= 2;
  }
  for (; bit; bit /= 2) m[0] = larger_bits<T>(m[0], __shfl_xor_sync(kFull, m[0], bit));
  return one_of<T>(m[0]);
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// A row's scale and what its values are multiplied by (0: codes are 0).
template <bool kE4m3>
__device__ __forceinline__ void scale_of(uint32_t top, float& scale, float& by) {
  const float largest = kE4m3 ? 448.f : 127.f, a = __uint_as_float(top);
  by = __fdiv_rn(largest, a);
  scale = __fdiv_rn(a, largest);
  if (top >= 0x7F800000u) {
    by = 0.f;
    scale = __uint_as_float(0x7FC00000u);
  } else if (scale == 0.f || isinf(by)) {
    by = scale = 0.f;
  }
}

// Codes of eight values. I8: adding 1.5 * 2^23 leaves the nearest whole number,
// ties to even, in a float's low bits; products are at most 127 and its last
// place, so nothing has to be cut.
template <bool kE4m3>
__device__ __forceinline__ uint2 codes8(const float* x, float by) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* y = x + 4 * h;
    if (kE4m3) {
      w[h] = e4m3_pair(y[0] * by, y[1] * by) | e4m3_pair(y[2] * by, y[3] * by) << 16;
    } else {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(__fadd_rn(__fmul_rn(y[j], by), 12582912.f));
      w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
  }
  return by > 0.f ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
}

// Where a row of the batch has its token: found one row ahead of the data, so
// that the table's answer is there when the loads before it are.
struct Place {
  uint32_t page, slot;
  bool held;  // it has one
};

// The row's request is the one it is in, or a later one; `i` and `q` follow.
// `position`: of a valid request's row.
template <typename F>
__device__ __forceinline__ Place find_place(const CacheView& v, uint32_t r, uint32_t& i, Request& q,
                                            bool& mine, bool fresh, F position) {
  while (i + 1 < v.n && (int32_t)r >= __ldg(v.start + i + 1)) q = read_request(v, ++i, fresh);
  mine = q.ok && r >= q.first && r - q.first < q.rows;
  Place w = {0, 0, false};
  if (mine) {
    const uint64_t at = position(i, q, r - q.first);
    if (at < q.length) {
      const uint32_t column = (uint32_t)at / v.page_tokens;
      w.slot = (uint32_t)at - column * v.page_tokens;
      w.page = (uint32_t)__ldg(v.table + (uint64_t)q.seq * v.columns + column);
      w.held = true;
    }
  }
  return w;
}

// One warp: rows [r0, r1) of the batch, the first of which is in request i. kType:
// what the pages hold; kUnroll: heads' rows of a lane under way.
template <typename Src, int kType, int kUnroll>
__device__ __forceinline__ void write_rows(const MoveParams& p, uint32_t r0, uint32_t r1, uint32_t i) {
  constexpr bool kCodes = kType == DB_E4M3 || kType == DB_I8;
  const CacheView& v = p.view;
  const uint32_t lane = threadIdx.x & 31;
  // kHalf heads' keys and as many values at a time: a lane has eight values of
  // head h0 + j * per + lane / lanes
  constexpr int kHalf = kUnroll / 2;
  const uint32_t lanes = p.lanes, at = (lane & (lanes - 1)) * 8, per = 32 / lanes, first_head = lane / lanes;
  const uint32_t heads = p.c.heads;
  const bool mine = at < p.c.width;
  const uint64_t k_next = per * p.k.head_stride, v_next = per * p.v.head_stride, next = per * p.head_step;
  const char* const k_from = (const char*)p.k.base + first_head * p.k.head_stride + at * sizeof(Src);
  const char* const v_from = (const char*)p.v.base + first_head * p.v.head_stride + at * sizeof(Src);
  const uint64_t in_page = first_head * p.head_step + at * (kCodes ? 1 : 2);
  const auto position = [&](uint32_t, const Request& q, uint32_t j) { return (uint64_t)q.length - q.rows + j; };
  Request q = read_request(v, i, true);
  bool has;
  Place w = find_place(v, r0, i, q, has, true, position);
  for (uint32_t r = r0; r < r1; ++r) {
    Place now = w;
    const bool go = has;
    for (uint32_t h0 = 0; h0 < heads; h0 += per * kHalf) {
      Eight<Src> e[kUnroll];
      if (go) {
        const char* const kf = k_from + r * p.k.row_stride + h0 * p.k.head_stride;
        const char* const vf = v_from + r * p.v.row_stride + h0 * p.v.head_stride;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
#pragma unroll
          for (uint32_t z = 0; z < sizeof(Src) / 2; ++z) e[j].w[z] = e[j + kHalf].w[z] = make_uint4(0, 0, 0, 0);
          if (h0 + j * per >= heads) continue;
          const bool real = mine && h0 + j * per + first_head < heads;
          if (real) {
            e[j] = load8<Src>(kf + j * k_next);
            e[j + kHalf] = load8<Src>(vf + j * v_next);
          }
        }
      }
      if (h0 == 0) {
        if (r + 1 < r1) w = find_place(v, r + 1, i, q, has, true, position);
        if (go && now.held && now.page >= v.n_pages) {
          now.held = false;
          if (lane == 0) report_table(v.ctr);
        }
      }
      if (!go) break;
      const uint64_t off = now.slot * p.token_step + h0 * p.head_step + in_page;
      char* const kt = (char*)p.c.k + now.page * p.c.k_stride + off;
      char* const vt = (char*)p.c.v + now.page * p.c.v_stride + off;
      float by[kUnroll];
      if (kCodes) {
        // A lane divides for one of the lane group's rows (few lanes: for each).
        const uint32_t of = lane & (lanes - 1);
        float my_scale = 0.f, my_by = 0.f;
        if (lanes >= kUnroll) {
          uint32_t top[kUnroll];
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) top[j] = largest_bits(e[j]);
          scale_of<kType == DB_E4M3>(largest_of_rows<Src, kUnroll>(top, lanes), my_scale, my_by);
          const uint32_t every = lanes / kUnroll, row = of / every;
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) by[j] = __shfl_sync(kFull, my_by, (lane & ~(lanes - 1)) | j * every);
          const bool val = row >= kHalf;
          const uint32_t head = h0 + (val ? row - kHalf : row) * per + first_head;
          if (row * every == of && head < heads && now.held) {
            char* const to = (char*)(val ? p.c.v_scale : p.c.k_scale) + now.page * (val ? p.c.v_scale_stride : p.c.k_scale_stride);
            ((float*)to)[now.slot * p.scale_token_step + head * p.scale_head_step] = my_scale;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) {
            if (h0 + (j >= kHalf ? j - kHalf : j) * per >= heads) continue;
            uint32_t top[1] = {largest_bits(e[j])};
            scale_of<kType == DB_E4M3>(largest_of_rows<Src, 1>(top, lanes), my_scale, by[j]);
            const bool val = j >= kHalf;
            const uint32_t head = h0 + (val ? j - kHalf : j) * per + first_head;
            if (of == 0 && head < heads && now.held) {
              char* const to = (char*)(val ? p.c.v_scale : p.c.k_scale) + now.page * (val ? p.c.v_scale_stride : p.c.k_scale_stride);
              ((float*)to)[now.slot * p.scale_token_step + head * p.scale_head_step] = my_scale;
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int jj = j >= kHalf ? j - kHalf : j;
        if (h0 + jj * per >= heads) continue;
        char* const to = (j >= kHalf ? vt : kt) + jj * next;
        float x[8];
        floats8(e[j], x);
        if (kCodes) {
          const uint2 c = codes8<kType == DB_E4M3>(x, by[j]);
          if (mine && now.held && h0 + jj * per + first_head < heads) *(uint2*)to = c;
        } else if (mine && now.held && h0 + jj * per + first_head < heads) {
          typedef typename std::conditional<kType == DB_F16, __half, __nv_bfloat16>::type H;
          store8<H>(to, x);
        }
      }
    }
  }
}

// Eight cached values, as they lie in memory and as floats.
template <int kType>
struct Held {
  typedef typename std::conditional<kType == DB_E4M3 || kType == DB_I8, uint2, uint4>::type type;
};

template <int kType>
__device__ __forceinline__ void held_floats(const typename Held<kType>::type& c, float scale, float* x) {
  if constexpr (kType == DB_E4M3 || kType == DB_I8) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (kType == DB_E4M3) {
        const float2 a = unpack2<__half>(e4m3x2_to_f16x2(w[h])), b = unpack2<__half>(e4m3x2_to_f16x2(w[h] >> 16));
        x[4 * h] = a.x * scale, x[4 * h + 1] = a.y * scale, x[4 * h + 2] = b.x * scale, x[4 * h + 3] = b.y * scale;
      } else {
        // a code and 128 as the low bits of 2^23
        const uint32_t u = w[h] ^ 0x80808080u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[4 * h + j] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + j)), 8388736.f), scale);
      }
    }
  } else {
    typedef typename std::conditional<kType == DB_F16, __half, __nv_bfloat16>::type H;
    Eight<H> e;
    e.w[0] = c;
    floats8(e, x);
  }
}

template <typename Dst, int kType, int kUnroll>
__device__ __forceinline__ void read_rows(const MoveParams& p, uint32_t r0, uint32_t r1, uint32_t i) {
  constexpr bool kCodes = kType == DB_E4M3 || kType == DB_I8;
  constexpr uint32_t kBytes = kCodes ? 1 : 2;
  typedef typename Held<kType>::type V;
  const CacheView& v = p.view;
  const uint32_t lane = threadIdx.x & 31;
  constexpr int kHalf = kUnroll / 2;
  const uint32_t lanes = p.lanes, at = (lane & (lanes - 1)) * 8, per = 32 / lanes, first_head = lane / lanes;
  const uint32_t heads = p.c.heads;
  const bool mine = at < p.c.width;
  const uint64_t k_next = per * p.k.head_stride, v_next = per * p.v.head_stride, next = per * p.head_step;
  char* const k_to = (char*)p.k.base + first_head * p.k.head_stride + at * sizeof(Dst);
  char* const v_to = (char*)p.v.base + first_head * p.v.head_stride + at * sizeof(Dst);
  const uint64_t in_page = first_head * p.head_step + at * kBytes;
  const auto position = [&](uint32_t i, const Request&, uint32_t j) {
    return (uint64_t)(p.first ? (uint32_t)__ldg(p.first + i) : 0) + j;
  };
  Request q = read_request(v, i, false);
  bool has;
  Place w = find_place(v, r0, i, q, has, false, position);
  for (uint32_t r = r0; r < r1; ++r) {
    Place now = w;
    const bool go = has;
    if (now.held && now.page >= v.n_pages) {
      now.held = false;
      if (lane == 0) report_table(v.ctr);
    }
    for (uint32_t h0 = 0; h0 < heads; h0 += per * kHalf) {
      V c[kUnroll];
      float scale[kUnroll];
      const uint64_t off = now.slot * p.token_step + h0 * p.head_step + in_page;
      const char* const kf = (const char*)p.c.k + now.page * p.c.k_stride + off;
      const char* const vf = (const char*)p.c.v + now.page * p.c.v_stride + off;
      const uint32_t of = now.slot * p.scale_token_step + (h0 + first_head) * p.scale_head_step;
      const float* const ks = (const float*)((const char*)p.c.k_scale + now.page * p.c.k_scale_stride) + (kCodes ? of : 0);
      const float* const vs = (const float*)((const char*)p.c.v_scale + now.page * p.c.v_scale_stride) + (kCodes ? of : 0);
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        if (h0 + j * per >= heads) break;
        c[j] = c[j + kHalf] = V{};
        scale[j] = scale[j + kHalf] = 0.f;
        if (go && mine && now.held && h0 + j * per + first_head < heads) {
          c[j] = __ldcs((const V*)(kf + j * next));
          c[j + kHalf] = __ldcs((const V*)(vf + j * next));
          if (kCodes) {
            scale[j] = ks[j * per * p.scale_head_step];
            scale[j + kHalf] = vs[j * per * p.scale_head_step];
          }
        }
      }
      if (h0 == 0 && r + 1 < r1) w = find_place(v, r + 1, i, q, has, false, position);
      if (!go) break;
      char* const kt = k_to + r * p.k.row_stride + h0 * p.k.head_stride;
      char* const vt = v_to + r * p.v.row_stride + h0 * p.v.head_stride;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int jj = j >= kHalf ? j - kHalf : j;
        if (mine && h0 + jj * per + first_head < heads) {
          float x[8];
          held_floats<kType>(c[j], scale[j], x);
          store8<Dst>(j >= kHalf ? vt + jj * v_next : kt + jj * k_next, x);
        }
      }
    }
  }
}

// A row's request is found by a search that takes starts for ascending. Where they are
// not it may miss some, so the first CTAs have no rows of the batch: they look all starts
// over while the others work, and where one descends they share out every valid
// request's rows. (What others have done is done again, with the same result; rows and
// slots of several requests are any one's.) They go through the rows with as few
// registers as that takes: with the loop of the others, or calling it, those had fewer
// (192,000 rows written 201 and 199 us, 197 so and without menders; 384,000 read 257
// and 262, 256 so, 254 without).
constexpr uint32_t kMenders = 16, kMendingWarps = kMenders * kWarps;

template <typename F>
__device__ __forceinline__ void mend(const CacheView& v, bool fresh, F rows) {
  const uint32_t lane = threadIdx.x & 31, warp = blockIdx.x * kWarps + threadIdx.x / 32;
#pragma unroll 1
  for (uint32_t i0 = 0; i0 < v.n; i0 += 32) {
    const uint32_t i = i0 + lane;
    Request q = {};
    if (i < v.n) q = read_request(v, i, fresh);
    // a warp's share of a request: neighbouring rows; of a short one other warps' turn each time
    const uint32_t each = (q.rows + kMendingWarps - 1) / kMendingWarps;
    const uint64_t at = (uint64_t)((warp + i) % kMendingWarps) * each;
#pragma unroll 1
    for (uint32_t votes = __ballot_sync(kFull, at < q.rows); votes; votes &= votes - 1) {
      const uint32_t from = __ffs(votes) - 1;
      const uint32_t r0 = __shfl_sync(kFull, q.first + (uint32_t)at, from);
      const uint32_t r1 = __shfl_sync(kFull, q.first + (uint32_t)min(at + each, (uint64_t)q.rows), from);
      rows(r0, r1, i0 + from);
      __syncwarp();
    }
  }
}

// Whether a mender has work.
__device__ __forceinline__ bool starts_descend(const CacheView& v) {
  bool any = false;
#pragma unroll 8
  for (uint32_t i = threadIdx.x; i < v.n; i += kThreads) any |= __ldg(v.start + i) > __ldg(v.start + i + 1);
  return __syncthreads_or(any);
}

// A warp's rows of the batch; false: it has none.
__device__ __forceinline__ bool own_rows(const MoveParams& p, uint32_t& r0, uint32_t& r1) {
  const uint64_t at = ((uint64_t)(blockIdx.x - kMenders) * kWarps + threadIdx.x / 32) * p.chunk;
  r0 = (uint32_t)at;
  r1 = (uint32_t)min(at + p.chunk, (uint64_t)p.view.rows);
  return at < p.view.rows;
}

template <typename Src, int kType>
__global__ void __launch_bounds__(kThreads, 3) cache_write_kernel(const __grid_constant__ MoveParams p) {
  wait_for_prerequisites();
  dependents_may_launch();
  report_requests(p.view, (uint64_t)blockIdx.x * kThreads + threadIdx.x, (uint64_t)gridDim.x * kThreads, true);
  uint32_t r0, r1;
  if (blockIdx.x < kMenders) {
    if (starts_descend(p.view))
      mend(p.view, true, [&](uint32_t a, uint32_t b, uint32_t i) { write_rows<Src, kType, 2>(p, a, b, i); });
  } else if (own_rows(p, r0, r1)) {
    write_rows<Src, kType, sizeof(Src) == 4 ? 4 : 8>(p, r0, r1, find_request(p.view.start, p.view.n, r0));
  }
}

template <typename Dst, int kType>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ MoveParams p) {
  wait_for_prerequisites();
  dependents_may_launch();
  report_requests(p.view, (uint64_t)blockIdx.x * kThreads + threadIdx.x, (uint64_t)gridDim.x * kThreads, false);
  uint32_t r0, r1;
  if (blockIdx.x < kMenders) {
    if (starts_descend(p.view))
      mend(p.view, false, [&](uint32_t a, uint32_t b, uint32_t i) { read_rows<Dst, kType, 2>(p, a, b, i); });
  } else if (own_rows(p, r0, r1)) {
    read_rows<Dst, kType, 8>(p, r0, r1, find_request(p.view.start, p.view.n, r0));
  }
}

MoveParams move_params(const CacheView& v, const db_cache_layer* c, const db_cache_rows* k,
                       const db_cache_rows* vals) {
  MoveParams p = {};
  p.view = v;
  p.c = *c;
  p.k = *k;
  p.v = *vals;
  const uint64_t row = (uint64_t)c->width * item_bytes(c->type);
  p.token_step = c->heads_first ? row : c->heads * row;
  p.head_step = c->heads_first ? v.page_tokens * row : row;
  p.scale_token_step = c->heads_first ? 1 : c->heads;
  p.scale_head_step = c->heads_first ? v.page_tokens : 1;
  p.lanes = 2;
  while (p.lanes * 8 < c->width) p.lanes *= 2;
  return p;
}

// A warp for each row up to 24 CTAs an SM, several times what is resident, then
// neighbouring rows, whose places are neighbours too.
int launch_move(void (*kernel)(MoveParams), MoveParams& p, cudaStream_t s) {
  const uint64_t most = (uint64_t)24 * num_sms(), want = ((uint64_t)p.view.rows + kWarps - 1) / kWarps;
  const uint64_t grid = want < 1 ? 1 : want < most ? want : most;
  p.chunk = (uint32_t)((p.view.rows + grid * kWarps - 1) / (grid * kWarps));
  if (!p.chunk) p.chunk = 1;
  return launch_dependent(kernel, (unsigned)grid + kMenders, kThreads, 0, s, p);
}

template <typename Row>
void (*write_kernel(uint32_t type))(MoveParams) {
  switch (type) {
    case DB_BF16:
      return cache_write_kernel<Row, DB_BF16>;
    case DB_F16:
      return cache_write_kernel<Row, DB_F16>;
    case DB_E4M3:
      return cache_write_kernel<Row, DB_E4M3>;
    default:
      return cache_write_kernel<Row, DB_I8>;
  }
}

template <typename Row>
void (*read_kernel(uint32_t type))(MoveParams) {
  switch (type) {
    case DB_BF16:
      return cache_read_kernel<Row, DB_BF16>;
    case DB_F16:
      return cache_read_kernel<Row, DB_F16>;
    case DB_E4M3:
      return cache_read_kernel<Row, DB_E4M3>;
    default:
      return cache_read_kernel<Row, DB_I8>;
  }
}

// ----------------------------------------------------------------------- keep
constexpr uint32_t kKeepThreads = 128;

struct KeepParams {
  CacheView view;
  const int32_t* path;
  const int32_t* accepted;
  db_page_pool pool;
  uint32_t planes, segments, token_bytes;
  uint64_t seg_bytes;
  uint32_t vectors;  // of a token's run
  uint32_t lanes;    // a power of two: threads of a run, which take vectors one after the other
  db_page_cut* cut;
};

template <int kVec>
struct Bytes;
template <>
struct Bytes<16> {
  typedef uint4 type;
};
template <>
struct Bytes<8> {
  typedef uint2 type;
};
template <>
struct Bytes<4> {
  typedef uint32_t type;
};
template <>
struct Bytes<2> {
  typedef uint16_t type;
};
template <>
struct Bytes<1> {
  typedef uint8_t type;
};

// A CTA takes one request and every gridDim.y-th share of its planes and
// segments. It lists the tokens that move (128 of the path at a time) in
// shared memory; a thread then carries its bytes of a run through the list in
// ascending order, 8 under way. A token goes to a place that is not above its
// own, and places ascend, so nothing is overwritten before it has been read,
// and no thread touches another one's bytes.
template <int kVec>
__global__ void __launch_bounds__(kKeepThreads) cache_keep_kernel(const KeepParams p) {
  typedef typename Bytes<kVec>::type V;
  __shared__ uint64_t s_src[kKeepThreads], s_dst[kKeepThreads];
  __shared__ uint32_t s_warp[kKeepThreads / 32];
  wait_for_prerequisites();
  dependents_may_launch();
  const CacheView& v = p.view;
  const uint32_t i = blockIdx.x, tid = threadIdx.x;
  Request q = read_request(v, i, true);
  const uint32_t kept = q.ok ? (uint32_t)__ldg(p.accepted + i) : 0;
  bool ok = q.ok && kept <= q.rows;
  if (ok) {  // the path ascends below the request's rows
    bool bad = false;
    for (uint32_t k = tid; k < kept; k += kKeepThreads) {
      const int32_t x = __ldg(p.path + q.first + k);
      bad |= x < 0 || (uint32_t)x >= q.rows || (k && x <= __ldg(p.path + q.first + k - 1));
    }
    ok = !__syncthreads_or(bad);
  }
  const uint32_t base = q.length - q.rows;
  if (tid == 0 && blockIdx.y == 0) {
    if (v.status) v.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    if (p.cut) p.cut[i] = db_page_cut{q.seq, ok ? base + kept : 0xFFFFFFFFu};
    if (v.ctr) {
      if (ok && q.rows) atomicAdd((unsigned long long*)&v.ctr->total, (unsigned long long)q.rows);
      if (!ok) atomicAdd((unsigned long long*)&v.ctr->n_invalid, 1ull);
    }
  }
  if (!ok) return;
  const uint32_t runs = p.planes * p.segments, per = kKeepThreads / p.lanes;
  const uint32_t lane = tid & (p.lanes - 1);
  for (uint32_t k0 = 0; k0 < kept; k0 += kKeepThreads) {
    const uint32_t k = k0 + tid;
    bool moves = false;
    uint64_t src = 0, dst = 0;
    if (k < kept) {
      const uint32_t x = (uint32_t)__ldg(p.path + q.first + k);
      if (x != k) {
        const uint32_t a = base + x, b = base + k, ca = a / v.page_tokens, cb = b / v.page_tokens;
        const uint32_t pa = (uint32_t)__ldg(v.table + (uint64_t)q.seq * v.columns + ca);
        const uint32_t pb = (uint32_t)__ldg(v.table + (uint64_t)q.seq * v.columns + cb);
        moves = pa < v.n_pages && pb < v.n_pages;
        if (!moves) report_table(v.ctr);
        src = pa * p.pool.page_stride + (uint64_t)(a - ca * v.page_tokens) * p.token_bytes;
        dst = pb * p.pool.page_stride + (uint64_t)(b - cb * v.page_tokens) * p.token_bytes;
      }
    }
    uint32_t place, count;
    block_excl_scan<kKeepThreads / 32>(moves, place, count, s_warp);
    if (moves) {
      s_src[place] = src;
      s_dst[place] = dst;
    }
    __syncthreads();
    if (count)
      for (uint32_t run = blockIdx.y * per + tid / p.lanes; run < runs; run += gridDim.y * per) {
        const uint32_t plane = run / p.segments, seg = run - plane * p.segments;
        char* const at = (char*)p.pool.base + plane * p.pool.plane_stride + seg * p.seg_bytes;
        for (uint32_t w = lane; w < p.vectors; w += p.lanes) {
          char* const mine = at + (uint64_t)w * kVec;
          for (uint32_t m0 = 0; m0 < count; m0 += 8) {
            V x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (m0 + j < count) x[j] = *(const V*)(mine + s_src[m0 + j]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (m0 + j < count) *(V*)(mine + s_dst[m0 + j]) = x[j];
          }
        }
      }
    __syncthreads();
  }
}

template <int kVec>
int launch_keep(KeepParams& p, cudaStream_t s) {
  p.vectors = p.token_bytes / kVec;
  p.lanes = 1;
  while (p.lanes < kKeepThreads && p.lanes < p.vectors) p.lanes *= 2;
  const uint64_t per = kKeepThreads / p.lanes, all = ((uint64_t)p.planes * p.segments + per - 1) / per;
  // CTAs for 8 an SM, a share of at least one run for each thread
  const uint64_t most = ((uint64_t)8 * num_sms() + p.view.n - 1) / p.view.n;
  uint64_t y = all < most ? all : most;
  if (y > 65535) y = 65535;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.view.n, (unsigned)y);
  cfg.blockDim = dim3(kKeepThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_keep_kernel<kVec>, p);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_result();
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_cache_write(const db_page_tables* t, const db_cache_batch* b, const db_cache_layer* c,
                              const db_cache_rows* k, const db_cache_rows* v, uint32_t type,
                              uint8_t* status, db_counters* ctr, void* stream) {
  CacheView view;
  if (check_cache(t, b, status, ctr, &view) || check_layer(t, c)) return -EINVAL;
  if (check_rows(k, b->rows, c->heads, c->width, type, false) ||
      check_rows(v, b->rows, c->heads, c->width, type, false))
    return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (const int e = zero_counters(ctr, s)) return e;
  if (!b->n) return 0;
  MoveParams p = move_params(view, c, k, v);
  switch (type) {
    case DB_BF16:
      return launch_move(write_kernel<__nv_bfloat16>(c->type), p, s);
    case DB_F16:
      return launch_move(write_kernel<__half>(c->type), p, s);
    default:
      return launch_move(write_kernel<float>(c->type), p, s);
  }
}

extern "C" int db_cache_read(const db_page_tables* t, const db_cache_batch* b, const int32_t* first,
                             const db_cache_layer* c, const db_cache_rows* k, const db_cache_rows* v,
                             uint32_t type, uint8_t* status, db_counters* ctr, void* stream) {
  CacheView view;
  if (check_cache(t, b, status, ctr, &view) || check_layer(t, c) || !aligned(first, 4)) return -EINVAL;
  if (check_rows(k, b->rows, c->heads, c->width, type, true) ||
      check_rows(v, b->rows, c->heads, c->width, type, true))
    return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (const int e = zero_counters(ctr, s)) return e;
  if (!b->n) return 0;
  MoveParams p = move_params(view, c, k, v);
  p.first = first;
  switch (type) {
    case DB_BF16:
      return launch_move(read_kernel<__nv_bfloat16>(c->type), p, s);
    case DB_F16:
      return launch_move(read_kernel<__half>(c->type), p, s);
    default:
      return launch_move(read_kernel<float>(c->type), p, s);
  }
}

extern "C" int db_cache_keep(const db_page_tables* t, const db_cache_batch* b, const int32_t* path,
                             const int32_t* accepted, const db_page_pool* pool,
                             const db_page_shape* shape, db_page_cut* cut, uint8_t* status,
                             db_counters* ctr, void* stream) {
  CacheView view;
  if (check_cache(t, b, status, ctr, &view)) return -EINVAL;
  if (!pool || !shape || !pool->base || !shape->planes || !shape->segments || !shape->token_bytes)
    return -EINVAL;
  const uint64_t limit = 1ull << 31, rows = (uint64_t)shape->segments * shape->page_tokens;
  if (shape->page_tokens != t->page_tokens || shape->planes > 65536 || rows > limit) return -EINVAL;
  const uint64_t page_bytes = rows * shape->token_bytes;
  if (page_bytes > limit || page_bytes * shape->planes > limit) return -EINVAL;
  if (pool->n_pages < t->n_pages || pool->n_pages > 0xFFFFFFFFull) return -EINVAL;
  if (pool->n_pages > 1 && pool->page_stride < page_bytes) return -EINVAL;
  if (shape->planes > 1 && pool->plane_stride < page_bytes) return -EINVAL;
  if (!aligned(path, 4) || !aligned(accepted, 4) || !aligned(cut, 8)) return -EINVAL;
  if (b->n && (!accepted || (b->rows && !path))) return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (const int e = zero_counters(ctr, s)) return e;
  if (!b->n) return 0;
  KeepParams p = {};
  p.view = view;
  p.path = path;
  p.accepted = accepted;
  p.pool = *pool;
  p.planes = shape->planes;
  p.segments = shape->segments;
  p.token_bytes = shape->token_bytes;
  p.seg_bytes = (uint64_t)shape->page_tokens * shape->token_bytes;
  p.cut = cut;
  // Every run starts on a multiple of the lowest set bit of all of these.
  uint64_t all = (uint64_t)(uintptr_t)pool->base | p.token_bytes;
  if (p.planes > 1) all |= pool->plane_stride;
  if (pool->n_pages > 1) all |= pool->page_stride;
  if (!(all & 15)) return launch_keep<16>(p, s);
  if (!(all & 7)) return launch_keep<8>(p, s);
  if (!(all & 3)) return launch_keep<4>(p, s);
  if (!(all & 1)) return launch_keep<2>(p, s);
  return launch_keep<1>(p, s);
}
