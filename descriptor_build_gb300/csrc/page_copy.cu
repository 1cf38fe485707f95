// Copies of cache pages (include/pagecache.h: db_page_copy).
//
// A record's work in one plane is a fixed number of slots, each a vector of
// kVec bytes: `runs` runs of `len` bytes, every run rounded up to whole
// vectors. Slots are numbered through records and planes, a warp takes 256 of
// them at a time, 8 loads in flight a lane, and stores them.
#include "common.cuh"
#include "pagecache.h"

namespace db {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kBatch = 8;                   // vectors a lane has in flight
constexpr uint32_t kWarpSlots = 32 * kBatch;     // slots a warp takes at a time

struct CopyParams {
  const db_page_move* moves;
  const uint32_t* n_moves;
  uint32_t max_moves;
  db_page_pool src, dst;
  uint32_t planes, segments, page_tokens, token_bytes;
  uint64_t seg_bytes, page_bytes;
  uint64_t slots;  // of a record in one plane: a multiple of kWarpSlots, or a power of two below it
  db_counters* ctr;
};

template <int kVec>
struct Vec;
template <>
struct Vec<16> {
  typedef uint4 type;
};
template <>
struct Vec<8> {
  typedef uint2 type;
};
template <>
struct Vec<4> {
  typedef uint32_t type;
};
template <>
struct Vec<2> {
  typedef uint16_t type;
};
template <>
struct Vec<1> {
  typedef uint8_t type;
};

// Where slot v of a record in a plane is: bytes [at, at + bytes) of the page.
struct Piece {
  uint64_t at;
  uint32_t bytes;  // 0: none
};

template <int kVec>
__device__ __forceinline__ Piece piece(const CopyParams& p, uint32_t tokens, uint64_t v) {
  Piece x = {0, 0};
  uint64_t len = p.page_bytes, run = 0;
  if (tokens < p.page_tokens) {
    len = (uint64_t)tokens * p.token_bytes;
    if (!len) return x;
    const uint64_t per = (len + kVec - 1) / kVec;
    if (p.segments > 1) {
      if ((v | per) >> 32) {
        run = v / per;
      } else {
        run = (uint32_t)v / (uint32_t)per;
      }
      v -= run * per;
      if (run >= p.segments) return x;
    }
  }
  const uint64_t off = v * kVec;
  if (off >= len) return x;
  x.at = run * p.seg_bytes + off;
  x.bytes = len - off < kVec ? (uint32_t)(len - off) : kVec;
  return x;
}

template <int kVec>
__global__ void __launch_bounds__(kThreads) page_copy_kernel(const CopyParams p) {
  typedef typename Vec<kVec>::type V;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t n = min(__ldcg(p.n_moves), p.max_moves);
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t all = (uint64_t)n * p.planes * p.slots;
  const uint64_t stride = (uint64_t)gridDim.x * (kThreads / 32) * kWarpSlots;
  uint64_t x0 = ((uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kWarpSlots;
  for (; x0 < all; x0 += stride) {
    V v[kBatch];
    uint64_t to[kBatch];
    uint32_t bytes[kBatch];
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
      const uint64_t x = x0 + 32 * j + lane;
      bytes[j] = 0;
      to[j] = 0;
      if (x < all) {
        const uint64_t rp = x / p.slots, r = rp / p.planes;
        const uint64_t plane = rp - r * p.planes;
        const uint4 m = *(reinterpret_cast<const uint4*>(p.moves) + r);
        if (m.x < p.src.n_pages && m.y < p.dst.n_pages) {
          const Piece c = piece<kVec>(p, m.z, x - rp * p.slots);
          bytes[j] = c.bytes;
          const char* from = (const char*)p.src.base + plane * p.src.plane_stride +
                             m.x * p.src.page_stride + c.at;
          to[j] = (uint64_t)((char*)p.dst.base + plane * p.dst.plane_stride +
                             m.y * p.dst.page_stride + c.at);
          if (c.bytes == kVec) {
            v[j] = *(const V*)from;
          } else {
            for (uint32_t k = 0; k < c.bytes; ++k) ((char*)to[j])[k] = from[k];
          }
        }
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j)
      if (bytes[j] == kVec) *(V*)to[j] = v[j];
  }
  if (p.ctr && blockIdx.x == 0) {
    __shared__ unsigned int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    uint32_t bad = 0;
    for (uint32_t r = threadIdx.x; r < n; r += kThreads) {
      const uint4 m = *(reinterpret_cast<const uint4*>(p.moves) + r);
      bad += m.x >= p.src.n_pages || m.y >= p.dst.n_pages;
    }
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();
    if (threadIdx.x == 0) *p.ctr = db_counters{(uint64_t)n - s_bad, s_bad, 0, 0};
  }
}

bool pool_ok(const db_page_pool* q, const db_page_shape* f, uint64_t page_bytes) {
  if (!q || !q->base || !q->n_pages || q->n_pages > 0xFFFFFFFFull) return false;
  if (q->n_pages > 1 && q->page_stride < page_bytes) return false;
  if (f->planes > 1 && q->plane_stride < page_bytes) return false;
  return true;
}

template <int kVec>
int launch_copy(CopyParams& p, cudaStream_t s) {
  const uint64_t per = (p.seg_bytes + kVec - 1) / kVec * p.segments;
  if (per > kWarpSlots / 2) {
    p.slots = (per + kWarpSlots - 1) / kWarpSlots * kWarpSlots;
  } else {
    p.slots = 1;
    while (p.slots < per) p.slots *= 2;
  }
  const uint64_t warps = ((uint64_t)p.max_moves * p.planes * p.slots + kWarpSlots - 1) / kWarpSlots;
  const uint64_t want = (warps + kThreads / 32 - 1) / (kThreads / 32), most = 8ull * num_sms();
  return launch_dependent(page_copy_kernel<kVec>, (unsigned)(want < most ? want : most), kThreads,
                          0, s, p);
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_page_copy(const db_page_move* moves, uint32_t max_moves, const uint32_t* n_moves,
                            const db_page_pool* src, const db_page_pool* dst,
                            const db_page_shape* shape, db_counters* ctr, void* stream) {
  if (!shape || !shape->planes || !shape->segments || !shape->page_tokens || !shape->token_bytes)
    return -EINVAL;
  // A page stays below 2^32 bytes, a record below 2^40 in all its planes.
  const uint64_t rows = (uint64_t)shape->segments * shape->page_tokens;
  if (rows > 0xFFFFFFFFull || rows * shape->token_bytes > 0xFFFFFFFFull || shape->planes > 65536)
    return -EINVAL;
  const uint64_t page_bytes = rows * shape->token_bytes;
  if (!pool_ok(src, shape, page_bytes) || !pool_ok(dst, shape, page_bytes)) return -EINVAL;
  if (!n_moves || !aligned(n_moves, 4) || !aligned(ctr, 8)) return -EINVAL;
  if (max_moves && (!moves || !aligned(moves, 16))) return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!max_moves) {
    if (!ctr) return 0;
    const cudaError_t e = cudaMemsetAsync(ctr, 0, sizeof(*ctr), s);
    return e == cudaSuccess ? 0 : cuda_failure(e);
  }
  CopyParams p = {};
  p.moves = moves;
  p.n_moves = n_moves;
  p.max_moves = max_moves;
  p.src = *src;
  p.dst = *dst;
  p.planes = shape->planes;
  p.segments = shape->segments;
  p.page_tokens = shape->page_tokens;
  p.token_bytes = shape->token_bytes;
  p.seg_bytes = (uint64_t)shape->page_tokens * shape->token_bytes;
  p.page_bytes = page_bytes;
  p.ctr = ctr;
  // Every run starts on a multiple of the lowest set bit of all of these.
  uint64_t all = (uint64_t)(uintptr_t)src->base | (uint64_t)(uintptr_t)dst->base;
  if (p.planes > 1) all |= src->plane_stride | dst->plane_stride;
  if (src->n_pages > 1) all |= src->page_stride;
  if (dst->n_pages > 1) all |= dst->page_stride;
  if (p.segments > 1) all |= p.seg_bytes;
  if (!(all & 15)) return launch_copy<16>(p, s);
  if (!(all & 7)) return launch_copy<8>(p, s);
  if (!(all & 3)) return launch_copy<4>(p, s);
  if (!(all & 1)) return launch_copy<2>(p, s);
  return launch_copy<1>(p, s);
}
