// Copies of cache pages (include/pagecache.h: db_page_copy).
//
// A record is `planes` copies of either the whole page, one run of bytes, or
// its first tokens, a run in each of `segments`. Two kernels share the rest:
//
//  - page_copy_wide_kernel, for pages (or segments, where there are several)
//    of kWideBytes and more: a warp takes chunks of 4 KiB of one run, finds
//    record, plane and segment once, and moves 8 vectors of 16 bytes a lane,
//    all loads in flight before the first store. Few runs get a warp for each
//    chunk; where that would be more than 64 warps an SM, half as many, so that
//    partial pages leave fewer warps without work (1,023 times 15 of 32 KiB in
//    4 planes: 16.5, and 13.5 so; with a quarter 12, but whole pages 0.5 % more);
//  - page_copy_fine_kernel, for smaller ones and for addresses that are not
//    multiples of 16: a CTA works on one plane and segment at a time, in which
//    as many lanes as a run has vectors (up to a warp) take a record, so that
//    short runs share a warp and records are found without a division.
//
// Both are bound by memory: a page's bytes are read once and written once.
// Times below are of one GB300, in microseconds.
#include "common.cuh"
#include "pagecache.h"

namespace db {
namespace {

constexpr uint32_t kThreads = 128;
constexpr uint32_t kBatch = 8;  // vectors a lane has in flight

struct CopyParams {
  const db_page_move* moves;
  const uint32_t* n_moves;
  uint32_t max_moves;
  db_page_pool src, dst;
  uint32_t planes, segments, page_tokens, token_bytes;
  uint64_t seg_bytes;
  uint32_t step;   // wide: warps of a run
  uint32_t lanes;  // fine: lanes of a run
  db_counters* ctr;
};

// The counters, by one CTA when its copies are made: it reads every record,
// with 128 threads and no other work beside. 32,400 records take 11 longer so
// than without counters when their pages are of 64 bytes (5.0 -> 16.0), a
// million 800 longer (51.6 -> 853); behind 32,400 pages of 32 KiB (312) nothing
// shows.
__device__ __forceinline__ void count_records(const CopyParams& p, uint32_t n) {
  if (p.ctr && blockIdx.x == 0 && blockIdx.y == 0) {
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

// A load of page data: L1 holds none of it. (Not the read-only path: source
// and destination may be one pool.)
__device__ __forceinline__ ulonglong2 ld_page16(const void* p, uint64_t pol) {
  ulonglong2 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v2.u64 {%0, %1}, [%2], %3;"
               : "=l"(v.x), "=l"(v.y)
               : "l"(p), "l"(pol)
               : "memory");
  return v;
}

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

// ---------------------------------------------------------------------- fine
// CTAs an SM of the largest grid: with 16, 537 MB of 64-byte pages take 138 and
// 925 MB of partial pages of 1,536 bytes 185, with 64 117 and 165 (4.6 and 5.6
// TB/s), with 256 117 and 186.
constexpr uint32_t kFineCtas = 64;

// Runs of one plane and one segment: `lanes` lanes take a record's run, kUnroll
// vectors a lane, kBatch / kUnroll records at a time.
template <int kVec, int kUnroll>
__global__ void __launch_bounds__(kThreads) page_copy_fine_kernel(const CopyParams p) {
  typedef typename Vec<kVec>::type V;
  constexpr int kRecords = kBatch / kUnroll;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t n = min(__ldcg(p.n_moves), p.max_moves);
  const uint32_t lane = threadIdx.x & (p.lanes - 1), per = kThreads / p.lanes;
  const uint64_t stride = (uint64_t)gridDim.x * per;
  for (uint32_t y = blockIdx.y; y < p.planes * p.segments; y += gridDim.y) {
    const uint32_t plane = y / p.segments, seg = y - plane * p.segments;
    const char* const from = (const char*)p.src.base + plane * p.src.plane_stride + seg * p.seg_bytes;
    char* const to = (char*)p.dst.base + plane * p.dst.plane_stride + seg * p.seg_bytes;
    for (uint64_t r0 = (uint64_t)blockIdx.x * per + threadIdx.x / p.lanes; r0 < n; r0 += stride * kRecords) {
      const char* src[kRecords];
      char* dst[kRecords];
      uint32_t len[kRecords];
#pragma unroll
      for (int i = 0; i < kRecords; ++i) {
        const uint64_t r = r0 + i * stride;
        len[i] = 0;
        src[i] = from;
        dst[i] = to;
        if (r < n) {
          const uint4 m = *(reinterpret_cast<const uint4*>(p.moves) + r);
          if (m.x < p.src.n_pages && m.y < p.dst.n_pages) {
            src[i] = from + m.x * p.src.page_stride;
            dst[i] = to + m.y * p.dst.page_stride;
            len[i] = min(m.z, p.page_tokens) * p.token_bytes;
          }
        }
      }
      for (uint32_t at = lane * kVec; at < (uint32_t)p.seg_bytes; at += p.lanes * kVec * kUnroll) {
        V v[kBatch];
#pragma unroll
        for (int j = 0; j < (int)kBatch; ++j) {
          const uint32_t off = at + j % kUnroll * p.lanes * kVec;
          if (off + kVec <= len[j / kUnroll]) v[j] = *(const V*)(src[j / kUnroll] + off);
        }
#pragma unroll
        for (int j = 0; j < (int)kBatch; ++j) {
          const uint32_t off = at + j % kUnroll * p.lanes * kVec, end = len[j / kUnroll];
          if (off + kVec <= end) {
            *(V*)(dst[j / kUnroll] + off) = v[j];
          } else {  // the run's last bytes
            uint32_t k = off;
            if (kVec > 4)
              for (; k + 4 <= end; k += 4)
                *(uint32_t*)(dst[j / kUnroll] + k) = *(const uint32_t*)(src[j / kUnroll] + k);
            for (; k < end; ++k) dst[j / kUnroll][k] = src[j / kUnroll][k];
          }
        }
      }
    }
  }
  count_records(p, n);
}

// ---------------------------------------------------------------------- wide
constexpr uint32_t kChunk = 32 * kBatch * 16;  // bytes a warp moves at a time
// Runs from here on go to the wide kernel. The other one takes 235 for partial
// segments of 5.6 KB and 346 for 4 KB ones, this one 246 and 351; for whole 32
// KiB pages it is 547 against 538 above, and for six pages 5.3 against 2.6.
constexpr uint64_t kWideBytes = 8192;
// CTAs an SM of the largest grid. How many records there are is on the device,
// so the grid is bounded and loops; 8 CTAs are resident, and several times as
// many even out what the loops leave at the end. 3,500 pages of 16 planes of
// 32 KiB (3.67 GB read and written): 580 with one grid of residents, 557
// twice, 544 four times, 538 eight times (6.8 TB/s, the rate of a plain copy),
// 535 sixteen times; six pages alone take 0.3 less in CTAs of 128 threads
// than of 256. The same pages through shared memory by bulk copies (4 to 16 KiB,
// 3 to 12 CTAs an SM, 2 or 4 stages ahead) took 570 to 607, and 2.8 KB
// runs 75 and more where these loads and stores take 44.
constexpr uint32_t kWideCtas = 64;
__device__ __forceinline__ uint64_t div64(uint64_t a, uint32_t b) {
  return (a >> 32) ? a / b : (uint32_t)a / b;
}

__global__ void __launch_bounds__(kThreads) page_copy_wide_kernel(const CopyParams p) {
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t n = min(__ldcg(p.n_moves), p.max_moves);
  const uint32_t lane = threadIdx.x & 31, runs = p.planes * p.segments;
  const uint64_t all = (uint64_t)n * runs * p.step;
  const uint64_t stride = (uint64_t)gridDim.x * (kThreads / 32);
  const uint64_t pol = policy_evict_first();
  for (uint64_t x = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; x < all; x += stride) {
    const uint64_t run = div64(x, p.step), r = div64(run, runs);
    const uint32_t of = (uint32_t)(run - r * runs), plane = of / p.segments, seg = of - plane * p.segments;
    const uint4 m = *(reinterpret_cast<const uint4*>(p.moves) + r);
    if (m.x >= p.src.n_pages || m.y >= p.dst.n_pages) continue;
    const uint32_t len = min(m.z, p.page_tokens) * p.token_bytes;
    const char* const from = (const char*)p.src.base + plane * p.src.plane_stride + m.x * p.src.page_stride + seg * p.seg_bytes;
    char* const to = (char*)p.dst.base + plane * p.dst.plane_stride + m.y * p.dst.page_stride + seg * p.seg_bytes;
    for (uint32_t off = (uint32_t)(x - run * p.step) * kChunk; off < len; off += p.step * kChunk) {
      ulonglong2 v[kBatch];
      if (len - off >= kChunk) {
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) v[j] = ld_page16(from + off + 16 * (32 * j + lane), pol);
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) st_stream16(to + off + 16 * (32 * j + lane), v[j].x, v[j].y, pol);
      } else {
        const uint32_t left = len - off, whole = left / 16;
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j)
          if (32 * j + lane < whole) v[j] = ld_page16(from + off + 16 * (32 * j + lane), pol);
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j)
          if (32 * j + lane < whole) st_stream16(to + off + 16 * (32 * j + lane), v[j].x, v[j].y, pol);
        if (lane < left % 16) to[off + 16 * whole + lane] = from[off + 16 * whole + lane];
      }
    }
  }
  count_records(p, n);
}

bool pool_ok(const db_page_pool* q, const db_page_shape* f, uint64_t page_bytes) {
  if (!q || !q->base || !q->n_pages || q->n_pages > 0xFFFFFFFFull) return false;
  if (q->n_pages > 1 && q->page_stride < page_bytes) return false;
  if (f->planes > 1 && q->plane_stride < page_bytes) return false;
  return true;
}

int launch_fine(void (*kernel)(CopyParams), int unroll, const CopyParams& p, cudaStream_t s) {
  const uint64_t per = kThreads / p.lanes * (kBatch / unroll);
  const uint64_t rows = (uint64_t)p.planes * p.segments, x = (p.max_moves + per - 1) / per;
  // CTAs along the records and along planes and segments, in all no more than
  // stay busy for several rounds. How many records there are is on the device:
  // where the list has room for many and holds few, the CTAs along the records
  // find none and the others go through planes and segments one by one. 6
  // records of 64 planes x 8 segments take 3.7 in a list of 6, 10.6 of 256, 27
  // of 4,096 and 516 of 100,000.
  const uint64_t most = (uint64_t)kFineCtas * num_sms();
  const uint64_t gx = x < most ? x : most;
  uint64_t gy = most / gx;
  gy = gy < 1 ? 1 : gy < rows ? gy : rows;
  if (gy > 65535) gy = 65535;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)gx, (unsigned)gy);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_result();
}

template <int kVec>
int launch_copy(CopyParams& p, cudaStream_t s) {
  const uint64_t vectors = (p.seg_bytes + kVec - 1) / kVec;
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < vectors) p.lanes *= 2;
  const uint64_t each = (vectors + p.lanes - 1) / p.lanes;
  if (each <= 1) return launch_fine(page_copy_fine_kernel<kVec, 1>, 1, p, s);
  if (each <= 2) return launch_fine(page_copy_fine_kernel<kVec, 2>, 2, p, s);
  if (each <= 4) return launch_fine(page_copy_fine_kernel<kVec, 4>, 4, p, s);
  return launch_fine(page_copy_fine_kernel<kVec, 8>, 8, p, s);
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_page_copy(const db_page_move* moves, uint32_t max_moves, const uint32_t* n_moves,
                            const db_page_pool* src, const db_page_pool* dst,
                            const db_page_shape* shape, db_counters* ctr, void* stream) {
  if (!shape || !shape->planes || !shape->segments || !shape->page_tokens || !shape->token_bytes)
    return -EINVAL;
  // A page's bytes in all planes are at most 2^31: what is numbered below stays within 64 bits.
  const uint64_t limit = 1ull << 31, rows = (uint64_t)shape->segments * shape->page_tokens;
  if (shape->planes > 65536 || rows > limit) return -EINVAL;
  const uint64_t page_bytes = rows * shape->token_bytes;
  if (page_bytes > limit || page_bytes * shape->planes > limit) return -EINVAL;
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
  p.ctr = ctr;
  // Every run starts on a multiple of the lowest set bit of all of these.
  uint64_t all = (uint64_t)(uintptr_t)src->base | (uint64_t)(uintptr_t)dst->base;
  if (p.planes > 1) all |= src->plane_stride | dst->plane_stride;
  if (src->n_pages > 1) all |= src->page_stride;
  if (dst->n_pages > 1) all |= dst->page_stride;
  if (p.segments > 1) all |= p.seg_bytes;
  if (!(all & 15) && p.seg_bytes >= kWideBytes) {
    const uint64_t runs = (uint64_t)max_moves * p.planes * p.segments;
    p.step = (uint32_t)((p.seg_bytes + kChunk - 1) / kChunk);
    if (runs * p.step > 64ull * num_sms()) p.step = (p.step + 1) / 2;
    const uint64_t warps = runs * p.step;
    const uint64_t want = (warps + kThreads / 32 - 1) / (kThreads / 32), most = (uint64_t)kWideCtas * num_sms();
    return launch_dependent(page_copy_wide_kernel, (unsigned)(want < most ? want : most), kThreads, 0, s, p);
  }
  if (!(all & 15)) return launch_copy<16>(p, s);
  if (!(all & 7)) return launch_copy<8>(p, s);
  if (!(all & 3)) return launch_copy<4>(p, s);
  if (!(all & 1)) return launch_copy<2>(p, s);
  return launch_copy<1>(p, s);
}
