// Shared by the calls on what a cache's pages hold (include/cachedata.h): the
// batch's requests, the places of tokens in the pages, host-side checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cachedata.h"
#include "common.cuh"

namespace db {

// What a kernel needs of the tables and the batch.
struct CacheView {
  const int32_t* table;
  const uint32_t* length;
  uint32_t n_seqs, columns, n_pages, page_tokens;
  const int32_t* seq;
  const int32_t* start;
  uint32_t n, rows;
  uint8_t* status;
  db_counters* ctr;
};

struct Request {
  uint32_t seq, first, rows;  // rows [first, first + rows) of the batch's arrays
  uint32_t length;            // the sequence's tokens
  bool ok;
};

// Request i; of a bad one ok is false and rows 0. `fresh`: its rows are the
// sequence's last tokens.
__device__ __forceinline__ Request read_request(const CacheView& v, uint32_t i, bool fresh) {
  Request r;
  const int32_t a = __ldg(v.start + i), b = __ldg(v.start + i + 1);
  r.seq = (uint32_t)__ldg(v.seq + i);
  r.first = (uint32_t)a;
  r.ok = r.seq < v.n_seqs && a >= 0 && a <= b && (uint32_t)b <= v.rows;
  r.rows = r.ok ? (uint32_t)(b - a) : 0;
  r.length = r.ok ? __ldg(v.length + r.seq) : 0;
  if (r.length >= 1u << 31 || r.length > (uint64_t)v.columns * v.page_tokens || (fresh && r.rows > r.length)) {
    r.ok = false;
    r.rows = 0;
  }
  return r;
}

// The largest i in [0, n) with start[i] <= row (0 when there is none): the
// request that has the row, if any has. Every lane of the warp calls it with
// the same row. 32-way search: three dependent loads for 32,768 requests.
__device__ __forceinline__ uint32_t find_request(const int32_t* start, uint32_t n, uint32_t row) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0, size = n;  // the answer is in [lo, lo + size)
  while (size > 1) {
    const uint32_t step = (size + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < size && (lane == 0 || __ldg(start + at) <= (int32_t)row);
    const uint32_t votes = __ballot_sync(kFull, below);
    // start ascends, so the votes are a run from lane 0 (a broken start still
    // leaves lo inside)
    const uint32_t last = 31 - __clz(votes);
    const uint32_t left = size - last * step;
    lo += last * step;
    size = left < step ? left : step;
  }
  return lo;
}

// Status and counters of the batch's requests, by the calling threads
// (x = index of the thread among `threads`). ctr was zeroed before the kernel.
__device__ __forceinline__ void report_requests(const CacheView& v, uint64_t x, uint64_t threads,
                                                bool fresh) {
  if (!v.status && !v.ctr) return;
  uint64_t rows = 0, bad = 0;
  for (uint64_t i = x; i < v.n; i += threads) {
    const Request r = read_request(v, (uint32_t)i, fresh);
    if (v.status) v.status[i] = r.ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    rows += r.rows;
    bad += !r.ok;
  }
  if (v.ctr) {
    if (rows) atomicAdd((unsigned long long*)&v.ctr->total, (unsigned long long)rows);
    if (bad) atomicAdd((unsigned long long*)&v.ctr->n_invalid, (unsigned long long)bad);
  }
}

__device__ __forceinline__ void report_table(db_counters* ctr) {
  if (ctr) atomicOr((unsigned int*)&ctr->err, DB_ERR_PAGE_TABLE);
}

// ------------------------------------------------------------------ conversions
template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_float(__half x) {
  return __half2float(x);
}

// Two neighbouring 16-bit values of a word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two E4M3 codes (the low 16 bits) as two f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

inline uint32_t item_bytes(uint32_t type) {
  return type == DB_F32 ? 4 : type == DB_BF16 || type == DB_F16 ? 2 : 1;
}

// ----------------------------------------------------------- host-side checks
// 0 or -EINVAL; fills the view.
int check_cache(const db_page_tables* t, const db_cache_batch* b, uint8_t* status, db_counters* ctr,
                CacheView* v);
int check_layer(const db_page_tables* t, const db_cache_layer* c);
int check_rows(const db_cache_rows* r, uint32_t rows, uint32_t heads, uint32_t width, uint32_t type,
               bool written);
// Zeroes the counters (NULL: nothing) on the stream.
int zero_counters(db_counters* ctr, cudaStream_t s);

}  // namespace db
