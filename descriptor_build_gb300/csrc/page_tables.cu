// Page tables of a cache in the device heap: extend, fork, free, compact
// (include/pagecache.h has the definitions).
//
// A plan is a prefix sum over what a call's requests ask for, and what follows
// is work on pieces of it, found again by a search. There are two ways to it,
// and no kernel of either waits on memory:
//
//  - Few requests: a gang. Every CTA of one launch plans the whole batch for
//    itself, in shared memory, and does its share of the pieces; the last CTA
//    to finish writes what the others may still have been reading.
//  - Many: a team. One cluster of CTAs, whose barriers are the hardware's,
//    plans together and does little work itself; a second kernel, launched as
//    a dependent of the first where the sizes of the call allow for more,
//    does it on the whole GPU (how much there is, only the device knows).
//
// Nothing depends on the order in which atomics land: a request's claim on
// its sequence and the holders of a shared page are a maximum and a count,
// references are sums, free pages are bits, and pages are taken by rank among
// the set bits.
#include "common.cuh"
#include "pagecache.h"

namespace db {
namespace {

// Times below are of one GB300, microseconds, of the sequence of calls named.
// They were taken when the choice was made, unless said otherwise.
//
// What bounds these kernels is latency: a few dependent trips to memory and
// the barriers of the plan between them. Freeing 98,304 pages in 96 CTAs (9.8)
// keeps a scheduler issuing in 10 % of its cycles, L1 18 % and L2 4 % busy; of
// 21 cycles between two instructions of a warp 11 are at barriers and 3 for
// loads. The scattered lines of those pages (a load and a store of a
// reference, an atomic on its free bit), one a clock, are 3,100 clocks of each
// of the 96 SMs, 1.6. 320,000 pages (11.4, 256 CTAs) are alike: L1 at 29 %,
// lines for 3.3 of the time. Only the second
// kernel of an extension is bound by something else, by issue (63 % of cycles,
// two searches a page). Bandwidth is far away (a freed or taken page is 24 bytes).
constexpr uint32_t kMaxTeam = 8;          // CTAs of the largest team (a portable cluster)
constexpr uint32_t kTeamThreads = 1024;   // threads of a CTA of a team, or of a gang that extends
// Threads of a CTA of a gang with few requests. A step of 48 sequences took
// 8.2 in CTAs of 256 or of 512 threads and 11.7 in one of 1,024, whose
// barriers and idle warps cost more than its width saves. Now it takes 7.8 in a
// pool of 32,768 pages, 8.6 in one of 32,800, whose extensions go to CTAs of
// 1,024 threads (a thread of the smaller ones keeps one quad of free words),
// and 9.0 in one of 131,072. Up to as many
// requests free and fork go to a gang: 1,023 of one prompt took 14.4 and 12.7
// in a gang of 1,024 threads and 13.3 and 11.0 as a team and a second kernel.
constexpr uint32_t kSmallThreads = 256;
// Requests of a group (see "row units"): 4, 8, 16 or 32 of them gave 61, 49,
// 46 or 50 for dropping and forking 1,023 samples anew (44 now, with 8), 21,
// 23, 25 or 33 for a decode step of 4,096 sequences (18.5 now), and 13, 14, 15
// or 34 for a turnover of 256 (12.4 now).
constexpr uint32_t kRows = 8;
constexpr uint32_t kSearch = 1024;        // starts that a second kernel keeps in shared memory
// Free words that a CTA of a gang counts (262,144 pages). Each CTA reads them
// all: an extension by 320,000 pages out of a million took 23.5 in a gang and
// takes 15 as a team and a second kernel, one by 98,000 of 262,144 takes 9.9
// and took 8.0 + 5.2. For 48 sequences the limit is low: a step takes 10.2 with
// 262,144 pages in a gang, 13.0 with 64 more as a team and a second kernel,
// and 11.9 with a million so; where the two meet was not measured.
constexpr uint32_t kGangWords = 8192;
constexpr uint32_t kTeamWords = 2048;     // free words that a CTA of a team keeps in shared memory
// A second kernel, or a gang of more than one CTA, is launched when the sizes
// of a call allow for more than this. It costs 1.2 on the device and 2.3 on
// the host when there turns out to be nothing to do; without it the 98,000
// entries of a prompt chunk took 18.6 to free in the team's SMs, with it 11.
constexpr uint32_t kRestUnits = 64, kRestPages = 16384, kRestMoves = 8192;
// With a second kernel there, a team still does this itself: entries for each
// of its CTAs (an SM takes about that many a microsecond), and pages.
constexpr uint32_t kOwnEntries = 1024, kOwnPages = 4096;
constexpr uint32_t kSoloEntries = 32768;  // table entries that a compaction's one CTA renames itself
constexpr uint32_t kNoMove = 0xFFFFFFFFu;
constexpr uint32_t kNoEntry = 0xFFFFFFFEu;   // a row without an entry in the column
constexpr uint32_t kBadEntry = 0xFFFFFFFFu;  // no page

// One request's place in the plan.
struct __align__(16) Plan {
  uint32_t row;   // row that is written
  uint32_t from;  // free, fork: first column; extend: the column of its first page
  uint32_t end;   // free, fork: past the last column; extend: pages of the requests before it
  uint32_t aux;   // extend: index of its move or kNoMove; fork: the parent's row
};

struct Head {
  unsigned long long released;  // a gang's sum over its CTAs, zero between calls
  uint32_t done;       // CTAs of a gang that are through, zero between calls
  uint32_t bad;        // a gang's error, zero between calls
  uint32_t units;      // left for the second kernel: units, pages or moves
  uint32_t used;       // extend: free words up to the last one used
  uint32_t n_live;     // compact: live pages
  uint32_t holes;      // compact: free pages below n_live
  uint32_t moved;      // compact: moves made
  uint32_t dst_last;   // compact: the last page moved to (with moved > 0)
  uint32_t src_first;  // compact: the lowest page moved from, or n_pages
};

struct Work {
  Head* head;
  uint32_t* claim;    // [n_seqs], zero between calls
  uint32_t* holders;  // [n_pages], zero between calls
  uint32_t* latest;   // [n_pages], zero between calls
  Plan* plan;         // [n_seqs]
  uint2* group;       // [n_seqs / kRows] {units before it, its first column}
  uint32_t* before;   // [n_words] free pages before each word
  uint32_t* bits;     // [n_words] extend: the free words before the call
  uint32_t* renamed;  // [n_pages] compact: where a moved page went
};

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t carve(char* ws, uint32_t n_seqs, uint32_t n_pages, Work* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws ? ws + at : nullptr;
    at += up256(bytes);
    return p;
  };
  Work x;
  x.head = (Head*)take(sizeof(Head));
  x.claim = (uint32_t*)take(4 * (size_t)n_seqs);
  x.holders = (uint32_t*)take(4 * (size_t)n_pages);
  x.latest = (uint32_t*)take(4 * (size_t)n_pages);
  x.plan = (Plan*)take(16 * (size_t)n_seqs);
  x.group = (uint2*)take(8 * (((size_t)n_seqs + kRows - 1) / kRows));
  const size_t words = ((size_t)n_pages + 31) / 32;
  x.before = (uint32_t*)take(4 * words);
  x.bits = (uint32_t*)take(4 * words);
  x.renamed = (uint32_t*)take(4 * (size_t)n_pages);
  if (w) *w = x;
  return at;
}

// ------------------------------------------------------------------ the team
struct TeamShared {
  uint32_t warp_a[2][32], warp_b[2][32];            // each warp's sums, two scans apart
  uint32_t cta_a[2][kMaxTeam], cta_b[2][kMaxTeam];  // each CTA's, written by it
};

// kSolo: the team is one CTA of kThreads.
template <uint32_t kThreads, bool kSolo>
struct Team {
  static constexpr uint32_t kWarps = kThreads / 32;
  uint32_t rank, size, round;
  TeamShared* s;

  __device__ __forceinline__ explicit Team(TeamShared* sh) : rank(0), size(1), round(0), s(sh) {
    if (!kSolo) {
      asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
      asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    }
  }
  // Every CTA of the cluster has started: its shared memory may be written.
  // Comes once, before the first sync or scan.
  __device__ __forceinline__ void started() const {
    if (!kSolo) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  __device__ __forceinline__ uint32_t id() const { return rank * kThreads + threadIdx.x; }
  __device__ __forceinline__ uint32_t threads() const { return size * kThreads; }
  // Requests are dealt evenly to the CTAs: a round takes per(n) * size of
  // them, thread t of CTA r the (r * per(n) + t)-th when t < per(n).
  __device__ __forceinline__ uint32_t per(uint32_t n) const {
    return kSolo ? kThreads : min(kThreads, ((n + size - 1) / size + 31) & ~31u);
  }
  // Barrier of the team; global and shared writes before it are seen after it.
  __device__ __forceinline__ void sync() const {
    if (kSolo) {
      __syncthreads();
    } else {
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                       : "memory");
    }
  }
  // Exclusive prefix of v in the order of CTAs and threads, and the sum; also
  // the sum of w, and the number of threads before with w != 0, when kPair.
  // Also a barrier of the team. The arrays of one scan are written again two
  // scans later, past the barrier of the one between.
  template <bool kPair>
  __device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* total, uint32_t w = 0,
                                           uint32_t* sum_w = nullptr, uint32_t* rank_w = nullptr) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = round++ & 1;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= (uint32_t)o) x += y;
    }
    const uint32_t ws = kPair ? __reduce_add_sync(kFull, w) : 0;
    if (lane == 31) {
      s->warp_a[k][warp] = x;
      if (kPair) s->warp_b[k][warp] = ws;
    }
    __syncthreads();
    const uint32_t a = lane < kWarps ? s->warp_a[k][lane] : 0;
    const uint32_t b = kPair && lane < kWarps ? s->warp_b[k][lane] : 0;
    uint32_t base_a = __reduce_add_sync(kFull, lane < warp ? a : 0), base_b = 0;
    if (rank_w) base_b = __reduce_add_sync(kFull, lane < warp ? b : 0);
    if (kSolo) {
      *total = __reduce_add_sync(kFull, a);
      if (kPair) *sum_w = __reduce_add_sync(kFull, b);
    } else {
      if (warp == 0) {
        const uint32_t sum_a = __reduce_add_sync(kFull, a);
        const uint32_t sum_b = kPair ? __reduce_add_sync(kFull, b) : 0;
        if (lane < size) {
          to_peer(&s->cta_a[k][rank], lane, sum_a);
          if (kPair) to_peer(&s->cta_b[k][rank], lane, sum_b);
        }
      }
      sync();
      const uint32_t c = lane < size ? s->cta_a[k][lane] : 0;
      base_a += __reduce_add_sync(kFull, lane < rank ? c : 0);
      *total = __reduce_add_sync(kFull, c);
      if (kPair) {
        const uint32_t d = lane < size ? s->cta_b[k][lane] : 0;
        if (rank_w) base_b += __reduce_add_sync(kFull, lane < rank ? d : 0);
        *sum_w = __reduce_add_sync(kFull, d);
      }
    }
    if (rank_w) *rank_w = base_b + __popc(__ballot_sync(kFull, w != 0) & lanemask_lt());
    return base_a + x - v;
  }
  // A word to the same place in a CTA of the cluster.
  __device__ __forceinline__ static void to_peer(uint32_t* mine, uint32_t peer, uint32_t v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(peer));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
  }
  __device__ __forceinline__ void to_all(uint32_t* mine, uint32_t v) const {
    for (uint32_t c = 0; c < size; ++c) to_peer(mine, c, v);
  }
};

// ---------------------------------------------------------- finding a piece
// The last i < n with start(i) <= e, where start does not decrease: every
// `step`-th start is in shared memory, and those between two of them lie in a
// line or two of memory.
struct Finder {
  const uint32_t* s_start;
  uint32_t n, kept, step;
  template <typename Start>
  __device__ __forceinline__ uint32_t find(uint32_t e, Start start) const {
    uint32_t lo = 0, hi = kept;  // s_start[lo] <= e < s_start[hi]
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      if (s_start[mid] <= e) lo = mid; else hi = mid;
    }
    if (step > 1) {
      lo *= step;
      hi = min(n, lo + step);
      while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (start(mid) <= e) lo = mid; else hi = mid;
      }
    }
    return lo;
  }
};

// Load the starts, at most `most` (every thread of a CTA; a barrier follows).
template <typename Start>
__device__ __forceinline__ Finder load_finder(uint32_t* s_start, uint32_t most, uint32_t n,
                                              Start start) {
  const uint32_t step = (n + most - 1) / most, kept = (n + step - 1) / step;
  for (uint32_t k = threadIdx.x; k < kept; k += blockDim.x) s_start[k] = start(k * step);
  return Finder{s_start, n, kept, step};
}

// The plan, in shared memory or in the workspace. (A team's barrier and the
// wait for the kernel before order these after the stores of other CTAs.)
__device__ __forceinline__ Plan ld_plan(const Plan* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return Plan{v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ void st_plan(Plan* p, const Plan& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v.row, v.from, v.end, v.aux);
}

// First come, first served: of the requests naming a sequence the first has
// the largest claim. 0 is no claim.
__device__ __forceinline__ void claim(uint32_t* c, uint32_t seq, uint32_t i) {
  atomicMax(&c[seq], 0xFFFFFFFFu - i);
}
__device__ __forceinline__ bool claimed(const uint32_t* c, uint32_t seq, uint32_t i) {
  return __ldcg(&c[seq]) == 0xFFFFFFFFu - i;
}

__device__ __forceinline__ uint32_t pages_of(uint64_t tokens, uint32_t page_tokens) {
  return tokens + page_tokens > 0xFFFFFFFFull
             ? (uint32_t)((tokens + page_tokens - 1) / page_tokens)
             : ((uint32_t)tokens + page_tokens - 1) / page_tokens;
}

// The j-th set bit (from 0) of v.
__device__ __forceinline__ uint32_t nth_bit(uint32_t v, uint32_t j) {
  uint32_t at = 0;
#pragma unroll
  for (uint32_t half = 16; half; half >>= 1) {
    const uint32_t c = __popc(v & ((1u << half) - 1));
    if (j >= c) {
      j -= c;
      at += half;
      v >>= half;
    }
  }
  return at;
}

// A count and an error, one warp's at a time, into the counters.
__device__ __forceinline__ void add_count(uint64_t* to, uint32_t count) {
  const uint32_t c = __reduce_add_sync(kFull, count);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd((unsigned long long*)to, (unsigned long long)c);
}
__device__ __forceinline__ void add_error(db_counters* ctr, bool bad) {
  if (__any_sync(kFull, bad) && (threadIdx.x & 31) == 0)
    atomicOr((unsigned long long*)&ctr->err, (unsigned long long)DB_ERR_PAGE_TABLE);
}

// -------------------------------------------------------------------- the gang
// Requests by what they name, in a CTA: open addressing with two places for
// each thread, so that a free one is always found. Numbers are below 2^31.
template <uint32_t kThreads>
struct Names {
  static constexpr uint32_t kPlaces = 2 * kThreads;
  uint32_t key[kPlaces], least[kPlaces], count[kPlaces];
  __device__ __forceinline__ void clear() {
    for (uint32_t k = threadIdx.x; k < kPlaces; k += kThreads) {
      key[k] = least[k] = 0xFFFFFFFFu;
      count[k] = 0;
    }
  }
  __device__ __forceinline__ uint32_t place(uint32_t name) {
    uint32_t k = name * 2654435761u >> 16 & (kPlaces - 1);
    for (uint32_t tries = 0; tries < kPlaces; ++tries) {
      const uint32_t was = atomicCAS(&key[k], 0xFFFFFFFFu, name);
      if (was == 0xFFFFFFFFu || was == name) break;
      k = (k + 1) & (kPlaces - 1);
    }
    return k;
  }
};

// Whether this CTA is the last of its gang to come here (a barrier of the CTA;
// what all of them have read before is read).
__device__ __forceinline__ bool last_of_gang(Head* head) {
  __shared__ uint32_t s_last;
  __syncthreads();
  if (gridDim.x == 1) return true;
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&head->done, 1u) == gridDim.x - 1;
    if (s_last) head->done = 0;
  }
  __syncthreads();
  return s_last;
}

// The same, with a count and an error of every CTA summed for the last one.
__device__ __forceinline__ bool last_of_gang(Head* head, uint32_t count, bool bad, uint64_t* total,
                                             bool* any_bad) {
  __shared__ uint32_t s_count, s_bad;
  if (threadIdx.x == 0) s_count = s_bad = 0;
  __syncthreads();
  const uint32_t c = __reduce_add_sync(kFull, count);
  const bool b = __any_sync(kFull, bad);
  if ((threadIdx.x & 31) == 0) {
    if (c) atomicAdd(&s_count, c);
    if (b) s_bad = 1;
  }
  __syncthreads();
  if (gridDim.x > 1 && threadIdx.x == 0) {
    if (s_count) atomicAdd(&head->released, (unsigned long long)s_count);
    if (s_bad) atomicOr(&head->bad, 1u);
  }
  if (!last_of_gang(head)) return false;
  *total = s_count;
  *any_bad = s_bad;
  if (gridDim.x > 1 && threadIdx.x == 0) {
    *total = atomicExch(&head->released, 0ull);
    *any_bad = atomicExch(&head->bad, 0u);
  }
  return true;
}

// ---------------------------------------------------------------- free words
// Word w of the free bits, without bits past n_pages.
__device__ __forceinline__ uint32_t ld_word(const uint32_t* bits, uint32_t w, uint32_t n_pages) {
  uint32_t v = __ldcg(&bits[w]);
  if (n_pages - 32 * w < 32) v &= (1u << (n_pages & 31)) - 1;
  return v;
}
// Words w to w + 3 of `all` (0 past them).
__device__ __forceinline__ uint4 ld_quad(const uint32_t* bits, uint32_t w, uint32_t all,
                                         uint32_t n_pages) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (w + 4 < all) {
    v = __ldcg(reinterpret_cast<const uint4*>(bits + w));
  } else {
    if (w < all) v.x = ld_word(bits, w, n_pages);
    if (w + 1 < all) v.y = ld_word(bits, w + 1, n_pages);
    if (w + 2 < all) v.z = ld_word(bits, w + 2, n_pages);
    if (w + 3 < all) v.w = ld_word(bits, w + 3, n_pages);
  }
  return v;
}

// A thread's share of the free bits: `quads` quads of consecutive words from
// `first` on, the first of which stays in registers.
struct Bits {
  uint32_t first, quads;
  uint32_t before;  // free pages before them
  uint32_t total;   // free pages of the cache
  uint4 v;
};

template <uint32_t kThreads, bool kSolo>
__device__ __forceinline__ Bits load_free(const Team<kThreads, kSolo>& team, const uint32_t* bits,
                                          uint32_t n_pages) {
  const uint32_t all = (n_pages + 31) / 32, threads = team.threads();
  Bits b;
  b.quads = (all + 4 * threads - 1) / (4 * threads);
  b.first = team.id() * b.quads * 4;
  b.v = ld_quad(bits, b.first, all, n_pages);
  return b;
}

// The free pages before them, and a vote of the team.
template <uint32_t kThreads, bool kSolo>
__device__ __forceinline__ bool scan_free(Team<kThreads, kSolo>& team, Bits& b,
                                          const uint32_t* bits, uint32_t n_pages, bool vote) {
  const uint32_t all = (n_pages + 31) / 32;
  uint32_t c = __popc(b.v.x) + __popc(b.v.y) + __popc(b.v.z) + __popc(b.v.w);
  for (uint32_t s = 1; s < b.quads; ++s) {
    const uint4 v = ld_quad(bits, b.first + 4 * s, all, n_pages);
    c += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
  }
  uint32_t votes;
  b.before = team.template scan<true>(c, &b.total, vote, &votes);
  return votes;
}

// f(first word, its quad, free pages before each of the four) for a thread's
// quads, in order, until f returns false.
template <typename F>
__device__ __forceinline__ void each_quad(const Bits& b, const uint32_t* bits, uint32_t n_pages,
                                          F f) {
  const uint32_t all = (n_pages + 31) / 32;
  uint32_t before = b.before;
  for (uint32_t s = 0; s < b.quads; ++s) {
    const uint32_t w = b.first + 4 * s;
    if (w >= all) return;
    const uint4 v = s ? ld_quad(bits, w, all, n_pages) : b.v;
    uint4 at;
    at.x = before;
    at.y = at.x + __popc(v.x);
    at.z = at.y + __popc(v.y);
    at.w = at.z + __popc(v.z);
    if (!f(w, v, at)) return;
    before = at.w + __popc(v.w);
  }
}

// A quad of words into an array of `all` words, 16-byte aligned.
__device__ __forceinline__ void st_quad(uint32_t* to, uint32_t w, uint32_t all, const uint4& v) {
  if (w + 4 <= all) {
    *reinterpret_cast<uint4*>(to + w) = v;
  } else {
    to[w] = v.x;
    if (w + 1 < all) to[w + 1] = v.y;
    if (w + 2 < all) to[w + 2] = v.z;
  }
}

struct WordStart {
  const uint32_t* before;
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const { return before[w]; }
};

// --------------------------------------------------------------- row units
// Free and fork work on columns [from, end) of each request's row. kRows
// requests in order are a group; the columns from the first to the last that
// any of them has, from a multiple of 32 on, are cut into units of 32, and a
// warp takes a unit: one column a lane, kRows rows in flight. Rows of one
// group often name the same page in one column (a common prefix, the
// children of one parent); its references then change by one atomic.
struct Rows {
  db_page_tables t;
  db_counters* ctr;
  uint8_t* status;
  uint32_t n;
  bool rest;  // a second kernel follows
  Work w;
};

// What a CTA keeps on chip of its requests' plan, of the last round.
template <uint32_t kThreads>
struct RowPlan {
  Plan plan[kThreads];
  uint32_t col[kThreads / kRows];
  uint32_t start[kThreads / kRows];
  uint32_t units;  // of this CTA
};

// Each thread's columns into the groups (visible past the next barrier).
// `units`, `entries`: those of the requests before, and then also of these.
template <uint32_t kThreads, bool kSolo>
__device__ __forceinline__ void plan_rows(Team<kThreads, kSolo>& team, const Rows& p,
                                          RowPlan<kThreads>* s, uint32_t i, bool mine,
                                          const Plan& pl, uint32_t* units, uint32_t* entries) {
  const uint32_t count = pl.from < pl.end ? pl.end - pl.from : 0;
  uint32_t lo = count ? pl.from : 0xFFFFFFFFu, hi = count ? pl.end : 0;
#pragma unroll
  for (uint32_t o = 1; o < kRows; o <<= 1) {
    lo = min(lo, __shfl_xor_sync(kFull, lo, o));
    hi = max(hi, __shfl_xor_sync(kFull, hi, o));
  }
  lo &= ~31u;
  const bool lead = threadIdx.x % kRows == 0, first = mine && lead;
  const uint32_t here = first && hi > lo ? (hi - lo + 31) / 32 : 0;
  uint32_t total, total_entries;
  const uint32_t x = team.template scan<true>(here, &total, count, &total_entries);
  s->plan[threadIdx.x] = pl;
  if (lead) {
    s->start[threadIdx.x / kRows] = x;
    s->col[threadIdx.x / kRows] = lo;
  }
  if (threadIdx.x == kThreads - kRows) s->units = x + here;  // past this CTA's last
  if (mine && p.rest) {
    st_plan(&p.w.plan[i], pl);
    if (first) p.w.group[i / kRows] = make_uint2(*units + x, lo);
  }
  *units += total;
  *entries += total_entries;
}

struct GroupStart {
  const uint2* group;
  __device__ __forceinline__ uint32_t operator()(uint32_t g) const { return group[g].x; }
};

// A CTA's own units, in shared memory. Starts do not decrease, so the number
// of those at or before u is found by votes, without a search's steps.
template <uint32_t kThreads>
struct OwnUnits {
  const RowPlan<kThreads>* s;
  struct Unit {
    const Plan* plan;
    uint32_t base;  // its first column
    __device__ __forceinline__ Plan row(uint32_t j) const { return ld_plan(plan + j); }
  };
  __device__ __forceinline__ Unit find(uint32_t u) const {
    uint32_t g = 0;
#pragma unroll
    for (uint32_t k = 0; k < kThreads / kRows; k += 32)
      g += __popc(__ballot_sync(kFull, s->start[k + (threadIdx.x & 31)] <= u));
    --g;
    return Unit{&s->plan[g * kRows], s->col[g] + (u - s->start[g]) * 32};
  }
};

// All units, in the workspace: a lane loads a row's plan and the others get
// it from there.
struct AllUnits {
  Finder f;
  const Plan* plan;
  const uint2* group;
  uint32_t n;
  struct Unit {
    Plan mine;
    uint32_t base;
    __device__ __forceinline__ Plan row(uint32_t j) const {
      return Plan{__shfl_sync(kFull, mine.row, j), __shfl_sync(kFull, mine.from, j),
                  __shfl_sync(kFull, mine.end, j), __shfl_sync(kFull, mine.aux, j)};
    }
  };
  __device__ __forceinline__ Unit find(uint32_t u) const {
    const uint32_t g = f.find(u, GroupStart{group}), lane = threadIdx.x & 31, i = g * kRows + lane;
    Plan pl = {0, 0, 0, 0};
    if (lane < kRows && i < n) pl = ld_plan(&plan[i]);
    const uint2 at = group[g];
    return Unit{pl, at.y + (u - at.x) * 32};
  }
};

__device__ __forceinline__ AllUnits all_units(const Rows& p, uint32_t* s_start) {
  AllUnits x;
  x.f = load_finder(s_start, kSearch, (p.n + kRows - 1) / kRows, GroupStart{p.w.group});
  x.plan = p.w.plan;
  x.group = p.w.group;
  x.n = p.n;
  __syncthreads();
  return x;
}

// The end of a planning team: each CTA's own units, or all units to the second
// kernel. A team that plans in more than one round always has one.
template <uint32_t kThreads, typename F>
__device__ __forceinline__ void own_units(const Team<kThreads, false>& team, const Rows& p,
                                          RowPlan<kThreads>* s, uint32_t units, uint32_t entries,
                                          F work) {
  const bool own = !p.rest || (p.n <= team.threads() && entries <= kOwnEntries * team.size);
  if (p.rest && team.id() == 0) p.w.head->units = own ? 0 : units;
  if (!own || !units) return;
  __syncthreads();
  work(OwnUnits<kThreads>{s}, s->start[0] + threadIdx.x / 32, kThreads / 32, s->units);
}

// ---------------------------------------------------------------------- free
struct FreeParams {
  Rows r;
  const db_page_cut* req;
};

// refs[p] -= the rows of the batch that drop p; p is free when nothing is left.
// A step of 48 sequences frees its 12 pages in 3.7 (one launch, warm), 192
// prompt chunks of 512 pages in 9.8, 64 sequences of 5,000 pages in 11.4.
template <typename X>
__device__ __forceinline__ void free_units(const Rows& p, const X& x, uint32_t first,
                                           uint32_t stride, uint32_t units, uint32_t* count,
                                           bool* error) {
  uint32_t released = 0;
  bool bad = false;
  const uint32_t lane = threadIdx.x & 31;
  for (uint32_t u = first; u < units; u += stride) {
    const auto at = x.find(u);
    const uint32_t c = at.base + lane;
    int32_t* entry[kRows];
    uint32_t page[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const Plan pl = at.row(j);
      entry[j] = &p.t.table[(uint64_t)pl.row * p.t.columns + c];
      if (c - pl.from >= pl.end - pl.from) entry[j] = nullptr;
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) page[j] = entry[j] ? (uint32_t)*entry[j] : kNoEntry;
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!entry[j]) continue;
      *entry[j] = DB_PAGE_NONE;
      if (page[j] == kNoEntry) page[j] = kBadEntry;
    }
    uint32_t refs[kRows], times[kRows];  // times: rows from j on that name the page, if j is the first
#pragma unroll
    for (int j = kRows - 1; j >= 0; --j)
      times[j] = j + 1 < (int)kRows && page[j + 1] == page[j] ? times[j + 1] + 1 : 1;
#pragma unroll
    for (int j = kRows - 1; j >= 0; --j) {
      if (page[j] == kNoEntry || (j && page[j] == page[j - 1])) {
        times[j] = 0;
      } else if (page[j] >= p.t.n_pages) {
        times[j] = 0;
        bad = true;
      } else if (times[j] == 1) {
        refs[j] = __ldcg(&p.t.refs[page[j]]);
      } else {  // shared within the unit: likely by others too
        refs[j] = atomicSub(&p.t.refs[page[j]], times[j]);
      }
    }
    // A single reference left is nobody else's to drop, in this call or
    // before: a store does, and most pages have one. The atomics are all under
    // way before the first answer is looked at.
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!times[j]) continue;
      if (times[j] == 1 && refs[j] > 1) {
        refs[j] = atomicSub(&p.t.refs[page[j]], 1u);
      } else if (refs[j] < times[j]) {  // more rows than references
        bad = true;
        if (times[j] > 1) atomicAdd(&p.t.refs[page[j]], times[j]);
      } else if (times[j] == 1) {
        p.t.refs[page[j]] = 0;
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!times[j] || refs[j] != times[j]) continue;
      atomicOr(&p.t.free[page[j] >> 5], 1u << (page[j] & 31));
      ++released;
    }
  }
  *count = released;
  *error = bad;
}

// The same for a row with at most kFewEntries of them, by one thread: where no
// request of a CTA has more (a decode step), units would be almost empty. 4,096
// sequences with 267 pages among them: 10.0 in units, 6.9 so. A gang does it
// so when it is one CTA, which the width of the table decides: a step of 64
// sequences with 256 columns takes 8.1, one of 72, in units of several CTAs,
// 9.8, of 128 11.1 and of 256 11.9.
constexpr uint32_t kFewEntries = 4;

__device__ __forceinline__ void free_few(const Rows& p, const Plan& pl, uint32_t* count,
                                         bool* error) {
  uint32_t released = 0;
  bool bad = false;
  int32_t* const row = &p.t.table[(uint64_t)pl.row * p.t.columns];
  uint32_t page[kFewEntries], refs[kFewEntries];
#pragma unroll
  for (uint32_t k = 0; k < kFewEntries; ++k) {
    page[k] = pl.from + k < pl.end ? (uint32_t)row[pl.from + k] : kBadEntry;
    if (pl.from + k < pl.end && page[k] >= p.t.n_pages) bad = true;
  }
#pragma unroll
  for (uint32_t k = 0; k < kFewEntries; ++k) {
    if (pl.from + k < pl.end) row[pl.from + k] = DB_PAGE_NONE;
    refs[k] = page[k] < p.t.n_pages ? __ldcg(&p.t.refs[page[k]]) : 0;
  }
#pragma unroll
  for (uint32_t k = 0; k < kFewEntries; ++k) {
    if (page[k] >= p.t.n_pages) continue;
    if (refs[k] > 1)
      refs[k] = atomicSub(&p.t.refs[page[k]], 1u);
    else if (refs[k] == 1)
      p.t.refs[page[k]] = 0;
    else
      bad = true;
  }
#pragma unroll
  for (uint32_t k = 0; k < kFewEntries; ++k) {
    if (page[k] >= p.t.n_pages || refs[k] != 1) continue;
    atomicOr(&p.t.free[page[k] >> 5], 1u << (page[k] & 31));
    ++released;
  }
  *count = released;
  *error = bad;
}

// The same, into the counters.
template <typename X>
__device__ __forceinline__ void free_and_count(const Rows& p, const X& x, uint32_t first,
                                               uint32_t stride, uint32_t units) {
  uint32_t released;
  bool bad;
  free_units(p, x, first, stride, units, &released, &bad);
  if (p.ctr) {
    add_count(&p.ctr->total, released);
    add_error(p.ctr, bad);
  }
}

template <uint32_t kThreads>
__global__ void __launch_bounds__(kThreads) page_free_gang_kernel(const FreeParams q) {
  __shared__ TeamShared s_team;
  __shared__ RowPlan<kThreads> s_plan;
  __shared__ Names<kThreads> s_names;
  const Rows& p = q.r;
  Team<kThreads, true> cta(&s_team);
  s_names.clear();
  __syncthreads();
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t i = threadIdx.x;
  const bool mine = i < p.n;
  uint2 r = make_uint2(0, 0);  // sequence, tokens kept
  uint32_t len = 0, at = 0;
  if (mine) r = __ldcg(reinterpret_cast<const uint2*>(&q.req[i]));
  const bool named = mine && r.x < p.t.n_seqs;
  if (named) {
    len = __ldcg(&p.t.length[r.x]);
    at = s_names.place(r.x);
    atomicMin(&s_names.least[at], i);
  }
  __syncthreads();
  const bool ok = named && s_names.least[at] == i;
  const bool cut = ok && r.y < len;
  Plan pl = {0, 0, 0, 0};
  if (cut)
    pl = Plan{r.x, pages_of(r.y, p.t.page_tokens),
              min(pages_of(len, p.t.page_tokens), p.t.columns), 0};
  uint32_t units = 0, entries = 0, released;
  bool bad;
  plan_rows(cta, p, &s_plan, i, mine, pl, &units, &entries);
  const uint32_t invalid = __syncthreads_count(mine && !ok);
  constexpr uint32_t kWarps = kThreads / 32;
  if (gridDim.x == 1 && !__syncthreads_or(pl.end > pl.from + kFewEntries))
    free_few(p, pl, &released, &bad);
  else
    free_units(p, OwnUnits<kThreads>{&s_plan}, i / 32 * gridDim.x + blockIdx.x, gridDim.x * kWarps,
               units, &released, &bad);
  uint64_t total;
  if (!last_of_gang(p.w.head, released, bad, &total, &bad)) return;
  if (cut) p.t.length[r.x] = r.y;
  if (mine && p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
  if (i == 0 && p.ctr)
    *p.ctr = db_counters{total, invalid, 0, bad ? (uint64_t)DB_ERR_PAGE_TABLE : 0};
}

__global__ void __launch_bounds__(kTeamThreads) page_free_team_kernel(const FreeParams q) {
  __shared__ TeamShared s_team;
  __shared__ RowPlan<kTeamThreads> s_plan;
  const Rows& p = q.r;
  Team<kTeamThreads, false> team(&s_team);
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t per = team.per(p.n), at = team.rank * per + threadIdx.x, step = per * team.size;
  const bool one = p.n <= step;  // a thread for every request
  if (p.ctr && team.id() == 0) *p.ctr = db_counters{0, 0, 0, 0};
  db_page_cut r = {0, 0};
  uint32_t len = 0;
  for (uint32_t i = at; threadIdx.x < per && i < p.n; i += step) {
    r = q.req[i];
    len = 0;
    if (r.seq < p.t.n_seqs) {
      claim(p.w.claim, r.seq, i);
      len = __ldcg(&p.t.length[r.seq]);
    }
  }
  team.started();
  team.sync();
  uint32_t units = 0, entries = 0, invalid = 0;
  Plan pl = {0, 0, 0, 0};
  for (uint32_t i0 = 0; i0 < p.n; i0 += step) {
    const uint32_t i = i0 + at;
    const bool mine = threadIdx.x < per && i < p.n;
    pl = Plan{0, 0, 0, 0};
    if (mine) {
      if (!one) {
        r = q.req[i];
        if (r.seq < p.t.n_seqs) len = __ldcg(&p.t.length[r.seq]);
      }
      const bool ok = r.seq < p.t.n_seqs && claimed(p.w.claim, r.seq, i);
      if (ok) {
        p.w.claim[r.seq] = 0;
        if (r.keep < len) {
          pl = Plan{r.seq, pages_of(r.keep, p.t.page_tokens),
                    min(pages_of(len, p.t.page_tokens), p.t.columns), 0};
          p.t.length[r.seq] = r.keep;
        }
      }
      invalid += !ok;
      if (p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    }
    plan_rows(team, p, &s_plan, i, mine, pl, &units, &entries);
  }
  if (p.ctr) add_count(&p.ctr->n_invalid, invalid);
  own_units(team, p, &s_plan, units, entries,
            [&](const OwnUnits<kTeamThreads>& x, uint32_t first, uint32_t stride, uint32_t end) {
              if (one && !__syncthreads_or(pl.end > pl.from + kFewEntries)) {
                uint32_t released;
                bool bad;
                free_few(p, pl, &released, &bad);
                if (p.ctr) {
                  add_count(&p.ctr->total, released);
                  add_error(p.ctr, bad);
                }
              } else {
                free_and_count(p, x, first, stride, end);
              }
            });
}

constexpr uint32_t kUnitThreads = 128;

__global__ void __launch_bounds__(kUnitThreads) page_free_units_kernel(const FreeParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = p.w.head->units, first = (blockIdx.x * kUnitThreads + threadIdx.x) / 32;
  if (blockIdx.x * (kUnitThreads / 32) >= units) return;
  const AllUnits x = all_units(p, s_start);
  free_and_count(p, x, first, gridDim.x * (kUnitThreads / 32), units);
}

// ---------------------------------------------------------------------- fork
struct ForkParams {
  Rows r;
  const db_page_fork_req* req;
};

// The child's row is the parent's, refs[p] += the children that take p. 32
// forks of 44 pages take 4.4, 1,023 of 1,024 pages (4 MB of tables written)
// 5.1 + 6.4 for the plan and the units.
template <typename X>
__device__ __forceinline__ bool fork_units(const Rows& p, const X& x, uint32_t first,
                                           uint32_t stride, uint32_t units) {
  const uint32_t lane = threadIdx.x & 31;
  bool bad = false;
  for (uint32_t u = first; u < units; u += stride) {
    const auto at = x.find(u);
    const uint32_t c = at.base + lane;
    const int32_t* from[kRows];
    int32_t* to[kRows];
    uint32_t page[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const Plan pl = at.row(j);
      from[j] = &p.t.table[(uint64_t)pl.aux * p.t.columns + c];
      to[j] = c < pl.end ? &p.t.table[(uint64_t)pl.row * p.t.columns + c] : nullptr;
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) page[j] = to[j] ? (uint32_t)*from[j] : kNoEntry;
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!to[j]) continue;
      *to[j] = (int32_t)page[j];
      if (page[j] >= p.t.n_pages) {
        bad = true;
        page[j] = kNoEntry;
      }
    }
    uint32_t times = 0;
#pragma unroll
    for (int j = kRows - 1; j >= 0; --j) {
      ++times;
      if (j && page[j] == page[j - 1]) continue;
      if (page[j] != kNoEntry) atomicAdd(&p.t.refs[page[j]], times);
      times = 0;
    }
  }
  return bad;
}

template <uint32_t kThreads>
__global__ void __launch_bounds__(kThreads) page_fork_gang_kernel(const ForkParams q) {
  __shared__ TeamShared s_team;
  __shared__ RowPlan<kThreads> s_plan;
  __shared__ Names<kThreads> s_names;
  const Rows& p = q.r;
  Team<kThreads, true> cta(&s_team);
  s_names.clear();
  __syncthreads();
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t i = threadIdx.x;
  const bool mine = i < p.n;
  uint4 r = make_uint4(0, 0, 0, 0);  // parent, child, tokens
  uint32_t held = 0, of = 0, at = 0;  // the child's and the parent's lengths
  if (mine) r = __ldcg(reinterpret_cast<const uint4*>(&q.req[i]));
  const bool named = mine && r.y < p.t.n_seqs;
  if (named) {
    held = __ldcg(&p.t.length[r.y]);
    if (r.x < p.t.n_seqs) of = __ldcg(&p.t.length[r.x]);
    at = s_names.place(r.y);
    atomicMin(&s_names.least[at], i);
  }
  __syncthreads();
  const bool ok = named && s_names.least[at] == i && r.x < p.t.n_seqs && r.x != r.y && held == 0 &&
                  r.z <= of;
  Plan pl = {0, 0, 0, 0};
  if (ok) pl = Plan{r.y, 0, min(pages_of(r.z, p.t.page_tokens), p.t.columns), r.x};
  uint32_t units = 0, entries = 0;
  plan_rows(cta, p, &s_plan, i, mine, pl, &units, &entries);
  const uint32_t invalid = __syncthreads_count(mine && !ok);
  constexpr uint32_t kWarps = kThreads / 32;
  bool bad = fork_units(p, OwnUnits<kThreads>{&s_plan}, i / 32 * gridDim.x + blockIdx.x,
                        gridDim.x * kWarps, units);
  uint64_t none;
  if (!last_of_gang(p.w.head, 0, bad, &none, &bad)) return;
  if (ok) p.t.length[r.y] = r.z;
  if (mine && p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
  if (i == 0 && p.ctr)
    *p.ctr = db_counters{entries, invalid, 0, bad ? (uint64_t)DB_ERR_PAGE_TABLE : 0};
}

__global__ void __launch_bounds__(kTeamThreads) page_fork_team_kernel(const ForkParams q) {
  __shared__ TeamShared s_team;
  __shared__ RowPlan<kTeamThreads> s_plan;
  const Rows& p = q.r;
  Team<kTeamThreads, false> team(&s_team);
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t per = team.per(p.n), at = team.rank * per + threadIdx.x, step = per * team.size;
  const bool one = p.n <= step;  // a thread for every request
  if (p.ctr && team.id() == 0) *p.ctr = db_counters{0, 0, 0, 0};
  db_page_fork_req r = {0, 0, 0, 0};
  uint32_t held = 0, of = 0;  // the child's and the parent's lengths
  auto look = [&](uint32_t i) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(&q.req[i]));
    r = db_page_fork_req{v.x, v.y, v.z, v.w};
    held = r.child < p.t.n_seqs ? __ldcg(&p.t.length[r.child]) : 0;
    of = r.parent < p.t.n_seqs ? __ldcg(&p.t.length[r.parent]) : 0;
  };
  for (uint32_t i = at; threadIdx.x < per && i < p.n; i += step) {
    look(i);
    if (r.child < p.t.n_seqs) claim(p.w.claim, r.child, i);
  }
  team.started();
  team.sync();
  uint32_t units = 0, entries = 0, invalid = 0;
  uint64_t taken = 0;
  Plan pl;
  for (uint32_t i0 = 0; i0 < p.n; i0 += step) {
    const uint32_t i = i0 + at;
    const bool mine = threadIdx.x < per && i < p.n;
    pl = Plan{kNoMove, 0, 0, 0};
    if (mine) {
      if (!one) look(i);
      bool ok = false;
      if (r.child < p.t.n_seqs && claimed(p.w.claim, r.child, i)) {
        p.w.claim[r.child] = 0;
        ok = r.parent < p.t.n_seqs && r.parent != r.child && held == 0 && r.tokens <= of;
      }
      if (ok) {
        pl = Plan{r.child, 0, min(pages_of(r.tokens, p.t.page_tokens), p.t.columns), r.parent};
        taken += pl.end;
      }
      invalid += !ok;
      if (p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    }
    plan_rows(team, p, &s_plan, i, mine, pl, &units, &entries);
  }
  if (p.ctr) {
    add_count(&p.ctr->n_invalid, invalid);
    const uint64_t c = warp_sum64(taken);
    if ((threadIdx.x & 31) == 0 && c)
      atomicAdd((unsigned long long*)&p.ctr->total, (unsigned long long)c);
  }
  // Every length was read before the last scan's barrier.
  if (one) {
    if (threadIdx.x < per && at < p.n && pl.row != kNoMove) p.t.length[pl.row] = r.tokens;
  } else {
    for (uint32_t i = at; threadIdx.x < per && i < p.n; i += step) {
      const uint32_t row = p.w.plan[i].row;
      if (row != kNoMove) p.t.length[row] = q.req[i].tokens;
    }
  }
  own_units(team, p, &s_plan, units, entries,
            [&](const OwnUnits<kTeamThreads>& x, uint32_t first, uint32_t stride, uint32_t end) {
              const bool bad = fork_units(p, x, first, stride, end);
              if (p.ctr) add_error(p.ctr, bad);
            });
}

__global__ void __launch_bounds__(kUnitThreads) page_fork_units_kernel(const ForkParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = p.w.head->units, first = (blockIdx.x * kUnitThreads + threadIdx.x) / 32;
  if (blockIdx.x * (kUnitThreads / 32) >= units) return;
  const AllUnits x = all_units(p, s_start);
  const bool bad = fork_units(p, x, first, gridDim.x * (kUnitThreads / 32), units);
  if (p.ctr) add_error(p.ctr, bad);
}

// -------------------------------------------------------------------- extend
struct ExtendParams {
  db_page_tables t;
  const db_page_grow* req;
  uint32_t n;
  db_page_move* moves;
  uint32_t* n_moves;
  uint8_t* status;
  db_counters* ctr;
  bool rest;  // a second kernel follows
  Work w;
};

// What a request asks for, from the state before the call.
struct Ask {
  uint32_t seq, now;  // its row, and its length after
  uint32_t had;       // pages before
  uint32_t grow;      // pages after - before
  uint32_t part;      // tokens in a partly filled last page that it adds to, or 0
  uint32_t last;      // that page
  uint32_t refs;      // its references
  bool named, fits, mine, ok, corrupt;
  __device__ __forceinline__ bool shares() const { return part && refs > 1; }
};

// Its sequence and pages, before it is known whose the sequence is;
__device__ __forceinline__ Ask ask(const ExtendParams& p, uint32_t i, bool any) {
  Ask a = {0, 0, 0, 0, 0, 0, 0, false, false, false, false, false};
  if (!any) return a;
  const uint2 r = __ldcg(reinterpret_cast<const uint2*>(&p.req[i]));
  a.seq = r.x;
  a.named = a.seq < p.t.n_seqs;
  if (!a.named) return a;
  const uint32_t len = __ldcg(&p.t.length[a.seq]), part = len % p.t.page_tokens;
  const uint64_t now = (uint64_t)len + r.y;
  a.fits = now <= (uint64_t)p.t.columns * p.t.page_tokens && now <= 0xFFFFFFFFull;
  if (!a.fits) return a;
  a.had = pages_of(len, p.t.page_tokens);
  a.now = (uint32_t)now;
  a.grow = pages_of(now, p.t.page_tokens) - a.had;
  if (r.y && part) {
    a.part = part;
    a.last = (uint32_t)__ldcg(&p.t.table[(uint64_t)a.seq * p.t.columns + a.had - 1]);
    a.corrupt = a.last >= p.t.n_pages;
    if (!a.corrupt) a.refs = __ldcg(&p.t.refs[a.last]);
  }
  return a;
}

// and with that.
__device__ __forceinline__ void settle(Ask* a, bool first) {
  a->mine = a->named && first;
  a->ok = a->mine && a->fits && !a->corrupt;
  a->corrupt &= a->mine;
  if (!a->ok) a->grow = a->part = 0;
}

struct PlanStart {
  const Plan* plan;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return plan[i].end; }
};

// Page e of the batch: the e-th free one, into the row it is for.
__device__ __forceinline__ void place_pages(const ExtendParams& p, const Finder& request,
                                            const Plan* plan, const Finder& word,
                                            const uint32_t* before, const uint32_t* bits,
                                            uint32_t first, uint32_t stride, uint32_t total) {
  for (uint32_t e = first; e < total; e += stride) {
    const uint32_t w = word.find(e, WordStart{before});
    const uint32_t page = 32 * w + nth_bit(bits[w], e - before[w]);
    const Plan pl = ld_plan(&plan[request.find(e, PlanStart{plan})]);
    const uint32_t j = e - pl.end;
    p.t.table[(uint64_t)pl.row * p.t.columns + pl.from + j] = (int32_t)page;
    p.t.refs[page] = 1;
    if (j == 0 && pl.aux != kNoMove) p.moves[pl.aux].dst = page;
  }
}

// What is left of a quad of free words when the batch takes `need` pages;
// *used: words up to the last one used, if that is in it.
__device__ __forceinline__ uint4 left_of(const uint4& v, const uint4& before, uint32_t need,
                                         uint32_t* used, uint32_t w) {
  if (before.w + __popc(v.w) < need) return make_uint4(0, 0, 0, 0);
  const uint32_t vs[4] = {v.x, v.y, v.z, v.w}, bs[4] = {before.x, before.y, before.z, before.w};
  uint32_t ls[4];
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {
    ls[k] = 0;
    if (bs[k] >= need) {
      ls[k] = vs[k];
    } else if (bs[k] + __popc(vs[k]) >= need) {
      ls[k] = vs[k] & ~((2u << nth_bit(vs[k], need - bs[k] - 1)) - 1);
      *used = w + k + 1;
    }
  }
  return make_uint4(ls[0], ls[1], ls[2], ls[3]);
}

// The e-th free page, found in the free words: the thread whose share has it,
// and then the quad of that share. (Writing the list of all pages taken first,
// word by word, took 25 for 320,000 pages, which were then placed in 5.)
template <uint32_t kThreads>
__device__ __forceinline__ uint32_t nth_page(const uint32_t* bits, uint32_t n_pages,
                                             const uint32_t* s_first, uint32_t quads, uint32_t e) {
  uint32_t lo = 0, hi = kThreads;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (s_first[mid] <= e) lo = mid; else hi = mid;
  }
  uint32_t w = lo * quads * 4;
  e -= s_first[lo];
  const uint32_t all = (n_pages + 31) / 32;
  for (uint32_t s = 0; s < quads; ++s, w += 4) {
    const uint4 v = ld_quad(bits, w, all, n_pages);
    const uint32_t x = __popc(v.x), y = x + __popc(v.y), z = y + __popc(v.z), end = z + __popc(v.w);
    if (e < end) {
      if (e < x) return 32 * w + nth_bit(v.x, e);
      if (e < y) return 32 * (w + 1) + nth_bit(v.y, e - x);
      if (e < z) return 32 * (w + 2) + nth_bit(v.z, e - y);
      return 32 * (w + 3) + nth_bit(v.w, e - z);
    }
    e -= end;
  }
  return n_pages;  // not reached: e is below the free pages counted
}

// A request needs ceil((length + tokens) / T) - ceil(length / T) pages, and one
// for a copy when it adds to a page that others hold: all of a page's holders
// but the last when all are in the batch, else all of them. Start of request i
// = the needs before it; page e of the batch = the e-th free one. 5.3 for 48
// sequences, 10.1 for 192 times 512 pages, 10.5 for 1,023 holders of one page
// that all copy it.
template <uint32_t kThreads>
__global__ void __launch_bounds__(kThreads) page_extend_gang_kernel(const ExtendParams p) {
  __shared__ TeamShared s_team;
  __shared__ Names<kThreads> s_names;
  __shared__ Plan s_plan[kThreads];
  __shared__ uint32_t s_first[kThreads];  // free pages before each thread's share of the words
  Team<kThreads, true> cta(&s_team);
  s_names.clear();
  __syncthreads();
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t i = threadIdx.x;
  const bool mine = i < p.n;
  Bits bits = load_free(cta, p.t.free, p.t.n_pages);
  Ask a = ask(p, i, mine);
  uint32_t at = 0;
  if (a.named) {
    at = s_names.place(a.seq);
    atomicMin(&s_names.least[at], i);
  }
  const bool shares = scan_free(cta, bits, p.t.free, p.t.n_pages, a.shares());
  settle(&a, a.named && s_names.least[at] == i);
  uint32_t need, n_moves = 0, rank = 0, start;
  bool cow = false;
  if (shares) {
    // How many of the batch's requests hold each shared page, and the last of them.
    __syncthreads();
    s_names.clear();
    __syncthreads();
    if (a.shares()) {
      at = s_names.place(a.last);
      atomicAdd(&s_names.count[at], 1u);
      atomicMin(&s_names.least[at], ~i);
    }
    __syncthreads();
    if (a.shares()) cow = !(s_names.count[at] == a.refs && s_names.least[at] == ~i);
    start = cta.template scan<true>(a.grow + cow, &need, cow, &n_moves, &rank);
  } else {
    start = cta.template scan<false>(a.grow, &need);
  }
  s_plan[i] = Plan{a.seq, a.had - cow, start, cow ? rank : kNoMove};
  s_first[i] = bits.before;
  const bool go = need <= bits.total;
  const uint32_t invalid = __syncthreads_count(mine && !a.ok);
  const bool corrupt = __syncthreads_or(a.corrupt);
  if (go)
    for (uint32_t e = (i / 32 * gridDim.x + blockIdx.x) * 32 + i % 32; e < need;
         e += gridDim.x * kThreads) {
      uint32_t lo = 0, hi = kThreads;
      while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (s_plan[mid].end <= e) lo = mid; else hi = mid;
      }
      const Plan pl = s_plan[lo];
      const uint32_t j = e - pl.end;
      if (j == 0 && pl.aux != kNoMove) continue;  // replaces an entry that a CTA may yet read
      const uint32_t page = nth_page<kThreads>(p.t.free, p.t.n_pages, s_first, bits.quads, e);
      p.t.table[(uint64_t)pl.row * p.t.columns + pl.from + j] = (int32_t)page;
      p.t.refs[page] = 1;
    }
  if (!last_of_gang(p.w.head)) return;
  const uint32_t copiers = __ballot_sync(kFull, cow && go);
  if (cow && go) {
    const uint32_t page = nth_page<kThreads>(p.t.free, p.t.n_pages, s_first, bits.quads, start);
    p.t.table[(uint64_t)a.seq * p.t.columns + a.had - 1] = (int32_t)page;
    p.t.refs[page] = 1;
    *reinterpret_cast<uint4*>(&p.moves[rank]) = make_uint4(a.last, page, a.part, 0);
    const uint32_t same = __match_any_sync(copiers, a.last);
    if ((same & lanemask_lt()) == 0) atomicSub(&p.t.refs[a.last], (uint32_t)__popc(same));
  }
  if (a.ok && go) p.t.length[a.seq] = a.now;
  if (mine && p.status) p.status[i] = !a.ok ? DB_PAGE_INVALID : go ? DB_PAGE_OK : DB_PAGE_SHORT;
  if (i == 0) {
    *p.n_moves = go ? n_moves : 0;
    if (p.ctr)
      *p.ctr = db_counters{need, invalid, go ? 0 : p.n - invalid,
                           corrupt ? (uint64_t)DB_ERR_PAGE_TABLE : 0};
  }
  __syncthreads();  // the pages are found
  if (go && bits.before < need)
    each_quad(bits, p.t.free, p.t.n_pages, [&](uint32_t w, const uint4& v, const uint4& before) {
      if (before.x >= need) return false;
      uint32_t used;
      st_quad(p.t.free, w, (p.t.n_pages + 31) / 32, left_of(v, before, need, &used, w));
      return true;
    });
}

__global__ void __launch_bounds__(kTeamThreads) page_extend_team_kernel(const ExtendParams p) {
  constexpr uint32_t kThreads = kTeamThreads, kWords = kTeamWords;
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kThreads];
  __shared__ Plan s_plan[kThreads];
  __shared__ __align__(16) uint32_t s_before[kWords], s_bits[kWords];
  __shared__ uint32_t s_used, s_end;
  Team<kThreads, false> team(&s_team);
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t id = team.id(), words = (p.t.n_pages + 31) / 32;
  const uint32_t per = team.per(p.n), at = team.rank * per + threadIdx.x;
  const uint32_t step = per * team.size;
  const bool one = p.n <= step;  // a thread for every request, which asks once
  Bits bits = load_free(team, p.t.free, p.t.n_pages);
  if (p.ctr && id == 0) *p.ctr = db_counters{0, 0, 0, 0};
  Ask a = ask(p, at, false);
  bool shares = false;
  for (uint32_t i = at; threadIdx.x < per && i < p.n; i += step) {
    a = ask(p, i, true);
    if (a.named) claim(p.w.claim, a.seq, i);
    shares |= a.shares();
  }
  team.started();
  // Also the barrier after the claims, and whether any request may share.
  shares = scan_free(team, bits, p.t.free, p.t.n_pages, shares);
  if (one && at < p.n && threadIdx.x < per) settle(&a, a.named && claimed(p.w.claim, a.seq, at));
  if (shares) {
    // How many of the batch's requests hold each shared page, and the last of
    // them; requests of a warp that hold the same one (samples of one prompt)
    // count together. (Whole warps take part in every round, so that a vote
    // can name the lanes of each match.)
    for (uint32_t i0 = 0; i0 < p.n; i0 += step) {
      const uint32_t i = i0 + at;
      if (!one) {
        const bool mine = threadIdx.x < per && i < p.n;
        a = ask(p, i, mine);
        if (mine) settle(&a, a.named && claimed(p.w.claim, a.seq, i));
      }
      const uint32_t sharers = __ballot_sync(kFull, a.shares());
      if (a.shares()) {
        const uint32_t same = __match_any_sync(sharers, a.last);
        if ((same & lanemask_lt()) == 0) {
          atomicAdd(&p.w.holders[a.last], (uint32_t)__popc(same));
          atomicMax(&p.w.latest[a.last], i + (31 - __clz(same)) - (threadIdx.x & 31));
        }
      }
    }
    team.sync();
  }
  uint32_t need = 0, n_moves = 0, move = kNoMove;
  for (uint32_t i0 = 0; i0 < p.n; i0 += step) {
    const uint32_t i = i0 + at;
    const bool mine = threadIdx.x < per && i < p.n;
    if (!one) {
      a = ask(p, i, mine);
      if (mine) settle(&a, a.named && claimed(p.w.claim, a.seq, i));
    }
    bool cow = false;
    uint32_t total, copies = 0, rank = 0, x;
    if (shares) {
      if (a.shares())
        cow = !(__ldcg(&p.w.holders[a.last]) == a.refs && __ldcg(&p.w.latest[a.last]) == i);
      x = team.template scan<true>(a.grow + cow, &total, cow, &copies, &rank);
    } else {
      x = team.template scan<false>(a.grow, &total);
    }
    move = cow ? n_moves + rank : kNoMove;
    const Plan pl = {a.seq, a.had - cow, need + x, move};
    s_plan[threadIdx.x] = pl;
    s_start[threadIdx.x] = pl.end;
    if (threadIdx.x == kThreads - 1) s_end = pl.end + a.grow + cow;
    if (mine && (p.rest || !one)) st_plan(&p.w.plan[i], pl);
    need += total;
    n_moves += copies;
  }
  const bool go = need <= bits.total;
  // The team places few pages, each CTA those of its requests: not when it
  // plans in more than one round, or needs more words than it keeps.
  const bool few = !p.rest || (one && need <= kOwnPages);
  if (id == 0) {
    *p.n_moves = go ? n_moves : 0;
    if (p.ctr) p.ctr->total = need;
  }
  // The words up to the last one used as they were, to find the pages in, and
  // without those taken.
  if (go && need && bits.before < need)
    each_quad(bits, p.t.free, p.t.n_pages, [&](uint32_t w, const uint4& v, const uint4& before) {
      if (before.x >= need) return false;
      st_quad(p.w.before, w, words, before);
      st_quad(p.w.bits, w, words, v);
      uint32_t used = 0;
      const uint4 left = left_of(v, before, need, &used, w);
      if (used) {
        team.to_all(&s_used, used);
        p.w.head->used = used;
      }
      st_quad(p.t.free, w, words, left);
      return true;
    });
  // Every request has been asked before the last scan. Lengths, moves and
  // status, and the workspace as the next call wants it.
  uint32_t invalid = 0, refused = 0;
  bool corrupt = false;
  for (uint32_t i0 = 0; i0 < p.n; i0 += step) {
    const uint32_t i = i0 + at;
    const bool mine = threadIdx.x < per && i < p.n;
    if (!one) {
      a = ask(p, i, mine);
      move = kNoMove;
      if (mine) {
        settle(&a, a.named && claimed(p.w.claim, a.seq, i));
        move = p.w.plan[i].aux;
      }
    }
    const uint32_t copiers = __ballot_sync(kFull, move != kNoMove);
    if (move != kNoMove) {  // at least one holder of every shared page copies, and clears for all
      p.w.holders[a.last] = 0;
      p.w.latest[a.last] = 0;
      if (go) {
        const uint32_t same = __match_any_sync(copiers, a.last);
        if ((same & lanemask_lt()) == 0) atomicSub(&p.t.refs[a.last], (uint32_t)__popc(same));
        p.moves[move].src = a.last;
        *reinterpret_cast<uint2*>(&p.moves[move].tokens) = make_uint2(a.part, 0);
      }
    }
    if (a.mine) p.w.claim[a.seq] = 0;
    if (a.ok && go) p.t.length[a.seq] = a.now;
    invalid += mine && !a.ok;
    refused += a.ok && !go;
    corrupt |= a.corrupt;
    if (mine && p.status) p.status[i] = !a.ok ? DB_PAGE_INVALID : go ? DB_PAGE_OK : DB_PAGE_SHORT;
  }
  if (p.ctr) {
    add_count(&p.ctr->n_invalid, invalid);
    add_count(&p.ctr->n_overflow, refused);
    add_error(p.ctr, corrupt);
  }
  team.sync();  // words are known, and the replaced entries have been read
  const uint32_t used = go && need ? s_used : 0;
  const bool own = few && used <= kWords;
  if (p.rest && id == 0) p.w.head->units = go && !own ? need : 0;
  if (!used || !own) return;
  for (uint32_t w = threadIdx.x; w < used; w += kThreads) {
    s_before[w] = p.w.before[w];
    s_bits[w] = p.w.bits[w];
  }
  __syncthreads();
  place_pages(p, Finder{s_start, kThreads, kThreads, 1}, s_plan, Finder{s_before, used, used, 1},
              s_before, s_bits, s_start[0] + threadIdx.x, kThreads, s_end);
}

constexpr uint32_t kPlaceThreads = 256;

__global__ void __launch_bounds__(kPlaceThreads) page_place_kernel(const ExtendParams p) {
  __shared__ uint32_t s_start[kSearch], s_word[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t total = p.w.head->units, used = p.w.head->used;
  if (blockIdx.x * kPlaceThreads >= total) return;
  const Finder r = load_finder(s_start, kSearch, p.n, PlanStart{p.w.plan});
  const Finder f = load_finder(s_word, kSearch, used, WordStart{p.w.before});
  __syncthreads();
  place_pages(p, r, p.w.plan, f, p.w.before, p.w.bits, blockIdx.x * kPlaceThreads + threadIdx.x,
              gridDim.x * kPlaceThreads, total);
}

// ------------------------------------------------------------------- compact
struct CompactParams {
  db_page_tables t, out;
  db_page_move* moves;
  uint32_t cap;
  uint32_t* n_moves;
  db_counters* ctr;
  bool rest;   // moves are left to a second kernel
  bool whole;  // the planning CTA does everything
  Work w;
};

// 131,072 pages, 32,000 moves, 1,024 rows of 512 entries: 12 for plan, moves
// and tables together, beside 628 for the moves' 4.25 GB. Listing free and live
// pages word by word in one CTA first took 50.
//
// Live pages before a word.
struct LiveStart {
  const uint32_t* before;
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const { return 32 * w - before[w]; }
};

// Move k: the k-th free page gets the k-th live one from above.
__device__ __forceinline__ void make_moves(const CompactParams& p, uint32_t* s_word,
                                           uint32_t* s_live, uint32_t n_live, uint32_t moved,
                                           uint32_t first, uint32_t stride) {
  const uint32_t words = (p.t.n_pages + 31) / 32;
  const Finder f = load_finder(s_word, kSearch, words, WordStart{p.w.before});
  const Finder g = load_finder(s_live, kSearch, words, LiveStart{p.w.before});
  __syncthreads();
  for (uint32_t k = first; k < moved; k += stride) {
    const uint32_t v = f.find(k, WordStart{p.w.before});
    const uint32_t dst = 32 * v + nth_bit(ld_word(p.t.free, v, p.t.n_pages), k - p.w.before[v]);
    const uint32_t e = n_live - 1 - k, w = g.find(e, LiveStart{p.w.before});
    const uint32_t src =
        32 * w + nth_bit(~ld_word(p.t.free, w, p.t.n_pages), e - (32 * w - p.w.before[w]));
    *reinterpret_cast<uint4*>(&p.moves[k]) = make_uint4(src, dst, DB_PAGE_ALL, 0);
    p.w.renamed[src] = dst;
    p.out.refs[dst] = p.t.refs[src];
    p.out.refs[src] = 0;
    if (k == moved - 1) {
      p.w.head->dst_last = dst;
      p.w.head->src_first = src;
    }
  }
}

// An array of n words from `in` to `out` through f, four at a time where both
// are aligned. f(index, word) may have out's word left as it is by `keep`.
template <typename F>
__device__ __forceinline__ void rewrite(const uint32_t* in, uint32_t* out, uint64_t n, uint64_t id,
                                        uint64_t step, F f) {
  uint64_t done = 0;
  if ((((uintptr_t)in | (uintptr_t)out) & 15) == 0) {
    done = n & ~3ull;
    for (uint64_t q = 4 * id; q < done; q += 4 * step) {
      const uint4 was = *reinterpret_cast<const uint4*>(in + q);
      uint4 is = was;
      bool skip = false;
      f(q, &is.x, &skip);
      f(q + 1, &is.y, &skip);
      f(q + 2, &is.z, &skip);
      f(q + 3, &is.w, &skip);
      if (skip) {  // words that are written elsewhere: each for itself
        for (uint32_t k = 0; k < 4; ++k) {
          uint32_t v = k == 0 ? was.x : k == 1 ? was.y : k == 2 ? was.z : was.w;
          bool leave = false;
          f(q + k, &v, &leave);
          if (!leave) out[q + k] = v;
        }
      } else if (in != out || is.x != was.x || is.y != was.y || is.z != was.z || is.w != was.w) {
        *reinterpret_cast<uint4*>(out + q) = is;
      }
    }
  }
  for (uint64_t q = done + id; q < n; q += step) {
    const uint32_t was = in[q];
    uint32_t is = was;
    bool skip = false;
    f(q, &is, &skip);
    if (!skip && (in != out || is != was)) out[q] = is;
  }
}

// Tables, references, free bits and lengths after the moves.
__device__ __forceinline__ void apply_moves(const CompactParams& p, uint32_t moved,
                                            uint32_t src_first, uint32_t dst_last, uint64_t id,
                                            uint64_t step) {
  const uint32_t n_pages = p.t.n_pages, words = (n_pages + 31) / 32;
  bool bad = false;
  rewrite((const uint32_t*)p.t.table, (uint32_t*)p.out.table, (uint64_t)p.t.n_seqs * p.t.columns,
          id, step, [&](uint64_t, uint32_t* v, bool*) {
            if (*v >= src_first && *v != (uint32_t)DB_PAGE_NONE) {
              if (*v < n_pages) *v = p.w.renamed[*v]; else bad = true;
            }
          });
  if (p.ctr) add_error(p.ctr, bad);
  if (p.out.refs != p.t.refs)
    rewrite(p.t.refs, p.out.refs, n_pages, id, step, [&](uint64_t q, uint32_t* v, bool* skip) {
      if (q >= src_first)
        *v = 0;
      else if (!*v && moved && q <= dst_last)
        *skip = true;  // moved to: written with the move
    });
  for (uint64_t w = id; w < words; w += step) {
    uint32_t v = p.t.free[w];
    const uint64_t at = 32 * w;
    if (moved) {
      if (at + 31 <= dst_last)
        v = 0;
      else if (at <= dst_last)
        v &= ~((2u << (dst_last - at)) - 1);
      if (at >= src_first)
        v = kFull;
      else if (at + 31 >= src_first)
        v |= ~((1u << (src_first - at)) - 1);
    }
    if (w == words - 1 && (n_pages & 31)) v &= (1u << (n_pages & 31)) - 1;
    p.out.free[w] = v;
  }
  if (p.out.length != p.t.length)
    for (uint64_t s = id; s < p.t.n_seqs; s += step) p.out.length[s] = p.t.length[s];
}

template <uint32_t kThreads, bool kSolo>
__global__ void __launch_bounds__(kThreads) page_compact_plan_kernel(const CompactParams p) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_word[kSearch], s_live[kSearch];
  Team<kThreads, kSolo> team(&s_team);
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t id = team.id(), n_pages = p.t.n_pages, words = (n_pages + 31) / 32;
  Bits bits = load_free(team, p.t.free, n_pages);
  team.started();
  scan_free(team, bits, p.t.free, n_pages, false);
  const uint32_t n_live = n_pages - bits.total;
  // M, the free pages below n_live: known to the thread that has the word.
  each_quad(bits, p.t.free, n_pages, [&](uint32_t w, const uint4& v, const uint4& before) {
    st_quad(p.w.before, w, words, before);
    if (n_live / 32 >= w && n_live / 32 < w + 4) {
      const uint32_t k = n_live / 32 - w, x = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
      p.w.head->holes = (k == 0 ? before.x : k == 1 ? before.y : k == 2 ? before.z : before.w) +
                        __popc(x & ((1u << (n_live & 31)) - 1));
    }
    return true;
  });
  team.sync();
  const uint32_t holes = n_live == n_pages ? 0 : __ldcg(&p.w.head->holes);
  const uint32_t moved = min(holes, p.cap);
  if (id == 0) {
    *p.n_moves = moved;
    p.w.head->moved = moved;
    p.w.head->n_live = n_live;
    if (moved == 0) {
      p.w.head->src_first = n_pages;
      p.w.head->dst_last = 0;
    }
    if (p.ctr) *p.ctr = db_counters{holes, 0, (uint64_t)holes - moved, 0};
  }
  if (p.rest) return;
  if (moved) make_moves(p, s_word, s_live, n_live, moved, id, team.threads());
  if (!kSolo || !p.whole) return;
  __syncthreads();
  apply_moves(p, moved, p.w.head->src_first, p.w.head->dst_last, id, kThreads);
}

__global__ void __launch_bounds__(256) page_compact_moves_kernel(const CompactParams p) {
  __shared__ uint32_t s_word[kSearch], s_live[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t moved = p.w.head->moved;
  if (blockIdx.x * 256 >= moved) return;
  make_moves(p, s_word, s_live, p.w.head->n_live, moved, blockIdx.x * 256 + threadIdx.x,
             gridDim.x * 256);
}

__global__ void __launch_bounds__(256) page_compact_apply_kernel(const CompactParams p) {
  wait_for_prerequisites();
  dependents_may_launch();
  apply_moves(p, p.w.head->moved, p.w.head->src_first, p.w.head->dst_last,
              (uint64_t)blockIdx.x * 256 + threadIdx.x, (uint64_t)gridDim.x * 256);
}

// ---------------------------------------------------------------- host side
template <typename P>
int launch_team(void (*kernel)(P), uint32_t ctas, uint32_t threads, cudaStream_t s,
                const P& params) {
  if (ctas == 1) return launch_dependent(kernel, 1, threads, 0, s, params);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_result();
}

int check_tables(const db_page_tables* t) {
  if (!t || !t->table || !t->length || !t->refs || !t->free) return -EINVAL;
  if (!aligned(t->table, 4) || !aligned(t->length, 4) || !aligned(t->refs, 4) ||
      !aligned(t->free, 16))
    return -EINVAL;
  if (!t->n_seqs || !t->columns || !t->n_pages || !t->page_tokens) return -EINVAL;
  if (t->n_pages > 0x7FFFFFFFu || t->n_seqs > 0x7FFFFFFFu) return -EINVAL;
  return 0;
}

int check_call(const db_page_tables* t, const void* req, uintptr_t req_align, uint32_t n,
               const db_counters* ctr, void* ws, size_t ws_bytes, Work* w) {
  const int rc = check_tables(t);
  if (rc) return rc;
  if (!ws || !aligned(ws, 256) || !aligned(ctr, 8)) return -EINVAL;
  if (n && (!req || !aligned(req, req_align))) return -EINVAL;
  if (n > t->n_seqs) return -EINVAL;
  if ((uint64_t)n * t->columns > 0xFFFFFFFFull) return -EINVAL;  // entries are counted in 32 bits
  if (ws_bytes < carve(nullptr, t->n_seqs, t->n_pages, nullptr)) return -ENOSPC;
  carve((char*)ws, t->n_seqs, t->n_pages, w);
  return 0;
}

// A call without requests zeroes what it would count.
int nothing(db_counters* ctr, uint32_t* n_moves, cudaStream_t s) {
  if (ctr) {
    const cudaError_t e = cudaMemsetAsync(ctr, 0, sizeof(*ctr), s);
    if (e != cudaSuccess) return cuda_failure(e);
  }
  if (n_moves) {
    const cudaError_t e = cudaMemsetAsync(n_moves, 0, sizeof(*n_moves), s);
    if (e != cudaSuccess) return cuda_failure(e);
  }
  return 0;
}

inline uint32_t most_of(uint32_t a, uint32_t b) { return a > b ? a : b; }

// CTAs of a team that wants `threads`.
uint32_t team_size(uint64_t threads) {
  uint32_t c = 1;
  while (c < kMaxTeam && (uint64_t)c * kTeamThreads < threads) c *= 2;
  return c;
}

// CTAs of `block` threads for at most `threads`, at most `each` an SM.
unsigned whole_grid(uint64_t threads, uint32_t block, uint32_t each) {
  const uint64_t want = (threads + block - 1) / block, most = (uint64_t)each * num_sms();
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

// CTAs of a gang with at most `pieces` pieces, `each` of which a CTA does at a
// time: one where they are few, else up to `most` an SM.
unsigned gang_size(uint64_t pieces, uint64_t few, uint32_t each, uint32_t most) {
  if (pieces <= few) return 1;
  const uint64_t want = (pieces + each - 1) / each, all = (uint64_t)most * num_sms();
  return (unsigned)(want < all ? want : all);
}

// Free and fork: a gang, or a team and then the whole GPU where there may be
// much to do.
template <typename P>
int launch_rows(void (*gang)(P), void (*team)(P), void (*rest)(P), cudaStream_t s, P& p) {
  const uint64_t units = ((uint64_t)p.r.n + kRows - 1) / kRows * (((uint64_t)p.r.t.columns + 31) / 32);
  if (p.r.n <= kSmallThreads)
    return launch_dependent(gang, gang_size(units, kRestUnits, kSmallThreads / 32, 2), kSmallThreads, 0, s, p);
  const uint32_t ctas = most_of(team_size(4 * (uint64_t)p.r.n), 2);
  p.r.rest = units > kRestUnits || p.r.n > ctas * kTeamThreads;
  const int e = launch_team(team, ctas, kTeamThreads, s, p);
  if (e || !p.r.rest) return e;
  return launch_dependent(rest, whole_grid(units * 32, kUnitThreads, 8), kUnitThreads, 0, s, p);
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_page_workspace_size(uint32_t n_seqs, uint32_t n_pages, size_t* bytes) {
  if (!bytes || !n_seqs || !n_pages || n_seqs > 0x7FFFFFFFu || n_pages > 0x7FFFFFFFu) return -EINVAL;
  *bytes = carve(nullptr, n_seqs, n_pages, nullptr);
  return 0;
}

extern "C" int db_page_free(const db_page_tables* t, const db_page_cut* req, uint32_t n,
                            uint8_t* status, db_counters* ctr, void* ws, size_t ws_bytes,
                            void* stream) {
  FreeParams p = {};
  const int rc = check_call(t, req, sizeof(*req), n, ctr, ws, ws_bytes, &p.r.w);
  if (rc) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, nullptr, s);
  p.r.t = *t;
  p.r.n = n;
  p.r.status = status;
  p.r.ctr = ctr;
  p.req = req;
  return launch_rows(page_free_gang_kernel<kSmallThreads>, page_free_team_kernel, page_free_units_kernel, s, p);
}

extern "C" int db_page_fork(const db_page_tables* t, const db_page_fork_req* req, uint32_t n,
                            uint8_t* status, db_counters* ctr, void* ws, size_t ws_bytes,
                            void* stream) {
  ForkParams p = {};
  const int rc = check_call(t, req, sizeof(*req), n, ctr, ws, ws_bytes, &p.r.w);
  if (rc) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, nullptr, s);
  p.r.t = *t;
  p.r.n = n;
  p.r.status = status;
  p.r.ctr = ctr;
  p.req = req;
  return launch_rows(page_fork_gang_kernel<kSmallThreads>, page_fork_team_kernel, page_fork_units_kernel, s, p);
}

extern "C" int db_page_extend(const db_page_tables* t, const db_page_grow* req, uint32_t n,
                              db_page_move* moves, uint32_t* n_moves, uint8_t* status,
                              db_counters* ctr, void* ws, size_t ws_bytes, void* stream) {
  ExtendParams p = {};
  const int rc = check_call(t, req, sizeof(*req), n, ctr, ws, ws_bytes, &p.w);
  if (rc) return rc;
  if (!n_moves || !aligned(n_moves, 4) || (n && (!moves || !aligned(moves, 16)))) return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, n_moves, s);
  p.t = *t;
  p.req = req;
  p.n = n;
  p.moves = moves;
  p.n_moves = n_moves;
  p.status = status;
  p.ctr = ctr;
  const uint64_t pages = (uint64_t)n * t->columns < t->n_pages ? (uint64_t)n * t->columns : t->n_pages;
  const uint32_t words = (t->n_pages + 31) / 32;
  if (n <= kSmallThreads && words <= 4 * kSmallThreads && pages <= kRestPages)
    return launch_dependent(page_extend_gang_kernel<kSmallThreads>, 1, kSmallThreads, 0, s, p);
  if (n <= kTeamThreads && words <= kGangWords)
    return launch_dependent(page_extend_gang_kernel<kTeamThreads>,
                            gang_size(pages, kRestPages, kTeamThreads, 1), kTeamThreads, 0, s, p);
  p.rest = pages > kRestPages || n > kMaxTeam * kTeamThreads || words > kTeamWords;
  uint32_t ctas = team_size(2ull * n > words / 4 ? 2ull * n : words / 4);
  if (ctas == 1) ctas = 2;
  const int e = launch_team(page_extend_team_kernel, ctas, kTeamThreads, s, p);
  if (e || !p.rest) return e;
  return launch_dependent(page_place_kernel, whole_grid(pages, kPlaceThreads, 8), kPlaceThreads, 0,
                          s, p);
}

extern "C" int db_page_compact(const db_page_tables* t, const db_page_tables* out,
                               db_page_move* moves, uint32_t cap, uint32_t* n_moves,
                               db_counters* ctr, void* ws, size_t ws_bytes, void* stream) {
  CompactParams p = {};
  int rc = check_call(t, nullptr, 1, 0, ctr, ws, ws_bytes, &p.w);
  if (rc) return rc;
  rc = check_tables(out);
  if (rc) return rc;
  if (out->n_seqs != t->n_seqs || out->columns != t->columns || out->n_pages != t->n_pages ||
      out->page_tokens != t->page_tokens)
    return -EINVAL;
  if (!n_moves || !aligned(n_moves, 4) || (cap && (!moves || !aligned(moves, 16)))) return -EINVAL;
  p.t = *t;
  p.out = *out;
  p.moves = moves;
  p.cap = cap;
  p.n_moves = n_moves;
  p.ctr = ctr;
  const cudaStream_t s = (cudaStream_t)stream;
  const uint64_t entries = (uint64_t)t->n_seqs * t->columns;
  const uint32_t most = cap < t->n_pages / 2 ? cap : t->n_pages / 2;
  const uint32_t ctas = team_size(((uint64_t)t->n_pages + 127) / 128);
  p.rest = most > kRestMoves;
  p.whole = ctas == 1 && !p.rest && entries <= kSoloEntries;
  int e = ctas == 1 ? launch_team(page_compact_plan_kernel<kTeamThreads, true>, 1, kTeamThreads, s, p)
                    : launch_team(page_compact_plan_kernel<kTeamThreads, false>, ctas, kTeamThreads, s, p);
  if (e || p.whole) return e;
  if (p.rest) e = launch_dependent(page_compact_moves_kernel, whole_grid(most, 256, 8), 256, 0, s, p);
  if (e) return e;
  const uint64_t work = entries > t->n_pages ? entries : t->n_pages;
  return launch_dependent(page_compact_apply_kernel, whole_grid((work + 3) / 4, 256, 8), 256, 0, s, p);
}
