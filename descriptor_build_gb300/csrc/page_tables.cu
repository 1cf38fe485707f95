// Page tables of a cache in the device heap: extend, fork, free, compact
// (include/pagecache.h has the definitions).
//
// A call's requests are planned by one team: a single CTA or one cluster of
// CTAs, whose barriers are the hardware's, so no kernel here waits on memory.
// The plan is a prefix sum over what the requests ask for, and what follows
// is work on pieces of it, found again by a search in shared memory. The team
// does that work itself when it is little; otherwise a second kernel does it
// on the whole GPU, launched as a dependent of the first when the sizes of
// the call allow for so much (how much there is, only the device knows).
//
// Nothing depends on the order in which atomics land: a request's claim on
// its sequence and the holders of a shared page are a maximum and a count,
// references are sums, free pages are bits, and pages are taken by rank among
// the set bits.
#include "common.cuh"
#include "pagecache.h"

namespace db {
namespace {

constexpr uint32_t kTeamThreads = 1024;
constexpr uint32_t kTeamWarps = kTeamThreads / 32;
#ifndef DB_PAGE_TEAM
#define DB_PAGE_TEAM 8
#endif
constexpr uint32_t kMaxTeam = DB_PAGE_TEAM;  // CTAs of the largest team
constexpr uint32_t kSearch = 4096;     // prefix entries kept in shared memory
constexpr uint32_t kRows = 8;          // requests of a group (see free_units)
constexpr uint32_t kNoMove = 0xFFFFFFFFu;
constexpr uint32_t kNoEntry = 0xFFFFFFFEu;   // a row without an entry in the column
constexpr uint32_t kBadEntry = 0xFFFFFFFFu;  // no page
#ifndef DB_PAGE_OWN
#define DB_PAGE_OWN 4
#endif
constexpr uint32_t kOwn = DB_PAGE_OWN;  // what a warp (unit) or thread (page) of the team does itself

// One request's place in the plan.
struct __align__(16) Plan {
  uint32_t row;   // row that is written
  uint32_t from;  // free, fork: first column; extend: the column of its first page
  uint32_t end;   // free, fork: past the last column; extend: pages of the requests before it
  uint32_t aux;   // extend: index of its move or kNoMove; fork: the parent's row
};

struct Head {
  uint32_t units;      // left for the second kernel
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
  uint32_t* pages;    // [n_pages] extend: the pages taken, by rank; compact: where a moved page went
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
  x.before = (uint32_t*)take(4 * (((size_t)n_pages + 31) / 32));
  x.pages = (uint32_t*)take(4 * (size_t)n_pages);
  if (w) *w = x;
  return at;
}

// ------------------------------------------------------------------ the team
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

struct Sum {
  uint64_t a;
  uint32_t b;
};

struct TeamShared {
  uint64_t warp_a[kTeamWarps];
  uint32_t warp_b[kTeamWarps];
  uint64_t cta_a[2];  // this CTA's sums, read by its peers; two rounds apart
  uint32_t cta_b[2];
  uint64_t base_a, total_a;
  uint32_t base_b, total_b;
};

struct Team {
  uint32_t rank, size, round;
  TeamShared* s;
  __device__ __forceinline__ explicit Team(TeamShared* sh)
      : rank(cluster_rank()), size(cluster_size()), round(0), s(sh) {}
  __device__ __forceinline__ uint32_t id() const { return rank * kTeamThreads + threadIdx.x; }
  __device__ __forceinline__ uint32_t threads() const { return size * kTeamThreads; }
  // Barrier of the team; global and shared writes before it are seen after it.
  __device__ __forceinline__ void sync() const {
    if (size == 1) {
      __syncthreads();
    } else {
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                       : "memory");
    }
  }
  // Exclusive prefix of one pair per thread in id() order, and the team's sum.
  __device__ __forceinline__ Sum scan(Sum v, Sum* total) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t a = v.a;
    uint32_t b = v.b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(kFull, a, o);
      const uint32_t y = __shfl_up_sync(kFull, b, o);
      if (lane >= (uint32_t)o) {
        a += x;
        b += y;
      }
    }
    __syncthreads();  // the last round's readers are done
    if (lane == 31) {
      s->warp_a[warp] = a;
      s->warp_b[warp] = b;
    }
    __syncthreads();
    const uint32_t k = round++ & 1;
    if (warp == 0) {
      const uint64_t wa = s->warp_a[lane];
      const uint32_t wb = s->warp_b[lane];
      uint64_t xa = wa;
      uint32_t xb = wb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(kFull, xa, o);
        const uint32_t y = __shfl_up_sync(kFull, xb, o);
        if (lane >= (uint32_t)o) {
          xa += x;
          xb += y;
        }
      }
      s->warp_a[lane] = xa - wa;
      s->warp_b[lane] = xb - wb;
      if (lane == 31) {
        s->cta_a[k] = xa;
        s->cta_b[k] = xb;
        s->base_a = 0;
        s->base_b = 0;
        s->total_a = xa;
        s->total_b = xb;
      }
    }
    sync();
    if (size > 1) {
      if (warp == 0) {
        uint64_t pa = 0;
        uint32_t pb = 0;
        if (lane < size) {
          uint32_t at, bt;
          asm("mapa.shared::cluster.u32 %0, %1, %2;"
              : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&s->cta_a[k])), "r"(lane));
          asm("mapa.shared::cluster.u32 %0, %1, %2;"
              : "=r"(bt) : "r"((uint32_t)__cvta_generic_to_shared(&s->cta_b[k])), "r"(lane));
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(pa) : "r"(at) : "memory");
          asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(pb) : "r"(bt) : "memory");
        }
        const uint64_t ta = warp_sum64(pa), ba = warp_sum64(lane < rank ? pa : 0);
        const uint32_t tb = warp_sum32(pb), bb = warp_sum32(lane < rank ? pb : 0);
        if (lane == 0) {
          s->base_a = ba;
          s->base_b = bb;
          s->total_a = ta;
          s->total_b = tb;
        }
      }
      __syncthreads();
    }
    total->a = s->total_a;
    total->b = s->total_b;
    Sum out;
    out.a = s->base_a + s->warp_a[warp] + a - v.a;
    out.b = s->base_b + s->warp_b[warp] + b - v.b;
    return out;
  }
};

// A scan may end with a peer still reading this CTA's shared memory: the last
// sync of a kernel's team comes after its last scan in every kernel below, so
// no CTA leaves before its peers have read it.

// ---------------------------------------------------------- finding a piece
// The last i with start(i) <= e, where start is not decreasing: every
// `step`-th start is in shared memory, all of them up to kSearch.
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

// Load the starts (every thread of a CTA; ends past a barrier).
template <typename Start>
__device__ __forceinline__ Finder load_finder(uint32_t* s_start, uint32_t n, Start start) {
  Finder f;
  f.s_start = s_start;
  f.n = n;
  f.step = (n + kSearch - 1) / kSearch;
  f.kept = (n + f.step - 1) / f.step;
  for (uint32_t k = threadIdx.x; k < f.kept; k += blockDim.x) s_start[k] = start(k * f.step);
  __syncthreads();
  return f;
}

__device__ __forceinline__ Plan ld_plan(const Plan* p) {
  const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
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
  return (tokens >> 32) || tokens + page_tokens > 0xFFFFFFFFull
             ? (uint32_t)((tokens + page_tokens - 1) / page_tokens)
             : ((uint32_t)tokens + page_tokens - 1) / page_tokens;
}

// Word w of the free bits, without bits past n_pages.
__device__ __forceinline__ uint32_t ld_word(const uint32_t* bits, uint32_t w, uint32_t n_pages) {
  uint32_t v = __ldcg(&bits[w]);
  if (n_pages - 32 * w < 32) v &= (1u << (n_pages & 31)) - 1;
  return v;
}

// Free pages before each word into `before`; returns their number.
__device__ __forceinline__ uint32_t scan_free(Team& team, const uint32_t* bits, uint32_t n_pages,
                                              uint32_t* before) {
  const uint32_t words = (n_pages + 31) / 32;
  uint32_t carry = 0;
  for (uint32_t w0 = 0; w0 < words; w0 += team.threads()) {
    const uint32_t w = w0 + team.id();
    const uint32_t c = w < words ? __popc(ld_word(bits, w, n_pages)) : 0;
    Sum total;
    const Sum x = team.scan(Sum{c, 0}, &total);
    if (w < words) before[w] = carry + (uint32_t)x.a;
    carry += (uint32_t)total.a;
  }
  return carry;
}

// A count and an error, one warp's at a time, into the counters.
__device__ __forceinline__ void add_count(uint64_t* to, uint32_t count) {
  const uint32_t c = warp_sum32(count);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd((unsigned long long*)to, (unsigned long long)c);
}
__device__ __forceinline__ void add_error(db_counters* ctr, bool bad) {
  if (__any_sync(kFull, bad) && (threadIdx.x & 31) == 0)
    atomicOr((unsigned long long*)&ctr->err, (unsigned long long)DB_ERR_PAGE_TABLE);
}

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
  Work w;
};

// Each thread's columns into the groups; ends with every group of these
// requests written (not yet visible to other CTAs). `carry`: units before.
__device__ __forceinline__ void plan_rows(Team& team, const Rows& p, uint32_t i, const Plan& pl,
                                          uint32_t* carry) {
  uint32_t lo = pl.from < pl.end ? pl.from : 0xFFFFFFFFu, hi = pl.from < pl.end ? pl.end : 0;
#pragma unroll
  for (uint32_t o = 1; o < kRows; o <<= 1) {
    lo = min(lo, __shfl_xor_sync(kFull, lo, o));
    hi = max(hi, __shfl_xor_sync(kFull, hi, o));
  }
  lo &= ~31u;
  const uint32_t units = hi > lo ? (hi - lo + 31) / 32 : 0;
  const bool first = i % kRows == 0;
  Sum total;
  const Sum x = team.scan(Sum{first ? units : 0, 0}, &total);
  if (i < p.n) {
    st_plan(&p.w.plan[i], pl);
    if (first) p.w.group[i / kRows] = make_uint2(*carry + (uint32_t)x.a, lo);
  }
  *carry += (uint32_t)total.a;
}

struct GroupStart {
  const uint2* group;
  __device__ __forceinline__ uint32_t operator()(uint32_t g) const { return __ldcg(&group[g].x); }
};

// The rows of unit u: lane j < kRows holds the j-th plan (empty if there is
// none); returns this lane's column.
__device__ __forceinline__ uint32_t load_unit(const Rows& p, const Finder& f, uint32_t u,
                                              uint32_t lane, Plan* pl) {
  const uint32_t g = f.find(u, GroupStart{p.w.group});
  const uint2 at = __ldcg(&p.w.group[g]);
  const uint32_t i = g * kRows + lane;
  *pl = Plan{0, 0, 0, 0};
  if (lane < kRows && i < p.n) *pl = ld_plan(&p.w.plan[i]);
  return at.y + (u - at.x) * 32 + lane;
}

// ---------------------------------------------------------------------- free
struct FreeParams {
  Rows r;
  const db_page_cut* req;
};

__device__ __forceinline__ void free_units(const Rows& p, const Finder& f, uint32_t first,
                                           uint32_t stride, uint32_t units) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t released = 0;
  bool bad = false;
  for (uint32_t u = first; u < units; u += stride) {
    Plan pl;
    const uint32_t c = load_unit(p, f, u, lane, &pl);
    uint32_t page[kRows];
    bool clear[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const uint32_t row = __shfl_sync(kFull, pl.row, j), from = __shfl_sync(kFull, pl.from, j);
      const uint32_t end = __shfl_sync(kFull, pl.end, j);
      page[j] = kNoEntry;
      if (c >= from && c < end) page[j] = (uint32_t)p.t.table[(uint64_t)row * p.t.columns + c];
      clear[j] = c >= from && c < end;
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const uint32_t row = __shfl_sync(kFull, pl.row, j);
      if (!clear[j]) continue;
      p.t.table[(uint64_t)row * p.t.columns + c] = DB_PAGE_NONE;
      if (page[j] == kNoEntry) page[j] = kBadEntry;
    }
    uint32_t old[kRows], times[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      times[j] = 0;
      if (page[j] == kNoEntry || (j && page[j] == page[j - 1])) continue;
      if (page[j] >= p.t.n_pages) {
        bad = true;
        continue;
      }
      uint32_t run = 1;
#pragma unroll
      for (uint32_t k = j + 1; k < kRows; ++k)
        if (run == k - j && page[k] == page[j]) ++run;
      times[j] = run;
      old[j] = atomicSub(&p.t.refs[page[j]], run);
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!times[j]) continue;
      if (old[j] == times[j]) {
        atomicOr(&p.t.free[page[j] >> 5], 1u << (page[j] & 31));
        ++released;
      } else if (old[j] < times[j]) {  // more rows than references: leave them as they were
        atomicAdd(&p.t.refs[page[j]], times[j]);
        bad = true;
      }
    }
  }
  if (p.ctr) {
    add_count(&p.ctr->total, released);
    add_error(p.ctr, bad);
  }
}

__global__ void __launch_bounds__(kTeamThreads) page_free_kernel(const FreeParams q) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  if (p.ctr && team.id() == 0) *p.ctr = db_counters{0, 0, 0, 0};
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t seq = q.req[i].seq;
    if (seq < p.t.n_seqs) claim(p.w.claim, seq, i);
  }
  team.sync();
  uint32_t units = 0, invalid = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += team.threads()) {
    const uint32_t i = i0 + team.id();
    Plan pl = {0, 0, 0, 0};
    if (i < p.n) {
      const db_page_cut r = q.req[i];
      const uint32_t len = r.seq < p.t.n_seqs ? p.t.length[r.seq] : 0;
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
    plan_rows(team, p, i, pl, &units);
  }
  if (p.ctr) add_count(&p.ctr->n_invalid, invalid);
  const bool own = units <= kOwn * (team.threads() / 32);
  if (team.id() == 0) p.w.head->units = own ? 0 : units;
  team.sync();
  if (!own || !units) return;
  const Finder f = load_finder(s_start, (p.n + kRows - 1) / kRows, GroupStart{p.w.group});
  free_units(p, f, team.id() / 32, team.threads() / 32, units);
}

__global__ void __launch_bounds__(256) page_free_units_kernel(const FreeParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = __ldcg(&p.w.head->units);
  if (blockIdx.x * 8 >= units) return;
  const Finder f = load_finder(s_start, (p.n + kRows - 1) / kRows, GroupStart{p.w.group});
  free_units(p, f, blockIdx.x * 8 + threadIdx.x / 32, gridDim.x * 8, units);
}

// ---------------------------------------------------------------------- fork
struct ForkParams {
  Rows r;
  const db_page_fork_req* req;
};

__device__ __forceinline__ void fork_units(const Rows& p, const Finder& f, uint32_t first,
                                           uint32_t stride, uint32_t units) {
  const uint32_t lane = threadIdx.x & 31;
  bool bad = false;
  for (uint32_t u = first; u < units; u += stride) {
    Plan pl;
    const uint32_t c = load_unit(p, f, u, lane, &pl);
    uint32_t page[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const uint32_t from = __shfl_sync(kFull, pl.aux, j), end = __shfl_sync(kFull, pl.end, j);
      page[j] = kNoEntry;
      if (c < end) page[j] = (uint32_t)p.t.table[(uint64_t)from * p.t.columns + c];
    }
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      const uint32_t row = __shfl_sync(kFull, pl.row, j), end = __shfl_sync(kFull, pl.end, j);
      if (c >= end) continue;
      p.t.table[(uint64_t)row * p.t.columns + c] = (int32_t)page[j];
      if (page[j] >= p.t.n_pages) {
        bad = true;
        page[j] = kNoEntry;
        continue;
      }
      if (j && page[j] == page[j - 1]) continue;
      uint32_t run = 1;
#pragma unroll
      for (uint32_t k = j + 1; k < kRows; ++k)
        if (run == k - j && page[k] == page[j]) ++run;
      atomicAdd(&p.t.refs[page[j]], run);
    }
  }
  if (p.ctr) add_error(p.ctr, bad);
}

__global__ void __launch_bounds__(kTeamThreads) page_fork_kernel(const ForkParams q) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  if (p.ctr && team.id() == 0) *p.ctr = db_counters{0, 0, 0, 0};
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t child = q.req[i].child;
    if (child < p.t.n_seqs) claim(p.w.claim, child, i);
  }
  team.sync();
  uint32_t units = 0, invalid = 0;
  uint64_t taken = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += team.threads()) {
    const uint32_t i = i0 + team.id();
    Plan pl = {kNoMove, 0, 0, 0};
    if (i < p.n) {
      const db_page_fork_req r = q.req[i];
      bool ok = false;
      if (r.child < p.t.n_seqs && claimed(p.w.claim, r.child, i)) {
        p.w.claim[r.child] = 0;
        ok = r.parent < p.t.n_seqs && r.parent != r.child && __ldcg(&p.t.length[r.child]) == 0 &&
             r.tokens <= __ldcg(&p.t.length[r.parent]);
      }
      if (ok) {
        pl = Plan{r.child, 0, min(pages_of(r.tokens, p.t.page_tokens), p.t.columns), r.parent};
        taken += pl.end;
      }
      invalid += !ok;
      if (p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    }
    plan_rows(team, p, i, pl, &units);
  }
  if (p.ctr) {
    add_count(&p.ctr->n_invalid, invalid);
    const uint64_t c = warp_sum64(taken);
    if ((threadIdx.x & 31) == 0 && c)
      atomicAdd((unsigned long long*)&p.ctr->total, (unsigned long long)c);
  }
  const bool own = units <= kOwn * (team.threads() / 32);
  if (team.id() == 0) p.w.head->units = own ? 0 : units;
  team.sync();  // every length is read
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t row = p.w.plan[i].row;
    if (row != kNoMove) p.t.length[row] = q.req[i].tokens;
  }
  if (!own || !units) return;
  const Finder f = load_finder(s_start, (p.n + kRows - 1) / kRows, GroupStart{p.w.group});
  fork_units(p, f, team.id() / 32, team.threads() / 32, units);
}

__global__ void __launch_bounds__(256) page_fork_units_kernel(const ForkParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = __ldcg(&p.w.head->units);
  if (blockIdx.x * 8 >= units) return;
  const Finder f = load_finder(s_start, (p.n + kRows - 1) / kRows, GroupStart{p.w.group});
  fork_units(p, f, blockIdx.x * 8 + threadIdx.x / 32, gridDim.x * 8, units);
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
  bool mine, ok, corrupt;
  __device__ __forceinline__ bool shares() const { return part && refs > 1; }
};

__device__ __forceinline__ Ask ask(const ExtendParams& p, uint32_t i) {
  Ask a = {0, 0, 0, 0, 0, 0, 0, false, false, false};
  if (i >= p.n) return a;
  const db_page_grow r = p.req[i];
  a.seq = r.seq;
  if (r.seq >= p.t.n_seqs) return a;
  const uint32_t len = p.t.length[r.seq];
  a.mine = claimed(p.w.claim, r.seq, i);
  const uint64_t now = (uint64_t)len + r.tokens;
  if (!a.mine || now > (uint64_t)p.t.columns * p.t.page_tokens || now > 0xFFFFFFFFull) return a;
  a.ok = true;
  a.now = (uint32_t)now;
  a.had = pages_of(len, p.t.page_tokens);
  a.grow = pages_of(now, p.t.page_tokens) - a.had;
  const uint32_t part = len % p.t.page_tokens;
  if (r.tokens && part) {
    a.last = (uint32_t)p.t.table[(uint64_t)r.seq * p.t.columns + a.had - 1];
    if (a.last >= p.t.n_pages) {
      a.ok = false;
      a.corrupt = true;
      a.grow = 0;
    } else {
      a.refs = __ldcg(&p.t.refs[a.last]);
      a.part = part;
    }
  }
  return a;
}

struct PlanStart {
  const Plan* plan;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return __ldcg(&plan[i].end); }
};

// Page e of the batch into its row.
__device__ __forceinline__ void place_pages(const ExtendParams& p, const Finder& f, uint32_t first,
                                            uint32_t stride, uint32_t total) {
  for (uint32_t e = first; e < total; e += stride) {
    const uint32_t page = __ldcg(&p.w.pages[e]);
    const Plan pl = ld_plan(&p.w.plan[f.find(e, PlanStart{p.w.plan})]);
    const uint32_t j = e - pl.end;
    p.t.table[(uint64_t)pl.row * p.t.columns + pl.from + j] = (int32_t)page;
    p.t.refs[page] = 1;
    if (j == 0 && pl.aux != kNoMove) p.moves[pl.aux].dst = page;
  }
}

__global__ void __launch_bounds__(kTeamThreads) page_extend_kernel(const ExtendParams p) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  const uint32_t id = team.id(), threads = team.threads();
  const bool one = p.n <= threads;  // every request has a thread: asked once, kept in registers
  if (p.ctr && id == 0) *p.ctr = db_counters{0, 0, 0, 0};
  for (uint32_t i = id; i < p.n; i += threads) {
    const uint32_t seq = p.req[i].seq;
    if (seq < p.t.n_seqs) claim(p.w.claim, seq, i);
  }
  const uint32_t avail = scan_free(team, p.t.free, p.t.n_pages, p.w.before);
  team.sync();
  // How many of the batch's requests hold each shared page, and the last of them.
  Ask a = {0, 0, 0, 0, 0, 0, 0, false, false, false};
  for (uint32_t i = id; i < p.n; i += threads) {
    a = ask(p, i);
    if (a.shares()) {
      atomicAdd(&p.w.holders[a.last], 1u);
      atomicMax(&p.w.latest[a.last], i);
    }
  }
  team.sync();
  uint64_t need = 0;
  uint32_t n_moves = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += threads) {
    const uint32_t i = i0 + id;
    if (!one) a = ask(p, i);
    const uint32_t cow = a.shares() && !(__ldcg(&p.w.holders[a.last]) == a.refs &&
                                     __ldcg(&p.w.latest[a.last]) == i);
    Sum total;
    const Sum x = team.scan(Sum{(uint64_t)a.grow + cow, cow}, &total);
    if (i < p.n)
      st_plan(&p.w.plan[i], Plan{a.seq, a.had - cow, (uint32_t)min(need + x.a, (uint64_t)0xFFFFFFFFu),
                                 cow ? n_moves + x.b : kNoMove});
    need += total.a;
    n_moves += total.b;
  }
  const bool go = need <= avail;
  const bool own = need <= (uint64_t)kOwn * threads;
  if (id == 0) {
    *p.n_moves = go ? n_moves : 0;
    p.w.head->units = go && !own ? (uint32_t)need : 0;
    if (p.ctr) p.ctr->total = need;
  }
  team.sync();
  // Lengths, moves and status, and the workspace as the next call wants it.
  uint32_t invalid = 0, refused = 0;
  bool corrupt = false;
  for (uint32_t i = id; i < p.n; i += threads) {
    if (!one) a = ask(p, i);
    const uint32_t m = p.w.plan[i].aux;
    if (m != kNoMove) {  // at least one holder of every shared page copies, and clears for all
      p.w.holders[a.last] = 0;
      p.w.latest[a.last] = 0;
      if (go) {
        atomicSub(&p.t.refs[a.last], 1u);
        p.moves[m].src = a.last;
        *reinterpret_cast<uint2*>(&p.moves[m].tokens) = make_uint2(a.part, 0);
      }
    }
    if (a.mine) p.w.claim[a.seq] = 0;
    if (a.ok && go) p.t.length[a.seq] = a.now;
    invalid += !a.ok;
    refused += a.ok && !go;
    corrupt |= a.corrupt;
    if (p.status) p.status[i] = !a.ok ? DB_PAGE_INVALID : go ? DB_PAGE_OK : DB_PAGE_SHORT;
  }
  if (p.ctr) {
    add_count(&p.ctr->n_invalid, invalid);
    add_count(&p.ctr->n_overflow, refused);
    add_error(p.ctr, corrupt);
  }
  if (!go || need == 0) return;
  // The pages taken, by rank: a word at a time, a page per lane.
  const uint32_t lane = threadIdx.x & 31, words = (p.t.n_pages + 31) / 32;
  for (uint32_t w0 = id - lane; w0 < words; w0 += threads) {
    const uint32_t w = w0 + lane;
    const uint32_t rank = w < words ? __ldcg(&p.w.before[w]) : 0xFFFFFFFFu;
    const uint32_t bits = w < words ? ld_word(p.t.free, w, p.t.n_pages) : 0;
    uint32_t active = __ballot_sync(kFull, bits && rank < need);
    uint32_t left = bits;
    while (active) {
      const uint32_t k = __ffs(active) - 1;
      active &= active - 1;
      const uint32_t v = __shfl_sync(kFull, bits, k);
      const uint32_t e = __shfl_sync(kFull, rank, k) + __popc(v & lanemask_lt());
      const bool mine = (v >> lane & 1) && e < need;
      const uint32_t taken = __ballot_sync(kFull, mine);
      if (mine) p.w.pages[e] = (w0 + k) * 32 + lane;
      if (lane == k) left &= ~taken;
    }
    if (left != bits) p.t.free[w] = left;
  }
  team.sync();  // the pages are known, and the replaced entries have been read
  if (!own) return;
  const Finder f = load_finder(s_start, p.n, PlanStart{p.w.plan});
  place_pages(p, f, id, threads, (uint32_t)need);
}

__global__ void __launch_bounds__(256) page_place_kernel(const ExtendParams p) {
  __shared__ uint32_t s_start[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t total = __ldcg(&p.w.head->units);
  if (blockIdx.x * 256 >= total) return;
  const Finder f = load_finder(s_start, p.n, PlanStart{p.w.plan});
  place_pages(p, f, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, total);
}

// ------------------------------------------------------------------- compact
struct CompactParams {
  db_page_tables t, out;
  db_page_move* moves;
  uint32_t cap;
  uint32_t* n_moves;
  db_counters* ctr;
  Work w;
};

__global__ void __launch_bounds__(kTeamThreads) page_compact_plan_kernel(const CompactParams p) {
  __shared__ TeamShared s_team;
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  const uint32_t id = team.id(), threads = team.threads();
  const uint32_t n_pages = p.t.n_pages, words = (n_pages + 31) / 32;
  const uint32_t n_live = n_pages - scan_free(team, p.t.free, n_pages, p.w.before);
  team.sync();
  // M: the free pages below n_live.
  uint32_t holes = 0;
  if (n_live < n_pages) {
    const uint32_t w = n_live / 32;
    holes = __ldcg(&p.w.before[w]) +
            __popc(ld_word(p.t.free, w, n_pages) & ((1u << (n_live & 31)) - 1));
  }
  const uint32_t moved = min(holes, p.cap);
  if (id == 0) {
    *p.n_moves = moved;
    p.w.head->moved = moved;
    if (moved == 0) {
      p.w.head->src_first = n_pages;
      p.w.head->dst_last = 0;
    }
    if (p.ctr) *p.ctr = db_counters{holes, 0, (uint64_t)holes - moved, 0};
  }
  const uint32_t lane = threadIdx.x & 31;
  for (uint32_t w0 = id - lane; w0 < words && moved; w0 += threads) {
    const uint32_t w = w0 + lane, first = 32 * w;
    const uint32_t bits = w < words ? ld_word(p.t.free, w, n_pages) : 0;
    const uint32_t before = w < words ? __ldcg(&p.w.before[w]) : 0;
    // free pages below n_live to move to, or live pages from n_live on to move from
    bool use = false;
    if (w < words) {
      if (first < n_live) use = bits && before < moved;
      if (first + 31 >= n_live) use |= bits != kFull;
    }
    uint32_t active = __ballot_sync(kFull, use);
    while (active) {
      const uint32_t k = __ffs(active) - 1;
      active &= active - 1;
      const uint32_t v = __shfl_sync(kFull, bits, k);
      const uint32_t page = (w0 + k) * 32 + lane;
      const uint32_t rank = __shfl_sync(kFull, before, k) + __popc(v & lanemask_lt());
      if (page < n_pages) {
        if (v >> lane & 1) {
          if (page < n_live && rank < moved) {
            p.moves[rank].dst = page;
            *reinterpret_cast<uint2*>(&p.moves[rank].tokens) = make_uint2(DB_PAGE_ALL, 0);
            if (rank == moved - 1) p.w.head->dst_last = page;
          }
        } else if (page >= n_live) {
          const uint32_t top = n_live - 1 - (page - rank);  // live pages above it
          if (top < moved) {
            p.moves[top].src = page;
            if (top == moved - 1) p.w.head->src_first = page;
          }
        }
      }
    }
  }
  team.sync();
  for (uint32_t k = id; k < moved; k += threads) {
    const uint2 m = __ldcg(reinterpret_cast<const uint2*>(&p.moves[k]));
    p.w.pages[m.x] = m.y;
    p.out.refs[m.y] = p.t.refs[m.x];
    p.out.refs[m.x] = 0;
  }
}

__global__ void __launch_bounds__(256) page_compact_apply_kernel(const CompactParams p) {
  wait_for_prerequisites();
  dependents_may_launch();
  const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x, step = (uint64_t)gridDim.x * 256;
  const uint32_t n_pages = p.t.n_pages;
  const uint32_t moved = __ldcg(&p.w.head->moved), src_first = __ldcg(&p.w.head->src_first);
  const uint32_t dst_last = __ldcg(&p.w.head->dst_last);
  const uint64_t entries = (uint64_t)p.t.n_seqs * p.t.columns;
  bool bad = false;
  for (uint64_t e = id; e < entries; e += step) {
    const uint32_t was = (uint32_t)p.t.table[e];
    uint32_t is = was;
    if (was >= src_first && was != (uint32_t)DB_PAGE_NONE) {
      if (was < n_pages) is = __ldcg(&p.w.pages[was]); else bad = true;
    }
    if (p.out.table != p.t.table || is != was) p.out.table[e] = (int32_t)is;
  }
  if (p.ctr) add_error(p.ctr, bad);
  if (p.out.refs != p.t.refs)
    for (uint64_t q = id; q < n_pages; q += step) {
      const uint32_t v = p.t.refs[q];
      if (q >= src_first)
        p.out.refs[q] = 0;
      else if (v || !moved || q > dst_last)  // the plan wrote the pages moved to
        p.out.refs[q] = v;
    }
  const uint32_t words = (n_pages + 31) / 32;
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

// ---------------------------------------------------------------- host side
template <typename P>
int launch_team(void (*kernel)(P), uint32_t ctas, cudaStream_t s, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTeamThreads);
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
  if (ctas > 8) cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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

// CTAs of the team for `n` requests, `words` of free bits and at most `units`
// pieces of a warp's work.
uint32_t team_size(uint64_t n, uint64_t words, uint64_t units) {
  uint64_t want = n > words ? n : words;
  if (units * 32 / kOwn > want) want = units * 32 / kOwn;
  uint32_t c = 1;
  while (c < kMaxTeam && (uint64_t)c * kTeamThreads < want) c *= 2;
  return c;
}

// CTAs of 256 threads for at most `threads`.
unsigned whole_grid(uint64_t threads) {
  const uint64_t want = (threads + 255) / 256, most = 8ull * num_sms();
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

// Free and fork: the team, and the whole GPU where there may be more than the
// team does itself.
template <typename P>
int launch_rows(void (*team)(P), void (*rest)(P), cudaStream_t s, const P& p) {
  const uint64_t units = ((uint64_t)p.r.n + kRows - 1) / kRows * (((uint64_t)p.r.t.columns + 31) / 32);
  const uint32_t ctas = team_size(p.r.n, 0, units);
  const int e = launch_team(team, ctas, s, p);
  if (e || units <= (uint64_t)kOwn * ctas * kTeamWarps) return e;
  return launch_dependent(rest, whole_grid(units * 32), 256, 0, s, p);
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
  if ((uint64_t)n * t->columns > 0xFFFFFFFFull) return -EINVAL;  // entries are numbered in 32 bits
  p.r.t = *t;
  p.r.n = n;
  p.r.status = status;
  p.r.ctr = ctr;
  p.req = req;
  return launch_rows(page_free_kernel, page_free_units_kernel, s, p);
}

extern "C" int db_page_fork(const db_page_tables* t, const db_page_fork_req* req, uint32_t n,
                            uint8_t* status, db_counters* ctr, void* ws, size_t ws_bytes,
                            void* stream) {
  ForkParams p = {};
  const int rc = check_call(t, req, sizeof(*req), n, ctr, ws, ws_bytes, &p.r.w);
  if (rc) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, nullptr, s);
  if ((uint64_t)n * t->columns > 0xFFFFFFFFull) return -EINVAL;  // entries are numbered in 32 bits
  p.r.t = *t;
  p.r.n = n;
  p.r.status = status;
  p.r.ctr = ctr;
  p.req = req;
  return launch_rows(page_fork_kernel, page_fork_units_kernel, s, p);
}

extern "C" int db_page_extend(const db_page_tables* t, const db_page_grow* req, uint32_t n,
                              db_page_move* moves, uint32_t* n_moves, uint8_t* status,
                              db_counters* ctr, void* ws, size_t ws_bytes, void* stream) {
  ExtendParams p = {};
  const int rc = check_call(t, req, 8, n, ctr, ws, ws_bytes, &p.w);
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
  const uint32_t ctas = team_size(n, (t->n_pages + 31) / 32, 0);
  const int e = launch_team(page_extend_kernel, ctas, s, p);
  if (e || pages <= (uint64_t)kOwn * ctas * kTeamThreads) return e;
  return launch_dependent(page_place_kernel, whole_grid(pages), 256, 0, s, p);
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
  const int e = launch_team(page_compact_plan_kernel, team_size(0, (t->n_pages + 31) / 32, 0), s, p);
  if (e) return e;
  const uint64_t entries = (uint64_t)t->n_seqs * t->columns;
  return launch_dependent(page_compact_apply_kernel,
                          whole_grid(entries > t->n_pages ? entries : t->n_pages), 256, 0, s, p);
}
