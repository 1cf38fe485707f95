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
constexpr uint32_t kMaxTeam = 8;       // CTAs of the largest team
constexpr uint32_t kSearch = 1024;     // starts kept in shared memory, the others are near one
constexpr uint32_t kRows = 8;          // requests of a group (see "row units")
constexpr uint32_t kSoloWords = 2048;  // free words of a team of one CTA
// What a team does itself when a second kernel is there for the rest: units of
// rows for each of its CTAs, pages for each of its threads. The second kernel
// is launched when the sizes of the call allow for more than kRest of them.
constexpr uint32_t kOwnUnits = 8, kOwnPages = 4;
constexpr uint32_t kRestUnits = 64, kRestPages = 16384;
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
  uint32_t units;      // left for the second kernel
  uint32_t moved;      // compact: moves made
  uint32_t dst_last;   // compact: the last page moved to (with moved > 0)
  uint32_t src_first;  // compact: the lowest page moved from, or n_pages
  uint32_t holes;      // compact: free pages below the number of live ones
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

// kSolo: the team is one CTA.
template <bool kSolo>
struct Team {
  uint32_t rank, size, round;
  TeamShared* s;
  __device__ __forceinline__ explicit Team(TeamShared* sh)
      : rank(kSolo ? 0 : cluster_rank()), size(kSolo ? 1 : cluster_size()), round(0), s(sh) {}
  __device__ __forceinline__ uint32_t id() const { return rank * kTeamThreads + threadIdx.x; }
  __device__ __forceinline__ uint32_t threads() const { return size * kTeamThreads; }
  // Barrier of the team; global and shared writes before it are seen after it.
  __device__ __forceinline__ void sync() const {
    if (kSolo) {
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
    if (!kSolo) {
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
// The last i < n with start(i) <= e, where start does not decrease: every
// `step`-th start is in shared memory (all of them up to kSearch), and those
// between two of them lie in a line or two of memory.
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

__device__ __forceinline__ Finder finder_of(const uint32_t* s_start, uint32_t n) {
  const uint32_t step = (n + kSearch - 1) / kSearch;
  return Finder{s_start, n, (n + step - 1) / step, step};
}

// Load the starts (every thread of a CTA; a barrier has to follow).
template <typename Start>
__device__ __forceinline__ Finder load_finder(uint32_t* s_start, uint32_t n, Start start) {
  const Finder f = finder_of(s_start, n);
  for (uint32_t k = threadIdx.x; k < f.kept; k += blockDim.x) s_start[k] = start(k * f.step);
  return f;
}

// What a team of one CTA keeps of its plan on chip instead of in the workspace.
struct SoloPlan {
  Plan plan[kTeamThreads];
  uint2 group[kTeamThreads / kRows];
};

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

// A thread's share of the free bits: `words` consecutive words from `first` on,
// one where the team has a thread for each, else a multiple of four, of which
// the first four stay in registers.
struct Bits {
  uint32_t first, words;
  uint32_t before;  // free pages before them
  uint32_t total;   // free pages of the cache
  uint4 v;
};

template <bool kSolo>
__device__ __forceinline__ Bits scan_free(Team<kSolo>& team, const uint32_t* bits,
                                          uint32_t n_pages) {
  const uint32_t all = (n_pages + 31) / 32, threads = team.threads();
  Bits b;
  b.words = all <= threads ? 1 : 4 * ((all + 4 * threads - 1) / (4 * threads));
  b.first = team.id() * b.words;
  b.v = make_uint4(0, 0, 0, 0);
  uint32_t c = 0;
  if (b.words == 1) {
    if (b.first < all) b.v.x = ld_word(bits, b.first, n_pages);
    c = __popc(b.v.x);
  } else {
    for (uint32_t s = 0; s < b.words && b.first + s < all; s += 4) {
      const uint32_t w = b.first + s;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (w + 4 < all) {
        v = __ldcg(reinterpret_cast<const uint4*>(bits + w));
      } else {
        v.x = ld_word(bits, w, n_pages);
        if (w + 1 < all) v.y = ld_word(bits, w + 1, n_pages);
        if (w + 2 < all) v.z = ld_word(bits, w + 2, n_pages);
        if (w + 3 < all) v.w = ld_word(bits, w + 3, n_pages);
      }
      c += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
      if (s == 0) b.v = v;
    }
  }
  Sum total;
  b.before = (uint32_t)team.scan(Sum{c, 0}, &total).a;
  b.total = (uint32_t)total.a;
  return b;
}

// f(word's index, its free bits, free pages before it) for every word, by whole
// warps (a lane without a word has no free bits and an index past the words).
template <typename F>
__device__ __forceinline__ void each_word(const Bits& b, const uint32_t* bits, uint32_t n_pages,
                                          F f) {
  const uint32_t all = (n_pages + 31) / 32;
  uint32_t before = b.before;
  for (uint32_t s = 0; s < b.words; ++s) {
    const uint32_t w = b.first + s;
    uint32_t v = s == 0 ? b.v.x : s == 1 ? b.v.y : s == 2 ? b.v.z : b.v.w;
    if (s >= 4) v = w < all ? ld_word(bits, w, n_pages) : 0;
    f(w, v, before);
    before += __popc(v);
  }
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
  bool rest;  // a second kernel follows
  Work w;
};

// Each thread's columns into the groups; ends with every group of these
// requests written (not yet visible to other CTAs). `carry`: units before.
template <bool kSolo>
__device__ __forceinline__ void plan_rows(Team<kSolo>& team, const Rows& p, SoloPlan* solo,
                                          uint32_t i, const Plan& pl, uint32_t* carry) {
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
    const uint2 g = make_uint2(*carry + (uint32_t)x.a, lo);
    st_plan(&p.w.plan[i], pl);  // for the second kernel, when there is one
    if (first) p.w.group[i / kRows] = g;
    if (kSolo) {
      st_plan(&solo->plan[i], pl);
      if (first) solo->group[i / kRows] = g;
    }
  }
  *carry += (uint32_t)total.a;
}

struct GroupStart {
  const uint2* group;
  __device__ __forceinline__ uint32_t operator()(uint32_t g) const { return group[g].x; }
};

// Where the units of a call are found.
struct Units {
  Finder f;
  const Plan* plan;
  const uint2* group;
  uint32_t n;
  // The rows of unit u: lane j < kRows holds the j-th plan (empty if there is
  // none); returns this lane's column.
  __device__ __forceinline__ uint32_t load(uint32_t u, uint32_t lane, Plan* pl) const {
    const uint32_t g = f.find(u, GroupStart{group});
    const uint2 at = group[g];
    const uint32_t i = g * kRows + lane;
    *pl = Plan{0, 0, 0, 0};
    if (lane < kRows && i < n) *pl = ld_plan(&plan[i]);
    return at.y + (u - at.x) * 32 + lane;
  }
};

__device__ __forceinline__ Units find_units(const Rows& p, const Plan* plan, const uint2* group,
                                            uint32_t* s_start) {
  Units x;
  x.plan = plan;
  x.group = group;
  x.n = p.n;
  x.f = load_finder(s_start, (p.n + kRows - 1) / kRows, GroupStart{group});
  __syncthreads();
  return x;
}

// ---------------------------------------------------------------------- free
struct FreeParams {
  Rows r;
  const db_page_cut* req;
};

__device__ __forceinline__ void free_units(const Rows& p, const Units& x, uint32_t first,
                                           uint32_t stride, uint32_t units) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t released = 0;
  bool bad = false;
  for (uint32_t u = first; u < units; u += stride) {
    Plan pl;
    const uint32_t c = x.load(u, lane, &pl);
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
    uint32_t refs[kRows], times[kRows];
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      times[j] = refs[j] = 0;
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
      refs[j] = __ldcg(&p.t.refs[page[j]]);
    }
    // References that are down to these rows' are nobody else's to drop, in
    // this call or before: a store does, and most pages have one reference.
#pragma unroll
    for (uint32_t j = 0; j < kRows; ++j) {
      if (!times[j]) continue;
      bool last = refs[j] == times[j];
      if (last) {
        p.t.refs[page[j]] = 0;
      } else if (refs[j] > times[j]) {
        last = atomicSub(&p.t.refs[page[j]], times[j]) == times[j];
      } else {  // more rows than references
        bad = true;
      }
      if (last) {
        atomicOr(&p.t.free[page[j] >> 5], 1u << (page[j] & 31));
        ++released;
      }
    }
  }
  if (p.ctr) {
    add_count(&p.ctr->total, released);
    add_error(p.ctr, bad);
  }
}

template <bool kSolo>
__global__ void __launch_bounds__(kTeamThreads) page_free_kernel(const FreeParams q) {
  __shared__ TeamShared s_team;
  __shared__ SoloPlan s_plan;
  __shared__ uint32_t s_start[kSolo ? kTeamThreads / kRows : kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  Team<kSolo> team(&s_team);
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
    plan_rows(team, p, &s_plan, i, pl, &units);
  }
  if (p.ctr) add_count(&p.ctr->n_invalid, invalid);
  const bool own = !p.rest || units <= kOwnUnits * team.size;
  if (team.id() == 0) p.w.head->units = own ? 0 : units;
  team.sync();
  if (!own || !units) return;
  const Units x = find_units(p, kSolo ? s_plan.plan : p.w.plan, kSolo ? s_plan.group : p.w.group,
                             s_start);
  free_units(p, x, team.id() / 32, team.threads() / 32, units);
}

__global__ void __launch_bounds__(256) page_free_units_kernel(const FreeParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = __ldcg(&p.w.head->units);
  if (blockIdx.x * 8 >= units) return;
  const Units x = find_units(p, p.w.plan, p.w.group, s_start);
  free_units(p, x, blockIdx.x * 8 + threadIdx.x / 32, gridDim.x * 8, units);
}

// ---------------------------------------------------------------------- fork
struct ForkParams {
  Rows r;
  const db_page_fork_req* req;
};

__device__ __forceinline__ void fork_units(const Rows& p, const Units& x, uint32_t first,
                                           uint32_t stride, uint32_t units) {
  const uint32_t lane = threadIdx.x & 31;
  bool bad = false;
  for (uint32_t u = first; u < units; u += stride) {
    Plan pl;
    const uint32_t c = x.load(u, lane, &pl);
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

template <bool kSolo>
__global__ void __launch_bounds__(kTeamThreads) page_fork_kernel(const ForkParams q) {
  __shared__ TeamShared s_team;
  __shared__ SoloPlan s_plan;
  __shared__ uint32_t s_start[kSolo ? kTeamThreads / kRows : kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  Team<kSolo> team(&s_team);
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
    plan_rows(team, p, &s_plan, i, pl, &units);
  }
  if (p.ctr) {
    add_count(&p.ctr->n_invalid, invalid);
    const uint64_t c = warp_sum64(taken);
    if ((threadIdx.x & 31) == 0 && c)
      atomicAdd((unsigned long long*)&p.ctr->total, (unsigned long long)c);
  }
  const bool own = !p.rest || units <= kOwnUnits * team.size;
  if (team.id() == 0) p.w.head->units = own ? 0 : units;
  // every length was read before the last scan
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t row = kSolo ? s_plan.plan[i].row : p.w.plan[i].row;
    if (row != kNoMove) p.t.length[row] = q.req[i].tokens;
  }
  team.sync();
  if (!own || !units) return;
  const Units x = find_units(p, kSolo ? s_plan.plan : p.w.plan, kSolo ? s_plan.group : p.w.group,
                             s_start);
  fork_units(p, x, team.id() / 32, team.threads() / 32, units);
}

__global__ void __launch_bounds__(256) page_fork_units_kernel(const ForkParams q) {
  __shared__ uint32_t s_start[kSearch];
  const Rows& p = q.r;
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t units = __ldcg(&p.w.head->units);
  if (blockIdx.x * 8 >= units) return;
  const Units x = find_units(p, p.w.plan, p.w.group, s_start);
  fork_units(p, x, blockIdx.x * 8 + threadIdx.x / 32, gridDim.x * 8, units);
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
  bool mine, ok, corrupt;
  __device__ __forceinline__ bool shares() const { return part && refs > 1; }
};

__device__ __forceinline__ Ask ask(const ExtendParams& p, uint32_t i) {
  Ask a = {0, 0, 0, 0, 0, 0, 0, false, false, false};
  if (i >= p.n) return a;
  const db_page_grow r = p.req[i];
  a.seq = r.seq;
  if (r.seq >= p.t.n_seqs) return a;
  const uint32_t len = p.t.length[r.seq], of = __ldcg(&p.w.claim[r.seq]);
  const uint64_t now = (uint64_t)len + r.tokens;
  const bool fits = now <= (uint64_t)p.t.columns * p.t.page_tokens && now <= 0xFFFFFFFFull;
  const uint32_t had = pages_of(len, p.t.page_tokens), part = len % p.t.page_tokens;
  // its page is looked up before it is known whose sequence it is
  uint32_t last = 0, refs = 0;
  if (fits && r.tokens && part) {
    last = (uint32_t)p.t.table[(uint64_t)r.seq * p.t.columns + had - 1];
    if (last < p.t.n_pages) refs = __ldcg(&p.t.refs[last]);
  }
  a.mine = of == 0xFFFFFFFFu - i;
  if (!a.mine || !fits) return a;
  a.corrupt = last >= p.t.n_pages;
  a.ok = !a.corrupt;
  if (!a.ok) return a;
  a.now = (uint32_t)now;
  a.had = had;
  a.grow = pages_of(now, p.t.page_tokens) - had;
  if (r.tokens) a.part = part;
  a.last = last;
  a.refs = refs;
  return a;
}

struct PlanStart {
  const Plan* plan;
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return plan[i].end; }
};
struct WordStart {
  const uint32_t* before;
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const { return before[w]; }
};

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

template <bool kSolo>
__global__ void __launch_bounds__(kTeamThreads) page_extend_kernel(const ExtendParams p) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kSolo ? kTeamThreads : kSearch], s_word[kSearch];
  __shared__ Plan s_plan[kSolo ? kTeamThreads : 1];
  __shared__ uint32_t s_before[kSolo ? kSoloWords : 1], s_bits[kSolo ? kSoloWords : 1];
  wait_for_prerequisites();
  dependents_may_launch();
  Team<kSolo> team(&s_team);
  const uint32_t id = team.id(), threads = team.threads();
  const uint32_t words = (p.t.n_pages + 31) / 32;
  const bool one = kSolo || p.n <= threads;  // a thread for every request, which asks once
  if (p.ctr && id == 0) *p.ctr = db_counters{0, 0, 0, 0};
  for (uint32_t i = id; i < p.n; i += threads) {
    const uint32_t seq = p.req[i].seq;
    if (seq < p.t.n_seqs) claim(p.w.claim, seq, i);
  }
  const Bits bits = scan_free(team, p.t.free, p.t.n_pages);  // its barrier is the claims'
  // How many of the batch's requests hold each shared page, and the last of
  // them; requests of a warp that hold the same one (samples of one prompt)
  // count together.
  Ask a = {0, 0, 0, 0, 0, 0, 0, false, false, false};
  bool shares = false;
  for (uint32_t i0 = 0; i0 < p.n; i0 += threads) {
    const uint32_t i = i0 + id;
    a = ask(p, i);
    if (a.shares()) {
      shares = true;
      const uint32_t same = __match_any_sync(__activemask(), a.last);
      if ((same & lanemask_lt()) == 0) {
        atomicAdd(&p.w.holders[a.last], (uint32_t)__popc(same));
        atomicMax(&p.w.latest[a.last], i + (31 - __clz(same)) - (threadIdx.x & 31));
      }
    }
  }
  if (kSolo) shares = __syncthreads_or(shares); else team.sync();
  uint64_t need = 0;
  uint32_t n_moves = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += threads) {
    const uint32_t i = i0 + id;
    if (!one) a = ask(p, i);
    uint32_t cow = 0;
    if ((!kSolo || shares) && a.shares())
      cow = !(__ldcg(&p.w.holders[a.last]) == a.refs && __ldcg(&p.w.latest[a.last]) == i);
    Sum total;
    const Sum x = team.scan(Sum{(uint64_t)a.grow + cow, cow}, &total);
    if (i < p.n) {
      const Plan pl = {a.seq, a.had - cow, (uint32_t)min(need + x.a, (uint64_t)0xFFFFFFFFu),
                       cow ? n_moves + x.b : kNoMove};
      st_plan(&p.w.plan[i], pl);
      if (kSolo) {
        st_plan(&s_plan[i], pl);
        s_start[i] = pl.end;
      }
    }
    need += total.a;
    n_moves += total.b;
  }
  const bool go = need <= bits.total;
  const bool own = !p.rest || need <= (uint64_t)kOwnPages * threads;
  if (id == 0) {
    *p.n_moves = go ? n_moves : 0;
    p.w.head->units = go && !own ? (uint32_t)need : 0;
    if (p.ctr) p.ctr->total = need;
  }
  // The words as they were, to find the pages in, and without those taken.
  if (go && need) {
    const uint32_t stop = (uint32_t)need;
    const Finder f = finder_of(s_word, words);
    each_word(bits, p.t.free, p.t.n_pages, [&](uint32_t w, uint32_t free, uint32_t before) {
      if (w >= words) return;
      if (kSolo) {
        s_before[w] = before;
        s_bits[w] = free;
        if (w % f.step == 0) s_word[w / f.step] = before;
      }
      if (!kSolo || !own) {
        p.w.before[w] = before;
        p.w.bits[w] = free;
      }
      if (free && before < stop) {
        uint32_t left = 0;
        if (before + __popc(free) > stop)
          left = free & ~((2u << nth_bit(free, stop - before - 1)) - 1);
        p.t.free[w] = left;
      }
    });
  }
  // Every request has been asked before the last scan. Lengths, moves and
  // status, and the workspace as the next call wants it.
  uint32_t invalid = 0, refused = 0;
  bool corrupt = false;
  for (uint32_t i = id; i < p.n; i += threads) {
    if (!one) a = ask(p, i);
    const uint32_t m = kSolo ? s_plan[i].aux : p.w.plan[i].aux;
    if (m != kNoMove) {  // at least one holder of every shared page copies, and clears for all
      p.w.holders[a.last] = 0;
      p.w.latest[a.last] = 0;
      if (go) {
        const uint32_t same = __match_any_sync(__activemask(), a.last);
        if ((same & lanemask_lt()) == 0) atomicSub(&p.t.refs[a.last], (uint32_t)__popc(same));
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
  team.sync();  // plan and words are known, and the replaced entries have been read
  if (!go || !need || !own) return;
  if (kSolo) {
    place_pages(p, Finder{s_start, p.n, p.n, 1}, s_plan, finder_of(s_word, words), s_before, s_bits,
                id, threads, (uint32_t)need);
  } else {
    const Finder r = load_finder(s_start, p.n, PlanStart{p.w.plan});
    const Finder f = load_finder(s_word, words, WordStart{p.w.before});
    __syncthreads();
    place_pages(p, r, p.w.plan, f, p.w.before, p.w.bits, id, threads, (uint32_t)need);
  }
}

__global__ void __launch_bounds__(256) page_place_kernel(const ExtendParams p) {
  __shared__ uint32_t s_start[kSearch], s_word[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint32_t total = p.w.head->units;
  if (blockIdx.x * 256 >= total) return;
  const Finder r = load_finder(s_start, p.n, PlanStart{p.w.plan});
  const Finder f = load_finder(s_word, (p.t.n_pages + 31) / 32, WordStart{p.w.before});
  __syncthreads();
  place_pages(p, r, p.w.plan, f, p.w.before, p.w.bits, blockIdx.x * 256 + threadIdx.x,
              gridDim.x * 256, total);
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

// Live pages before a word.
struct LiveStart {
  const uint32_t* before;
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const { return 32 * w - before[w]; }
};

template <bool kSolo>
__global__ void __launch_bounds__(kTeamThreads) page_compact_plan_kernel(const CompactParams p) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_word[kSearch], s_live[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  Team<kSolo> team(&s_team);
  const uint32_t id = team.id(), threads = team.threads();
  const uint32_t n_pages = p.t.n_pages, words = (n_pages + 31) / 32;
  const Bits bits = scan_free(team, p.t.free, n_pages);
  const uint32_t n_live = n_pages - bits.total;
  // M, the free pages below n_live: known to the thread that has the word.
  each_word(bits, p.t.free, n_pages, [&](uint32_t w, uint32_t free, uint32_t before) {
    if (w >= words) return;
    p.w.before[w] = before;
    if (w == n_live / 32)
      p.w.head->holes = before + __popc(free & ((1u << (n_live & 31)) - 1));
  });
  if (n_live == n_pages && id == 0) p.w.head->holes = 0;
  team.sync();
  const uint32_t holes = __ldcg(&p.w.head->holes), moved = min(holes, p.cap);
  if (id == 0) {
    *p.n_moves = moved;
    p.w.head->moved = moved;
    if (moved == 0) {
      p.w.head->src_first = n_pages;
      p.w.head->dst_last = 0;
    }
    if (p.ctr) *p.ctr = db_counters{holes, 0, (uint64_t)holes - moved, 0};
  }
  if (!moved) return;
  const Finder f = load_finder(s_word, words, WordStart{p.w.before});
  const Finder g = load_finder(s_live, words, LiveStart{p.w.before});
  __syncthreads();
  for (uint32_t k = id; k < moved; k += threads) {
    // the k-th free page, and the k-th live one from above
    const uint32_t v = f.find(k, WordStart{p.w.before});
    const uint32_t dst = 32 * v + nth_bit(ld_word(p.t.free, v, n_pages), k - p.w.before[v]);
    const uint32_t e = n_live - 1 - k, w = g.find(e, LiveStart{p.w.before});
    const uint32_t src = 32 * w + nth_bit(~ld_word(p.t.free, w, n_pages), e - (32 * w - p.w.before[w]));
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
      if (was < n_pages) is = __ldcg(&p.w.renamed[was]); else bad = true;
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

// CTAs of a team that wants `threads`.
uint32_t team_size(uint64_t threads) {
  uint32_t c = 1;
  while (c < kMaxTeam && (uint64_t)c * kTeamThreads < threads) c *= 2;
  return c;
}
inline uint64_t most_of(uint64_t a, uint64_t b) { return a > b ? a : b; }

// CTAs of 256 threads for at most `threads`.
unsigned whole_grid(uint64_t threads) {
  const uint64_t want = (threads + 255) / 256, most = 4ull * num_sms();
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

// Free and fork: the team, and the whole GPU where there may be much to do.
template <typename P>
int launch_rows(void (*solo)(P), void (*team)(P), void (*rest)(P), cudaStream_t s, P& p) {
  const uint64_t units = ((uint64_t)p.r.n + kRows - 1) / kRows * (((uint64_t)p.r.t.columns + 31) / 32);
  const uint32_t ctas = team_size(p.r.n);
  p.r.rest = units > kRestUnits;
  const int e = launch_team(ctas == 1 ? solo : team, ctas, s, p);
  if (e || !p.r.rest) return e;
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
  return launch_rows(page_free_kernel<true>, page_free_kernel<false>, page_free_units_kernel, s, p);
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
  return launch_rows(page_fork_kernel<true>, page_fork_kernel<false>, page_fork_units_kernel, s, p);
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
  const uint32_t words = (t->n_pages + 31) / 32;
  const uint32_t ctas = team_size(words > kSoloWords ? most_of(n, words / 4) + kTeamThreads : n);
  p.rest = pages > kRestPages;
  const int e = launch_team(ctas == 1 ? page_extend_kernel<true> : page_extend_kernel<false>, ctas, s, p);
  if (e || !p.rest) return e;
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
  const uint32_t ctas = team_size(((uint64_t)t->n_pages + 31) / 32);
  const int e = launch_team(ctas == 1 ? page_compact_plan_kernel<true> : page_compact_plan_kernel<false>,
                            ctas, s, p);
  if (e) return e;
  const uint64_t entries = (uint64_t)t->n_seqs * t->columns;
  return launch_dependent(page_compact_apply_kernel,
                          whole_grid(entries > t->n_pages ? entries : t->n_pages), 256, 0, s, p);
}
