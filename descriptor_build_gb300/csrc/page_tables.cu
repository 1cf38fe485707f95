// Page tables of a cache in the device heap: extend, fork, free, compact
// (include/pagecache.h has the definitions).
//
// A call's requests are planned by one team: a single CTA or one cluster of
// CTAs, whose barriers are the hardware's, so no kernel here waits on memory.
// The plan is a prefix sum over the requests (how many table entries or pages
// each of them has), and what follows is work on single entries found again
// in that prefix by a search in shared memory.
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
constexpr uint32_t kSearch = 4096;     // prefix entries kept in shared memory
constexpr uint32_t kNoMove = 0xFFFFFFFFu;

// One request's place in the plan.
struct __align__(16) Plan {
  uint32_t start;  // entries (or pages) of the requests before it
  uint32_t seq;    // row that is written
  uint32_t col;    // its first entry's column
  uint32_t aux;    // extend: index of its move or kNoMove; fork: the parent's row
};

// Workspace: header, then one claim a sequence, the holders of each page in
// the batch (count, latest), the plan, the free pages before each 128.
struct Head {
  unsigned long long total;  // entries of the plan
  uint32_t n_live;
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
  uint32_t* before;   // [n_quads] free pages before each quad of words
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
  x.before = (uint32_t*)take(4 * (((size_t)n_pages + 127) / 128));
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

// --------------------------------------------------------- finding an entry
// The request that entry e belongs to: the last i with start[i] <= e, among
// requests whose starts are in shared memory, every `step`-th of them when
// there are more than kSearch.
struct Finder {
  const uint32_t* s_start;
  const Plan* plan;
  uint32_t n, kept, step;
  __device__ __forceinline__ uint32_t find(uint32_t e) const {
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
        if (__ldcg(&plan[mid].start) <= e) lo = mid; else hi = mid;
      }
    }
    return lo;
  }
};

// Load the plan's starts (every thread of a CTA; ends past a barrier).
__device__ __forceinline__ Finder load_finder(uint32_t* s_start, const Plan* plan, uint32_t n) {
  Finder f;
  f.s_start = s_start;
  f.plan = plan;
  f.n = n;
  f.step = (n + kSearch - 1) / kSearch;
  f.kept = (n + f.step - 1) / f.step;
  for (uint32_t k = threadIdx.x; k < f.kept; k += blockDim.x)
    s_start[k] = __ldcg(&plan[k * f.step].start);
  __syncthreads();
  return f;
}

__device__ __forceinline__ Plan ld_plan(const Plan* p) {
  const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
  return Plan{v.x, v.y, v.z, v.w};
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
  return (uint32_t)((tokens + page_tokens - 1) / page_tokens);
}

// The four free words of quad q, with the bits past n_pages cleared.
__device__ __forceinline__ uint4 ld_quad(const uint32_t* bits, uint32_t q, uint32_t n_pages) {
  uint4 v = make_uint4(0, 0, 0, 0);
  const uint32_t words = (n_pages + 31) / 32, w = 4 * q;
  if (w + 3 < words) {
    v = __ldcg(reinterpret_cast<const uint4*>(bits) + q);
  } else {
    if (w < words) v.x = __ldcg(&bits[w]);
    if (w + 1 < words) v.y = __ldcg(&bits[w + 1]);
    if (w + 2 < words) v.z = __ldcg(&bits[w + 2]);
    if (w + 3 < words) v.w = __ldcg(&bits[w + 3]);
  }
  const uint32_t tail = n_pages & 31;
  if (tail && w + 4 >= words) {
    const uint32_t mask = (1u << tail) - 1, last = (words - 1) & 3;
    if (words > w) {
      if (last == 0) v.x &= mask;
      if (last == 1) v.y &= mask;
      if (last == 2) v.z &= mask;
      if (last == 3) v.w &= mask;
    }
  }
  return v;
}
__device__ __forceinline__ uint32_t popc4(const uint4& v) {
  return __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
}

// Free pages before each quad into `before`; returns their number.
__device__ __forceinline__ uint32_t scan_free(Team& team, const uint32_t* bits, uint32_t n_pages,
                                              uint32_t* before) {
  const uint32_t quads = (n_pages + 127) / 128;
  uint32_t carry = 0;
  for (uint32_t q0 = 0; q0 < quads; q0 += team.threads()) {
    const uint32_t q = q0 + team.id();
    const uint32_t c = q < quads ? popc4(ld_quad(bits, q, n_pages)) : 0;
    Sum total;
    const Sum x = team.scan(Sum{c, 0}, &total);
    if (q < quads) before[q] = carry + (uint32_t)x.a;
    carry += (uint32_t)total.a;
  }
  return carry;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, uint32_t k) {
  return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
}

// Add a CTA's per-thread count and error bits to the counters.
__device__ __forceinline__ void add_counts(uint64_t* total, uint64_t* err, uint32_t count,
                                           uint32_t bad) {
  const uint32_t c = warp_sum32(count);
  const uint32_t e = __any_sync(kFull, bad != 0);
  if ((threadIdx.x & 31) == 0) {
    if (c) atomicAdd((unsigned long long*)total, (unsigned long long)c);
    if (e) atomicOr((unsigned long long*)err, (unsigned long long)DB_ERR_PAGE_TABLE);
  }
}

// ---------------------------------------------------------------------- free
struct FreeParams {
  db_page_tables t;
  const db_page_cut* req;
  uint32_t n;
  uint8_t* status;
  db_counters* ctr;
  Work w;
};

// Entry e: its page loses a reference, and is free when that was the last.
__device__ __forceinline__ void free_entries(const FreeParams& p, const Finder& f, uint64_t total,
                                             uint64_t first, uint64_t stride) {
  uint32_t released = 0, bad = 0;
  for (uint64_t e = first; e < total; e += stride) {
    const Plan pl = ld_plan(&p.w.plan[f.find((uint32_t)e)]);
    int32_t* at = &p.t.table[(uint64_t)pl.seq * p.t.columns + pl.col + ((uint32_t)e - pl.start)];
    const uint32_t page = (uint32_t)*at;
    *at = DB_PAGE_NONE;
    if (page >= p.t.n_pages) {
      bad = 1;
      continue;
    }
    const uint32_t old = atomicSub(&p.t.refs[page], 1u);
    if (old == 1) {
      atomicOr(&p.t.free[page >> 5], 1u << (page & 31));
      ++released;
    } else if (old == 0) {  // a free page: leave it so
      atomicAdd(&p.t.refs[page], 1u);
      bad = 1;
    }
  }
  if (p.ctr) add_counts(&p.ctr->total, &p.ctr->err, released, bad);
}

__global__ void __launch_bounds__(kTeamThreads) page_free_plan_kernel(const FreeParams p) {
  __shared__ TeamShared s_team;
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t seq = p.req[i].seq;
    if (seq < p.t.n_seqs) claim(p.w.claim, seq, i);
  }
  team.sync();
  uint64_t carry = 0, invalid = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += team.threads()) {
    const uint32_t i = i0 + team.id();
    uint32_t from = 0, count = 0, seq = 0;
    bool ok = false;
    if (i < p.n) {
      const db_page_cut r = p.req[i];
      seq = r.seq;
      ok = seq < p.t.n_seqs && claimed(p.w.claim, seq, i);
      if (ok) {
        p.w.claim[seq] = 0;
        const uint32_t len = p.t.length[seq];
        if (r.keep < len) {
          from = pages_of(r.keep, p.t.page_tokens);
          count = min(pages_of(len, p.t.page_tokens), p.t.columns);
          count = count > from ? count - from : 0;
          p.t.length[seq] = r.keep;
        }
      }
      if (p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    }
    Sum total;
    const Sum x = team.scan(Sum{count, (uint32_t)(i < p.n && !ok)}, &total);
    if (i < p.n) p.w.plan[i] = Plan{(uint32_t)(carry + x.a), seq, from, 0};
    carry += total.a;
    invalid += total.b;
  }
  if (team.id() == 0) {
    p.w.head->total = carry;
    if (p.ctr) *p.ctr = db_counters{0, invalid, 0, 0};
  }
  team.sync();
}

__global__ void __launch_bounds__(256) page_free_entries_kernel(const FreeParams p) {
  __shared__ uint32_t s_start[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint64_t total = __ldcg(&p.w.head->total), first = (uint64_t)blockIdx.x * 256;
  if (first >= total) return;
  const Finder f = load_finder(s_start, p.w.plan, p.n);
  free_entries(p, f, total, first + threadIdx.x, (uint64_t)gridDim.x * 256);
}

// ---------------------------------------------------------------------- fork
struct ForkParams {
  db_page_tables t;
  const db_page_fork_req* req;
  uint32_t n;
  uint8_t* status;
  db_counters* ctr;
  Work w;
};

__device__ __forceinline__ void fork_entries(const ForkParams& p, const Finder& f, uint64_t total,
                                             uint64_t first, uint64_t stride) {
  uint32_t bad = 0;
  for (uint64_t e = first; e < total; e += stride) {
    const Plan pl = ld_plan(&p.w.plan[f.find((uint32_t)e)]);
    const uint32_t col = (uint32_t)e - pl.start;
    const int32_t page = p.t.table[(uint64_t)pl.aux * p.t.columns + col];
    p.t.table[(uint64_t)pl.seq * p.t.columns + col] = page;
    if ((uint32_t)page < p.t.n_pages)
      atomicAdd(&p.t.refs[page], 1u);
    else
      bad = 1;
  }
  if (p.ctr) add_counts(&p.ctr->total, &p.ctr->err, 0, bad);
}

__global__ void __launch_bounds__(kTeamThreads) page_fork_plan_kernel(const ForkParams p) {
  __shared__ TeamShared s_team;
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t child = p.req[i].child;
    if (child < p.t.n_seqs) claim(p.w.claim, child, i);
  }
  team.sync();
  uint64_t carry = 0, invalid = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += team.threads()) {
    const uint32_t i = i0 + team.id();
    db_page_fork_req r = {0, 0, 0, 0};
    uint32_t count = 0;
    bool ok = false;
    if (i < p.n) {
      r = p.req[i];
      if (r.child < p.t.n_seqs && claimed(p.w.claim, r.child, i)) {
        p.w.claim[r.child] = 0;
        ok = r.parent < p.t.n_seqs && r.parent != r.child && p.t.length[r.child] == 0 &&
             r.tokens <= p.t.length[r.parent];
      }
      if (ok) count = min(pages_of(r.tokens, p.t.page_tokens), p.t.columns);
      if (p.status) p.status[i] = ok ? DB_PAGE_OK : DB_PAGE_INVALID;
    }
    Sum total;
    const Sum x = team.scan(Sum{count, (uint32_t)(i < p.n && !ok)}, &total);
    if (i < p.n) p.w.plan[i] = Plan{(uint32_t)(carry + x.a), r.child, ok ? 1u : 0u, r.parent};
    carry += total.a;
    invalid += total.b;
  }
  if (team.id() == 0) {
    p.w.head->total = carry;
    if (p.ctr) *p.ctr = db_counters{carry, invalid, 0, 0};
  }
  team.sync();  // every length is read
  for (uint32_t i = team.id(); i < p.n; i += team.threads())
    if (p.w.plan[i].col) p.t.length[p.req[i].child] = p.req[i].tokens;
}

__global__ void __launch_bounds__(256) page_fork_entries_kernel(const ForkParams p) {
  __shared__ uint32_t s_start[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  const uint64_t total = __ldcg(&p.w.head->total), first = (uint64_t)blockIdx.x * 256;
  if (first >= total) return;
  const Finder f = load_finder(s_start, p.w.plan, p.n);
  fork_entries(p, f, total, first + threadIdx.x, (uint64_t)gridDim.x * 256);
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

// What request i asks for, from the state before the call.
struct Ask {
  bool ok;
  bool corrupt;     // its last page does not exist
  uint32_t had;     // pages before
  uint32_t grow;    // pages after - before
  uint32_t last;    // its last page, when `shared`
  uint32_t refs;    // of that page
  bool shared;      // it adds to a partly filled page with other holders
};

__device__ __forceinline__ Ask ask(const ExtendParams& p, uint32_t i, const db_page_grow& r) {
  Ask a = {false, false, 0, 0, 0, 0, false};
  if (r.seq >= p.t.n_seqs || !claimed(p.w.claim, r.seq, i)) return a;
  const uint64_t len = p.t.length[r.seq], now = len + r.tokens;
  if (now > (uint64_t)p.t.columns * p.t.page_tokens || now > 0xFFFFFFFFull) return a;
  a.ok = true;
  a.had = pages_of(len, p.t.page_tokens);
  a.grow = pages_of(now, p.t.page_tokens) - a.had;
  if (r.tokens && len % p.t.page_tokens) {
    a.last = (uint32_t)p.t.table[(uint64_t)r.seq * p.t.columns + a.had - 1];
    if (a.last >= p.t.n_pages) {
      a.ok = false;
      a.corrupt = true;
      a.grow = 0;
      return a;
    }
    a.refs = __ldcg(&p.t.refs[a.last]);
    a.shared = a.refs > 1;
  }
  return a;
}

__global__ void __launch_bounds__(kTeamThreads) page_extend_kernel(const ExtendParams p) {
  __shared__ TeamShared s_team;
  __shared__ uint32_t s_start[kSearch];
  wait_for_prerequisites();
  dependents_may_launch();
  Team team(&s_team);
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const uint32_t seq = p.req[i].seq;
    if (seq < p.t.n_seqs) claim(p.w.claim, seq, i);
  }
  const uint32_t avail = scan_free(team, p.t.free, p.t.n_pages, p.w.before);
  team.sync();
  // How many of the batch's requests hold each shared page, and the last of them.
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const Ask a = ask(p, i, p.req[i]);
    if (a.shared) {
      atomicAdd(&p.w.holders[a.last], 1u);
      atomicMax(&p.w.latest[a.last], i);
    }
  }
  team.sync();
  uint64_t total_need = 0, n_moves = 0, n_bad = 0, n_corrupt = 0;
  for (uint32_t i0 = 0; i0 < p.n; i0 += team.threads()) {
    const uint32_t i = i0 + team.id();
    Ask a = {false, false, 0, 0, 0, 0, false};
    db_page_grow r = {0, 0};
    uint32_t cow = 0;
    if (i < p.n) {
      r = p.req[i];
      a = ask(p, i, r);
      if (a.shared)
        cow = !(__ldcg(&p.w.holders[a.last]) == a.refs && __ldcg(&p.w.latest[a.last]) == i);
    }
    Sum total;
    const Sum x = team.scan(Sum{(uint64_t)a.grow + cow, cow}, &total);
    if (i < p.n)
      p.w.plan[i] = Plan{(uint32_t)min(total_need + x.a, (uint64_t)0xFFFFFFFFu), r.seq, a.had - cow,
                         cow ? (uint32_t)n_moves + x.b : kNoMove};
    total_need += total.a;
    n_moves += total.b;
    Sum bad;
    team.scan(Sum{(uint64_t)(i < p.n && !a.ok), (uint32_t)a.corrupt}, &bad);
    n_bad += bad.a;
    n_corrupt += bad.b;
  }
  const bool go = total_need <= avail;
  if (team.id() == 0) {
    *p.n_moves = go ? (uint32_t)n_moves : 0;
    if (p.ctr)
      *p.ctr = db_counters{total_need, n_bad, go ? 0 : p.n - n_bad,
                           n_corrupt ? (uint64_t)DB_ERR_PAGE_TABLE : 0};
  }
  team.sync();
  // Lengths, moves and status, and the workspace as the next call wants it.
  for (uint32_t i = team.id(); i < p.n; i += team.threads()) {
    const db_page_grow r = p.req[i];
    const bool mine = r.seq < p.t.n_seqs && claimed(p.w.claim, r.seq, i);
    bool ok = false;
    if (mine) {
      const uint32_t len = p.t.length[r.seq];
      const uint64_t now = (uint64_t)len + r.tokens;
      ok = now <= (uint64_t)p.t.columns * p.t.page_tokens && now <= 0xFFFFFFFFull;
      if (ok && r.tokens && len % p.t.page_tokens) {
        const uint32_t had = pages_of(len, p.t.page_tokens);
        const uint32_t last = (uint32_t)p.t.table[(uint64_t)r.seq * p.t.columns + had - 1];
        if (last >= p.t.n_pages) {
          ok = false;
        } else {
          p.w.holders[last] = 0;
          p.w.latest[last] = 0;
          const uint32_t m = p.w.plan[i].aux;
          if (go && m != kNoMove) {
            atomicSub(&p.t.refs[last], 1u);
            p.moves[m].src = last;
            p.moves[m].tokens = len % p.t.page_tokens;
            p.moves[m].rsvd = 0;
          }
        }
      }
      p.w.claim[r.seq] = 0;
      if (ok && go) p.t.length[r.seq] = (uint32_t)now;
    }
    if (p.status) p.status[i] = !ok ? DB_PAGE_INVALID : go ? DB_PAGE_OK : DB_PAGE_SHORT;
  }
  team.sync();  // the replaced entries have been read
  if (!go || total_need == 0) return;
  // The pages, by rank among the free ones: a warp takes 32 words, one word at
  // a time with a page per lane, so that neighbours write neighbours.
  const Finder f = load_finder(s_start, p.w.plan, p.n);
  const uint32_t lane = threadIdx.x & 31, words = (p.t.n_pages + 31) / 32;
  const uint32_t groups = (words + 31) / 32, warps = team.threads() / 32;
  for (uint32_t g = team.id() / 32; g < groups; g += warps) {
    uint32_t rank = __ldcg(&p.w.before[8 * g]);
    if (rank >= total_need) break;  // ranks grow with g
    const uint32_t w = 32 * g + lane;
    uint32_t bits = w < words ? __ldcg(&p.t.free[w]) : 0;
    if (w == words - 1 && (p.t.n_pages & 31)) bits &= (1u << (p.t.n_pages & 31)) - 1;
    uint32_t left = bits;
    for (uint32_t k = 0; k < 32; ++k) {
      const uint32_t v = __shfl_sync(kFull, bits, k);
      const uint32_t e = rank + __popc(v & lanemask_lt());
      const bool mine = (v >> lane & 1) && e < total_need;
      const uint32_t taken = __ballot_sync(kFull, mine);
      if (lane == k) left &= ~taken;
      if (mine) {
        const uint32_t page = (32 * g + k) * 32 + lane;
        const Plan pl = ld_plan(&p.w.plan[f.find(e)]);
        const uint32_t j = e - pl.start;
        p.t.table[(uint64_t)pl.seq * p.t.columns + pl.col + j] = (int32_t)page;
        p.t.refs[page] = 1;
        if (j == 0 && pl.aux != kNoMove) p.moves[pl.aux].dst = page;
      }
      rank += __popc(v);
      if (rank >= total_need) break;
    }
    if (left != bits) p.t.free[w] = left;
  }
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
  const uint32_t n_pages = p.t.n_pages;
  const uint32_t n_live = n_pages - scan_free(team, p.t.free, n_pages, p.w.before);
  team.sync();
  // M: the free pages below n_live.
  uint32_t holes;
  if (n_live == n_pages) {
    holes = 0;
  } else {
    const uint32_t q = n_live / 128;
    const uint4 v = ld_quad(p.t.free, q, n_pages);
    holes = __ldcg(&p.w.before[q]);
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t at = q * 128 + k * 32, x = word_of(v, k);
      if (n_live >= at + 32)
        holes += __popc(x);
      else if (n_live > at)
        holes += __popc(x & ((1u << (n_live - at)) - 1));
    }
  }
  const uint32_t moved = min(holes, p.cap);
  if (team.id() == 0) {
    *p.n_moves = moved;
    p.w.head->moved = moved;
    p.w.head->n_live = n_live;
    if (moved == 0) {
      p.w.head->src_first = n_pages;
      p.w.head->dst_last = 0;
    }
    if (p.ctr) *p.ctr = db_counters{holes, 0, (uint64_t)holes - moved, 0};
  }
  const uint32_t lane = threadIdx.x & 31, words = (n_pages + 31) / 32;
  const uint32_t groups = (words + 31) / 32, warps = team.threads() / 32;
  for (uint32_t g = team.id() / 32; g < groups && moved; g += warps) {
    uint32_t before = __ldcg(&p.w.before[8 * g]);
    const uint32_t w = 32 * g + lane;
    const uint32_t bits = w < words ? __ldcg(&p.t.free[w]) : 0;
    for (uint32_t k = 0; k < 32; ++k) {
      const uint32_t v = __shfl_sync(kFull, bits, k);
      const uint32_t page = (32 * g + k) * 32 + lane;
      const uint32_t rank = before + __popc(v & lanemask_lt());  // free pages before it
      if (page < n_pages) {
        if (v >> lane & 1) {
          if (page < n_live && rank < moved) {
            p.moves[rank].dst = page;
            p.moves[rank].tokens = DB_PAGE_ALL;
            p.moves[rank].rsvd = 0;
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
      before += __popc(v);
    }
  }
  team.sync();
  for (uint32_t k = team.id(); k < moved; k += team.threads()) {
    const uint32_t src = __ldcg(&p.moves[k].src), dst = __ldcg(&p.moves[k].dst);
    p.w.renamed[src] = dst;
    p.out.refs[dst] = p.t.refs[src];
    p.out.refs[src] = 0;
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
  uint32_t bad = 0;
  for (uint64_t e = id; e < entries; e += step) {
    const uint32_t was = (uint32_t)p.t.table[e];
    uint32_t is = was;
    if (was >= src_first && was != (uint32_t)DB_PAGE_NONE) {
      if (was < n_pages) is = __ldcg(&p.w.renamed[was]); else bad = 1;
    }
    if (p.out.table != p.t.table || is != was) p.out.table[e] = (int32_t)is;
  }
  if (p.ctr) add_counts(&p.ctr->total, &p.ctr->err, 0, bad);
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

uint32_t team_size() { return 1; }

// CTAs of an entries kernel over at most `entries`.
unsigned entry_grid(uint64_t entries) {
  const uint64_t want = (entries + 255) / 256, most = 8ull * num_sms();
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
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
  const int rc = check_call(t, req, 8, n, ctr, ws, ws_bytes, &p.w);
  if (rc) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, nullptr, s);
  if ((uint64_t)n * t->columns > 0xFFFFFFFFull) return -EINVAL;  // entries are numbered in 32 bits
  p.t = *t;
  p.req = req;
  p.n = n;
  p.status = status;
  p.ctr = ctr;
  const int e = launch_team(page_free_plan_kernel, team_size(), s, p);
  if (e) return e;
  return launch_dependent(page_free_entries_kernel, entry_grid((uint64_t)n * t->columns), 256, 0,
                          s, p);
}

extern "C" int db_page_fork(const db_page_tables* t, const db_page_fork_req* req, uint32_t n,
                            uint8_t* status, db_counters* ctr, void* ws, size_t ws_bytes,
                            void* stream) {
  ForkParams p = {};
  const int rc = check_call(t, req, 16, n, ctr, ws, ws_bytes, &p.w);
  if (rc) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  if (!n) return nothing(ctr, nullptr, s);
  if ((uint64_t)n * t->columns > 0xFFFFFFFFull) return -EINVAL;  // entries are numbered in 32 bits
  p.t = *t;
  p.req = req;
  p.n = n;
  p.status = status;
  p.ctr = ctr;
  const int e = launch_team(page_fork_plan_kernel, team_size(), s, p);
  if (e) return e;
  return launch_dependent(page_fork_entries_kernel, entry_grid((uint64_t)n * t->columns), 256, 0,
                          s, p);
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
  return launch_team(page_extend_kernel, team_size(), s, p);
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
  const int e = launch_team(page_compact_plan_kernel, team_size(), s, p);
  if (e) return e;
  const uint64_t entries = (uint64_t)t->n_seqs * t->columns;
  return launch_dependent(page_compact_apply_kernel,
                          entry_grid(entries > t->n_pages ? entries : t->n_pages), 256, 0, s, p);
}
