// Verification of drafted tokens (include/cachedata.h: db_draft_verify).
//
// A request's walk through its tree needs a few numbers, p and q at its
// drafted tokens, which are all fetched at once; then one row of p (and of q)
// from end to end for the token that is drawn where the walk ends, and one
// for each child that was refused by a drafter's probabilities. That row is
// what bounds the call: memory, or for few requests the latency of the chain
// start -> nodes -> p and q at their tokens -> row -> the drawn token.
//
// A cluster of CTAs works on one request. Each makes the same walk (the same
// numbers give the same decisions, so nothing has to be told), and sums its
// share of a row; every warp has a range of neighbouring tokens. The sums are
// of integers (multiples of 2^-44), which need no order, and say in which
// warp's range the drawn token lies: only that range is read again.
#include "cachedata.cuh"

namespace db {
namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kMaxNodes = 1024;
constexpr uint32_t kMaxCluster = 8;
// A request gets twice as many CTAs while each still has kMinTokens tokens and
// all together are at most kCtas an SM: a walk's rows follow one another, so a
// row should be short for each. 256 trees over 50,001 tokens: 117 us with at
// most 4 CTAs an SM, 76 with 8, 75 with 16; 48 chains over 32,000: 9.0 us with
// 4,096 tokens at least, 8.3 with 2,048.
constexpr uint32_t kMinTokens = 2048, kCtas = 16;
constexpr int kUnroll = 8;

struct VerifyParams {
  const int32_t* start;
  uint32_t n, rows;
  const int32_t* parent;
  const int32_t* token;
  const void* p;
  const void* q;
  uint64_t p_stride, q_stride;
  uint32_t vocab, cluster, range;  // range: tokens of a warp
  const float* u;
  int32_t* path;
  int32_t* accepted;
  int32_t* next;
  uint8_t* status;
  db_counters* ctr;
};

__device__ __forceinline__ float probability(float x) { return __saturatef(x); }  // NaN: 0

// Weights from 0 to 1 as multiples of 2^-44, rounded to nearest even, summed
// without conversions to 64 bits (a quarter of the rate and less): what is
// added to 6 is rounded to multiples of 2^-21, which end up in the float's low
// bits; the rest, at most 2^-22, is exact, and added to 1.5 * 2^-21 gives the
// multiples of 2^-44 in the same way. Constants are taken off for many at once.
constexpr float kHigh = 6.f, kLow = 1.5f / 2097152.f;
struct Parts {
  uint32_t high = 0, low = 0;  // of up to 32 weights
  __device__ __forceinline__ void add(float w) {
    const float t = __fadd_rn(w, kHigh);
    high += __float_as_uint(t) - __float_as_uint(kHigh);
    low += __float_as_uint(__fadd_rn(w - __fsub_rn(t, kHigh), kLow)) - __float_as_uint(kLow);
  }
  __device__ __forceinline__ uint64_t sum() const {
    return ((uint64_t)high << 23) + (uint64_t)(int64_t)(int32_t)low;
  }
};
__device__ __forceinline__ uint64_t fixed(float w) {
  Parts p;
  p.add(w);
  return p.sum();
}

struct Shared {
  int32_t parent[kMaxNodes];
  int32_t token[kMaxNodes];
  float u[kMaxNodes], pt[kMaxNodes], qt[kMaxNodes];
  int32_t path[kMaxNodes];
  // with a drafter: 1 / W of each step of w at the current node; without: the
  // refused children there
  union {
    float by[kMaxNodes];
    int32_t refused[kMaxNodes];
  };
  uint64_t sums[2][kMaxCluster * kWarps];  // of all warps of the cluster
  uint64_t scan[kWarps];
  uint64_t excl;
  uint32_t here, level, accepted, done, range;
};

// w of a token whose probabilities are p and q, after `level` refusals.
template <bool kDraft>
__device__ __forceinline__ float weight(float p, float q, const Shared& s, uint32_t level) {
  float w = p;
  if (kDraft)
    for (uint32_t k = 0; k < level; ++k) w = fmaxf(__fmaf_rn(w, s.by[k], -q), 0.f);
  return w;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of w over all tokens, a range for each warp of the cluster, in
// s.sums[turn]. (w without the refused children where there is no drafter.)
template <typename T, bool kDraft>
__device__ __forceinline__ void sum_row(const VerifyParams& a, Shared& s, uint32_t rank, uint64_t row,
                                        uint32_t level, uint32_t turn) {
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = rank * kWarps + warp;
  const T* const p = (const T*)a.p + row * a.p_stride;
  const T* const q = kDraft ? (const T*)a.q + row * a.q_stride : nullptr;
  const uint32_t t0 = min((uint64_t)g * a.range, (uint64_t)a.vocab), t1 = min(t0 + a.range, a.vocab);
  uint64_t sum = 0;
  const auto go_through = [&](auto weigh, bool with_q) __attribute__((always_inline)) {
    for (uint32_t t = t0 + lane; t < t1; t += 32 * kUnroll) {
      float x[kUnroll], y[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const bool in = t + 32 * k < t1;
        x[k] = in ? to_float(p[t + 32 * k]) : 0.f;
        y[k] = with_q && in ? to_float(q[t + 32 * k]) : 0.f;
      }
      Parts parts;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) parts.add(weigh(probability(x[k]), probability(y[k])));
      sum += parts.sum();
    }
  };
  // the first refusals without a loop over them for each token
  if (!kDraft || level == 0) {
    go_through([](float x, float) { return x; }, false);
  } else if (level == 1) {
    const float a0 = s.by[0];
    go_through([&](float x, float y) { return fmaxf(__fmaf_rn(x, a0, -y), 0.f); }, true);
  } else {
    go_through([&](float x, float y) { return weight<kDraft>(x, y, s, level); }, true);
  }
  sum = warp_sum64(sum);
  if (!kDraft)
    for (uint32_t k = 0; k < level; ++k) {
      const int32_t c = s.refused[k];
      if ((uint32_t)s.token[c] >= t0 && (uint32_t)s.token[c] < t1) sum -= fixed(s.pt[c]);
    }
  if (a.cluster == 1) {
    if (lane == 0) s.sums[turn][g] = sum;
    __syncthreads();
  } else {
    if (lane < a.cluster) {
      uint32_t to;
      asm("mapa.shared::cluster.u32 %0, %1, %2;"
          : "=r"(to)
          : "r"((uint32_t)__cvta_generic_to_shared(&s.sums[turn][g])), "r"(lane));
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(sum) : "memory");
    }
    cluster_barrier();
  }
}

// The sum of all ranges, by a whole warp; each lane gets what is before its
// four ranges and their sums.
__device__ __forceinline__ uint64_t total_of(const Shared& s, uint32_t turn, uint32_t ranges,
                                             uint64_t& before, uint64_t* mine) {
  const uint32_t lane = threadIdx.x & 31;
  uint64_t sum = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    mine[k] = 4 * lane + k < ranges ? s.sums[turn][4 * lane + k] : 0;
    sum += mine[k];
  }
  uint64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= (uint32_t)o) x += y;
  }
  before = x - sum;
  return __shfl_sync(kFull, x, 31);
}

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const VerifyParams a) {
  __shared__ Shared s;
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const uint32_t i = blockIdx.x / a.cluster, rank = blockIdx.x - i * a.cluster;
  wait_for_prerequisites();
  dependents_may_launch();
  const int32_t b0 = __ldg(a.start + i), b1 = __ldg(a.start + i + 1);
  const bool placed = b0 >= 0 && b0 <= b1 && (uint32_t)b1 <= a.rows;
  const uint32_t first = (uint32_t)b0, m = placed ? (uint32_t)(b1 - b0) : 0;
  bool bad = !m || m > kMaxNodes;
  if (!bad)
    for (uint32_t j = tid; j < m; j += kThreads) {
      const uint32_t r = first + j;
      int32_t above = j ? __ldg(a.parent + r) : -1, t = j ? __ldg(a.token + r) : 0;
      const bool wrong = j && ((uint32_t)above >= j || (uint32_t)t >= a.vocab);
      bad |= wrong;
      if (wrong) above = -1, t = 0;
      s.parent[j] = above;
      s.token[j] = t;
      s.u[j] = fminf(fmaxf(__ldg(a.u + r), 0.f), 0.99999994f);
      const uint64_t from = first + (above < 0 ? 0 : above);
      s.pt[j] = probability(to_float(((const T*)a.p)[from * a.p_stride + t]));
      s.qt[j] = kDraft ? probability(to_float(((const T*)a.q)[from * a.q_stride + t])) : 1.f;
    }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (rank == 0) {
      for (uint32_t j = tid; j < m; j += kThreads) a.path[first + j] = -1;
      if (tid == 0) {
        a.accepted[i] = 0;
        a.next[i] = -1;
        if (a.status) a.status[i] = DB_PAGE_INVALID;
        if (a.ctr) atomicAdd((unsigned long long*)&a.ctr->n_invalid, 1ull);
      }
    }
    return;
  }
  if (a.cluster > 1) cluster_barrier();  // all have started: their shared memory may be written

  // Warp 0 walks. `level` refusals at node `here`; W as a number.
  uint32_t here = 0, level = 0, accepted = 1, j = 1, turn = 0;
  double W = 1.0;
  if (tid == 0) s.path[0] = 0;
  for (;;) {
    if (warp == 0) {
      bool wants = false;
      while (j < m) {
        // the next child of `here` from node j on
        const uint32_t x = j + lane;
        const uint32_t votes = __ballot_sync(kFull, x < m && (uint32_t)s.parent[x] == here);
        if (!votes) {
          j += 32;
          continue;
        }
        const uint32_t c = j + __ffs(votes) - 1;
        j = c + 1;
        float w = weight<kDraft>(s.pt[c], s.qt[c], s, level);
        bool again = false;  // a token that was refused here before
        if (!kDraft)
          for (uint32_t k = 0; k < level; ++k) again |= s.token[s.refused[k]] == s.token[c];
        if (again) w = 0.f;
        if ((double)s.u[c] * (double)s.qt[c] * W < (double)w) {
          here = c;
          level = 0;
          W = 1.0;
          if (lane == 0) s.path[accepted] = (int32_t)c;
          ++accepted;
        } else if (kDraft) {
          if (lane == 0) s.by[level] = W > 0.0 ? (float)(1.0 / W) : 1.f;
          ++level;
          wants = true;
          break;
        } else if (!again) {
          if (lane == 0) s.refused[level] = (int32_t)c;
          ++level;
          W -= (double)w;
        }
        __syncwarp();
      }
      if (lane == 0) {
        s.here = here;
        s.level = level;
        s.accepted = accepted;
        s.done = !wants;
      }
    }
    __syncthreads();
    here = s.here;
    level = s.level;
    const bool done = s.done;
    if (!done || !(kDraft && level)) {
      turn ^= 1;
      sum_row<T, kDraft>(a, s, rank, (uint64_t)first + here, level, turn);
    }
    if (done) break;
    if (warp == 0) {
      uint64_t before, mine[4];
      W = (double)total_of(s, turn, a.cluster * kWarps, before, mine) * (1.0 / 17592186044416.0);
    }
    __syncthreads();
  }
  accepted = s.accepted;

  // The drawn token: its warp's range, then the range's tokens.
  const uint32_t ranges = a.cluster * kWarps;
  uint64_t target = 0;
  for (int tries = 0;; ++tries) {
    uint64_t before, mine[4];
    const uint64_t total = total_of(s, turn, ranges, before, mine);
    if (total || tries) {
      target = __umul64hi(total, __float2ull_rz(s.u[0] * 18446744073709551616.f));
      if (warp == 0) {
        if (!total) {
          if (lane == 0) s.range = ranges;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (target >= before && target - before < mine[k]) {
              s.range = 4 * lane + k;
              s.excl = before;
            }
            before += mine[k];
          }
        }
      }
      break;
    }
    level = 0;  // nothing is left: the target's own probabilities
    turn ^= 1;
    sum_row<T, kDraft>(a, s, rank, (uint64_t)first + here, 0, turn);
  }
  __syncthreads();
  const uint32_t range = s.range;
  if (range == ranges) {
    if (rank == 0 && tid == 0) a.next[i] = -1;
  } else if (range / kWarps == rank) {
    target -= s.excl;
    const T* const p = (const T*)a.p + ((uint64_t)first + here) * a.p_stride;
    const T* const q = kDraft ? (const T*)a.q + ((uint64_t)first + here) * a.q_stride : nullptr;
    const uint32_t t0 = range * a.range, t1 = min(t0 + a.range, a.vocab);
    const uint32_t each = (a.range + kThreads - 1) / kThreads;
    const uint32_t from = min(t0 + tid * each, t1), to = min(from + each, t1);
    const auto at = [&](uint32_t t) {
      if (!kDraft)
        for (uint32_t k = 0; k < level; ++k)
          if (s.token[s.refused[k]] == (int32_t)t) return (uint64_t)0;
      const float y = kDraft && level ? probability(to_float(q[t])) : 0.f;
      return fixed(weight<kDraft>(probability(to_float(p[t])), y, s, level));
    };
    uint64_t sum = 0, excl, all;
    for (uint32_t t = from; t < to; ++t) sum += at(t);
    block_excl_scan64<kWarps>(sum, excl, all, s.scan);
    if (target >= excl && target - excl < sum) {
      uint64_t x = excl;
      for (uint32_t t = from; t < to; ++t) {
        x += at(t);
        if (x > target) {
          a.next[i] = (int32_t)t;
          break;
        }
      }
    }
  }
  if (rank == 0) {
    for (uint32_t k = tid; k < m; k += kThreads) a.path[first + k] = k < accepted ? s.path[k] : -1;
    if (tid == 0) {
      a.accepted[i] = (int32_t)accepted;
      if (a.status) a.status[i] = DB_PAGE_OK;
      if (a.ctr) atomicAdd((unsigned long long*)&a.ctr->total, (unsigned long long)m);
    }
  }
}

template <typename T>
int launch_verify(VerifyParams& p, cudaStream_t s) {
  p.cluster = 1;
  while (p.cluster < kMaxCluster && p.n * (uint64_t)p.cluster * 2 <= kCtas * (uint64_t)num_sms() &&
         p.vocab / (p.cluster * 2) >= kMinTokens)
    p.cluster *= 2;
  const uint32_t warps = p.cluster * kWarps;
  p.range = (p.vocab + warps - 1) / warps;
  p.range = (p.range + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n * p.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = p.q ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, true>, p)
                            : cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, false>, p);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_result();
}

}  // namespace
}  // namespace db

using namespace db;

extern "C" int db_draft_verify(const int32_t* start, uint32_t n, uint32_t rows, const int32_t* parent,
                               const int32_t* token, const void* p, uint64_t p_stride, const void* q,
                               uint64_t q_stride, uint32_t type, uint32_t vocab, const float* u,
                               int32_t* path, int32_t* accepted, int32_t* next, uint8_t* status,
                               db_counters* ctr, void* stream) {
  if (type > DB_F32 || !vocab || vocab > 1u << 19 || n >= 1u << 28 || rows >= 1u << 31) return -EINVAL;
  const uint32_t size = item_bytes(type);
  if (!aligned(start, 4) || !aligned(parent, 4) || !aligned(token, 4) || !aligned(u, 4) ||
      !aligned(path, 4) || !aligned(accepted, 4) || !aligned(next, 4) || !aligned(ctr, 8) ||
      !aligned(p, size) || !aligned(q, size))
    return -EINVAL;
  if (n && (!start || !accepted || !next)) return -EINVAL;
  if (n && rows && (!parent || !token || !p || !u || !path)) return -EINVAL;
  if (rows > 1 && (p_stride < vocab || (q && q_stride < vocab))) return -EINVAL;
  if (p_stride >= 1ull << 32 || q_stride >= 1ull << 32) return -EINVAL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (const int e = zero_counters(ctr, s)) return e;
  if (!n) return 0;
  VerifyParams a = {};
  a.start = start;
  a.n = n;
  a.rows = rows;
  a.parent = parent;
  a.token = token;
  a.p = p;
  a.q = q;
  a.p_stride = p_stride;
  a.q_stride = q_stride;
  a.vocab = vocab;
  a.u = u;
  a.path = path;
  a.accepted = accepted;
  a.next = next;
  a.status = status;
  a.ctr = ctr;
  switch (type) {
    case DB_BF16:
      return launch_verify<__nv_bfloat16>(a, s);
    case DB_F16:
      return launch_verify<__half>(a, s);
    default:
      return launch_verify<float>(a, s);
  }
}
