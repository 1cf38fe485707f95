// Attention over a paged cache for many query rows (cache_attention.cuh: the
// mathematics and the way work is cut): 128 rows of an item at a time, with
// tcgen05 products.
//
// A CTA has three kinds of warps that hand tiles of 64 tokens on by mbarriers:
//   loaders (4 warps)   keys and values from their pages into a ring of tiles,
//                       16-bit rows by asynchronous copies, 8-bit codes through
//                       registers, where they are widened
//   one issuing thread  S = Q K^T into TMEM (two buffers), O += P V from TMEM
//   weights (4 warps)   a thread for each query row: S -> maxima, weights P
//                       (over S in TMEM) and their sum
// so that the product of one tile runs while weights of the one before are
// made, and two CTAs share an SM. A row's maximum is followed only when it has
// risen by 2^8 (weights then are at most 2^8, which every type here holds as
// exactly as 1), so O is hardly ever rescaled.
//
// Tiles lie as the tensor cores' 128-byte swizzle wants them: panels of 64
// values, a row of 128 bytes for each token, 16-byte chunks exchanged by the
// row's number; keys are read along their rows (K-major), values across
// (MN-major).
#pragma once

#include <type_traits>

#include "cache_attention.cuh"

namespace db {

template <uint32_t kPad, bool kCodes>
struct Many {
  static constexpr uint32_t kRows = 128;
  static constexpr uint32_t kThreads = 288;
  static constexpr uint32_t kLoaders = 128, kWeights = 128;
  static constexpr uint32_t kUnit = kTile * kPad * 2;  // keys or values of a tile
  static constexpr uint32_t kUnits = kPad >= 128 ? 4 : 6;
  static constexpr uint32_t kLag = kCodes ? 2 : 3;     // units under way before one is handed on
  static constexpr uint32_t kQuery = kRows * kPad * 2;
  static constexpr uint32_t kMeta = 8;                 // tiles that notes are kept of
  static constexpr uint32_t kColumns = kPad <= 128 ? 256 : 512;  // of TMEM
  static constexpr uint32_t kBytes = kUnits * kUnit + kQuery + 1024;
  // no more than two CTAs an SM, which is what TMEM holds
  static constexpr uint32_t kAsk = kBytes < 80 * 1024 ? 80 * 1024 : kBytes;
};

// What the weights' warps need to know of a tile, by the loaders.
struct alignas(16) TileNotes {  // scales are read by fours
  int2 place[kTile];              // page (or -1) and slot of a token
  float k_scale[kTile], v_scale[kTile];
  uint32_t real[2], odd[2];       // bits of tokens: that are there; whose values are not all finite
  uint32_t exponent[2];           // of the largest scale of values
};

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for a phase; gives up after a second, or when another thread has.
static __device__ __noinline__ bool barrier_wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* failed) {
  const uint64_t began = globaltimer_ns();
  for (;;) {
    for (int k = 0; k < 32; ++k)
      if (barrier_try(bar, parity)) return true;
    if (*failed) return false;
    if (globaltimer_ns() - began > kWaitLimitNs) {
      *failed = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile uint32_t* failed) {
  if (barrier_try(bar, parity)) return true;
  return barrier_wait_long(bar, parity, failed);
}
__device__ __forceinline__ void group_sync(uint32_t id, uint32_t threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, and whether `yes` held in all of them.
__device__ __forceinline__ bool group_all(uint32_t id, uint32_t threads, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)yes)
      : "memory");
  return r;
}
__device__ __forceinline__ void writes_to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (TMEM) += A B: A from shared memory or from TMEM.
__device__ __forceinline__ void tensor_multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tensor_multiply_t(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
// A tile in shared memory: 128-byte swizzle, groups of 8 rows 1024 bytes
// apart; `panel`: bytes between panels where they lie along the rows' number.
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at, uint32_t panel) {
  return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)((panel >> 4) & 0x3FFF) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// The product's kind: 32-bit sums of 16-bit values (f16 0, bf16 1), M = 128.
__device__ __forceinline__ uint32_t product_kind(uint32_t type, uint32_t n, bool across) {
  return 1u << 4 | type << 7 | type << 10 | (across ? 1u << 16 : 0) | (n / 8) << 17 | (128u / 16) << 24;
}

#define DB_OUT8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define DB_IN8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : DB_OUT8(r, 0), DB_OUT8(r, 8), DB_OUT8(r, 16), DB_OUT8(r, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      DB_IN8(r, 0), DB_IN8(r, 8), DB_IN8(r, 16), DB_IN8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : DB_OUT8(r, 0), DB_OUT8(r, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      DB_IN8(r, 0), DB_IN8(r, 8)
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_load1(uint32_t at) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

constexpr float kSlack = 8.f;          // a maximum is followed when it has risen by this much (log2)

template <typename T, uint32_t kPad, bool kCodes>
__global__ void __launch_bounds__(288, kPad <= 128 ? 2 : 1) attention_many_kernel(const AttnParams p) {
  typedef Many<kPad, kCodes> F;
  typedef typename std::conditional<kCodes, __half, T>::type W;  // of weights and values
  constexpr uint32_t kTypeQ = std::is_same<T, __half>::value ? 0 : 1, kTypeW = std::is_same<W, __half>::value ? 0 : 1;
  constexpr uint32_t kPanel = kTile * 128, kQueryPanel = F::kRows * 128;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ TileNotes s_notes[F::kMeta];
  __shared__ uint64_t s_full[F::kUnits], s_empty[F::kUnits], s_scores[2], s_weights[2], s_output[2], s_query, s_drained;
  __shared__ uint32_t s_tmem, s_last;
  __shared__ volatile uint32_t s_failed;
  const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  unsigned char* const smem = smem_raw + ((1024 - (smem_at(smem_raw) & 1023)) & 1023);
  const uint32_t ring = smem_at(smem), query = ring + F::kUnits * F::kUnit;

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&s_tmem)), "n"(F::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (uint32_t k = 0; k < F::kUnits; ++k) {
      barrier_init(smem_at(&s_full[k]), F::kLoaders);
      barrier_init(smem_at(&s_empty[k]), 1);
    }
    for (int k = 0; k < 2; ++k) {
      barrier_init(smem_at(&s_scores[k]), 2);  // the products, and the notes that came with the keys
      barrier_init(smem_at(&s_weights[k]), F::kWeights);
      // one for even and one for odd tiles: a wait by parity must not be two
      // phases behind, and not every product is waited for (those of two tiles
      // before are over when a tile's scores come)
      barrier_init(smem_at(&s_output[k]), 1);
    }
    barrier_init(smem_at(&s_query), 1);
    barrier_init(smem_at(&s_drained), 1);
    s_failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_prerequisites();
  dependents_may_launch();
  tensor_fence_before();
  const Share share = plan_share<F::kRows, F::kThreads>(p);
  __syncthreads();
  tensor_fence_after();
  const uint32_t tmem = s_tmem, scores = tmem, output = tmem + 2 * kTile;
  const uint32_t steps = p.c.width / 16;
  const bool e4m3 = p.c.type == DB_E4M3;

  // All kinds of warps go through the same items and tiles.
  uint64_t at = share.lo, before = share.before;
  uint32_t request = share.request;
  uint32_t items = 0, tiles = 0, units = 0;  // behind this CTA
  bool go = true;
  while (go && at < share.hi) {
    const Request r = attention_request(p, request);
    const Extent e = extent_of<F::kRows>(p, r);
    if (at - before >= e.units) {
      before += e.units;
      ++request;
      continue;
    }
    const uint64_t x = at - before;
    const uint32_t t0 = (uint32_t)(x % e.tiles);
    const uint32_t item = (uint32_t)(x / e.tiles), head = item / e.blocks, rb = item - head * e.blocks;
    const uint32_t t1 = (uint32_t)min((uint64_t)e.tiles, t0 + (share.hi - at)), n = t1 - t0;
    const uint32_t rows = min(F::kRows, r.rows * p.group - rb * F::kRows);
    const uint32_t base = r.length - r.rows;  // tokens before the request's own

    if (warp >= 4 && warp < 8) {
      // ------------------------------------------------------------- loaders
      const uint32_t me = tid - 128;
      const int32_t* const table = p.view.table + (uint64_t)r.seq * p.view.columns;
      const char* const keys = (const char*)p.c.k + head * p.head_step;
      const char* const values = (const char*)p.c.v + head * p.head_step;
      const auto look = [&](uint32_t t) {  // threads 0 to 63: a token's place
        int2 w = make_int2(-1, 0);
        const uint32_t position = t * kTile + me;
        if (me < kTile && t < t1 && position < r.length) {
          const uint32_t column = position / p.view.page_tokens;
          const uint32_t page = (uint32_t)__ldg(table + column);
          if (page < p.view.n_pages)
            w = make_int2((int)page, (int)(position - column * p.view.page_tokens));
          else
            w.y = -1;
        }
        return w;
      };
      const auto note = [&](uint32_t t, int2 w) {
        if (t >= t1) return;
        TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
        if (me < kTile) {
          m.place[me] = w;
          const uint32_t real = __ballot_sync(kFull, w.x >= 0);
          if (lane == 0) {
            m.real[me / 32] = real;
            m.odd[me / 32] = 0;
          }
          if (w.y < 0) report_table(p.view.ctr);
        }
      };
      constexpr uint32_t kChunks = kPad / 8, kRawChunks = kCodes ? kPad / 16 : kChunks;
      constexpr uint32_t kStep = F::kLoaders / kRawChunks, kEach = kTile / kStep;  // tokens apart, copies a thread
      const uint32_t chunk = me % kRawChunks, token0 = me / kRawChunks;
      const bool mine = chunk < (kCodes ? p.c.width / 16 : p.c.width / 8);
      uint4 raw[2][kCodes ? kEach : 1];
      float scale[2] = {0.f, 0.f};

      // unit u of the item: its tile, and whether it is of keys
      const auto unit_of = [&](uint32_t u, uint32_t& t, bool& key) {
        key = u == 0 || ((u & 1) && u != 2 * n - 1);
        t = t0 + (u == 0 ? 0 : u == 2 * n - 1 ? n - 1 : key ? (u + 1) / 2 : u / 2 - 1);
      };
      const auto issue = [&](uint32_t u, uint4* to, float& sc) {
        uint32_t t;
        bool key;
        unit_of(u, t, key);
        TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
        const char* const from = key ? keys : values;
        const uint64_t step = key ? p.c.k_stride : p.c.v_stride;
        const uint32_t slot = (units + u) % F::kUnits;
        if (!kCodes) {
          if (!barrier_wait(smem_at(&s_empty[slot]), ((units + u) / F::kUnits + 1) & 1, &s_failed)) return;
        }
#pragma unroll
        for (uint32_t k = 0; k < kEach; ++k) {
          const uint32_t token = token0 + k * kStep;
          const int2 w = m.place[token];
          const bool real = w.x >= 0 && (key || !((m.odd[token / 32] >> (token & 31)) & 1));
          const char* const source =
              from + (real ? (uint64_t)w.x * step + (uint64_t)w.y * p.token_step : 0) + (mine ? chunk * 16 : 0);
          if (kCodes) {
            to[k] = real && mine ? __ldg((const uint4*)source) : make_uint4(0, 0, 0, 0);
          } else if (mine) {
            copy16(ring + slot * F::kUnit + chunk / 8 * kPanel + token * 128 + ((chunk & 7) ^ (token & 7)) * 16, source, real);
          }
        }
        if (!kCodes) copies_commit();
        if (key) {
          if (kCodes) {
            const uint32_t token = me % kTile;
            const bool val = me >= kTile;
            const int2 w = m.place[token];
            const char* const s = (const char*)(val ? p.c.v_scale : p.c.k_scale);
            sc = w.x >= 0 ? __ldg((const float*)(s + (uint64_t)w.x * (val ? p.c.v_scale_stride : p.c.k_scale_stride)) +
                                  w.y * p.scale_token_step + head * p.scale_head_step)
                          : 0.f;
          }
          // Values of a tile that not every row sees: those that are not
          // finite stay out of the product.
          if ((t + 1) * kTile > base || (m.real[0] & m.real[1]) != 0xFFFFFFFFu) {
            for (uint32_t k = 0; k < kEach; ++k) {
              const uint32_t token = token0 + k * kStep;
              const int2 w = m.place[token];
              if (w.x < 0 || !mine) continue;
              const uint4 v = __ldg((const uint4*)(values + (uint64_t)w.x * p.c.v_stride + (uint64_t)w.y * p.token_step + chunk * 16));
              bool odd;
              if (kCodes) {
                const auto nan4 = [](uint32_t c) { return ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
                odd = e4m3 && (nan4(v.x) | nan4(v.y) | nan4(v.z) | nan4(v.w));
              } else {
                odd = not_finite2<W>(v.x) || not_finite2<W>(v.y) || not_finite2<W>(v.z) || not_finite2<W>(v.w);
              }
              if (odd) atomicOr(&m.odd[token / 32], 1u << (token & 31));
            }
          }
        }
      };
      const auto finish = [&](uint32_t u, const uint4* got, float sc) {
        uint32_t t;
        bool key;
        unit_of(u, t, key);
        const uint32_t slot = (units + u) % F::kUnits;
        if (u == 0) {
          // the item's queries, when the products with the ones before are made
          if (items && !barrier_wait(smem_at(&s_query), (items - 1) & 1, &s_failed)) return;
          const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.f ? 0u : 0xFFFFFFFFu;
#pragma unroll 4
          for (uint32_t c = me; c < F::kRows * kChunks; c += F::kLoaders) {
            const uint32_t row = c / kChunks, ch = c % kChunks, all = rb * F::kRows + row;
            const bool real = row < rows && ch < p.c.width / 8;
            const uint32_t nd = real ? all / p.group : 0, qh = head * p.group + (real ? all - nd * p.group : 0);
            uint4 v = real ? __ldg((const uint4*)((const char*)p.q.base + (uint64_t)(r.first + nd) * p.q.row_stride +
                                                  qh * p.q.head_stride + ch * 16))
                           : make_uint4(0, 0, 0, 0);
            v.x = (v.x ^ flip) & keep, v.y = (v.y ^ flip) & keep, v.z = (v.z ^ flip) & keep, v.w = (v.w ^ flip) & keep;
            *(uint4*)(smem + F::kUnits * F::kUnit + ch / 8 * kQueryPanel + row * 128 + ((ch & 7) ^ (row & 7)) * 16) = v;
          }
        }
        if (kCodes) {
          if (!barrier_wait(smem_at(&s_empty[slot]), ((units + u) / F::kUnits + 1) & 1, &s_failed)) return;
          if (mine) {
#pragma unroll
            for (uint32_t k = 0; k < kEach; ++k) {
              const uint32_t token = token0 + k * kStep;
              uint2 a, b, c, d;
              if (key) {
                a = widen4<T>(got[k].x, e4m3), b = widen4<T>(got[k].y, e4m3), c = widen4<T>(got[k].z, e4m3), d = widen4<T>(got[k].w, e4m3);
              } else {
                a = widen4<W>(got[k].x, e4m3), b = widen4<W>(got[k].y, e4m3), c = widen4<W>(got[k].z, e4m3), d = widen4<W>(got[k].w, e4m3);
              }
              unsigned char* const to = smem + slot * F::kUnit + chunk / 4 * kPanel + token * 128;
              *(uint4*)(to + (((2 * chunk) & 7) ^ (token & 7)) * 16) = make_uint4(a.x, a.y, b.x, b.y);
              *(uint4*)(to + (((2 * chunk + 1) & 7) ^ (token & 7)) * 16) = make_uint4(c.x, c.y, d.x, d.y);
            }
          }
          if (key) {
            TileNotes& m = s_notes[(tiles + t - t0) % F::kMeta];
            if (me < kTile) {
              // an infinite scale stands for values of both signs, whose
              // products have no sum
              m.k_scale[me] = __fmaf_rn(sc, 0.f, sc) * fabsf(p.scale_log2);
            } else {
              m.v_scale[me - kTile] = sc;
              const uint32_t ex = (__float_as_uint(sc) >> 23) & 0xFFu;
              const uint32_t most = __reduce_max_sync(kFull, ex == 0xFFu ? 0u : ex);
              if (lane == 0) m.exponent[(me - kTile) / 32] = most;
            }
          }
        } else if (u + F::kLag < 2 * n) {
          copies_wait<F::kLag - 1>();
        } else {
          copies_wait<0>();
        }
        writes_to_async_proxy();
        barrier_arrive(smem_at(&s_full[slot]));
      };

      note(t0, look(t0));
      note(t0 + 1, look(t0 + 1));
      int2 ahead = make_int2(-1, 0);
      group_sync(2, F::kLoaders);
      for (uint32_t u = 0; u < 2 * n + F::kLag; u += 2) {
        // two units, keys of tile t0 + u / 2 + 1 among them
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const uint32_t v = u + h;
          if (v >= F::kLag && v - F::kLag < 2 * n) finish(v - F::kLag, raw[h], scale[h]);
          if (v < 2 * n) issue(v, raw[h], scale[h]);
          if (h == 0) ahead = look(t0 + u / 2 + 2);
          if (h == 1) note(t0 + u / 2 + 2, ahead);
          group_sync(2, F::kLoaders);
        }
      }
      go = group_all(2, F::kLoaders, !s_failed);
    } else if (warp == 8) {
      // ------------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t kind_s = product_kind(kTypeQ, kTile, false), kind_o = product_kind(kTypeW, p.c.width, true);
        const auto unit_at = [&](uint32_t u, uint32_t& slot) {  // waits until a unit is there
          slot = (units + u) % F::kUnits;
          return barrier_wait(smem_at(&s_full[slot]), ((units + u) / F::kUnits) & 1, &s_failed);
        };
        const auto score = [&](uint32_t k) {
          uint32_t slot;
          if (!unit_at(k ? 2 * k - 1 : 0, slot)) return false;
          tensor_fence_after();
          const uint32_t buffer = (tiles + k) & 1;
          for (uint32_t st = 0; st < steps; ++st) {
            const uint32_t off = (st & 3) * 32;
            tensor_multiply(scores + buffer * kTile, tile_descriptor(query + (st / 4) * kQueryPanel + off, 16),
                            tile_descriptor(ring + slot * F::kUnit + (st / 4) * kPanel + off, 16), kind_s, st > 0);
          }
          tensor_commit(smem_at(&s_scores[buffer]));
          tensor_commit(smem_at(&s_empty[slot]));
          barrier_arrive(smem_at(&s_scores[buffer]));
          if (k == n - 1) tensor_commit(smem_at(&s_query));
          return true;
        };
        bool ok = score(0);
        for (uint32_t k = 0; ok && k < n; ++k) {
          if (k + 1 < n) ok = score(k + 1);
          if (!ok) break;
          const uint32_t buffer = (tiles + k) & 1;
          uint32_t slot;
          ok = unit_at(k + 1 < n ? 2 * k + 2 : 2 * n - 1, slot) &&
               barrier_wait(smem_at(&s_weights[buffer]), ((tiles + k) >> 1) & 1, &s_failed);
          if (!ok) break;
          tensor_fence_after();
#pragma unroll
          for (uint32_t st = 0; st < kTile / 16; ++st)
            tensor_multiply_t(output, scores + buffer * kTile + st * 8,
                              tile_descriptor(ring + slot * F::kUnit + st * 2048, kPanel), kind_o, true);
          tensor_commit(smem_at(&s_empty[slot]));
          tensor_commit(smem_at(&s_output[buffer]));
        }
        go = ok;
      }
      go = __shfl_sync(kFull, go, 0);
    } else {
      // -------------------------------------------------------------- weights
      const uint32_t row = tid, lanes = (warp * 32) << 16;
      const bool row_real = row < rows;
      const uint32_t all = rb * F::kRows + (row_real ? row : 0), node = all / p.group;
      const uint32_t* const mask = p.mask ? p.mask + (uint64_t)(r.first + node) * p.mask_words : nullptr;
      const float factor = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
      // Weights are exp2(score - ref). ref is a score that was the largest, and
      // for codes also takes in the size of the values' scales, which P has as
      // a factor, so that P stays in the middle of f16's range.
      float top = -INFINITY, sum = 0.f;
      uint32_t exponent = 0;
      {
        uint32_t zero[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) zero[j] = 0;
        for (uint32_t c = 0; c < p.c.width; c += 16) tmem_store16(output + lanes + c, zero);
        tmem_stored();
      }
      bool ok = true;
      for (uint32_t k = 0; k < n; ++k) {
        const uint32_t tile = tiles + k, buffer = tile & 1, t = t0 + k;
        const uint32_t here = scores + buffer * kTile + lanes;
        ok = barrier_wait(smem_at(&s_scores[buffer]), (tile >> 1) & 1, &s_failed);
        if (!__all_sync(kFull, ok)) break;
        tensor_fence_after();
        const TileNotes& m = s_notes[tile % F::kMeta];
        // which tokens this row sees
        const bool masked = (t + 1) * kTile > base || (m.real[0] & m.real[1]) != 0xFFFFFFFFu;
        uint32_t sees[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (masked) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int32_t own = (int32_t)(t * kTile + 32 * h - base);  // the node of the word's first token
            uint32_t bits;
            if (own <= -32) {
              bits = 0xFFFFFFFFu;
            } else if (!mask) {
              const int32_t upto = (int32_t)node - own + 1;
              bits = upto <= 0 ? 0u : upto >= 32 ? 0xFFFFFFFFu : (1u << upto) - 1;
            } else {
              const int32_t word = own >> 5;  // -1: tokens before the request's
              const uint32_t a = word < 0 ? 0xFFFFFFFFu : (uint32_t)word < p.mask_words ? __ldg(mask + word) : 0u;
              const uint32_t b = (uint32_t)(word + 1) < p.mask_words ? __ldg(mask + word + 1) : 0u;
              bits = __funnelshift_r(a, b, (uint32_t)own & 31);
            }
            sees[h] = bits & m.real[h];
          }
        }
        // The scores of half a tile; they are fetched twice, for the maximum
        // and for the weights: 32 registers instead of 64 let two CTAs share
        // an SM without spills.
        const auto fetch = [&](int h, float* s) {
          tmem_load32(here + 32 * h, (uint32_t*)s);
          tmem_loaded();
          if (kCodes) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 y = ((const float4*)m.k_scale)[8 * h + j];
              s[4 * j] *= y.x, s[4 * j + 1] *= y.y, s[4 * j + 2] *= y.z, s[4 * j + 3] *= y.w;
            }
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((sees[h] >> j) & 1)) s[j] = -INFINITY;
          }
        };
        float most = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float s[32];
          fetch(h, s);
          float other = s[1];
          most = fmaxf(most, s[0]);
#pragma unroll
          for (int j = 2; j < 32; j += 2) most = fmaxf(most, s[j]), other = fmaxf(other, s[j + 1]);
          most = fmaxf(most, other);
        }
        if (!kCodes) most *= factor;
        const float ref_before = top + (kCodes ? (float)((int)exponent - 127) : 0.f);
        bool move = most > top + kSlack || (top == -INFINITY && most > -INFINITY);
        if (move) top = most;
        if (kCodes) {
          const uint32_t ex = min(max(max(m.exponent[0], m.exponent[1]), 31u), 227u);
          if (exponent == 0 || ex > exponent + kScaleSlack) {
            exponent = ex;
            move = true;
          }
        }
        const float ref = top == -INFINITY ? 0.f : top + (kCodes ? (float)((int)exponent - 127) : 0.f);
        const uint64_t odd = masked ? (uint64_t)m.odd[0] | (uint64_t)m.odd[1] << 32 : 0;
        if (__any_sync(kFull, move && k) || odd) {
          // O belongs to this warp while no product adds to it
          if (k) {
            ok = barrier_wait(smem_at(&s_output[buffer ^ 1]), ((tile - 1) >> 1) & 1, &s_failed);
            if (!__all_sync(kFull, ok)) break;
            tensor_fence_after();
          }
          const float down = move ? exp2_of(ref_before - ref) : 1.f;
          if (k) sum *= down;
          for (uint32_t c = 0; c < p.c.width; c += 16) {
            uint32_t o[16];
            tmem_load16(output + lanes + c, o);
            tmem_loaded();
            if (k) {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * down);
            }
            // Rare: values that are not finite, which the product was not given,
            // for the rows that see them.
            for (uint64_t left = odd; left; left &= left - 1) {
              const uint32_t token = __ffsll((long long)left) - 1;
              __syncwarp();
              const float score = __uint_as_float(tmem_load1(here + token));
              tmem_loaded();
              const int2 place = m.place[token];
              const char* const from = (const char*)p.c.v + head * p.head_step + (uint64_t)place.x * p.c.v_stride +
                                       (uint64_t)place.y * p.token_step;
              const float weight = exp2_of(__fmaf_rn(score, kCodes ? m.k_scale[token] : factor, -ref)) *
                                   (kCodes ? m.v_scale[token] : 1.f);
              if ((sees[token / 32] >> (token & 31)) & 1) {
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  float2 v;
                  if (kCodes)
                    v = unpack2<__half>(e4m3x2_to_f16x2(*(const uint16_t*)(from + c + j)));
                  else
                    v = unpack2<T>(*(const uint32_t*)(from + 2 * (c + j)));
                  o[j] = __float_as_uint(__uint_as_float(o[j]) + weight * v.x);
                  o[j + 1] = __float_as_uint(__uint_as_float(o[j + 1]) + weight * v.y);
                }
              }
            }
            __syncwarp();
            tmem_store16(output + lanes + c, o);
          }
          tmem_stored();
        }
        float more = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float s[32];
          uint32_t w[16];
          fetch(h, s);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float y[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) y[g] = exp2_of(kCodes ? s[j + g] - ref : __fmaf_rn(s[j + g], factor, -ref));
            sum += y[0] + y[1];
            more += y[2] + y[3];
            if (kCodes) {
              const float4 z = ((const float4*)m.v_scale)[8 * h + j / 4];
              y[0] *= z.x, y[1] *= z.y, y[2] *= z.z, y[3] *= z.w;
              if (masked) {  // the scale of what is not seen may be NaN
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  if (!((sees[h] >> (j + g)) & 1)) y[g] = 0.f;
              }
            }
            w[j / 2] = pack2<W>(y[0], y[1]);
            w[j / 2 + 1] = pack2<W>(y[2], y[3]);
          }
          __syncwarp();
          tmem_store16(here + 16 * h, w);  // over scores that have been fetched
        }
        sum += more;
        tmem_stored();
        tensor_fence_before();
        barrier_arrive(smem_at(&s_weights[buffer]));
      }
      if (ok) ok = barrier_wait(smem_at(&s_output[(tiles + n - 1) & 1]), ((tiles + n - 1) >> 1) & 1, &s_failed);
      go = group_all(1, F::kWeights, ok);
      if (go) {
        tensor_fence_after();
        const float ref = top == -INFINITY ? -INFINITY : top + (kCodes ? (float)((int)exponent - 127) : 0.f);
        const bool whole = t0 == 0 && t1 == e.tiles;
        const auto query_head = [&](uint32_t row_, uint32_t& nd) {
          const uint32_t a = rb * F::kRows + row_;
          nd = a / p.group;
          return head * p.group + (a - nd * p.group);
        };
        float* const mine = p.partial + (uint64_t)(2 * blockIdx.x + (t0 == 0)) * partial_floats(F::kRows, kPad);
        uint32_t nd;
        const uint32_t qh = query_head(row_real ? row : 0, nd);
        char* const to = (char*)p.out.base + (uint64_t)(r.first + nd) * p.out.row_stride + qh * p.out.head_stride;
        const float by = sum == 0.f ? 0.f : 1.f / sum;
        for (uint32_t c = 0; c < p.c.width; c += 16) {
          uint32_t o[16];
          __syncwarp();
          tmem_load16(output + lanes + c, o);
          tmem_loaded();
          if (!row_real) continue;
          const float* const f = (const float*)o;
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              *(uint4*)(to + (c + j) * 2) =
                  make_uint4(pack2<T>(f[j] * by, f[j + 1] * by), pack2<T>(f[j + 2] * by, f[j + 3] * by),
                             pack2<T>(f[j + 4] * by, f[j + 5] * by), pack2<T>(f[j + 6] * by, f[j + 7] * by));
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              __stcg((float4*)(mine + row * kPad + c + j), make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]));
          }
        }
        const auto statistics = [&](uint32_t nd_, uint32_t qh_, float m_, float l_) {
          if (p.lse)
            p.lse[(uint64_t)(r.first + nd_) * (p.c.heads * p.group) + qh_] =
                l_ == 0.f ? -INFINITY : m_ * 0.6931471805599453f + logf(l_);
        };
        if (whole) {
          if (row_real) statistics(nd, qh, ref, sum);
        } else {
          if (row_real) {
            __stcg(mine + F::kRows * kPad + row, ref);
            __stcg(mine + F::kRows * kPad + F::kRows + row, sum);
          }
          __threadfence();
          group_sync(1, F::kWeights);
          const uint64_t first = at - t0;
          const uint32_t c0 = owner_of(share, first), c1 = owner_of(share, first + e.tiles - 1);
          if (tid == 0) {
            const unsigned int seen = atomicAdd(p.arrived + c0, 1u);
            s_last = seen == c1 - c0;
            if (s_last) p.arrived[c0] = 0;
          }
          group_sync(1, F::kWeights);
          if (s_last) {
            __threadfence();
            constexpr uint32_t kQuads = kPad / 4;
            for (uint32_t c = tid; c < rows * kQuads; c += F::kWeights) {
              const uint32_t row_ = c / kQuads, quad = c % kQuads;
              if (quad * 4 >= p.c.width) continue;
              float l, m;
              const float4 v = join_parts<F::kRows, kPad>(p, c0, c1, row_, quad, m, l);
              uint32_t nd_;
              const uint32_t qh_ = query_head(row_, nd_);
              const float by_ = l == 0.f ? 0.f : 1.f / l;
              *(uint2*)((char*)p.out.base + (uint64_t)(r.first + nd_) * p.out.row_stride + qh_ * p.out.head_stride + quad * 8) =
                  make_uint2(pack2<T>(v.x * by_, v.y * by_), pack2<T>(v.z * by_, v.w * by_));
              if (quad == 0) statistics(nd_, qh_, m, l);
            }
          }
          group_sync(1, F::kWeights);  // s_last has been read
        }
      }
    }
    at += n;
    ++items;
    tiles += n;
    units += 2 * n;
  }
  // nothing is under way when the shared memory and TMEM are given back
  if (warp >= 4 && warp < 8) copies_wait<0>();
  if (tid == 256) {
    tensor_commit(smem_at(&s_drained));
    const uint64_t began = globaltimer_ns();
    while (!barrier_try(smem_at(&s_drained), 0) && globaltimer_ns() - began < kWaitLimitNs) {
    }
  }
  if (!go && tid == 0 && p.view.ctr) atomicOr((unsigned int*)&p.view.ctr->err, DB_ERR_TIMEOUT);
  tensor_fence_before();
  __syncthreads();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(F::kColumns));
}

template <typename T, uint32_t kPad, bool kCodes>
int launch_many(const AttnParams& p, unsigned grid, cudaStream_t s) {
  typedef Many<kPad, kCodes> F;
  const cudaError_t e = cudaFuncSetAttribute(attention_many_kernel<T, kPad, kCodes>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, F::kAsk);
  if (e != cudaSuccess) return cuda_failure(e);
  return launch_dependent(attention_many_kernel<T, kPad, kCodes>, grid, F::kThreads, F::kAsk, s, p);
}

template <uint32_t kPad>
int launch_attention(const AttnParams& p, uint32_t type, uint32_t blocks, unsigned grid, cudaStream_t s) {
  const bool codes = item_bytes(p.c.type) == 1;
  if (blocks == kManyBlocks) {
    if (type == DB_BF16)
      return codes ? launch_many<__nv_bfloat16, kPad, true>(p, grid, s) : launch_many<__nv_bfloat16, kPad, false>(p, grid, s);
    return codes ? launch_many<__half, kPad, true>(p, grid, s) : launch_many<__half, kPad, false>(p, grid, s);
  }
  if (type == DB_BF16)
    return codes ? launch_blocks<__nv_bfloat16, kPad, true>(p, blocks, grid, s)
                 : launch_blocks<__nv_bfloat16, kPad, false>(p, blocks, grid, s);
  return codes ? launch_blocks<__half, kPad, true>(p, blocks, grid, s)
               : launch_blocks<__half, kPad, false>(p, blocks, grid, s);
}

}  // namespace db
