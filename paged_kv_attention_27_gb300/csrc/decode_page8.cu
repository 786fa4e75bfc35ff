// Batch decode over a page-scaled FP8 cache: out = softmax(sm_scale q K^T) V
// with K = s_k(page, head) * codes and V = s_v(page, head) * codes.
//
// A work item is (request, kv head, chunk of keys); the g query heads of the
// kv head share every page that is loaded. HBM-bound: 2 bytes per key and
// dimension for K and V together against 4 g flops, so an SM has about 1400
// cycles per 32 KB tile of 128 keys (head_dim 128) and may not spend
// instructions per byte. Hence both products run on tcgen05 with the cache
// bytes as they arrive, nothing is converted, and the roles of rows and
// columns are swapped against prefill: keys (or dimensions) are the 128 M
// rows, heads the N columns.
//   S[key][head]  = K (A, K-major, e4m3) x Q^T (B, e4m3)
//   O[dim][head] += V^T (A, MN-major, e4m3) x P^T (B, e4m3)
// The 16-bit q and the fp32 weights enter as sums of e4m3 terms, each in its
// own column: x = t0 + t1 / 16 (+ t2 / 256), t0 = e4m3(x), t1 = e4m3(16 (x -
// t0)), ... Two terms carry the 8 significand bits of bf16, three the 11 of
// fp16: q (times a power of two that puts its largest element at 224..448)
// enters exactly, and weights are rounded as bf16 (fp16) weights would be. N
// is at least 16 for M = 128, so up to 8 heads x 2 terms cost nothing extra.
//
// Scales: the score of a key is multiplied by its page's s_k with the softmax
// scale. The page's s_v joins the weight before it is rounded:
//   w = 2^(s + log2 s_v - m),  m the running maximum of s + log2 s_v,
//   O = sum w code,  l = sum w r / s_v (r: s_v of the item's first page),
//   out = O r / l,   lse = ln 2 (m + log2 l - log2 r):
// one exponential per score, and both sums keep their leading bits where a
// request's V scales are up to 2^80 apart (l then stays below 2^118, and a
// weight of 2^-80 is far from underflow).
//
// Roles (8 warps): 0-3 softmax (thread = key of the tile = TMEM lane), then
// the epilogue (thread = dimension); 4 copies pages by TMA and page scales by
// cp.async into a ring; 5 issues the MMAs (the scores of tile j + 1 before the
// output of tile j, with two score buffers); 6 merges the states of requests
// whose last chunk this CTA finished, beside the next items; 7 turns the next
// item's q into terms. The launch is persistent: a CTA takes items from a
// counter and the ring runs on from item to item. (With q and the merge on the
// softmax warps, an item's start and end cost as much as four tiles.)
//
// Measured, calls back to back with their work-list copies: 64 requests of
// 512-4096 keys, 32/32 heads of 128 (828 MB) 132 us, 0.92 of the copy bandwidth;
// 128 requests of 128-16384 keys, 64/8 heads (870 MB) 152 us, 0.84; 56 requests,
// 16/8 heads of 256, fp16, window of 4096 (598 MB) 100.3 us, 0.88. Long keys
// alone run at 0.97-0.99; the rest is items' starts and ends and the last items.
#include <cfloat>
#include <type_traits>

#include "elem.cuh"
#include "page8.cuh"
#include "ptx_page8.cuh"

namespace fi {

namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kItemRing = 8;
// A weight is at most 2^kGrow (the running maximum moves when a score passes it
// by more, which costs a tile as much again: with 1 in place of 4 the batch of
// 64/8 heads took 4 % longer), and is stored times kWeightUnit: at most 256,
// below E4M3's 448. What the last term rounds off is then at most 2^-18 (three
// terms: 2^-22) of the largest weight, or 2^-8 (2^-12) of the weight itself.
constexpr float kGrow = 4.f;
constexpr float kWeightUnit = 16.f;

template <int D, int G, class E>
struct D8Cfg {
  static constexpr int T = kPage8DecodeTile;                // keys per tile
  static constexpr int TERMS = std::is_same<E, Bf16>::value ? 2 : 3;
  static constexpr int COLS = G * TERMS;                    // column term * G + head
  static constexpr int N = COLS <= 16 ? 16 : 32;
  static constexpr int ROWB = D < 128 ? D : 128;            // bytes of a shared-memory row
  static constexpr int DB = D <= 128 ? 1 : D / 128;         // 128-byte slices of a key
  static constexpr uint32_t SWZ = ROWB == 128 ? 2 : 4;      // 128- or 64-byte swizzle
  static constexpr uint32_t ATOM = 8 * ROWB;
  static constexpr int KBYTES = T * D;                      // one K (or V) tile
  static constexpr int STAGE = 2 * KBYTES;
  static constexpr int CTAS = D <= 128 ? 2 : 1;             // per SM
  static constexpr int NST = D == 64 ? 6 : 3;
  static constexpr int QBYTES = N * D;
  static constexpr int PBYTES = T * N;
  static constexpr int OFF_Q = NST * STAGE;                 // two buffers
  static constexpr int OFF_P = OFF_Q + 2 * QBYTES;          // two buffers
  static constexpr int SMEM = OFF_P + 2 * PBYTES + 1024;
  static constexpr int THREADS = 256;
  static constexpr uint32_t TMEM_COLS = N * (2 + DB) <= 64 ? 64 : 128;
  static constexpr uint32_t IDESC_S = idesc_e4m3(128, N, 0, 0);
  static constexpr uint32_t IDESC_O = idesc_e4m3(128, 16, 1, 1);
  static_assert(SMEM * CTAS <= 227 * 1024, "shared-memory budget");
  static_assert(COLS <= 32 && N * (2 + DB) <= 128, "");
};

struct D8Barriers {
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t k_full[6], v_full[6], empty[6];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2];
  uint64_t m_full[2], m_empty[2];   // finished chunks for the merging warp
  uint64_t drain;
};

// A float in [0, inf) orders as its bits.
__device__ __forceinline__ float warp_max(float x) {
  int k = __float_as_int(x);
  k = k < 0 ? k ^ 0x7fffffff : k;
  k = __reduce_max_sync(0xffffffffu, k);
  return __int_as_float(k < 0 ? k ^ 0x7fffffff : k);
}

__device__ __forceinline__ float pow2i(int k) { return __uint_as_float(uint32_t(127 + k) << 23); }

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

template <int D, int G, class E>
__global__ void __launch_bounds__(D8Cfg<D, G, E>::THREADS, D8Cfg<D, G, E>::CTAS)
decode_page8_kernel(const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, DecodeParams prm) {
  using C = D8Cfg<D, G, E>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) D8Barriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ WorkItem item_ring[kItemRing];             // req < 0: no more
  __shared__ __align__(8) float2 scale_sh[C::NST][8];   // per page of a tile: s_k (-1: no page), s_v
  __shared__ float q_unit[2][G];                        // score scale of a head, by item parity
  __shared__ float red[4][G], sum_sh[4][G];             // per warp: maxima of a tile, sums of an item
  __shared__ int2 merge_sh[2];                          // merge task (-1: no more), kv head

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = prm.wait_limit_ns;
  const int P = prm.page_size, ppt = C::T / P;
  const int hkv = prm.num_qo_heads / G;

  // item n of this CTA (for a whole warp, or for one thread)
  auto take_item = [&](int n, WorkItem& w) {
    if (!mbar_sleep_bounded(smem_u32(&bars.item_full[n % kItemRing]), (n / kItemRing) & 1, limit,
                            &abort_flag))
      return false;
    w = item_ring[n % kItemRing];
    return true;
  };
  auto take_item_warp = [&](int n, WorkItem& w) {
    const bool good = take_item(n, w);
    if (!__all_sync(0xffffffffu, good)) return false;
    if (lane == 0) mbar_arrive(smem_u32(&bars.item_empty[n % kItemRing]));
    return true;
  };
  // tiles of an item: its keys from the start of its first page
  auto lead_of = [&](const WorkItem& w) { return w.tok_begin % P; };
  auto tiles_of = [&](const WorkItem& w) {
    const int n = w.tok_end - w.tok_begin;
    return n > 0 ? (n + lead_of(w) + C::T - 1) / C::T : 0;
  };

  // The next kernel of the stream may start its set-up beside this one, as this
  // one's runs beside the copy of its work list.
  if (threadIdx.x == 0) {
    pdl_trigger();
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(smem_u32(&bars.item_full[s]), 1);
      mbar_init(smem_u32(&bars.item_empty[s]), 6);      // 4 softmax warps, the MMA and q warps
    }
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(smem_u32(&bars.k_full[s]), 1 + ppt);    // K's bytes, and each page's scales
      mbar_init(smem_u32(&bars.v_full[s]), 1);
      mbar_init(smem_u32(&bars.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars.q_full[s]), 1);
      mbar_init(smem_u32(&bars.q_empty[s]), 5);         // the last scores; the 4 softmax warps
      mbar_init(smem_u32(&bars.s_full[s]), 1);
      mbar_init(smem_u32(&bars.p_full[s]), 4);
      mbar_init(smem_u32(&bars.pv_done[s]), 1);
      mbar_init(smem_u32(&bars.m_full[s]), 4);
      mbar_init(smem_u32(&bars.m_empty[s]), 1);
    }
    mbar_init(smem_u32(&bars.drain), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  // rows of Q that no head uses stay zero
  for (int i = threadIdx.x; i < 2 * C::QBYTES / 16; i += C::THREADS)
    st_shared_zero16(base + C::OFF_Q + i * 16);
  fence_proxy_async_smem();
  if (warp == 5) {
    tmem_alloc(smem_u32(&tmem_base_sh), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const uint32_t o_col0 = tmem + 2 * C::N;
  int issued = 0;   // the producer: tiles whose copies it has issued

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    WorkItem w = prm.items[blockIdx.x], wn;   // (the grid has no more CTAs than items)
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
    const uint32_t box = uint32_t(P) * C::ROWB;
    // The next item is taken in three steps with copies in between, so that the
    // latencies of the counter and of the work list hide behind them.
    int v_next = 0;
    auto count = [&] {
      if (lane == 0) v_next = int(gridDim.x + atomicAdd(prm.work_counter, 1u));
    };
    auto look_up = [&](int v, WorkItem& w) {
      if (v < prm.n_items) w = prm.items[v];
      else w.req = -1;
    };
    auto publish = [&](int n, const WorkItem& w) {   // as item n of this CTA
      if (n >= kItemRing && !mbar_sleep_warp(smem_u32(&bars.item_empty[n % kItemRing]),
                                             ((n / kItemRing) & 1) ^ 1, limit, &abort_flag))
        return false;
      if (lane == 0) {
        item_ring[n % kItemRing] = w;
        mbar_arrive(smem_u32(&bars.item_full[n % kItemRing]));
      }
      return true;
    };
    auto pages_in = [&](const WorkItem& w, int j) { return min(ppt, w.n_pages - j * ppt); };
    int g = 0;
    bool ok = publish(0, w);
    int next_page = lane < pages_in(w, 0) ? prm.page_indices[w.page_begin + lane] : -1;
    for (int n = 0; ok && w.req >= 0; ++n) {
      const int nt = tiles_of(w);
      const int c1 = prm.layout == FI_LAYOUT_NHD ? w.head : 0;
      const int c2 = prm.layout == FI_LAYOUT_NHD ? 0 : w.head;
      auto first_pages = [&] {
        next_page = wn.req >= 0 && lane < pages_in(wn, 0) ? prm.page_indices[wn.page_begin + lane] : -1;
      };
      count();
      if (nt == 0) {
        look_up(__shfl_sync(0xffffffffu, v_next, 0), wn);
        first_pages();
        ok = publish(n + 1, wn);
        if (!ok) break;
      }
      for (int j = 0; j < nt; ++j, ++g) {
        const int st = g % C::NST;
        const int page = next_page;
        const bool mine = lane < pages_in(w, j);
        const bool valid = mine && page >= 0 && page < prm.num_pages;
        if (mine && !valid) atomicOr(prm.err, kErrBounds);
        next_page = -1;
        if (j + 1 < nt) {
          if (lane < pages_in(w, j + 1))
            next_page = prm.page_indices[w.page_begin + (j + 1) * ppt + lane];
        } else if (j > 0) {
          first_pages();
        }
        const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, valid))) * C::DB * box;
        if (g >= C::NST && !mbar_sleep_warp(smem_u32(&bars.empty[st]), ((g / C::NST) & 1) ^ 1, limit,
                                           &abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t kf = smem_u32(&bars.k_full[st]), vf = smem_u32(&bars.v_full[st]);
        const bool skip = g == 0 && prm.fault_kind == 1 && blockIdx.x == 0;
        if (lane == 0) {
          if (!skip) mbar_arrive_expect_tx(kf, bytes);
          mbar_arrive_expect_tx(vf, bytes);
        }
        __syncwarp();
        if (lane < ppt) {
          if (valid) {
            const uint32_t dst = base + st * C::STAGE + lane * box;
#pragma unroll
            for (int b = 0; b < C::DB; ++b) {
              if (!skip) tma_load_4d(dst + b * C::T * C::ROWB, &k_map, kf, b * 128, c1, c2, page);
            }
#pragma unroll
            for (int b = 0; b < C::DB; ++b)
              tma_load_4d(dst + C::KBYTES + b * C::T * C::ROWB, &v_map, vf, b * 128, c1, c2, page);
            const size_t at = size_t(page) * hkv + w.head;
            const uint32_t sc = smem_u32(&scale_sh[st][lane]);
            cp_async4(sc, prm.k_head_scale + at);
            cp_async4(sc + 4, prm.v_head_scale + at);
            cp_async_arrive(kf);
          } else {
            scale_sh[st][lane] = make_float2(-1.f, 1.f);
            mbar_arrive(kf);
          }
        }
        issued = g + 1;
        if (j == 0) look_up(__shfl_sync(0xffffffffu, v_next, 0), wn);
        if (nt == 1) first_pages();
        if ((j == 1 || nt == 1) && !publish(n + 1, wn)) {
          ok = false;
          break;
        }
      }
      w = wn;
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      atomicOr(prm.err, kErrTimeout);
    }
    cp_async_wait_all();
    __syncwarp();
  } else if (warp == 5) {
    // -------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint64_t kd0 = sdesc_swz(base, 16, C::ATOM, C::SWZ);
      // head_dim 64: the second 64 of the 128 M rows repeat the first (their
      // accumulator rows are not read)
      const uint64_t vd0 = sdesc_swz(base + C::KBYTES, 0, C::ATOM, C::SWZ);
      const uint64_t qd0 = sdesc_swz(base + C::OFF_Q, 16, C::ATOM, C::SWZ);
      const uint64_t pd0 = sdesc_swz(base + C::OFF_P, 128, 128, 0);
      bool ok = true;
      int g = 0;
      auto scores = [&](int q_buf) {     // S of tile g
        const int st = g % C::NST;
        if (!mbar_sleep_bounded(smem_u32(&bars.k_full[st]), (g / C::NST) & 1, limit, &abort_flag))
          return false;
        tc_fence_after();
        const uint64_t kd = kd0 + uint64_t((st * C::STAGE) >> 4);
        const uint64_t qd = qd0 + uint64_t((q_buf * C::QBYTES) >> 4);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const int b = k * 32 / 128, o = k * 32 % 128;
          tc_mma_f8_ss(tmem + (g & 1) * C::N, kd + uint64_t((b * C::T * C::ROWB + o) >> 4),
                       qd + uint64_t((b * C::N * C::ROWB + o) >> 4), C::IDESC_S, k > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars.s_full[g & 1]));
        return true;
      };
      auto outputs = [&](int t, bool first) {   // O += V^T P^T of tile t
        const int st = t % C::NST;
        if (!mbar_sleep_bounded(smem_u32(&bars.v_full[st]), (t / C::NST) & 1, limit, &abort_flag) ||
            !mbar_sleep_bounded(smem_u32(&bars.p_full[t & 1]), (t >> 1) & 1, limit, &abort_flag))
          return false;
        tc_fence_after();
        const uint64_t vd = vd0 + uint64_t((st * C::STAGE) >> 4);
        const uint64_t pd = pd0 + uint64_t(((t & 1) * C::PBYTES) >> 4);
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
#pragma unroll
          for (int c = 0; c < C::N / 16; ++c)
#pragma unroll
            for (int k = 0; k < C::T / 32; ++k)
              tc_mma_f8_ss(o_col0 + b * C::N + c * 16,
                           vd + uint64_t((b * C::T * C::ROWB + k * 32 * C::ROWB) >> 4),
                           pd + uint64_t((c * C::T * 16 + k * 32 * 16) >> 4), C::IDESC_O,
                           (!first || k > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars.empty[st]));
        tc_commit(smem_u32(&bars.pv_done[t & 1]));
        return true;
      };
      for (int n = 0; ok; ++n) {
        WorkItem w;
        ok = take_item(n, w);
        if (!ok) break;
        mbar_arrive(smem_u32(&bars.item_empty[n % kItemRing]));
        if (w.req < 0) break;
        const int nt = tiles_of(w);
        ok = mbar_sleep_bounded(smem_u32(&bars.q_full[n & 1]), (n >> 1) & 1, limit, &abort_flag);
        for (int j = 0; ok && j < nt; ++j, ++g) {
          ok = scores(n & 1);
          if (ok && j + 1 == nt) tc_commit(smem_u32(&bars.q_empty[n & 1]));
          if (ok && j > 0) ok = outputs(g - 1, j == 1);
        }
        if (ok && nt == 0) mbar_arrive(smem_u32(&bars.q_empty[n & 1]));
        if (ok && nt > 0) ok = outputs(g - 1, nt == 1);
      }
      if (!ok) {
        abort_flag = 1;
        atomicOr(prm.err, kErrTimeout);
      }
      // every MMA issued so far completes before the TMEM is released
      tc_commit(smem_u32(&bars.drain));
      mbar_sleep_bounded(smem_u32(&bars.drain), 0, limit, nullptr);
    }
    __syncwarp();
  } else if (warp == 7) {
    // ----------------------------------------------------------------- q terms
    const float scale0 = prm.sm_scale * kLog2e;
    // the g heads' elements are consecutive: 32 / g lanes per head
    constexpr int LPH = 32 / G, EPL = D / LPH, WORDS = EPL / 2;
    const int h = lane / LPH, off = lane % LPH * EPL;
    bool ok = true;
    for (int n = 0;; ++n) {
      WorkItem w;
      if (n > 0) ok = take_item_warp(n, w);
      else w = prm.items[blockIdx.x];   // (read before it is published)
      if (!ok || w.req < 0) break;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const uint16_t*>(prm.q) +
          (size_t(w.q_row) * prm.num_qo_heads + w.head * G) * D + lane * EPL);
      uint32_t u[WORDS];
      if constexpr (WORDS >= 4) {
#pragma unroll
        for (int e = 0; e < WORDS; e += 4) {
          const uint4 y = *reinterpret_cast<const uint4*>(src + e);
          u[e] = y.x; u[e + 1] = y.y; u[e + 2] = y.z; u[e + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < WORDS; ++e) u[e] = src[e];
      }
      if (n == 0) ok = take_item_warp(0, w);
      if (n >= 2) ok = mbar_sleep_warp(smem_u32(&bars.q_empty[n & 1]), ((n - 2) >> 1) & 1, limit,
                                       &abort_flag);
      if (!ok) break;
      float x[EPL];
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        x[e] = e % 2 == 0 ? E::lo(u[e / 2]) : E::hi(u[e / 2]);
        const float b = fabsf(x[e]);
        a = b < INFINITY ? fmaxf(a, b) : a;
      }
#pragma unroll
      for (int d = LPH / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      const uint32_t au = __float_as_uint(a);
      // the smallest k >= -100 with a <= 448 * 2^k
      const int k = max(int(au >> 23) - 127 - 8 + ((au & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
      const float inv = pow2i(-k);
#pragma unroll
      for (int e = 0; e < EPL; ++e)   // (the conversion saturates infinities: NaN instead)
        x[e] = fabsf(x[e]) < INFINITY ? x[e] * inv : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int tm = 0; tm < C::TERMS; ++tm) {
        const int row = tm * G + h;
        const int sw = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
        uint32_t code[(EPL + 3) / 4];
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
          const uint32_t c = E4m3::from_f32x2(x[e], x[e + 1]);
          const uint32_t f = E4m3::to_f16x2(c);
          x[e] = (x[e] - Fp16::lo(f)) * 16.f;
          x[e + 1] = (x[e + 1] - Fp16::hi(f)) * 16.f;
          if (e % 4 == 0) code[e / 4] = c;
          else code[e / 4] |= c << 16;
        }
        uint8_t* buf = gen + C::OFF_Q + (n & 1) * C::QBYTES + row * C::ROWB;
        constexpr int PIECE = EPL < 16 ? EPL : 16;
#pragma unroll
        for (int e = 0; e < EPL; e += PIECE) {
          const int at = off + e, byte = at % C::ROWB;
          uint8_t* dst = buf + at / 128 * C::N * C::ROWB + (((byte >> 4) ^ sw) << 4) + (byte & 15);
          if constexpr (PIECE == 16)
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(code[e / 4], code[e / 4 + 1], code[e / 4 + 2], code[e / 4 + 3]);
          else if constexpr (PIECE == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
          else if constexpr (PIECE == 4) *reinterpret_cast<uint32_t*>(dst) = code[0];
          else *reinterpret_cast<uint16_t*>(dst) = uint16_t(code[0]);
        }
      }
      if (lane % LPH == 0) q_unit[n & 1][h] = scale0 * pow2i(k);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_full[n & 1]));
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      atomicOr(prm.err, kErrTimeout);
    }
  } else if (warp == 6) {
    // ----------------------------------------------------------------- merging
    // The CTA whose chunk completes a row merges the row's states in slot order
    // (whichever CTA that is, the result is the same): all heads at once, 32 / G
    // states at a time, with a running maximum per head.
    constexpr int SPB = 32 / G;            // states per block: a lane has one (state, head)'s lse
    constexpr int NV = (G * D + 127) / 128;   // float4 pieces per lane and state
    const int h_of = lane % G;
    const bool has = G * D >= 128 || lane * 4 < G * D;
    // the head of piece v of this lane
    auto head_of = [&](int v) { return G == 1 ? 0 : (v * 128 + lane * 4) / D; };
    for (int k = 0;; ++k) {
      // (nothing may be split for as long as the whole launch takes)
      if (!mbar_sleep_warp(smem_u32(&bars.m_full[k & 1]), (k >> 1) & 1, 64 * limit, &abort_flag)) break;
      const int2 e = merge_sh[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.m_empty[k & 1]));
      if (e.x < 0) break;
      const MergeTask mt = prm.merges[e.x];
      uint32_t before = 0;
      if (lane == 0) {
        __threadfence();   // this CTA's states, before the count
        before = atomicAdd(&prm.merge_counters[e.x * hkv + e.y], 1u);
        __threadfence();   // and the other CTAs' states after it
      }
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != uint32_t(mt.n_states - 1)) continue;
      const size_t row = size_t(mt.out_row) * prm.num_qo_heads + e.y * G;
      const size_t slot0 = size_t(mt.slot_base) * prm.num_qo_heads + e.y * G;
      const size_t step = size_t(prm.num_qo_heads);
      // of head h_of: the maximum of lse, and sum 2^(lse - top) (log2 units)
      float top = -INFINITY, sum = 0.f;
      float4 acc[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < mt.n_states; i0 += SPB) {
        const int i = i0 + lane / G;
        const float s = i < mt.n_states ? __ldcg(&prm.partial_lse[slot0 + i * step + h_of]) * kLog2e
                                        : -INFINITY;
        float top2 = s == s ? s : INFINITY;      // (a NaN: kept out of fmaxf, see below)
#pragma unroll
        for (int d = G; d < 32; d <<= 1) top2 = fmaxf(top2, __shfl_xor_sync(0xffffffffu, top2, d));
        top2 = fmaxf(top, top2);
        // 2^(x - x) = NaN for x = inf makes the row NaN; -inf: no keys so far
        const float old = top == -INFINITY ? (top2 == INFINITY ? top2 - top2 : 0.f) : ex2(top - top2);
        const float f = top2 == -INFINITY ? 0.f : ex2(s - top2);
        top = top2;
        float block = f;
#pragma unroll
        for (int d = G; d < 32; d <<= 1) block += __shfl_xor_sync(0xffffffffu, block, d);
        sum = fmaf(sum, old, block);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float o = __shfl_sync(0xffffffffu, old, head_of(v));
          acc[v].x *= o; acc[v].y *= o; acc[v].z *= o; acc[v].w *= o;
        }
#pragma unroll 2
        for (int c = 0; c < SPB; ++c) {
          if (i0 + c >= mt.n_states) break;
          float4 x[NV];
#pragma unroll
          for (int v = 0; v < NV; ++v)
            x[v] = has ? __ldcg(reinterpret_cast<const float4*>(prm.partial_o +
                                                                (slot0 + (i0 + c) * step) * D) +
                                v * 32 + lane)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const float p = __shfl_sync(0xffffffffu, f, c * G + head_of(v));
            acc[v].x = fmaf(p, x[v].x, acc[v].x);
            acc[v].y = fmaf(p, x[v].y, acc[v].y);
            acc[v].z = fmaf(p, x[v].z, acc[v].z);
            acc[v].w = fmaf(p, x[v].w, acc[v].w);
          }
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float o = __shfl_sync(0xffffffffu, inv, head_of(v));
        if (has)
          reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(prm.out) + row * D)[v * 32 + lane] =
              make_uint2(E::pack2(acc[v].x * o, acc[v].y * o), E::pack2(acc[v].z * o, acc[v].w * o));
      }
      if (lane < G && prm.lse)
        prm.lse[row + lane] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * kLn2;
    }
  } else {
    // ------------------------------------------------------ softmax + epilogue
    const int t = threadIdx.x;                          // key of the tile, then dimension
    const uint32_t lane_off = uint32_t(warp * 32) << 16;
    // The four warps meet at named barriers, so none of them leaves alone: after
    // a wait that ran out (`ok` false; no wait waits any more) a warp goes on,
    // and the vote at the next item's start ends all four.
    bool ok = true;
    int g = 0;
    auto sync4 = [] { named_bar_sync(1, 128); };
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      if (ok && !mbar_sleep_warp(smem_u32(&bar), parity, limit, &abort_flag)) {
        ok = false;
        abort_flag = 1;
      }
    };
    int merges = 0;
    for (int n = 0;; ++n) {
      WorkItem w;
      w.req = -1;
      if (ok) ok = take_item_warp(n, w);
      ok = !named_bar_or(1, 128, !ok);
      if (!ok || w.req < 0) break;
      const int nt = tiles_of(w), lead = lead_of(w);
      wait(bars.q_full[n & 1], (n >> 1) & 1);
      float unit[G], m[G], l[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        unit[h] = q_unit[n & 1][h];
        m[h] = -INFINITY;
        l[h] = 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_empty[n & 1]));
      float ref = 1.f;   // r
      for (int j = 0; j < nt; ++j, ++g) {
        const int st = g % C::NST;
        // this key's page scales
        wait(bars.k_full[st], (g / C::NST) & 1);
        const float2 sc = scale_sh[st][t / P];
        if (j == 0) {
          const float2 s0 = scale_sh[st][0];
          ref = s0.x < 0.f ? 1.f : s0.y;
        }
        const int i = j * C::T + t - lead;              // key number from tok_begin
        const bool seen = i >= 0 && i < w.tok_end - w.tok_begin && sc.x >= 0.f;
        const float lv = lg2(sc.y), per_v = fminf(__fdividef(ref, sc.y), 1.2676506e30f);
        wait(bars.s_full[g & 1], (g >> 1) & 1);
        tc_fence_after();
        uint32_t r[C::N];
        if constexpr (C::N == 16) tmem_ld16(tmem + lane_off + (g & 1) * C::N, r);
        else tmem_ld32(tmem + lane_off + (g & 1) * C::N, r);
        tmem_wait_ld();
        float u[G];      // score + log2 s_v
        bool grow = false;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float x = __uint_as_float(r[h]);
          x = fmaf(__uint_as_float(r[G + h]), 0.0625f, x);
          if (C::TERMS == 3) x = fmaf(__uint_as_float(r[2 * G + h]), 0.00390625f, x);
          u[h] = seen ? fmaf(x, sc.x * unit[h], lv) : -INFINITY;
          grow |= u[h] > m[h] + kGrow;
        }
        if (named_bar_or(1, 128, grow)) {
          // new maxima over the tile's keys, and O and l on the new scale
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float a = warp_max(u[h] == u[h] ? u[h] : -INFINITY);   // (without NaN)
            if (lane == 0) red[warp][h] = a;
          }
          sync4();
          float alpha[G];
          bool live = false;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float a = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]));
            const float m2 = fmaxf(m[h], a);
            alpha[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - m2);
            l[h] *= alpha[h];
            live |= alpha[h] != 1.f;
            m[h] = m2;
          }
          if (j > 0 && live) {
            wait(bars.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < C::DB; ++b) {
              uint32_t o[C::N];
              const uint32_t at = o_col0 + lane_off + b * C::N;
              if constexpr (C::N == 16) tmem_ld16(at, o);
              else tmem_ld32(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < C::COLS; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c % G]);
              if constexpr (C::N == 16) tmem_st16(at, o);
              else tmem_st32(at, o);
            }
            tmem_wait_st();
          }
        }
        // weights, as e4m3 terms into P^T
        uint32_t pw[C::N / 4];
#pragma unroll
        for (int c = 0; c < C::N / 4; ++c) pw[c] = 0u;
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          float x[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 2 && h + e < G; ++e) {
            x[e] = ex2(u[h + e] - (m[h + e] == -INFINITY ? 0.f : m[h + e]));
            l[h + e] = fmaf(x[e], per_v, l[h + e]);
            x[e] *= kWeightUnit;
          }
#pragma unroll
          for (int tm = 0; tm < C::TERMS; ++tm) {
            uint32_t c = E4m3::from_f32x2(x[0], x[1]);
            if (tm + 1 < C::TERMS) {
              const uint32_t f = E4m3::to_f16x2(c);
              x[0] = (x[0] - Fp16::lo(f)) * 16.f;
              x[1] = (x[1] - Fp16::hi(f)) * 16.f;
            }
            if (G == 1) c &= 0xffu;
            const int at = tm * G + h;
            pw[at / 4] |= c << (8 * (at % 4));
          }
        }
        // P^T: per key 16 bytes of each block of 16 columns; its buffer was
        // last read by the output MMAs of tile g - 2
        if (g >= 2) wait(bars.pv_done[g & 1], ((g - 2) >> 1) & 1);
        uint8_t* pb = gen + C::OFF_P + (g & 1) * C::PBYTES + t * 16;
#pragma unroll
        for (int c = 0; c < C::N / 16; ++c)
          *reinterpret_cast<uint4*>(pb + c * C::T * 16) =
              make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
        // V rows of keys outside the item hold stale bytes, maybe NaN codes,
        // which a zero weight would not cancel
        if (__any_sync(0xffffffffu, !seen)) {
          wait(bars.v_full[st], (g / C::NST) & 1);
          if (!seen) {
#pragma unroll
            for (int b = 0; b < C::DB; ++b)
#pragma unroll
              for (int c = 0; c < C::ROWB / 16; ++c)   // (spread over the banks)
                st_shared_zero16(base + st * C::STAGE + C::KBYTES + (b * C::T + t) * C::ROWB +
                                 ((c + lane) % (C::ROWB / 16)) * 16);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[g & 1]));
      }
      // ---- epilogue: the sums of the four warps' keys
      {
        // halving the heads a lane adds up with each exchange: after log2 G of
        // them a lane has one head, in the bits of its number from 16 down
        float x[G];
#pragma unroll
        for (int h = 0; h < G; ++h) x[h] = l[h];
        int head = 0, d = 16;
#pragma unroll
        for (int c = G / 2; c > 0; c /= 2, d >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int h = 0; h < c; ++h)
            x[h] = (up ? x[h + c] : x[h]) + __shfl_xor_sync(0xffffffffu, up ? x[h] : x[h + c], d);
          head += up ? c : 0;
        }
#pragma unroll
        for (int e = 16; e > 0; e >>= 1)
          if (e <= 16 / G) x[0] += __shfl_xor_sync(0xffffffffu, x[0], e);
        if ((lane & (32 / G - 1)) == 0) sum_sh[warp][head] = x[0];
      }
      sync4();
      float f[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        l[h] = (sum_sh[0][h] + sum_sh[1][h]) + (sum_sh[2][h] + sum_sh[3][h]);
        // (a NaN sum, from a NaN in q or in the cache, stays one)
        f[h] = l[h] == 0.f ? 0.f : __fdividef(prm.v_scale * ref, kWeightUnit * l[h]);
      }
      const bool split = w.slot >= 0;
      const size_t orow = size_t(split ? w.slot : w.q_row) * prm.num_qo_heads + w.head * G;
      if (nt > 0) wait(bars.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < C::DB; ++b) {
        uint32_t o[C::N];
        if (nt > 0) {
          const uint32_t at = o_col0 + lane_off + b * C::N;
          if constexpr (C::N == 16) tmem_ld16(at, o);
          else tmem_ld32(at, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < C::N; ++c) o[c] = 0u;
        }
        if (t < D && ok) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            float x = __uint_as_float(o[h]);
            x = fmaf(__uint_as_float(o[G + h]), 0.0625f, x);
            if (C::TERMS == 3) x = fmaf(__uint_as_float(o[2 * G + h]), 0.00390625f, x);
            x *= f[h];
            const size_t at = (orow + h) * D + b * 128 + t;
            if (split) prm.partial_o[at] = x;
            else reinterpret_cast<uint16_t*>(prm.out)[at] = E::one(x);
          }
        }
      }
      float* lse = split ? prm.partial_lse : prm.lse;
      if (lse) {
        const float lr = lg2(ref);
#pragma unroll
        for (int h = 0; h < G; ++h)
          if (t == h) lse[orow + h] = l[h] == 0.f ? -INFINITY : (m[h] + (lg2(l[h]) - lr)) * kLn2;
      }
      tc_fence_before();
      if (split) {
        const int e = merges & 1;
        if (merges >= 2) wait(bars.m_empty[e], ((merges - 2) >> 1) & 1);
        if (t == 0) merge_sh[e] = make_int2(w.merge, w.head);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.m_full[e]));
        ++merges;
      }
    }
    // no more merges
    {
      const int e = merges & 1;
      if (merges >= 2) wait(bars.m_empty[e], ((merges - 2) >> 1) & 1);
      if (t == 0) merge_sh[e] = make_int2(-1, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.m_full[e]));
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      atomicOr(prm.err, kErrTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // every copy that was issued lands before the CTA exits, also after a timeout
  if (warp == 4 && lane == 0) {
    for (int j = max(0, issued - C::NST); j < issued; ++j) {
      if (!(j == 0 && prm.fault_kind == 1 && blockIdx.x == 0))   // K never issued
        mbar_sleep_bounded(smem_u32(&bars.k_full[j % C::NST]), (j / C::NST) & 1, limit, nullptr);
      mbar_sleep_bounded(smem_u32(&bars.v_full[j % C::NST]), (j / C::NST) & 1, limit, nullptr);
    }
  }
}

template <int D, int G, class E>
cudaError_t launch_t(const CUtensorMap& km, const CUtensorMap& vm, const DecodeParams& p,
                     int n_items, int num_sms, bool overlap, cudaStream_t stream) {
  using C = D8Cfg<D, G, E>;
  auto kern = decode_page8_kernel<D, G, E>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = once_per_device(configured, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  DecodeParams q = p;
  q.n_items = n_items;
  const long long slots = (long long)num_sms * C::CTAS;
  return launch_overlapping(kern, int(slots < n_items ? slots : n_items), C::THREADS, C::SMEM,
                            overlap, stream, km, vm, q);
}

template <int D, class E>
cudaError_t launch_g(int group, const CUtensorMap& km, const CUtensorMap& vm,
                     const DecodeParams& p, int n_items, int num_sms, bool overlap,
                     cudaStream_t stream) {
  switch (group) {
    case 1: return launch_t<D, 1, E>(km, vm, p, n_items, num_sms, overlap, stream);
    case 2: return launch_t<D, 2, E>(km, vm, p, n_items, num_sms, overlap, stream);
    case 4: return launch_t<D, 4, E>(km, vm, p, n_items, num_sms, overlap, stream);
    case 8: return launch_t<D, 8, E>(km, vm, p, n_items, num_sms, overlap, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <class E>
cudaError_t launch_d(int head_dim, int group, const CUtensorMap& km, const CUtensorMap& vm,
                     const DecodeParams& p, int n_items, int num_sms, bool overlap,
                     cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_g<64, E>(group, km, vm, p, n_items, num_sms, overlap, stream);
    case 128: return launch_g<128, E>(group, km, vm, p, n_items, num_sms, overlap, stream);
    case 256: return launch_g<256, E>(group, km, vm, p, n_items, num_sms, overlap, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_page8(int head_dim, int group, int dtype, const CUtensorMap& km,
                                const CUtensorMap& vm, const DecodeParams& p, int n_items,
                                int num_sms, bool overlap, cudaStream_t stream) {
  if (n_items <= 0 || num_sms <= 0) return cudaSuccess;
  switch (dtype) {
    case FI_DTYPE_BF16: return launch_d<Bf16>(head_dim, group, km, vm, p, n_items, num_sms, overlap, stream);
    case FI_DTYPE_FP16: return launch_d<Fp16>(head_dim, group, km, vm, p, n_items, num_sms, overlap, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fi
