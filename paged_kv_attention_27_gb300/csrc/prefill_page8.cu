// Variable-length batch prefill over a page-scaled FP8 cache: chunks of query
// rows, causal or not, against K = s_k(page, head) * codes, V alike.
//
// A work item is (rows of a request, kv head): rows x the g query heads of the
// kv head fill the M rows of two 128-row tiles (one at head_dim 256), heads
// inner, so that every K/V tile that is loaded serves all of them; a draft's
// few rows and a long prompt run the same way. Where the rows fill one M tile
// only, the second stream of scores and outputs can take every other K/V tile
// of the same rows (a tile's chain score -> softmax -> output is serial, and two
// of them keep the SM busy); the two states are merged at the end. That is a
// kernel of its own (SOLO): 48 drafts of 1-9 rows 158 -> 129 us, but launches
// whose items fill both tiles 3 % slower, so the planner picks it where an
// eighth of the work or more is in items of one M tile.
//
// Arithmetic: the scores' MMAs take the K codes as they arrive (kind::f8f6f4).
// A q row, times the power of two that puts its largest element at 224..448,
// enters as a sum of e4m3 terms t0 = e4m3(x), t1 = e4m3(x - t0), ...: two carry
// the 8 significand bits of bf16, three the 11 of fp16, down to E4M3's finest
// step of 2^-9, so that an element is off by at most 2^-10, 2^-17 of the row's
// largest. Two e4m3 MMAs cost what one 16-bit MMA would, and K is neither
// widened nor stored twice. The outputs' MMAs multiply fp16 weights by V codes
// that a warpgroup widens to fp16, exactly (splitting the weights instead would
// cost the softmax warps three times the instructions that widening costs).
// The page's s_k joins the row's score scale, one factor per 16 columns. The
// page's s_v joins the weight before it is rounded to fp16:
//   w = 2^(s + log2 s_v - m),  m the running maximum of s + log2 s_v,
//   O = sum w code,  l = sum w r / s_v (r: s_v of the item's first page),
//   out = O r / l,   lse = ln 2 (m + log2 l - log2 r):
// one exponential per score, and both sums keep their leading bits where a
// request's V scales are up to 2^80 apart (l then stays below 2^118, and a
// weight of 2^-80 is far from underflow).
//
// Roles (16 warps): 8 softmax warps, then the epilogue. They work on one M tile
// after the other, two threads per row (TMEM lane), each on half of the keys:
// while they are on one tile, the other's MMAs run. (A warpgroup per tile, a
// thread per row, was slower: the warpgroups have to take turns for that
// overlap, and one warp per scheduler waits for its own instructions.) A warp
// each to issue a tile's MMAs and one to copy K/V pages and their scales (two in
// the SOLO kernel: a TMA box takes about 130 cycles to issue, so that one warp
// was slower than its tiles, 133 -> 129 us; elsewhere a second one costs 0.4 %);
// a warpgroup to turn q into terms and widen V.
//
// Measured, calls back to back: two chunks of 400-512 rows on 20000-32000 keys,
// 64/8 heads of 128, 938 us (1000 TFLOP/s, 0.54 of the measured bf16 burst
// rate); four prompts of 3300-4096 tokens 1008 us (0.52); 48 drafts of 1-9 rows
// on 300-8192 keys, 32/8 heads, 126 us (0.30 of the copy bandwidth). Bound by
// the chain of a tile: scores seen by the softmax, 1400 cycles of softmax, 300
// until its P is seen, 1150 for the output MMAs until the next scores' may go,
// 765 for those; the two M tiles' chains overlap, a pair takes 3850-4000 cycles,
// 41 % of them with the tensor pipe busy.
#include <cfloat>
#include <climits>
#include <type_traits>

#include "elem.cuh"
#include "page8.cuh"
#include "ptx_page8.cuh"

namespace fi {

namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 units: the maximum moves when a score passes it by more; weights stay
// at or below 2^8, inside fp16
constexpr float kRescaleThreshold = 8.0f;
constexpr int kItemRing = 8;
// tiles whose page scales are kept: K of tile t is copied once S of tile t - 3
// is complete, which was issued after the softmax of tile t - 4
constexpr int kScaleRing = 4;

template <int D, class E>
struct P8Cfg {
  static constexpr int TILES = D <= 128 ? 2 : 1;
  static constexpr int TERMS = std::is_same<E, Bf16>::value ? 2 : 3;
  static constexpr int M = 128;
  static constexpr int N = D <= 128 ? 128 : 64;             // keys per tile
  static constexpr int NG = N / 16;                         // 16-column groups (pages) of a tile
  static constexpr int ROWB = D < 128 ? D : 128;            // bytes of a shared-memory row of codes
  static constexpr int BLK = D <= 128 ? 1 : D / 128;        // 128-byte slices of a row of codes
  static constexpr uint32_t SWZ = ROWB == 128 ? 2 : 4;      // 128- or 64-byte swizzle
  static constexpr uint32_t ATOM = 8 * ROWB;
  static constexpr int CODES = N * D;                       // one K (or V) tile of codes
  static constexpr int V = N * D * 2;                       // one widened V tile
  static constexpr int QT = M * D;                          // one term of a tile's q
  static constexpr int Q = TERMS * QT;
  static constexpr int NK = TERMS == 3 && D >= 128 ? 2 : 3; // K tiles in flight
  static constexpr int NVR = TERMS == 3 && D >= 128 ? 1 : 2;   // V code tiles in flight
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + TILES * Q;
  static constexpr int OFF_V = OFF_K + NK * CODES;          // two
  static constexpr int OFF_VR = OFF_V + 2 * V;
  static constexpr int USED = OFF_VR + NVR * CODES;
  static constexpr int SMEM = (USED < 120 * 1024 ? 120 * 1024 : USED) + 1024;   // one CTA per SM
  static_assert(SMEM <= 220 * 1024, "shared-memory budget (and up to 6 KB of static arrays)");
  static constexpr int SOFT = 8;                            // softmax warps: two threads per row
  static constexpr int H = N / 2, HG = NG / 2;              // columns (16-column groups) per thread
  static constexpr int W_MMA = SOFT, W_KV = SOFT + 2, W_WIDE = SOFT + 4;
  static constexpr int THREADS = 32 * (SOFT + 8);
  // registers per thread at launch and, per warpgroup, after the split
  static constexpr uint32_t LAUNCH_REGS = 128, SOFT_REGS = 160, HELP_REGS = 80, WIDE_REGS = 112;
  static_assert(2 * SOFT_REGS + HELP_REGS + WIDE_REGS <= 4 * LAUNCH_REGS, "");
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t col_s(int i) { return uint32_t(i * N); }
  __host__ __device__ static constexpr uint32_t col_o(int i) { return uint32_t(TILES * N + i * D); }
  static_assert(TILES * (N + D) <= 512, "TMEM budget");
  static constexpr uint32_t IDESC_QK = idesc_e4m3(M, N, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_f16kind(M, D, 0, 1, Fp16::kMmaFmt);
};

struct P8Barriers {
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t q_full, q_empty;
  uint64_t k_full[3], k_empty[3], vr_full[2], vr_empty[2];     // tiles of codes
  uint64_t v_full[2], v_empty[2];                              // widened tiles
  uint64_t s_full[2], p_full[2], pv_done[2], o_final[2], drain[2];
  uint64_t sc_full[kScaleRing];                                // a tile's page scales
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

template <int D, class E, bool SOLO>
__global__ void __launch_bounds__(P8Cfg<D, E>::THREADS, 1)
prefill_page8_kernel(const void* q, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, PrefillParams prm) {
  using C = P8Cfg<D, E>;
  constexpr int COPIERS = SOLO ? 2 : 1;   // warps that copy K/V pages
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) P8Barriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int item_ring[kItemRing];
  __shared__ __align__(8) float2 raw_scale[C::NK][8];       // per page of a K tile: s_k, s_v
  __shared__ __align__(16) float4 scale_sh[kScaleRing][8];  // per 16 columns: s_k (-1: no page),
                                                            // log2 s_v, r / s_v, r
  __shared__ int lost_sh[kScaleRing];                       // the tile has a page outside the cache
  __shared__ float pair_sh[2][2][128];                      // a row's halves: maxima, sums
  __shared__ uint8_t q_exp[2][C::TILES * 128];              // q rows' exponents + 128, by item parity

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = prm.wait_limit_ns;
  const int P = prm.page_size, ppt = C::N / P;
  const int g = prm.group;
  const int R = C::M / g;                                   // query rows per tile
  const int hkv = prm.num_qo_heads / g;

  auto item_at = [&](int n, int& idx) {
    if (!mbar_sleep_bounded(smem_u32(&bars.item_full[n % kItemRing]), (n / kItemRing) & 1, limit,
                           &abort_flag))
      return false;
    idx = *reinterpret_cast<volatile int*>(&item_ring[n % kItemRing]);
    return true;
  };
  auto item_done = [&](int n) { mbar_arrive(smem_u32(&bars.item_empty[n % kItemRing])); };
  // item n for a whole warp (lane 0 waits)
  auto take_item = [&](int n, int& idx) {
    int v = -1;
    bool good = true;
    if (lane == 0) {
      good = item_at(n, v);
      item_done(n);
    }
    idx = __shfl_sync(0xffffffffu, v, 0);
    return __shfl_sync(0xffffffffu, good, 0) != 0;
  };
  auto tiles_of = [&](const WorkItem& w) { return (w.tok_end - w.tok_begin + C::N - 1) / C::N; };
  // whether tile i of the item has a row (tile 0 always does)
  auto active = [&](const WorkItem& w, int i) {
    return i == 0 || w.q_row + R < prm.qo_indptr[w.req + 1];
  };
  auto fail = [&] {
    abort_flag = 1;
    atomicOr(prm.err, kErrTimeout);
  };

  // (see the decode kernel)
  if (threadIdx.x == 0) {
    pdl_trigger();
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(smem_u32(&bars.item_full[s]), 1);
      // softmax warps, MMA warps, the widening warps, a second copying warp
      mbar_init(smem_u32(&bars.item_empty[s]), C::SOFT + C::TILES + 4 + COPIERS - 1);
    }
    mbar_init(smem_u32(&bars.q_full), 4);
    mbar_init(smem_u32(&bars.q_empty), C::TILES);
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(smem_u32(&bars.k_full[s]), COPIERS + ppt);  // the bytes, and each page's scales
      mbar_init(smem_u32(&bars.k_empty[s]), C::TILES + 4);  // S of the tiles; the scales' readers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars.vr_full[s]), COPIERS);
      mbar_init(smem_u32(&bars.vr_empty[s]), 4);
      mbar_init(smem_u32(&bars.v_full[s]), 4);
      mbar_init(smem_u32(&bars.v_empty[s]), C::TILES);
      mbar_init(smem_u32(&bars.s_full[s]), 1);
      mbar_init(smem_u32(&bars.p_full[s]), 8);
      mbar_init(smem_u32(&bars.pv_done[s]), 1);
      mbar_init(smem_u32(&bars.o_final[s]), 1);
      mbar_init(smem_u32(&bars.drain[s]), 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(smem_u32(&bars.sc_full[s]), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_u32(&tmem_base_sh), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  int issued = 0;    // the K/V copy warp: tiles whose copies it has issued

  if (warp >= C::W_WIDE) {
    // ------------------------------------------------------------------ widening
    if constexpr (C::WIDE_REGS < C::LAUNCH_REGS) setmaxnreg_dec<C::WIDE_REGS>();
    const int ct = threadIdx.x - C::W_WIDE * 32;            // 0..127
    // Codes -> fp16 rows as the TMA would write them (128-byte swizzled slices
    // of 64 dimensions). A warp's lanes take 8 rows x 4 chunks of 16 codes:
    // reads and writes then touch all banks evenly. Rows from `valid` on, and
    // those of pages outside the cache (bits of `lost`), become zero.
    // A thread keeps its chunk; its rows are 128 / CH apart, so that each address
    // is the first one plus a constant.
    constexpr int CH = D / 16;                              // 16-code chunks per row
    constexpr int STEP = 128 / CH, ITER = C::N / STEP;
    const int w_row = ((ct >> 3) / CH) * 8 + (ct & 7), w_ch = (ct >> 3) % CH;
    const uint32_t w_src = base + C::OFF_VR + (w_ch >> 3) * C::N * 128 + w_row * C::ROWB +
                           (((w_ch & 7) ^ (C::ROWB == 128 ? (w_row & 7) : ((w_row >> 1) & 3))) << 4);
    const uint32_t w_dst = base + C::OFF_V + (w_ch >> 2) * C::N * 128 + w_row * 128;
    const uint32_t w_lo = w_dst + ((((w_ch & 3) * 2) ^ (w_row & 7)) << 4);
    const uint32_t w_hi = w_dst + ((((w_ch & 3) * 2 + 1) ^ (w_row & 7)) << 4);
    auto widen = [&](int from, int to, int valid, uint32_t lost) {
      const uint32_t src = w_src + from * C::CODES, lo = w_lo + to * C::V, hi = w_hi + to * C::V;
      constexpr int AT_ONCE = ITER < 8 ? ITER : 8;
#pragma unroll
      for (int i0 = 0; i0 < ITER; i0 += AT_ONCE) {
        uint4 u[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) u[i] = lds128(src + (i0 + i) * STEP * C::ROWB);
        if (valid < C::N || lost != 0u) {
#pragma unroll
          for (int i = 0; i < AT_ONCE; ++i) {
            const int row = w_row + (i0 + i) * STEP;
            if (row >= valid || ((lost >> (row >> 4)) & 1u)) u[i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
          const uint2 a = E4m3::to_f16x4(u[i].x), b = E4m3::to_f16x4(u[i].y);
          const uint2 c = E4m3::to_f16x4(u[i].z), d = E4m3::to_f16x4(u[i].w);
          st_shared_v4(lo + (i0 + i) * STEP * 128, make_uint4(a.x, a.y, b.x, b.y));
          st_shared_v4(hi + (i0 + i) * STEP * 128, make_uint4(c.x, c.y, d.x, d.y));
        }
      }
    };
    bool ok = true;
    int gt = 0;   // tiles of earlier items
    const int g_log = __ffs(g) - 1;   // g is a power of two
    int it = -1, it_next = -1;
    ok = take_item(0, it);
    WorkItem w, wn;
    if (ok && it >= 0) w = prm.items[it];
    for (int n = 0; ok && it >= 0; ++n) {
      const int nt = tiles_of(w);
      // the item's M rows: query rows x heads, heads inner
      auto m_rows = [&](const WorkItem& y) {
        return min(C::TILES * C::M, (prm.qo_indptr[y.req + 1] - y.q_row) << g_log);
      };
      // The next item, when this one's work is under way: its q into L2.
      auto look_ahead = [&] {
        if (!take_item(n + 1, it_next)) return false;
        if (it_next >= 0) {
          wn = prm.items[it_next];
          const int lines = m_rows(wn) * (D * 2 / 128);
          for (int i = ct; i < lines; i += 128) {
            const int x = i / (D * 2 / 128);
            const uint16_t* at = reinterpret_cast<const uint16_t*>(q) +
                                 (size_t(wn.q_row + (x >> g_log)) * prm.num_qo_heads + wn.head * g +
                                  (x & (g - 1))) * D + i % (D * 2 / 128) * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
          }
        }
        return true;
      };
      // ---- q as terms: D / 16 lanes per row, 16 elements each; two rows' loads
      // ahead of the two rows at work, the first ones before the previous item
      // has let go of q (loaded row by row and in 32-bit arithmetic this took 29K
      // cycles, and the item waited for 20K of them)
      {
        constexpr int LPR = D / 16, STEP_ROWS = 128 / LPR, PASSES = C::TILES * C::M / STEP_ROWS;
        constexpr int BATCH = 2;
        static_assert(PASSES % BATCH == 0, "");
        const int used = m_rows(w);       // (rows behind the last one are never stored)
        const int ch = lane % LPR, x0 = ct / LPR;
        uint4 u[BATCH][2];
        auto load = [&](int b) {
#pragma unroll
          for (int e = 0; e < BATCH; ++e) {
            const int x = x0 + (b * BATCH + e) * STEP_ROWS;
            u[e][0] = u[e][1] = make_uint4(0u, 0u, 0u, 0u);
            if (x < used) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  reinterpret_cast<const uint16_t*>(q) +
                  (size_t(w.q_row + (x >> g_log)) * prm.num_qo_heads + w.head * g + (x & (g - 1))) * D +
                  ch * 16);
              u[e][0] = src[0];
              u[e][1] = src[1];
            }
          }
        };
        load(0);
        if (n >= 1 && !mbar_sleep_warp(smem_u32(&bars.q_empty), (n - 1) & 1, limit, &abort_flag)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int b = 0; b * BATCH * STEP_ROWS < used; ++b) {
          uint4 v[BATCH][2];
#pragma unroll
          for (int e = 0; e < BATCH; ++e) {
            v[e][0] = u[e][0];
            v[e][1] = u[e][1];
          }
          load(b + 1);
#pragma unroll
          for (int e4 = 0; e4 < BATCH; ++e4) {
            const int x = x0 + (b * BATCH + e4) * STEP_ROWS;
            const int i = x / C::M, row = x % C::M;
            const uint32_t q2[8] = {v[e4][0].x, v[e4][0].y, v[e4][0].z, v[e4][0].w,
                                    v[e4][1].x, v[e4][1].y, v[e4][1].z, v[e4][1].w};
            // |x| of bf16 and fp16 orders as its 15 bits
            uint32_t top2 = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) top2 = __vmaxu2(top2, q2[e] & 0x7fff7fffu);
#pragma unroll
            for (int d = LPR / 2; d > 0; d >>= 1)
              top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, d));
            const uint32_t top = max(top2 >> 16, top2 & 0xffffu);
            constexpr uint32_t kInf = std::is_same<E, Bf16>::value ? 0x7f80u : 0x7c00u;
            const bool odd = top >= kInf;   // a NaN or an infinity in the row
            // the smallest k >= -100 with a <= 448 * 2^k (such a row is NaN whatever its k)
            const uint32_t au = odd ? 0x3f800000u : __float_as_uint(E::lo(top));
            const int k = max(int(au >> 23) - 127 - 8 + ((au & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
            const float up = __uint_as_float(uint32_t(127 - k) << 23);
            uint32_t h2[8];                 // the row as fp16 pairs: exact, above its grid of 2^-24
#pragma unroll
            for (int e = 0; e < 8; ++e) h2[e] = Fp16::pack2(E::lo(q2[e]) * up, E::hi(q2[e]) * up);
            if (odd) {   // (the conversion to e4m3 saturates infinities: NaN instead)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if ((q2[e] & 0x7fffu) >= kInf) h2[e] = (h2[e] & 0xffff0000u) | 0x7e00u;
                if ((q2[e] >> 16 & 0x7fffu) >= kInf) h2[e] = (h2[e] & 0xffffu) | 0x7e000000u;
              }
            }
            const int sw = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
            const uint32_t dst = base + C::OFF_Q + i * C::Q + (ch >> 3) * C::M * 128 +
                                 row * C::ROWB + (((ch & 7) ^ sw) << 4);
#pragma unroll
            for (int tm = 0; tm < C::TERMS; ++tm) {
              uint32_t code[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const uint32_t c0 = E4m3::from_f16x2(h2[e]), c1 = E4m3::from_f16x2(h2[e + 1]);
                code[e / 2] = c0 | (c1 << 16);
                if (tm + 1 < C::TERMS) {   // what the term leaves, exactly
                  h2[e] = Fp16::sub2(h2[e], E4m3::to_f16x2(c0));
                  h2[e + 1] = Fp16::sub2(h2[e + 1], E4m3::to_f16x2(c1));
                }
              }
              st_shared_v4(dst + tm * C::QT, make_uint4(code[0], code[1], code[2], code[3]));
            }
            if (ch == 0) q_exp[n & 1][x] = uint8_t(k + 128);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.q_full));
      }
      float ref = 1.f;
      if (nt == 0) ok = look_ahead();
      for (int j = 0; j < nt; ++j) {
        const int t = gt + j, ks = t % C::NK, rs = t % C::NVR, st = t & 1;
        const int valid = min(C::N, w.tok_end - w.tok_begin - j * C::N);
        // the tile's page scales, which come with K
        if (!mbar_sleep_warp(smem_u32(&bars.k_full[ks]), (t / C::NK) & 1, limit, &abort_flag)) {
          ok = false;
          break;
        }
        uint32_t lost = 0u;   // by 16 columns
        {
          const bool in = lane < C::NG && lane * 16 < valid;
          const float2 s = in ? raw_scale[ks][lane * 16 / P] : make_float2(1.f, 1.f);
          const bool gone = in && s.x < 0.f;
          lost = __ballot_sync(0xffffffffu, gone);
          if (j == 0) ref = __shfl_sync(0xffffffffu, gone ? 1.f : s.y, 0);
          if (ct < 32) {      // the first warp writes them
            if (ct < C::NG)
              scale_sh[t % kScaleRing][lane] =
                  make_float4(gone ? 0.f : s.x, gone ? 0.f : lg2(s.y),
                              fminf(ref / s.y, 1.2676506e30f), ref);
            if (ct == 0) lost_sh[t % kScaleRing] = int(lost);
            __syncwarp();
            if (ct == 0) mbar_arrive(smem_u32(&bars.sc_full[t % kScaleRing]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.k_empty[ks]));
        }
        if (!mbar_sleep_warp(smem_u32(&bars.vr_full[rs]), (t / C::NVR) & 1, limit, &abort_flag) ||
            (t >= 2 && !mbar_sleep_warp(smem_u32(&bars.v_empty[st]), ((t >> 1) & 1) ^ 1, limit,
                                       &abort_flag))) {
          ok = false;
          break;
        }
        widen(rs, st, valid, lost);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars.vr_empty[rs]));
          mbar_arrive(smem_u32(&bars.v_full[st]));
        }
        if (j == 0 && !look_ahead()) {
          ok = false;
          break;
        }
      }
      gt += nt;
      w = wn;
      it = it_next;
    }
    if (!ok && lane == 0) fail();
  } else if (warp >= C::W_MMA) {
    setmaxnreg_dec<C::HELP_REGS>();
    if (warp >= C::W_KV && warp < C::W_KV + COPIERS) {
      // -------------------------------------------------------------- K/V copies
      // Each warp has its share of a tile's pages; the first hands out the items.
      const int share = ppt / COPIERS, slot0 = (warp - C::W_KV) * share;
      if (lane == 0) {
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
      }
      const uint32_t box = uint32_t(P) * C::ROWB;
      auto publish = [&](int n, int value) {
        if (n >= kItemRing &&
            !mbar_sleep_bounded(smem_u32(&bars.item_empty[n % kItemRing]),
                               ((n / kItemRing) & 1) ^ 1, limit, &abort_flag))
          return false;
        item_ring[n % kItemRing] = value;
        mbar_arrive(smem_u32(&bars.item_full[n % kItemRing]));
        return true;
      };
      auto next_item = [&](int n, int& idx) {
        if (warp != C::W_KV) return take_item(n, idx);
        int v = -1;
        bool good = true;
        if (lane == 0) {
          v = n == 0 ? int(blockIdx.x) : int(gridDim.x + atomicAdd(prm.work_counter, 1u));
          if (v >= prm.n_items) v = -1;
          good = publish(n, v);
        }
        idx = __shfl_sync(0xffffffffu, v, 0);
        return __shfl_sync(0xffffffffu, good, 0) != 0;
      };
      // whether this lane has a page of tile j
      auto has_page = [&](const WorkItem& w, int j) {
        return lane < share && (slot0 + lane) * P < w.tok_end - w.tok_begin - j * C::N;
      };
      int it = -1, t = 0;
      bool ok = next_item(0, it);
      WorkItem w;
      if (ok && it >= 0) w = prm.items[it];
      int next_page = -1;
      if (ok && it >= 0 && has_page(w, 0)) next_page = prm.page_indices[w.page_begin + slot0 + lane];
      for (int n = 0; ok && it >= 0; ++n) {
        const int nt = tiles_of(w);
        const int c1 = prm.layout == FI_LAYOUT_NHD ? w.head : 0;
        const int c2 = prm.layout == FI_LAYOUT_NHD ? 0 : w.head;
        int it_next = -1;
        if (!next_item(n + 1, it_next)) {
          ok = false;
          break;
        }
        WorkItem wn;
        if (it_next >= 0) wn = prm.items[it_next];
        if (nt == 0)
          next_page = it_next >= 0 && has_page(wn, 0) ? prm.page_indices[wn.page_begin + slot0 + lane]
                                                      : -1;
        for (int j = 0; j < nt; ++j, ++t) {
          const int ks = t % C::NK, rs = t % C::NVR;
          const int page = next_page;
          const bool mine = has_page(w, j);
          const bool valid = mine && page >= 0 && page < prm.num_pages;
          if (mine && !valid) atomicOr(prm.err, kErrBounds);
          next_page = -1;
          if (j + 1 < nt) {
            if (has_page(w, j + 1))
              next_page = prm.page_indices[w.page_begin + (j + 1) * ppt + slot0 + lane];
          } else if (it_next >= 0 && has_page(wn, 0)) {
            next_page = prm.page_indices[wn.page_begin + slot0 + lane];
          }
          const uint32_t bytes =
              uint32_t(__popc(__ballot_sync(0xffffffffu, valid))) * C::BLK * box;
          const bool skip = t == 0 && prm.fault_kind == 1 && blockIdx.x == 0;
          const uint32_t kf = smem_u32(&bars.k_full[ks]), vf = smem_u32(&bars.vr_full[rs]);
          if (t >= C::NK && !mbar_sleep_warp(smem_u32(&bars.k_empty[ks]), ((t / C::NK) & 1) ^ 1, limit,
                                            &abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0 && !skip) mbar_arrive_expect_tx(kf, bytes);
          __syncwarp();
          if (valid && !skip) {
            const uint32_t dst = base + C::OFF_K + ks * C::CODES + (slot0 + lane) * box;
#pragma unroll
            for (int b = 0; b < C::BLK; ++b)
              tma_load_4d(dst + b * C::N * 128, &k_map, kf, b * 128, c1, c2, page);
          }
          if (lane < share) {
            if (valid) {
              const size_t at = size_t(page) * hkv + w.head;
              const uint32_t sc = smem_u32(&raw_scale[ks][slot0 + lane]);
              cp_async4(sc, prm.k_head_scale + at);
              cp_async4(sc + 4, prm.v_head_scale + at);
              cp_async_arrive(kf);
            } else {
              raw_scale[ks][slot0 + lane] = make_float2(-1.f, 1.f);
              mbar_arrive(kf);
            }
          }
          issued = t + 1;
          if (t >= C::NVR && !mbar_sleep_warp(smem_u32(&bars.vr_empty[rs]), ((t / C::NVR) & 1) ^ 1,
                                             limit, &abort_flag)) {
            ok = false;
            issued = -issued;   // K of this tile, not V
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(vf, bytes);
          __syncwarp();
          if (valid) {
            const uint32_t dst = base + C::OFF_VR + rs * C::CODES + (slot0 + lane) * box;
#pragma unroll
            for (int b = 0; b < C::BLK; ++b)
              tma_load_4d(dst + b * C::N * 128, &v_map, vf, b * 128, c1, c2, page);
          }
        }
        w = wn;
        it = it_next;
      }
      if (!ok && lane == 0) fail();
      cp_async_wait_all();
      __syncwarp();
    } else if (warp < C::W_MMA + C::TILES) {
      // ------------------------------------------------------------- MMA issuers
      const int i = warp - C::W_MMA;
      if (lane == 0) {
        const uint64_t qd0 = sdesc_swz(base + C::OFF_Q, 16, C::ATOM, C::SWZ);
        const uint64_t kd0 = sdesc_swz(base + C::OFF_K, 16, C::ATOM, C::SWZ);
        const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, C::N * 128, 1024);
        const uint32_t s_col = tmem + C::col_s(i), o_col = tmem + C::col_o(i);
        auto wait = [&](uint64_t& bar, uint32_t parity) {
          return mbar_sleep_bounded(smem_u32(&bar), parity, limit, &abort_flag);
        };
        bool ok = true;
        int t = 0;      // tiles of earlier items
        int mine = 0;   // of which this stream took
        for (int n = 0; ok; ++n) {
          int it = -1;
          ok = item_at(n, it);
          item_done(n);
          if (!ok || it < 0) break;
          const WorkItem w = prm.items[it];
          const int nt = tiles_of(w);
          ok = wait(bars.q_full, n & 1);
          // Both M tiles have rows: each stream takes every K/V tile. One has:
          // stream 0 does, or (SOLO) the streams share that M tile's q and take
          // turns. (Separate loops: this thread is on the tiles' chains, and the
          // conditions in one common loop cost 4 % of a launch.)
          const bool both = C::TILES == 1 || active(w, 1);
          const uint64_t qd = qd0 + (both ? uint64_t((i * C::Q) >> 4) : 0);
          int of_item = 0;   // tiles of this item that this stream has taken
          // another stream's tile: this one's share of its release
          auto pass = [&] {
            ok = wait(bars.k_full[t % C::NK], (t / C::NK) & 1);
            if (ok) mbar_arrive(smem_u32(&bars.k_empty[t % C::NK]));
            ok = ok && wait(bars.v_full[t & 1], (t >> 1) & 1);
            if (ok) mbar_arrive(smem_u32(&bars.v_empty[t & 1]));
          };
          // a tile, once its K is there; `next`: the next tile is this stream's too
          auto take = [&](bool last, bool next) {
            const int st = t & 1, ph = (t >> 1) & 1, ks = t % C::NK;
            // S and P share columns, and the softmax rescales O after S is
            // full: the previous O += P V completes first
            if (ok && mine >= 1) ok = wait(bars.pv_done[i], (mine - 1) & 1);
            if (!ok) return;
            tc_fence_after();
            const uint64_t kd = kd0 + uint64_t((ks * C::CODES) >> 4);
#pragma unroll
            for (int tm = 0; tm < C::TERMS; ++tm)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                const int b = k * 32 / 128, o = k * 32 % 128;
                tc_mma_f8_ss(s_col, qd + uint64_t((tm * C::QT + b * C::M * 128 + o) >> 4),
                             kd + uint64_t((b * C::N * 128 + o) >> 4), C::IDESC_QK,
                             (tm > 0 || k > 0) ? 1u : 0u);
              }
            tc_commit(smem_u32(&bars.s_full[i]));
            tc_commit(smem_u32(&bars.k_empty[ks]));
            if (last) tc_commit(smem_u32(&bars.q_empty));
            // (the next K and this V are waited for while the softmax runs)
            if (next) ok = wait(bars.k_full[(t + 1) % C::NK], ((t + 1) / C::NK) & 1);
            if (ok) ok = wait(bars.v_full[st], ph);
            if (ok) ok = wait(bars.p_full[i], mine & 1);
            if (!ok) return;
            tc_fence_after();
            const uint64_t vd = vd0 + uint64_t((st * C::V) >> 4);
#pragma unroll
            for (int k = 0; k < C::N / 16; ++k)
              tc_mma_ts(o_col, s_col + k * 8, vd + uint64_t((k * 16 * 128) >> 4), C::IDESC_PV,
                        (of_item > 0 || k > 0) ? 1u : 0u);
            tc_commit(smem_u32(&bars.v_empty[st]));
            tc_commit(smem_u32(&bars.pv_done[i]));
            ++mine;
            ++of_item;
          };
          if (both || (!SOLO && i == 0)) {
            if (nt > 0) ok = ok && wait(bars.k_full[t % C::NK], (t / C::NK) & 1);
            for (int j = 0; ok && j < nt; ++j, ++t) take(j == nt - 1, j + 1 < nt);
          } else if (!SOLO) {
            for (int j = 0; ok && j < nt; ++j, ++t) pass();
            if (ok && nt > 0) mbar_arrive(smem_u32(&bars.q_empty));
          } else {
            for (int j = 0; ok && j < nt; ++j, ++t) {
              if ((j & 1) == i) {
                ok = wait(bars.k_full[t % C::NK], (t / C::NK) & 1);
                take(j == nt - 1, false);
              } else {
                pass();
                if (ok && j == nt - 1) mbar_arrive(smem_u32(&bars.q_empty));
              }
            }
          }
          if (!ok) break;
          if (nt == 0) tc_commit(smem_u32(&bars.q_empty));
          else if (of_item > 0) tc_commit(smem_u32(&bars.o_final[i]));
        }
        if (!ok) fail();
        // every MMA issued so far completes before the TMEM is released
        tc_commit(smem_u32(&bars.drain[i]));
        mbar_sleep_bounded(smem_u32(&bars.drain[i]), 0, limit, nullptr);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<C::SOFT_REGS>();
    // ------------------------------------------------------- softmax + epilogue
    const int half = warp >> 2;                       // which half of a row's columns
    const int t = (warp & 3) * 32 + lane;             // M row of a tile = TMEM lane
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const float scale0 = prm.sm_scale * kLog2e;
    // The two warps of 32 rows meet at a named barrier, so neither leaves an
    // item alone: after a wait that ran out (`ok` false; no wait waits any more)
    // a warp goes through the rest of its item, and the vote at the next item's
    // start ends both.
    const int pair_bar = 1 + (warp & 3);
    bool ok = true;
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      if (ok && !mbar_sleep_warp(smem_u32(&bar), parity, limit, &abort_flag)) {
        ok = false;
        abort_flag = 1;
      }
    };
    // A value of the row's other half (two buffers in turn: the next value may
    // be written while the other warp still reads this one).
    int swaps = 0;
    auto swap = [&](float mine) {
      float(*buf)[128] = pair_sh[swaps++ & 1];
      buf[half][t] = mine;
      tc_fence_before();
      named_bar_sync(pair_bar, 64);
      tc_fence_after();
      return buf[half ^ 1][t];
    };
    int gt = 0;                    // tiles of keys of earlier items
    int done0 = 0, done1 = 0;      // of which each stream took
    int outs0 = 0, outs1 = 0;      // items of which each stream took a tile
    for (int n = 0;; ++n) {
      int it = -1;
      if (ok) ok = take_item(n, it);
      ok = !named_bar_or(pair_bar, 64, !ok);
      if (!ok || it < 0) break;
      const WorkItem w = prm.items[it];
      const int nt = tiles_of(w);
      const int q_start = prm.qo_indptr[w.req], q_end = prm.qo_indptr[w.req + 1];
      const int np_req = prm.page_indptr[w.req + 1] - prm.page_indptr[w.req];
      const int kv_len = np_req > 0 ? (np_req - 1) * P + prm.last_page_len[w.req] : 0;
      const bool both = C::TILES == 1 || w.q_row + R < q_end;           // every M tile has a row
      // key position of this thread's row of tile 0 (tile 1: R rows on), and
      // the keys it may see, in columns of this thread's half
      const int row0 = w.q_row + t / g;
      const int pos0 = kv_len - (q_end - q_start) + (row0 - q_start);
      const int off = w.tok_begin + half * C::H;
      // tiles of keys that cross a bound of some row of this warp: from `last`
      // on, and with a window before `first` (a row past the request's last one
      // counts as the last one)
      const int col_row = prm.causal ? pos0 : kv_len - 1;
      const int low = __reduce_min_sync(0xffffffffu, min(col_row, kv_len - 1));
      const int high = __reduce_max_sync(0xffffffffu, pos0) + (C::TILES - 1) * R;
      const int last = low - off < C::H - 1 ? 0 : (low - off - (C::H - 1)) / C::N + 1;
      const int first = prm.window_left >= 0 ? (high - prm.window_left - off + C::N - 1) / C::N : 0;
      float unit0 = 0.f, unit1 = 0.f, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float ref = 1.f;             // r
      for (int j = 0; j < nt; ++j, ++gt) {
        wait(bars.sc_full[gt % kScaleRing], (gt / kScaleRing) & 1);
        const uint32_t lost = uint32_t(lost_sh[gt % kScaleRing]) >> (half * C::HG);
        const float4* sc = scale_sh[gt % kScaleRing] + half * C::HG;
        // (one copy of this code, for the instruction cache: unrolled over the
        // M tiles, or with a second copy for masked tiles, it was slower)
        // (the streams that have this tile, a bit each)
        const int act = both ? 3 : 1 << (j & 1);
#pragma unroll 1
        for (int i = 0; i < (SOLO || both ? C::TILES : 1); ++i) {
          if (SOLO && ((act >> i) & 1) == 0) continue;
          wait(bars.s_full[i], (i == 0 ? done0++ : done1++) & 1);
          tc_fence_after();
          float unit = i == 0 ? unit0 : unit1;
          float m = i == 0 ? m0 : m1, l = i == 0 ? l0 : l1;
          if (j == 0 || (SOLO && !both && j == 1)) {
            // (the first scores are there, so q's terms and exponents are.
            // Waiting for q_full itself here would be wrong: where items have
            // one tile of keys, q_full runs on to the next item's phase while
            // this warp is still in the previous item's epilogue)
            unit = scale0 * __uint_as_float(uint32_t(int(q_exp[n & 1][(!SOLO || both ? i * 128 : 0) + t]) - 1) << 23);
            if (i == 0) unit0 = unit;
            else unit1 = unit;
            if (j == 0) ref = scale_sh[gt % kScaleRing][0].w;
          }
          const uint32_t s_col = tmem + lane_off + C::col_s(i);
          const uint32_t o_col = tmem + lane_off + C::col_o(i) + half * (D / 2);
          const bool need_mask = j >= last || j < first || lost != 0u;
          {
            uint32_t sr[C::H / 32][32];
#pragma unroll
            for (int c = 0; c < C::H / 32; ++c) tmem_ld32(s_col + half * C::H + c * 32, sr[c]);
            tmem_wait_ld();
            if (need_mask) {
              const int pos = pos0 + (!SOLO || both ? i * R : 0), col0 = off + j * C::N;
              const int hi = min(prm.causal ? pos : kv_len - 1, kv_len - 1) - col0;
              const int lo = prm.window_left >= 0 ? max(pos - prm.window_left - col0, 0) : 0;
#pragma unroll
              for (int k = 0; k < C::H; ++k)
                if (k > hi || k < lo || ((lost >> (k >> 4)) & 1u)) sr[k >> 5][k & 31] = 0xff800000u;
            }
            // s + log2 s_v of a group's largest score; the scale is at least
            // FLT_MIN (a hidden score is -inf, and -inf * 0 would be NaN)
            float cu[C::HG], lv[C::HG];
            float m_tile = -INFINITY;
#pragma unroll
            for (int p = 0; p < C::HG; ++p) {
              const float2 s = *reinterpret_cast<const float2*>(sc + p);
              cu[p] = fmaxf(s.x * unit, FLT_MIN);
              lv[p] = s.y;
              float a = -INFINITY, b = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const int k = p * 16 + e;
                a = fmax3(a, __uint_as_float(sr[k >> 5][k & 31]),
                          __uint_as_float(sr[k >> 5][(k + 1) & 31]));
                b = fmax3(b, __uint_as_float(sr[k >> 5][(k + 2) & 31]),
                          __uint_as_float(sr[k >> 5][(k + 3) & 31]));
              }
              m_tile = fmaxf(m_tile, fmaf(fmaxf(a, b), cu[p], lv[p]));
            }
            const float m_other = swap(m_tile);
            const float m_new = fmax3(m, m_tile, m_other);
            const bool grow = m_new > m + kRescaleThreshold;
            const bool o_live = grow && m != -INFINITY;
            float alpha = 1.f;
            if (grow) {
              alpha = ex2(m - m_new);
              l *= alpha;
              m = m_new;
            }
            // O is settled: this S was issued after the previous O += P V had
            // completed. Each warp rescales half of the columns.
            if (__any_sync(0xffffffffu, o_live)) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t r[16];
                tmem_ld16(o_col + c * 16, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                tmem_st16(o_col + c * 16, r);
              }
              tmem_wait_st();
            }
            const float mm = m == -INFINITY ? 0.f : m;
            // P over S's first columns: both halves of S were read before the
            // barrier above
#pragma unroll
            for (int p = 0; p < C::HG; p += 2) {
              uint32_t wv[16];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float b = lv[p + h] - mm;
                const float2 c2 = make_float2(cu[p + h], cu[p + h]), b2 = make_float2(b, b);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const int k = (p + h) * 16 + e;
                  const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[k >> 5][k & 31]),
                                                          __uint_as_float(sr[k >> 5][(k + 1) & 31])),
                                              c2, b2);
                  const float2 y = make_float2(ex2(x.x), ex2(x.y));
                  sum = __fadd2_rn(sum, y);
                  wv[h * 8 + e / 2] = Fp16::pack2(y.x, y.y);
                }
                l = fmaf(sum.x + sum.y, sc[p + h].z, l);
              }
              tmem_st16(s_col + half * (C::H / 2) + p * 8, wv);
            }
            tmem_wait_st();
          }
          if (i == 0) {
            m0 = m;
            l0 = l;
          } else {
            m1 = m;
            l1 = l;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[i]));
        }
      }
      // ---- epilogue, half of the columns per warp (a piece of a split item
      // writes the rows' fp32 states)
      // One M tile: the streams' states are added up, with weights f0 and f1.
      float f0 = 1.f, f1 = 0.f;
      const bool merge2 = SOLO && !both && nt > 1;
      if (merge2) {
        const float m2 = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.f : ex2(m0 - m2);
        f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m2);
        l0 = l0 * f0 + l1 * f1;
        m0 = m2;
      }
#pragma unroll 1
      for (int i = 0; i < (both ? C::TILES : 1); ++i) {
        if (nt > 0) wait(bars.o_final[i], (i == 0 ? outs0++ : outs1++) & 1);
        if (merge2) wait(bars.o_final[1], outs1++ & 1);
        const float m = i == 0 ? m0 : m1, l = i == 0 ? l0 : l1;
        const float l_other = swap(l);
        const float sum = half == 0 ? l + l_other : l_other + l;
        const uint32_t o_col = tmem + lane_off + C::col_o(i) + half * (D / 2);
        const int row_in = i * R + t / g;               // query row within the item
        const int q_row = w.q_row + row_in;
        const bool row_ok = q_row < q_end;
        const float inv = sum == 0.f ? 0.f : prm.v_scale * ref / sum;
        const int head = w.head * g + t % g;
        const bool piece = w.merge > 0;
        const size_t orow =
            piece ? size_t(w.slot) + size_t(row_in) * size_t(w.merge) : size_t(q_row);
        const size_t at = orow * prm.num_qo_heads + head;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r[32];
          if (nt > 0) {
            tmem_ld32(o_col + c * 32, r);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (merge2) {
            uint32_t x[32];
            tmem_ld32(tmem + lane_off + C::col_o(C::TILES - 1) + half * (D / 2) + c * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              r[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), f1, __uint_as_float(r[e]) * f0));
          }
          const float* f = reinterpret_cast<const float*>(r);
          const size_t to = at * D + half * (D / 2) + c * 32;
          if (row_ok && piece) {
            float4* dst = reinterpret_cast<float4*>(prm.piece_o + to);
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
              dst[q4] = make_float4(f[q4 * 4] * inv, f[q4 * 4 + 1] * inv, f[q4 * 4 + 2] * inv,
                                    f[q4 * 4 + 3] * inv);
          } else if (row_ok) {
            uint4* dst =
                reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(prm.out) + to);
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const float* x = f + q4 * 8;
              dst[q4] =
                  make_uint4(E::pack2(x[0] * inv, x[1] * inv), E::pack2(x[2] * inv, x[3] * inv),
                             E::pack2(x[4] * inv, x[5] * inv), E::pack2(x[6] * inv, x[7] * inv));
            }
          }
        }
        float* lse = piece ? prm.piece_lse : prm.lse;
        if (half == 0 && row_ok && lse)
          lse[at] = sum == 0.f ? -INFINITY : (m + (lg2(sum) - lg2(ref))) * kLn2;
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // every copy that was issued lands before the CTA exits, also after a timeout
  if (warp >= C::W_KV && warp < C::W_KV + COPIERS && lane == 0) {
    const bool no_v = issued < 0;   // of the last tile
    if (no_v) issued = -issued;
    for (int j = max(0, issued - C::NK); j < issued; ++j) {
      if (!(j == 0 && prm.fault_kind == 1 && blockIdx.x == 0))   // K never issued
        mbar_sleep_bounded(smem_u32(&bars.k_full[j % C::NK]), (j / C::NK) & 1, limit, nullptr);
    }
    const int nv = no_v ? issued - 1 : issued;
    for (int j = max(0, nv - C::NVR); j < nv; ++j)
      mbar_sleep_bounded(smem_u32(&bars.vr_full[j % C::NVR]), (j / C::NVR) & 1, limit, nullptr);
  }
}

template <int D, class E, bool SOLO>
cudaError_t launch_t(const void* q, const CUtensorMap& km, const CUtensorMap& vm,
                     const PrefillParams& p, int grid, bool overlap, cudaStream_t stream) {
  using C = P8Cfg<D, E>;
  auto kern = prefill_page8_kernel<D, E, SOLO>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = once_per_device(configured, [&] {
    // the warpgroups' register split assumes this launch allocation
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, kern);
    if (r != cudaSuccess) return r;
    if (fa.numRegs != int(C::LAUNCH_REGS)) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  return launch_overlapping(kern, grid, C::THREADS, C::SMEM, overlap, stream, q, km, vm, p);
}

template <class E>
cudaError_t launch_d(int head_dim, bool solo, const void* q, const CUtensorMap& km,
                     const CUtensorMap& vm, const PrefillParams& p, int grid, bool overlap,
                     cudaStream_t stream) {
  switch (head_dim) {
    case 64: return solo ? launch_t<64, E, true>(q, km, vm, p, grid, overlap, stream)
                         : launch_t<64, E, false>(q, km, vm, p, grid, overlap, stream);
    case 128: return solo ? launch_t<128, E, true>(q, km, vm, p, grid, overlap, stream)
                          : launch_t<128, E, false>(q, km, vm, p, grid, overlap, stream);
    case 256: return launch_t<256, E, false>(q, km, vm, p, grid, overlap, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefill_page8(int head_dim, int dtype, bool solo, const void* q,
                                 const CUtensorMap& km, const CUtensorMap& vm,
                                 const PrefillParams& p, int num_sms, bool overlap,
                                 cudaStream_t stream) {
  const int grid = p.n_items < num_sms ? p.n_items : num_sms;
  if (grid <= 0) return cudaSuccess;
  switch (dtype) {
    case FI_DTYPE_BF16: return launch_d<Bf16>(head_dim, solo, q, km, vm, p, grid, overlap, stream);
    case FI_DTYPE_FP16: return launch_d<Fp16>(head_dim, solo, q, km, vm, p, grid, overlap, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fi
