// fi_append_paged_kv: new K and V rows into a paged cache, as they are or as
// E4M3 codes with a power-of-two scale per (page, kv head).
//
// Quantised: with m the largest finite |x| of the rows that a page receives,
// s' = 2^k is the smallest power of two with m <= 448 2^k: for m = 1.f 2^e
// that is k = e - 8 where 1.f <= 1.75 (448 = 1.75 2^8), else e - 7, read off
// m's bits. Codes are x 2^-k, an exact product, rounded once by the hardware
// conversion. A page that already held rows keeps the larger scale; where its
// own was smaller its codes are multiplied by old / new, again exact for
// powers of two, and rounded.
//
// Bound: bytes (4 read and 2 written per element pair) for prompts, latency
// for a decode step. A run (the rows of one page) of one kv head and of K or
// V is one warp's work, all rows loaded before the first is used: the maximum
// is known before anything is stored, each element is read once, and there is
// no reduction across warps. Blocks take 16 rows of the call; a decode step,
// where they are 16 runs, spreads each over up to 2 * num_kv_heads blocks.
//
// Measured, calls back to back: 8 prompts of 1000-4096 tokens, 8 heads of 128
// (125 MB) 25.7 us, 4.9 TB/s, 0.72 of the copy bandwidth (blocks of 8 rows 2 %
// slower, of 32 rows 11 %; what is left is a warp's chain of loads, maximum,
// conversion and stores, and the launch); 128 single tokens 12.8 us a call, of
// which the GPU is busy for 4.
#include <cuda_runtime.h>

#include <type_traits>

#include "elem.cuh"
#include "page8.cuh"
#include "ptx_page8.cuh"

namespace fi {

namespace {

using namespace dev;

constexpr int kWarps = 8;
constexpr int kRows = 16;            // rows of the call per block
constexpr int kMinExp = -100;        // the smallest scale is 2^kMinExp

// The exponent k of the smallest power of two with m <= 448 * 2^k (m >= 0, finite).
__device__ __forceinline__ int scale_exponent(float m) {
  const uint32_t u = __float_as_uint(m);
  const int k = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, kMinExp);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float(uint32_t(127 + k) << 23); }

// Eight floats -> eight E4M3 codes.
__device__ __forceinline__ uint2 codes8(const float (&f)[8]) {
  return make_uint2(E4m3::from_f32x2(f[0], f[1]) | (E4m3::from_f32x2(f[2], f[3]) << 16),
                    E4m3::from_f32x2(f[4], f[5]) | (E4m3::from_f32x2(f[6], f[7]) << 16));
}

// Registers: a run of up to 8 passes leaves room for five blocks per SM (4: 2 %
// slower, 6: 18 %, spilling).
template <int D, int P>
constexpr int min_blocks() {
  return P * D / 256 <= 8 ? 5 : P * D / 256 <= 16 ? 2 : 1;
}

// One run, one kv head, K or V: rows [t, t + n) of the call into page `page`
// from slot `first` on.
template <int D, class E, int P>
__device__ __forceinline__ void append_run(const uint16_t* src, int64_t row_stride, int first,
                                           int n, uint8_t* dst, int64_t slot_stride, float* scale,
                                           int lane) {
  constexpr int LPR = D / 8;            // lanes per row, 8 elements each
  constexpr int RPP = 32 / LPR;         // rows per pass
  constexpr int PASSES = P / RPP;       // a whole page
  constexpr int HELD = PASSES < 16 ? PASSES : 16;   // in registers; the rest is read twice
  const int row0 = lane / LPR, col = (lane % LPR) * 8;
  // pass i has row i * RPP + row0 of the run
  auto load = [&](int i) {
    const int r = i * RPP + row0;
    return r < n ? *reinterpret_cast<const uint4*>(src + r * row_stride + col)
                 : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 x[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) x[i] = load(i);
  const float old = first > 0 ? *scale : 0.f;
  // |x| of bf16 and fp16 orders as its 15 bits: the largest of all elements,
  // two at a time
  constexpr uint32_t kInf = std::is_same<E, Bf16>::value ? 0x7f80u : 0x7c00u;
  uint32_t top2 = 0u;
  auto largest = [&](const uint4& y) {
    top2 = __vmaxu2(top2, y.x & 0x7fff7fffu);
    top2 = __vmaxu2(top2, y.y & 0x7fff7fffu);
    top2 = __vmaxu2(top2, y.z & 0x7fff7fffu);
    top2 = __vmaxu2(top2, y.w & 0x7fff7fffu);
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) largest(x[i]);
  if (PASSES > HELD && n > HELD * RPP) {
#pragma unroll 4
    for (int i = HELD; i < PASSES; ++i) largest(load(i));
  }
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 >> 16, top2 & 0xffffu));
  float m = E::lo(top);
  bool odd = top >= kInf;   // a NaN, an infinity, or a scale that is no power of two
  if (odd) {                // (rare) the largest of the finite ones
    m = 0.f;
#pragma unroll 1
    for (int i = 0; i < PASSES; ++i) {
      float f[8];
      unpack8<E>(load(i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fabsf(f[e]) < INFINITY ? fmaxf(m, fabsf(f[e])) : m;
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  }
  const int k = scale_exponent(m);
  float s = pow2(k), inv = pow2(-k);
  if (first > 0) {
    if (old >= s) {
      s = old;
      inv = 1.f / old;   // exact for a power of two
      odd |= (__float_as_uint(old) & 0x7fffffu) != 0u;
    } else {
      // the older rows' codes on the larger scale
      const float ratio = old / s;
      for (int r = row0; r < first; r += RPP) {
        uint2* at = reinterpret_cast<uint2*>(dst + r * slot_stride + col);
        float f[8];
        E4m3::unpack8(*at, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= ratio;
        *at = codes8(f);
      }
    }
  }
  if (lane == 0 && !(first > 0 && s == old)) *scale = s;
  auto store = [&](int i, const uint4& y) {
    const int r = i * RPP + row0;
    if (r >= n) return;
    float f[8];
    unpack8<E>(y, f);
    if (!odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
    } else {   // (the conversion saturates infinities: make them NaN)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = fabsf(f[e]) < INFINITY ? f[e] / s : __uint_as_float(0x7fc00000u);
    }
    *reinterpret_cast<uint2*>(dst + (first + r) * slot_stride + col) = codes8(f);
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) store(i, x[i]);
  if (PASSES > HELD && n > HELD * RPP) {
#pragma unroll 4
    for (int i = HELD; i < PASSES; ++i) store(i, load(i));
  }
}

template <int D, class E, int P>
__global__ void __launch_bounds__(32 * kWarps, min_blocks<D, P>()) append_scaled_kernel(AppendParams p) {
  __shared__ int start_sh[kRows], n_sh[kRows], count_sh;
  __shared__ int64_t slot_sh[kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * kRows;
  // (the launch may start beside the one in front of it)
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    // bit i of `more`: row t0 + i continues row t0 + i - 1 within a page (64
    // rows: this block's and the longest run that can follow from its last one)
    static_assert(kRows + 32 <= 64, "");
    int64_t slot[2];
    uint64_t more = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int t = t0 + 32 * w + lane;
      slot[w] = t < p.num_tokens ? p.slot_map[t] : -1;
      int64_t before = __shfl_up_sync(0xffffffffu, slot[w], 1);
      const int64_t last = __shfl_sync(0xffffffffu, slot[0], 31);
      if (lane == 0) before = w == 1 ? last : t > 0 ? p.slot_map[t - 1] : -2;
      const bool on = slot[w] >= 0 && slot[w] % P != 0 && before + 1 == slot[w];
      more |= uint64_t(__ballot_sync(0xffffffffu, on)) << (32 * w);
    }
    const bool in = lane < kRows && slot[0] >= 0 && slot[0] < int64_t(p.num_pages) * P;
    if (lane < kRows && slot[0] >= int64_t(p.num_pages) * P) atomicOr(p.err, kErrBounds);
    const bool start = in && !((more >> lane) & 1u);
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    if (start) {
      const int at = __popc(starts & ((1u << lane) - 1u));
      start_sh[at] = t0 + lane;
      slot_sh[at] = slot[0];
      n_sh[at] = __ffsll(~(more >> (lane + 1)));   // (bits past the last one are clear)
    }
    if (lane == 0) count_sh = __popc(starts);
  }
  __syncthreads();
  const int H2 = 2 * p.num_kv_heads;
  const int tasks = count_sh * H2;
  // tasks of one run are adjacent: its heads' rows are adjacent in memory
  for (int task = blockIdx.y * kWarps + warp; task < tasks; task += gridDim.y * kWarps) {
    const int run = task / H2, hk = task - run * H2;
    const bool is_v = hk >= p.num_kv_heads;
    const int h = is_v ? hk - p.num_kv_heads : hk;
    const int t = start_sh[run], n = n_sh[run];
    const int64_t slot = slot_sh[run];
    const int64_t page = slot / P;
    const int first = int(slot - page * P);
    const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? p.v_new : p.k_new) +
                          int64_t(t) * p.token_stride + int64_t(h) * D;
    uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                   page * p.page_stride + int64_t(h) * p.head_stride;
    float* scale = (is_v ? p.v_scale : p.k_scale) + page * p.num_kv_heads + h;
    append_run<D, E, P>(src, p.token_stride, first, n, dst, p.slot_stride, scale, lane);
  }
}

// A 16-bit cache: each 16-byte piece of each row to its slot.
template <int D>
__global__ void __launch_bounds__(256) append_copy_kernel(AppendParams p) {
  constexpr int LPR = D / 8;
  pdl_trigger();
  pdl_wait();
  const int per_row = 2 * p.num_kv_heads * LPR;   // K pieces, then V pieces
  const int64_t total = int64_t(p.num_tokens) * per_row;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * 256) {
    const int t = int(i / per_row);
    int c = int(i - int64_t(t) * per_row);
    const int64_t slot = p.slot_map[t];
    if (slot < 0) continue;
    const int64_t page = slot / p.page_size;
    if (page >= p.num_pages) {
      if (c == 0) atomicOr(p.err, kErrBounds);
      continue;
    }
    const bool is_v = c >= per_row / 2;
    if (is_v) c -= per_row / 2;
    const int h = c / LPR, col = (c - h * LPR) * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(
        reinterpret_cast<const uint16_t*>(is_v ? p.v_new : p.k_new) +
        int64_t(t) * p.token_stride + int64_t(h) * D + col);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) +
                              page * p.page_stride + int64_t(h) * p.head_stride +
                              (slot - page * p.page_size) * p.slot_stride + col) = x;
  }
}

template <int D, class E>
cudaError_t launch_scaled(const AppendParams& p, cudaStream_t stream) {
  const int groups = (p.num_tokens + kRows - 1) / kRows;
  // about eight blocks for each of 152 SMs, and no more blocks per group than
  // a run has (kv head, K or V) tasks
  int y = 152 * 8 / groups;
  y = y < 1 ? 1 : (y > 2 * p.num_kv_heads ? 2 * p.num_kv_heads : y);
  return launch_overlapping(
      p.page_size == 16 ? append_scaled_kernel<D, E, 16> : append_scaled_kernel<D, E, 32>,
      dim3(groups, y), 32 * kWarps, 0, true, stream, p);
}

template <int D>
cudaError_t launch_d(int dtype, int kv_dtype, const AppendParams& p, cudaStream_t stream) {
  if (kv_dtype == FI_DTYPE_E4M3_PAGE) {
    return dtype == FI_DTYPE_BF16 ? launch_scaled<D, Bf16>(p, stream)
                                  : launch_scaled<D, Fp16>(p, stream);
  }
  const int64_t total = int64_t(p.num_tokens) * 2 * p.num_kv_heads * (D / 8);
  const int64_t blocks = (total + 255) / 256;
  return launch_overlapping(append_copy_kernel<D>,
                            dim3(unsigned(blocks < 152 * 32 ? blocks : 152 * 32)), 256, 0, true,
                            stream, p);
}

}  // namespace

cudaError_t launch_append(int head_dim, int dtype, int kv_dtype, const AppendParams& p,
                          cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_d<64>(dtype, kv_dtype, p, stream);
    case 128: return launch_d<128>(dtype, kv_dtype, p, stream);
    case 256: return launch_d<256>(dtype, kv_dtype, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fi
