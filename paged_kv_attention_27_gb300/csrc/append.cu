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
#include <cuda_runtime.h>

#include "elem.cuh"
#include "kernels.cuh"

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

// Whether row t begins a run: it does not continue row t - 1 within a page.
__device__ __forceinline__ bool run_start(const int64_t* slots, int t, int P) {
  const int64_t s = slots[t];
  return s >= 0 && (t == 0 || s % P == 0 || slots[t - 1] + 1 != s);
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
  const int row0 = lane / LPR, col = (lane % LPR) * 8;
  // pass i holds row i * RPP + row0 of the run
  uint4 x[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RPP + row0;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < n) x[i] = *reinterpret_cast<const uint4*>(src + r * row_stride + col);
  }
  const float old = first > 0 ? *scale : 0.f;
  float m = 0.f;
  bool odd = false;   // a NaN, an infinity, or a scale that is no power of two
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float f[8];
    unpack8<E>(x[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(f[e]);
      const bool fine = a < INFINITY;
      odd |= !fine;
      m = fine ? fmaxf(m, a) : m;
    }
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
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
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RPP + row0;
    if (r >= n) continue;
    float f[8];
    unpack8<E>(x[i], f);
    if (!odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
    } else {   // (the conversion saturates infinities: make them NaN)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = fabsf(f[e]) < INFINITY ? f[e] / s : __uint_as_float(0x7fc00000u);
    }
    *reinterpret_cast<uint2*>(dst + (first + r) * slot_stride + col) = codes8(f);
  }
}

template <int D, class E, int P>
__global__ void __launch_bounds__(32 * kWarps) append_scaled_kernel(AppendParams p) {
  __shared__ int start_sh[kRows], n_sh[kRows], count_sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * kRows;
  if (warp == 0) {
    const int t = t0 + lane;
    const bool in = lane < kRows && t < p.num_tokens;
    const int64_t slot = in ? p.slot_map[t] : -1;
    bool start = in && run_start(p.slot_map, t, P);
    if (in && slot >= int64_t(p.num_pages) * P) {
      atomicOr(p.err, kErrBounds);
      start = false;
    }
    int n = 0;
    if (start) {
      const int most = min(P - int(slot % P), p.num_tokens - t);
      n = 1;
      while (n < most && p.slot_map[t + n] == slot + n) ++n;
    }
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    if (start) {
      const int at = __popc(starts & ((1u << lane) - 1u));
      start_sh[at] = t;
      n_sh[at] = n;
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
    const int64_t slot = p.slot_map[t];
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
void launch_scaled(const AppendParams& p, cudaStream_t stream) {
  const int groups = (p.num_tokens + kRows - 1) / kRows;
  // about eight blocks for each of 152 SMs, and no more blocks per group than
  // a run has (kv head, K or V) tasks
  int y = 152 * 8 / groups;
  y = y < 1 ? 1 : (y > 2 * p.num_kv_heads ? 2 * p.num_kv_heads : y);
  const dim3 grid(groups, y);
  if (p.page_size == 16) append_scaled_kernel<D, E, 16><<<grid, 32 * kWarps, 0, stream>>>(p);
  else append_scaled_kernel<D, E, 32><<<grid, 32 * kWarps, 0, stream>>>(p);
}

template <int D>
void launch_d(int dtype, int kv_dtype, const AppendParams& p, cudaStream_t stream) {
  if (kv_dtype == FI_DTYPE_E4M3_PAGE) {
    if (dtype == FI_DTYPE_BF16) launch_scaled<D, Bf16>(p, stream);
    else launch_scaled<D, Fp16>(p, stream);
    return;
  }
  const int64_t total = int64_t(p.num_tokens) * 2 * p.num_kv_heads * (D / 8);
  const int64_t blocks = (total + 255) / 256;
  append_copy_kernel<D><<<int(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_append(int head_dim, int dtype, int kv_dtype, const AppendParams& p,
                          cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  switch (head_dim) {
    case 64: launch_d<64>(dtype, kv_dtype, p, stream); break;
    case 128: launch_d<128>(dtype, kv_dtype, p, stream); break;
    case 256: launch_d<256>(dtype, kv_dtype, p, stream); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace fi
