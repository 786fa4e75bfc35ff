// fi_page_table_step: a serving step's page table, row offsets and slot map
// from the requests' lengths.
//
// With P tokens per page, request b holds ceil(kv_len / P) pages before the
// step and ceil((kv_len + new_len) / P) after it. Four running sums over the
// batch place everything: pages taken, pages returned, pages held, new rows.
//
// The call is bound by latency, not by bytes (256 requests of up to 8K
// tokens: 180 KB), so it is one launch: every block computes the four sums of
// the whole batch for itself (a few loads per thread, out of L2 after the
// first block) and then fills its share of the outputs, finding the request
// of an entry by bisection in the sums. Nothing that a block reads is written
// by another one: entry j of a request's row is read from the block table
// where the request had it and from the ring where it is new. Lengths and
// ring state may be updated in place: then they are written once all blocks
// have read them, after a cluster barrier where one cluster has all blocks,
// by the last block of a ticket counter (which wraps to zero) otherwise.
//
// Measured, calls back to back: 256 requests of up to 8K tokens and one new
// token each (180 KB) 7.8 us, 1536 of 2048 requests with up to 64 new tokens
// (1.3 MB) 12.2 us. Blocks of 512 threads with 2048 entries each; 1024 threads
// and 4096 entries took 10.2 and 14.3 us (a barrier waits for twice the warps),
// 256 threads 8.2 and 14.4 us.
#include <cuda_runtime.h>

#include "page8.cuh"
#include "ptx_page8.cuh"

namespace fi {

namespace {

constexpr int kThreads = 512;
constexpr int kPerBlock = 2048;   // output entries per block that the grid is sized for
constexpr int kMaxBlocks = 152;
constexpr int kCluster = 8;       // blocks of the largest portable cluster
constexpr long long kMaxLen = 0x3fffffff;   // INT32_MAX / 2 tokens, as fi_plan accepts

// Sums that stop at 2^31 - 1 (more than any capacity holds).
struct Sums {
  uint32_t take, give, has, rows;
};
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  return min(a + b, 0x7fffffffu);
}
__device__ __forceinline__ void add(Sums& a, const Sums& b) {
  a.take = sat_add(a.take, b.take);
  a.give = sat_add(a.give, b.give);
  a.has = sat_add(a.has, b.has);
  a.rows = sat_add(a.rows, b.rows);
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, a.take, d), __shfl_up_sync(0xffffffffu, a.give, d),
              __shfl_up_sync(0xffffffffu, a.has, d), __shfl_up_sync(0xffffffffu, a.rows, d)};
}
// Inclusive sums over a warp.
__device__ __forceinline__ Sums warp_scan(Sums a, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(a, d);
    if (lane >= d) add(a, o);
  }
  return a;
}

// The rows whose ranges of `ends` (non-decreasing inclusive sums) hold the
// items i[c], i[c] < ends[n - 1]: the number of sums at or below each, by
// bisection, C searches side by side. `first` is the largest power of two <= n.
template <int C>
__device__ __forceinline__ void owners(const int32_t* ends, int n, int first, const int32_t (&i)[C],
                                       int (&r)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) r[c] = 0;
  for (int s = first; s > 0; s >>= 1) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (r[c] + s <= n && ends[r[c] + s - 1] <= i[c]) r[c] += s;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) r[c] = min(r[c], n - 1);   // (items behind the last one)
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads) page_step_kernel(PageStepParams p) {
  extern __shared__ int32_t sh[];
  // per request: inclusive sums, slot, length before; and the slots met so far
  // (a bit each)
  int32_t* take_end = sh;
  int32_t* give_end = take_end + p.batch;
  int32_t* has_end = give_end + p.batch;
  int32_t* row_end = has_end + p.batch;
  int32_t* slot_sh = row_end + p.batch;
  int32_t* old_sh = slot_sh + p.batch;
  uint32_t* met = reinterpret_cast<uint32_t*>(old_sh + p.batch);
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ uint32_t err_sh;
  __shared__ int last_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.page_size;
  // consecutive requests per thread; the first one's loads go out at once
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  // (the launch may start beside the one in front of it)
  dev::pdl_trigger();
  for (int i = tid; i < (p.max_requests + 31) / 32; i += kThreads) met[i] = 0u;
  if (tid == 0) err_sh = 0u;
  dev::pdl_wait();
  const int head = p.ring_state[0], count = p.ring_state[1], cap = p.ring_capacity;
  __syncthreads();

  uint32_t err = 0u;
  if (head < 0 || head >= cap || count < 0 || count > cap) err |= kErrBounds;
  // what a request takes, returns, has and adds, from its slot and length
  auto sums_of = [&](int slot, int old, int add_len) {
    Sums s = {0u, 0u, 0u, 0u};
    if (slot >= 0) {
      const int had = (old + P - 1) / P, has = (old + add_len + P - 1) / P;
      s.take = uint32_t(max(has - had, 0));
      s.give = uint32_t(max(had - has, 0));
      s.has = uint32_t(has);
      s.rows = uint32_t(max(add_len, 0));
    }
    return s;
  };
  Sums mine = {0u, 0u, 0u, 0u};
  for (int b = b0; b < b1; ++b) {
    int slot = p.slots ? p.slots[b] : b;
    const int add_len = p.new_len[b];
    int old = 0;
    if (slot >= p.max_requests) {
      err |= kErrBounds;
      slot = -1;
    } else if (slot >= 0) {
      const uint32_t bit = 1u << (slot & 31);
      if (atomicOr(&met[slot >> 5], bit) & bit) err |= kErrBounds;
      old = p.kv_len[slot];
      const long long len = (long long)old + add_len, most = (long long)p.max_pages * P;
      if (old < 0 || old > most || old > kMaxLen || len < 0 || len > kMaxLen) err |= kErrBounds;
      else if (len > most) err |= kErrPages;
    }
    slot_sh[b] = slot;
    old_sh[b] = old;
    if (!err) add(mine, sums_of(slot, old, add_len));
  }
  const Sums upto = warp_scan(mine, lane);
  if (lane == 31) warp_sums[warp] = upto;
  if (err) atomicOr(&err_sh, err);
  __syncthreads();
  // the warps' sums: lane w has those of warps 0..w
  constexpr int kWarps = kThreads / 32;
  const Sums warps =
      warp_scan(kWarps == 32 || lane < kWarps ? warp_sums[lane % kWarps] : Sums{0u, 0u, 0u, 0u}, lane);
  auto of_lane = [&](int w) {
    return Sums{__shfl_sync(0xffffffffu, warps.take, w), __shfl_sync(0xffffffffu, warps.give, w),
                __shfl_sync(0xffffffffu, warps.has, w), __shfl_sync(0xffffffffu, warps.rows, w)};
  };
  const Sums total = of_lane(31);
  Sums at = of_lane(warp > 0 ? warp - 1 : 0);
  if (warp == 0) at = Sums{0u, 0u, 0u, 0u};
  const Sums before = shfl_up(upto, 1);
  if (lane > 0) add(at, before);
  err = err_sh;
  if (!err && (total.take > uint32_t(count) || total.has > uint32_t(p.page_capacity) ||
               total.rows > uint32_t(p.token_capacity)))
    err |= kErrPages;
  if (!err && (long long)count + total.give > cap) err |= kErrBounds;
  const bool ok = err == 0u;   // the same in every thread of every block
  if (blockIdx.x == 0 && tid == 0 && !ok) atomicOr(p.err, err);

  for (int b = b0; b < b1; ++b) {
    const int slot = slot_sh[b], old = old_sh[b];
    const int add_len = slot >= 0 ? p.new_len[b] : 0;
    if (ok) {
      add(at, sums_of(slot, old, add_len));
      take_end[b] = int32_t(at.take);
      give_end[b] = int32_t(at.give);
      has_end[b] = int32_t(at.has);
      row_end[b] = int32_t(at.rows);
    }
    if (blockIdx.x == 0) {
      const int len = ok ? old + add_len : 0;
      p.page_indptr[b + 1] = ok ? int32_t(at.has) : 0;
      p.qo_indptr[b + 1] = ok ? int32_t(at.rows) : 0;
      p.last_page_len[b] = len > 0 ? (len - 1) % P + 1 : 0;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.page_indptr[0] = 0;
    p.qo_indptr[0] = 0;
  }
  __syncthreads();

  // entry head + i of the ring, i <= cap
  auto ring_at = [&](uint32_t i) {
    const uint32_t x = uint32_t(head) + i;
    return p.free_ring + (x >= uint32_t(cap) ? x - uint32_t(cap) : x);
  };
  auto row_of = [&](int slot) { return p.block_table + (long long)slot * p.max_pages; };
  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  const int n_rows = ok ? int(total.rows) : 0;
  const int first = 1 << (31 - __clz(p.batch));
  if (ok) {
    constexpr int C = 4;
    for (int i0 = gtid; i0 < int(total.has); i0 += C * gsize) {
      int32_t i[C];
      int r[C], page[C];
      int32_t* entry[C];
      bool fresh[C];
#pragma unroll
      for (int c = 0; c < C; ++c) i[c] = i0 + c * gsize;
      owners(has_end, p.batch, first, i, r);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = i[c] - (r[c] > 0 ? has_end[r[c] - 1] : 0);
        const int had = (old_sh[r[c]] + P - 1) / P;
        entry[c] = row_of(slot_sh[r[c]]) + j;
        fresh[c] = j >= had;
        page[c] = -1;
        if (i[c] < int(total.has))
          page[c] = fresh[c] ? *ring_at(uint32_t((r[c] > 0 ? take_end[r[c] - 1] : 0) + j - had))
                             : *entry[c];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (i[c] >= int(total.has)) continue;
        if (fresh[c]) *entry[c] = page[c];
        p.page_indices[i[c]] = page[c];
      }
    }
    for (int i0 = gtid; i0 < int(total.give); i0 += gsize) {
      const int32_t i[1] = {i0};
      int r[1];
      owners(give_end, p.batch, first, i, r);
      const int x = r[0];
      const int has = has_end[x] - (x > 0 ? has_end[x - 1] : 0);
      const int j = has + i0 - (x > 0 ? give_end[x - 1] : 0);
      *ring_at(uint32_t(count) + uint32_t(i0)) = row_of(slot_sh[x])[j];
    }
  }
  {
    constexpr int C = 2;
    for (int t0 = gtid; t0 < p.token_capacity; t0 += C * gsize) {
      int32_t t[C];
      int r[C], pos[C];
      long long where[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        t[c] = t0 + c * gsize;
        pos[c] = 0;
        where[c] = -1;
      }
      if (t0 < n_rows) {
        owners(row_end, p.batch, first, t, r);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (t[c] >= n_rows) continue;
          const int x = r[c];
          pos[c] = old_sh[x] + t[c] - (x > 0 ? row_end[x - 1] : 0);
          const int j = pos[c] / P, had = (old_sh[x] + P - 1) / P;
          const int page = j < had ? row_of(slot_sh[x])[j]
                                   : *ring_at(uint32_t((x > 0 ? take_end[x - 1] : 0) + j - had));
          where[c] = (long long)page * P + pos[c] % P;
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t[c] >= p.token_capacity) continue;
        p.slot_map[t[c]] = where[c];
        if (p.positions) p.positions[t[c]] = pos[c];
      }
    }
  }

  // every block has read the old lengths and ring state: now the new ones
  bool writes;
  if (CLUSTER) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
    writes = blockIdx.x == 0;
  } else {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      last_sh = atomicInc(p.ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    writes = last_sh != 0;
  }
  if (!writes) return;
  for (int b = b0; b < b1; ++b) {
    const int slot = slot_sh[b];
    if (slot >= 0) p.kv_len_out[slot] = old_sh[b] + (ok ? p.new_len[b] : 0);
  }
  if (tid == 0) {
    const uint32_t next = uint32_t(head) + total.take;
    p.ring_state_out[0] = ok ? int32_t(next >= uint32_t(cap) ? next - uint32_t(cap) : next) : head;
    p.ring_state_out[1] = ok ? int32_t(count - int(total.take) + int(total.give)) : count;
  }
}

template <bool CLUSTER>
cudaError_t launch(const PageStepParams& p, int grid, size_t smem, cudaStream_t stream) {
  auto kern = page_step_kernel<CLUSTER>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = once_per_device(configured, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kStepMaxBatch * 24 + kStepMaxRequests / 8);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(grid);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_page_step(const PageStepParams& p, cudaStream_t stream) {
  const size_t smem = size_t(p.batch) * 24 + size_t((p.max_requests + 31) / 32) * 4;
  const long long entries = (long long)p.page_capacity + p.token_capacity;
  long long grid = (entries + kPerBlock - 1) / kPerBlock;
  grid = grid < 1 ? 1 : (grid > kMaxBlocks ? kMaxBlocks : grid);
  return grid <= kCluster ? launch<true>(p, int(grid), smem, stream)
                          : launch<false>(p, int(grid), smem, stream);
}

}  // namespace fi
