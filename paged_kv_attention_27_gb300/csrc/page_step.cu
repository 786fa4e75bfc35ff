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
// ring state may be updated in place; the block that finishes last (a ticket
// counter that wraps to zero) writes them.
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace fi {

namespace {

constexpr int kThreads = 1024;
constexpr int kPerBlock = 4096;   // output entries per block that the grid is sized for
constexpr int kMaxBlocks = 152;
constexpr long long kMaxLen = 0x3fffffff;   // INT32_MAX / 2 tokens, as fi_plan accepts

struct Sums {
  long long take, give, has, rows;
};

__device__ __forceinline__ long long shfl_up_ll(long long v, int d) {
  return __shfl_up_sync(0xffffffffu, v, d);
}

// The row whose range of `ends` (non-decreasing inclusive sums) holds item i,
// i < ends[n - 1].
__device__ __forceinline__ int owner(const int32_t* ends, int n, int32_t i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_step_kernel(PageStepParams p) {
  extern __shared__ int32_t sh[];
  // inclusive sums per request, and the slots met so far (a bit each)
  int32_t* take_end = sh;
  int32_t* give_end = take_end + p.batch;
  int32_t* has_end = give_end + p.batch;
  int32_t* row_end = has_end + p.batch;
  uint32_t* met = reinterpret_cast<uint32_t*>(row_end + p.batch);
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ uint32_t err_sh;
  __shared__ int last_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.page_size;

  for (int i = tid; i < (p.max_requests + 31) / 32; i += kThreads) met[i] = 0u;
  if (tid == 0) err_sh = 0u;
  __syncthreads();

  const int head = p.ring_state[0], count = p.ring_state[1], cap = p.ring_capacity;
  uint32_t err = 0u;
  if (head < 0 || head >= cap || count < 0 || count > cap) err |= kErrBounds;
  auto slot_of = [&](int b) { return p.slots ? p.slots[b] : b; };
  // consecutive requests per thread
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  Sums mine = {0, 0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int slot = slot_of(b);
    int had = 0, has = 0, rows = 0;
    if (slot >= p.max_requests) {
      err |= kErrBounds;
    } else if (slot >= 0) {
      if (atomicOr(&met[slot >> 5], 1u << (slot & 31)) & (1u << (slot & 31))) err |= kErrBounds;
      const long long old = p.kv_len[slot], add = p.new_len[b], len = old + add;
      const long long most = (long long)p.max_pages * P;
      if (old < 0 || old > most || old > kMaxLen || len < 0 || len > kMaxLen) err |= kErrBounds;
      else if (len > most) err |= kErrPages;
      else {
        had = int((old + P - 1) / P);
        has = int((len + P - 1) / P);
        rows = int(add > 0 ? add : 0);
      }
    }
    mine.take += max(has - had, 0);
    mine.give += max(had - has, 0);
    mine.has += has;
    mine.rows += rows;
  }
  // exclusive sums over the block's threads
  Sums upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = {shfl_up_ll(upto.take, d), shfl_up_ll(upto.give, d), shfl_up_ll(upto.has, d),
                    shfl_up_ll(upto.rows, d)};
    if (lane >= d) {
      upto.take += o.take;
      upto.give += o.give;
      upto.has += o.has;
      upto.rows += o.rows;
    }
  }
  if (lane == 31) warp_sums[warp] = upto;
  if (err) atomicOr(&err_sh, err);
  __syncthreads();
  Sums total = {0, 0, 0, 0}, base = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) base = total;
    const Sums o = warp_sums[w];
    total.take += o.take;
    total.give += o.give;
    total.has += o.has;
    total.rows += o.rows;
  }
  err = err_sh;
  if (total.take > count || total.has > p.page_capacity || total.rows > p.token_capacity)
    err |= kErrPages;
  if (count - total.take + total.give > cap || count + total.give > cap) err |= kErrBounds;
  const bool ok = err == 0u;   // the same in every thread of every block
  if (blockIdx.x == 0 && tid == 0 && !ok) atomicOr(p.err, err);

  // entry head + i of the ring, i <= cap
  auto ring_at = [&](uint32_t i) {
    const uint32_t at = uint32_t(head) + i;
    return p.free_ring + (at >= uint32_t(cap) ? at - uint32_t(cap) : at);
  };

  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  {
    long long take = base.take + upto.take - mine.take, give = base.give + upto.give - mine.give;
    long long has_at = base.has + upto.has - mine.has, row_at = base.rows + upto.rows - mine.rows;
    for (int b = b0; b < b1; ++b) {
      const int slot = slot_of(b);
      int had = 0, has = 0, rows = 0, len = 0;
      if (ok && slot >= 0) {
        const int old = p.kv_len[slot], add = p.new_len[b];
        len = old + add;
        had = (old + P - 1) / P;
        has = (len + P - 1) / P;
        rows = max(add, 0);
      }
      take += max(has - had, 0);
      give += max(had - has, 0);
      has_at += has;
      row_at += rows;
      if (ok) {
        take_end[b] = int32_t(take);
        give_end[b] = int32_t(give);
        has_end[b] = int32_t(has_at);
        row_end[b] = int32_t(row_at);
      }
      if (blockIdx.x == 0) {
        p.page_indptr[b + 1] = ok ? int32_t(has_at) : 0;
        p.qo_indptr[b + 1] = ok ? int32_t(row_at) : 0;
        p.last_page_len[b] = len > 0 ? (len - 1) % P + 1 : 0;
      }
    }
    if (blockIdx.x == 0 && tid == 0) {
      p.page_indptr[0] = 0;
      p.qo_indptr[0] = 0;
    }
  }
  __syncthreads();

  const int n_rows = ok ? int(total.rows) : 0;
  if (ok) {
    for (int i = gtid; i < int(total.has); i += gsize) {
      const int r = owner(has_end, p.batch, i);
      const int slot = slot_of(r);
      const int j = i - (r > 0 ? has_end[r - 1] : 0);
      const int had = (p.kv_len[slot] + P - 1) / P;
      int32_t* entry = p.block_table + (long long)slot * p.max_pages + j;
      int page;
      if (j < had) {
        page = *entry;
      } else {
        page = *ring_at(uint32_t((r > 0 ? take_end[r - 1] : 0) + j - had));
        *entry = page;
      }
      p.page_indices[i] = page;
    }
    for (int i = gtid; i < int(total.give); i += gsize) {
      const int r = owner(give_end, p.batch, i);
      const int slot = slot_of(r);
      const int has = has_end[r] - (r > 0 ? has_end[r - 1] : 0);
      const int j = has + i - (r > 0 ? give_end[r - 1] : 0);
      *ring_at(uint32_t(count) + uint32_t(i)) =
          p.block_table[(long long)slot * p.max_pages + j];
    }
  }
  for (int t = gtid; t < p.token_capacity; t += gsize) {
    long long where = -1;
    int pos = 0;
    if (t < n_rows) {
      const int r = owner(row_end, p.batch, t);
      const int slot = slot_of(r), old = p.kv_len[slot];
      pos = old + t - (r > 0 ? row_end[r - 1] : 0);
      const int j = pos / P, had = (old + P - 1) / P;
      const int page = j < had ? p.block_table[(long long)slot * p.max_pages + j]
                               : *ring_at(uint32_t((r > 0 ? take_end[r - 1] : 0) + j - had));
      where = (long long)page * P + pos % P;
    }
    p.slot_map[t] = where;
    if (p.positions) p.positions[t] = pos;
  }

  // every block has read the old lengths and ring state: the last one to get
  // here writes the new ones
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last_sh = gridDim.x == 1 || atomicInc(p.ticket, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last_sh) return;
  for (int b = b0; b < b1; ++b) {
    const int slot = slot_of(b);
    if (slot >= 0 && slot < p.max_requests)
      p.kv_len_out[slot] = p.kv_len[slot] + (ok ? p.new_len[b] : 0);
  }
  if (tid == 0) {
    p.ring_state_out[0] = ok ? int32_t((head + total.take) % cap) : head;
    p.ring_state_out[1] = ok ? int32_t(count - total.take + total.give) : count;
  }
}

}  // namespace

cudaError_t launch_page_step(const PageStepParams& p, cudaStream_t stream) {
  const size_t smem = size_t(p.batch) * 16 + size_t((p.max_requests + 31) / 32) * 4;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(page_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kStepMaxBatch * 16 + kStepMaxRequests / 8);
  });
  if (e != cudaSuccess) return e;
  const long long entries = (long long)p.page_capacity + p.token_capacity;
  long long grid = (entries + kPerBlock - 1) / kPerBlock;
  grid = grid < 1 ? 1 : (grid > kMaxBlocks ? kMaxBlocks : grid);
  page_step_kernel<<<int(grid), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fi
