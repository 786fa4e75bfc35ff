// Launches of the kernels over a page-scaled FP8 cache and of the calls that
// prepare a step.
#pragma once
#include <type_traits>

#include "kernels.cuh"
#include "page8.h"

namespace fi {

// Over a page-scaled FP8 cache (decode_page8.cu, prefill_page8.cu); the
// params' k_head_scale / v_head_scale are then [num_pages][num_kv_heads].
// overlap: the launch may start beside the one in front of it (the copy of its
// work list), for which the kernels wait after their set-up.
cudaError_t launch_decode_page8(int head_dim, int group, int dtype, const CUtensorMap& km,
                                const CUtensorMap& vm, const DecodeParams& p, int n_items,
                                int num_sms, bool overlap, cudaStream_t stream);
// solo: items whose rows fill one of the two M tiles share it between both
// streams (PlanHandle::prefill_solo)
cudaError_t launch_prefill_page8(int head_dim, int dtype, bool solo, const void* q,
                                 const CUtensorMap& km, const CUtensorMap& vm,
                                 const PrefillParams& p, int num_sms, bool overlap,
                                 cudaStream_t stream);

// launch_merge behind the page-scaled prefill kernel.
cudaError_t launch_merge_page8(const MergeParams& p, int n_rows, bool overlap, cudaStream_t stream);

template <class... Args>
cudaError_t launch_overlapping(void (*kern)(Args...), dim3 grid, int threads, size_t smem,
                               bool overlap, cudaStream_t stream,
                               const std::common_type_t<Args>&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The work-list image of a page-scaled plan goes up by a kernel (merge.cu):
// a small one as its parameter, a larger one read from pinned host memory.
// `bytes` is a multiple of 16.
constexpr size_t kImageParamBytes = 3840;
struct ImageParam {
  uint32_t words[kImageParamBytes / 4];
};
cudaError_t launch_image(const ImageParam& image, size_t bytes, void* dst, cudaStream_t stream);
cudaError_t launch_image_copy(const void* src, size_t bytes, void* dst, cudaStream_t stream);

// fi_page_table_step (page_step.cu): the arguments of the call, and the step
// workspace's error word and ticket.
struct PageStepParams {
  int32_t batch;
  const int32_t* slots;
  const int32_t* new_len;
  int32_t max_requests;
  int32_t max_pages;
  int32_t page_size;
  const int32_t* kv_len;
  int32_t* kv_len_out;
  int32_t* block_table;
  int32_t* free_ring;
  int32_t ring_capacity;
  const int32_t* ring_state;
  int32_t* ring_state_out;
  int32_t* page_indptr;
  int32_t* page_indices;
  int32_t page_capacity;
  int32_t* last_page_len;
  int32_t* qo_indptr;
  int64_t* slot_map;
  int32_t* positions;
  int32_t token_capacity;
  uint32_t* err;
  uint32_t* ticket;
};
cudaError_t launch_page_step(const PageStepParams& p, cudaStream_t stream);

// fi_append_paged_kv (append.cu). Strides in elements: of a token row of k/v,
// and of the cache's pages, slots and kv heads.
struct AppendParams {
  int32_t num_tokens;
  const int64_t* slot_map;
  const void* k_new;
  const void* v_new;
  int64_t token_stride;
  int32_t num_kv_heads;
  void* k_cache;
  void* v_cache;
  int64_t page_stride, slot_stride, head_stride;
  int32_t num_pages;
  int32_t page_size;
  float* k_scale;
  float* v_scale;
  uint32_t* err;
};
// kv_dtype: dtype (the rows are copied) or FI_DTYPE_E4M3_PAGE
cudaError_t launch_append(int head_dim, int dtype, int kv_dtype, const AppendParams& p,
                          cudaStream_t stream);

}  // namespace fi
