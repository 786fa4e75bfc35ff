// Sizes, limits and plan data of the page-scaled FP8 cache and of the calls
// that prepare a step (plain C++: the planner includes it).
#pragma once
#include "fi_internal.h"

namespace fi {

// A further bit of the error word: fi_page_table_step ran out of pages.
constexpr uint32_t kErrPages = 4u;

// Step workspace (fi_page_table_step, fi_append_paged_kv): the error word, and
// the ticket counter of fi_page_table_step's blocks at this offset.
constexpr size_t kStepTicketOffset = 64;
constexpr int32_t kStepMaxBatch = 8192;
constexpr int32_t kStepMaxRequests = 262144;
constexpr int32_t kStepMaxPageSize = 1024;
constexpr int32_t kStepMaxEntries = 1 << 30;   // of the ring, page_indices, slot_map

// The kernels over a page-scaled FP8 cache: tokens per tile of the decode
// kernel; M rows (query rows x the g heads of a kv head) of a prefill item.
constexpr int kPage8DecodeTile = 128;
inline int page8_decode_ctas(int head_dim) { return head_dim <= 128 ? 2 : 1; }   // per SM
inline int page8_prefill_rows(int head_dim) { return head_dim <= 128 ? 256 : 128; }

// Whether much of a page-scaled prefill plan's work is in items whose rows fill
// one of the kernel's two M tiles (plan.cpp).
bool page8_prefill_solo(const Plan& p, const int32_t* qo_indptr);

// What fi_plan allocates.
struct PlanHandle : fi_plan_s {
  bool prefill_solo = false;
};

}  // namespace fi
