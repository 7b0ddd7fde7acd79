// Checks of arguments, their messages and the plan as the kernels take it, shared by the C ABI of
// the operators around the layer pass and of the training step.
#pragma once

#include <math.h>
#include <stdint.h>

#include "block_kernels.h"
#include "moe_layer.h"

namespace moe_checks {

constexpr int kMaxExperts = 256;

template <class... A>
moe_status fail(moe_status s, const char* fmt, A... a) {
  return (moe_status)moe::set_last_error(s, fmt, a...);
}

inline moe_status ok() { return (moe_status)moe::set_last_error(MOE_OK, "%s", ""); }

inline moe_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// p is there and a multiple of `a` (a power of two); optional: may be NULL
inline bool good(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }
inline bool optional(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool valid_dtype(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

// H elements of either type are whole 16-byte vectors; the kernels count a
// token tensor's pieces of 256 elements, and a row's last one, in 32 bits
inline moe_status check_rows(const char* what, int64_t T, int H) {
  if (T < 0) return fail(MOE_EINVAL, "%s: T = %lld < 0", what, (long long)T);
  if (T >= (int64_t)1 << 31) return fail(MOE_EUNSUPPORTED, "%s: T must be < 2^31", what);
  if (H < 8 || H % 8 != 0)
    return fail(MOE_EUNSUPPORTED, "%s: H = %d must be a positive multiple of 8", what, H);
  if (T * H >= (int64_t)1 << 39) return fail(MOE_EUNSUPPORTED, "%s: T*H must be < 2^39", what);
  return MOE_OK;
}

inline moe_status check_routing(const char* what, int64_t T, int E, int K) {
  if (T < 0) return fail(MOE_EINVAL, "%s: T = %lld < 0", what, (long long)T);
  if (E < 1 || K < 1 || K > E)
    return fail(MOE_EINVAL, "%s: need 1 <= K <= E (K = %d, E = %d)", what, K, E);
  if (E > kMaxExperts) return fail(MOE_EUNSUPPORTED, "%s: E = %d > %d", what, E, kMaxExperts);
  if (T >= (int64_t)1 << 31 || T * K >= (int64_t)1 << 31)
    return fail(MOE_EUNSUPPORTED, "%s: T*K must be < 2^31", what);
  return MOE_OK;
}

// The plan says nothing of its padding scheme: cap is at least what one of the
// two needs (the kernels check every row index against cap).
inline moe_status check_plan(const char* what, const moe_plan* plan, int64_t T, int K, int E) {
  if (!plan) return fail(MOE_EINVAL, "%s: plan is NULL", what);
  if (plan->block_m < 1 || plan->block_m > 1024)
    return fail(MOE_EUNSUPPORTED, "%s: block_m = %d outside 1..1024", what, plan->block_m);
  const int32_t* arrs[5] = {plan->expert_counts, plan->expert_offsets, plan->sorted_ids,
                            plan->block_expert, plan->inv_pos};
  const char* names[5] = {"expert_counts", "expert_offsets", "sorted_ids", "block_expert",
                          "inv_pos"};
  for (int i = 0; i < 5; ++i)
    if (!good(arrs[i], 4))
      return fail(MOE_EINVAL, "%s: plan->%s is NULL or misaligned", what, names[i]);
  if (plan->cap % plan->block_m != 0)
    return fail(MOE_EINVAL, "%s: plan->cap = %lld is not a multiple of block_m = %d", what,
                (long long)plan->cap, plan->block_m);
  const int64_t a = moe_align_capacity_ex(T, K, E, plan->block_m, MOE_PAD_BLOCK);
  const int64_t b = moe_align_capacity_ex(T, K, E, plan->block_m, MOE_PAD_MAX);
  const int64_t need = a < b ? a : b;
  if (plan->cap < need)
    return fail(MOE_ECAPACITY, "%s: plan->cap = %lld < %lld required", what, (long long)plan->cap,
                (long long)need);
  if (plan->cap >= (int64_t)1 << 31)
    return fail(MOE_EUNSUPPORTED, "%s: plan->cap must be < 2^31", what);
  return MOE_OK;
}

inline moe_status null_pointer(const char* what) {
  return fail(MOE_EINVAL, "%s: NULL or misaligned pointer", what);
}

inline moe::RowMap plan_rows(const moe_plan* plan, int K) {
  moe::RowMap rm{};
  rm.counts = plan->expert_counts;
  rm.offsets = plan->expert_offsets;
  rm.sorted_ids = plan->sorted_ids;
  rm.block_expert = plan->block_expert;
  rm.inv_pos = plan->inv_pos;
  rm.K = K;
  rm.block_m = plan->block_m;
  rm.min_rows = 1;
  rm.max_rows = INT32_MAX;
  return rm;
}

}  // namespace moe_checks
