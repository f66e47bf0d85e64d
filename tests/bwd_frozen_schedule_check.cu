// Host-only check of the backward's unit schedule without dW (a frozen head), run by
// tests/test_bwd_frozen_schedule.py on the CPU: bwd_schedule_check.cu's conditions on
// the plan that has no dW units.
#include "rlk_bwd.cuh"

namespace rlk {
inline BwdPlan plan_without_dw(long long T, long long H, long long V, long long ldx) {
  return make_bwd_plan(T, H, V, ldx, false);
}
}  // namespace rlk

#define make_bwd_plan plan_without_dw
#include "bwd_schedule_check.cu"
