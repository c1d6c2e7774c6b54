// Grouping rows by an index on the device: counts, a sorted order and a list
// of tiles of rows that share one index (routed experts, per-row adapters).
#include "awq_device.h"
#include "awq_internal.h"
#include "k_groups.h"

namespace awqk {

__global__ __launch_bounds__(kPlanThreads) void k_group_plan(const int32_t* __restrict__ ids, int S, int E,
                                                             int tile_rows, GroupPlan plan) {
  extern __shared__ int group_lds[];
  group_plan_block(ids, S, E, tile_rows, plan, group_lds);
}

}  // namespace awqk

namespace awq {

hipError_t launch_group_plan(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const awqk::GroupPlan& plan,
                             hipStream_t st) {
  hipLaunchKernelGGL(awqk::k_group_plan, dim3(1), dim3(awqk::kPlanThreads), awqk::group_plan_lds((int)E), st, ids,
                     (int)S, (int)E, tile_rows, plan);
  return hipGetLastError();
}

}  // namespace awq
