// Grouping rows by an index on the device: a sorted order and a list of tiles
// of rows that share one index (routed experts, per-row adapters).
#include "awq_device.h"
#include "awq_internal.h"
#include "k_groups.h"

namespace awqk {

__global__ __launch_bounds__(kPlanThreads) void k_group_sort(const int32_t* __restrict__ ids, int S, int E, int chunks,
                                                             int tile_rows, GroupPlan plan) {
  extern __shared__ int group_lds[];
  group_sort_block(ids, S, E, blockIdx.x, chunks, tile_rows, plan, group_lds);
}

__global__ __launch_bounds__(kPlanThreads) void k_group_place(const int32_t* __restrict__ ids, int S, int E, int chunks,
                                                              int tile_rows, GroupPlan plan) {
  extern __shared__ int group_lds[];
  group_place_block(ids, S, E, blockIdx.x, chunks, tile_rows, plan, group_lds);
}

}  // namespace awqk

namespace awq {
using namespace awqk;

hipError_t launch_group_place(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const GroupPlan& plan,
                              hipStream_t st) {
  const int chunks = group_chunks(S);
  if (chunks == 1) return hipSuccess;
  hipLaunchKernelGGL(k_group_place, dim3(chunks), dim3(kPlanThreads), group_plan_lds((int)E), st, ids, (int)S, (int)E,
                     chunks, tile_rows, plan);
  return hipGetLastError();
}

hipError_t launch_group_plan(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const GroupPlan& plan,
                             hipStream_t st) {
  const int chunks = group_chunks(S);
  hipLaunchKernelGGL(k_group_sort, dim3(chunks), dim3(kPlanThreads), group_plan_lds((int)E), st, ids, (int)S, (int)E,
                     chunks, tile_rows, plan);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_group_place(ids, S, E, tile_rows, plan, st);
}

}  // namespace awq
