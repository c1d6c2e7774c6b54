// Grouping rows by an index (k_groups.hip).
#pragma once

#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

// One tile: rows [first, first + rows) of the sorted order, all of group
// `group` (E: the rows whose index is outside [0, E)).
struct GroupTile {
  int group, first, rows;
  int before, tiles;           // tiles of all groups before this one, tiles of this group
  int pad[3];
};

// In the caller's workspace.  perm: the rows in sorted order (within a group
// in any order: no result depends on it); tiles: at most group_tiles_max of
// them, ntile[0] in use, ntile[1] of them in groups below E.
struct GroupPlan {
  int* perm;
  GroupTile* tiles;
  int* ntile;
};

constexpr int kPlanThreads = 1024;

inline int64_t group_tiles_max(int64_t S, int64_t E, int tile_rows) {
  return S / tile_rows + (S < E + 1 ? S : E + 1);
}
inline size_t group_plan_lds(int E) { return (size_t)(2 * E + 3 + 32) * 4; }
inline size_t group_plan_bytes(int64_t S, int64_t E, int tile_rows) {
  return awq::align_up((size_t)S * 4, 256) +
         awq::align_up((size_t)group_tiles_max(S, E, tile_rows) * sizeof(GroupTile), 256) + 256;
}
inline GroupPlan group_plan_at(void* ws, int64_t S, int64_t E, int tile_rows) {
  GroupPlan p;
  char* w = reinterpret_cast<char*>(ws);
  p.ntile = reinterpret_cast<int*>(w);
  p.perm = reinterpret_cast<int*>(w + 256);
  p.tiles = reinterpret_cast<GroupTile*>(w + 256 + awq::align_up((size_t)S * 4, 256));
  return p;
}

// Adds 1 to counter[g] for every lane with g >= 0 and returns the counter
// before the lane's own addition.  A wave of one g (runs of equal indices are
// common) adds once: lanes at one counter would take their turns.
__device__ __forceinline__ int group_add(int* counter, int g) {
  const int lane = threadIdx.x & 63;
  const int lead = __builtin_amdgcn_readfirstlane(g);
  if (__all(g == lead)) {
    if (lead < 0) return 0;
    int base = 0;
    if (lane == 0) base = atomicAdd(&counter[lead], 64);
    return __builtin_amdgcn_readfirstlane(base) + lane;
  }
  return g >= 0 ? atomicAdd(&counter[g], 1) : 0;
}

// One block of kPlanThreads: a counting sort of the S indices in LDS
// (group_plan_lds bytes at lds).  The positions inside a group come from LDS
// atomics.  Eight indices per thread are loaded together.
__device__ inline void group_plan_block(const int32_t* __restrict__ ids, int S, int E, int tile_rows,
                                        const GroupPlan& plan, int* lds) {
  int* start = lds;                    // counts, then first positions
  int* tstart = lds + E + 1;           // first tile of each group, and the end
  int* wsum = lds + 2 * E + 3;         // [16] rows, [16] tiles per wave
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  for (int g = tid; g <= E; g += kPlanThreads) start[g] = 0;
  __syncthreads();
  constexpr int kU = 8;
  int g8[kU];
  auto load8 = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s0 + u * kPlanThreads + tid;
      const int id = ids[s < S ? s : 0];
      g8[u] = s >= S ? -1 : id < 0 || id >= E ? E : id;
    }
  };
  for (int s0 = 0; s0 < S; s0 += kU * kPlanThreads) {
    load8(s0);
#pragma unroll
    for (int u = 0; u < kU; ++u) (void)group_add(start, g8[u]);
  }
  __syncthreads();
  // exclusive prefix sums of the counts and of the tile counts: each thread
  // takes a run of groups
  const int per = (E + kPlanThreads) / kPlanThreads;
  const int g0 = tid * per < E + 1 ? tid * per : E + 1, g1 = g0 + per < E + 1 ? g0 + per : E + 1;
  int n = 0, t = 0;
  for (int g = g0; g < g1; ++g) {
    n += start[g];
    t += (start[g] + tile_rows - 1) / tile_rows;
  }
  int ni = n, ti = t;                  // inclusive over the wave
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int a = __shfl_up(ni, off), b = __shfl_up(ti, off);
    if (lane >= off) {
      ni += a;
      ti += b;
    }
  }
  if (lane == 63) {
    wsum[wv] = ni;
    wsum[16 + wv] = ti;
  }
  __syncthreads();
  int nb = ni - n, tb = ti - t;
  for (int w = 0; w < wv; ++w) {
    nb += wsum[w];
    tb += wsum[16 + w];
  }
  for (int g = g0; g < g1; ++g) {
    const int c = start[g], tc = (c + tile_rows - 1) / tile_rows;
    tstart[g] = tb;
    if (g == E) {
      tstart[E + 1] = tb + tc;
      plan.ntile[0] = tb + tc;
      plan.ntile[1] = tb;
    }
    start[g] = nb;
    nb += c;
    tb += tc;
  }
  __syncthreads();
  // one tile per thread: its group is the last whose first tile is not past it
  const int tiles = tstart[E + 1];
  for (int i = tid; i < tiles; i += kPlanThreads) {
    int lo = 0, hi = E + 1;            // tstart[lo] <= i < tstart[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tstart[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int k = i - tstart[lo];
    const int end = lo == E ? S : start[lo + 1];
    GroupTile q;
    q.group = lo;
    q.first = start[lo] + k * tile_rows;
    q.rows = end - q.first < tile_rows ? end - q.first : tile_rows;
    q.before = tstart[lo];
    q.tiles = tstart[lo + 1] - tstart[lo];
    q.pad[0] = q.pad[1] = q.pad[2] = 0;
    plan.tiles[i] = q;
  }
  __syncthreads();
  for (int s0 = 0; s0 < S; s0 += kU * kPlanThreads) {
    if (S > kU * kPlanThreads) load8(s0);          // else still held from the counting
    int at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) at[u] = group_add(start, g8[u]);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (g8[u] >= 0) plan.perm[at[u]] = s0 + u * kPlanThreads + tid;
  }
}

}  // namespace awqk

namespace awq {
hipError_t launch_group_plan(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const awqk::GroupPlan& plan,
                             hipStream_t st);
}  // namespace awq
