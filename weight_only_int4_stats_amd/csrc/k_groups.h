// Grouping rows by an index (k_groups.hip): rows sorted by group and tiles of
// rows that share one.
#pragma once

#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

// One tile: rows [first, first + rows) of the sorted order, all of group
// `group` (E: the rows whose index is outside [0, E)).
struct GroupTile {
  int group, first, rows;
  int before, tiles;           // tiles of all groups before this one, tiles of this group
  int gfirst, grows;           // the group's rows
  int pad;
};

// In the caller's workspace.  perm: the rows in sorted order (within a group
// in any order: no result depends on it); tiles: at most group_tiles_max of
// them, ntile[0] in use, ntile[1] of them in groups below E.  Many rows are
// sorted in chunks first: lperm (each chunk's rows in its order) and lstart
// [chunks][E + 2] (where its groups start).
struct GroupPlan {
  int* perm;
  GroupTile* tiles;
  int* ntile;
  int* lperm;
  int* lstart;
};

constexpr int kPlanThreads = 1024;

// One block sorts up to 4096 rows alone; more are sorted in up to 64 chunks,
// one per block, and put together by a second launch.  (32768 rows of 64
// groups in one block: 50 us; the second launch takes 6.)
inline int group_chunks(int64_t S) {
  if (S <= 4096) return 1;
  const int64_t c = (S + 2047) / 2048;
  return (int)(c < 64 ? c : 64);
}
inline int64_t group_tiles_max(int64_t S, int64_t E, int tile_rows) {
  return S / tile_rows + (S < E + 1 ? S : E + 1);
}
inline size_t group_plan_lds(int E) { return (size_t)(3 * (E + 2) + 32) * 4; }
inline size_t group_plan_bytes(int64_t S, int64_t E, int tile_rows) {
  const size_t perm = awq::align_up((size_t)S * 4, 256);
  const int chunks = group_chunks(S);
  return 256 + perm + awq::align_up((size_t)group_tiles_max(S, E, tile_rows) * sizeof(GroupTile), 256) +
         awq::align_up((size_t)chunks * (size_t)(E + 2) * 4, 256) + (chunks > 1 ? perm : 0);
}
inline GroupPlan group_plan_at(void* ws, int64_t S, int64_t E, int tile_rows) {
  GroupPlan p;
  char* w = reinterpret_cast<char*>(ws);
  p.ntile = reinterpret_cast<int*>(w);
  p.perm = reinterpret_cast<int*>(w += 256);
  p.tiles = reinterpret_cast<GroupTile*>(w += awq::align_up((size_t)S * 4, 256));
  p.lstart = reinterpret_cast<int*>(w += awq::align_up((size_t)group_tiles_max(S, E, tile_rows) * sizeof(GroupTile), 256));
  p.lperm = reinterpret_cast<int*>(w + awq::align_up((size_t)group_chunks(S) * (size_t)(E + 2) * 4, 256));
  return p;
}

// The lanes of the wave whose g equals this lane's (bits: how many of g's bits
// can differ).  Lanes that added to one LDS counter together would take their
// turns there, so one lane adds for all of them.
__device__ __forceinline__ uint64_t same_lanes(int g, int bits) {
  uint64_t m = ~0ull;
  for (int i = 0; i < bits; ++i) {
    const bool bit = (g >> i) & 1;
    const uint64_t b = __ballot(bit);
    m &= bit ? b : ~b;
  }
  return m;
}

// Exclusive prefix sum over n values v[0 .. n) of LDS, in place, by the whole
// block of kPlanThreads (wsum: 16 ints); returns the total.
__device__ inline int block_prefix(int* v, int n, int* wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = tid * per < n ? tid * per : n, i1 = i0 + per < n ? i0 + per : n;
  int own = 0;
  for (int i = i0; i < i1; ++i) own += v[i];
  int incl = own;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int a = __shfl_up(incl, off);
    if (lane >= off) incl += a;
  }
  if (lane == 63) wsum[wv] = incl;
  __syncthreads();
  int at = incl - own, total = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wv) at += wsum[w];
    total += wsum[w];
  }
  for (int i = i0; i < i1; ++i) {
    const int c = v[i];
    v[i] = at;
    at += c;
  }
  __syncthreads();
  return total;
}

// Lists the tiles from the groups' sizes in tstart[0 .. E] (LDS; tiles per
// group on the way out) and first rows start[0 .. E + 1].
__device__ inline void group_tiles(int* start, int* tstart, int E, int tile_rows, const GroupPlan& plan, int* wsum, bool list) {
  const int tid = threadIdx.x;
  const int tiles = block_prefix(tstart, E + 1, wsum);
  if (!list) return;
  if (tid == 0) {
    tstart[E + 1] = tiles;
    plan.ntile[0] = tiles;
    plan.ntile[1] = tstart[E];
  }
  __syncthreads();
  // one tile per thread: its group is the last whose first tile is not past it
  for (int i = tid; i < tiles; i += kPlanThreads) {
    int lo = 0, hi = E + 1;            // tstart[lo] <= i < tstart[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tstart[mid] <= i) lo = mid;
      else hi = mid;
    }
    GroupTile q;
    q.group = lo;
    q.first = start[lo] + (i - tstart[lo]) * tile_rows;
    q.rows = start[lo + 1] - q.first < tile_rows ? start[lo + 1] - q.first : tile_rows;
    q.before = tstart[lo];
    q.tiles = tstart[lo + 1] - tstart[lo];
    q.gfirst = start[lo];
    q.grows = start[lo + 1] - start[lo];
    q.pad = 0;
    plan.tiles[i] = q;
  }
}

// Chunk c of the rows by one block of kPlanThreads: a counting sort in LDS
// (group_plan_lds bytes at lds).  One chunk: the whole plan.
__device__ inline void group_sort_block(const int32_t* __restrict__ ids, int S, int E, int c, int chunks, int tile_rows,
                                        const GroupPlan& plan, int* lds) {
  int* start = lds;                    // [E + 2] counts, then first positions, and the end
  int* tstart = lds + E + 2;           // [E + 2] the same for tiles (one chunk)
  int* wsum = lds + 3 * (E + 2);
  const int tid = threadIdx.x, lane = tid & 63;
  const int lo = (int)((int64_t)c * S / chunks), hi = (int)((int64_t)(c + 1) * S / chunks);
  const int bits = 32 - __builtin_clz(E + 1);      // of 0 .. E + 1; E + 1: past the last row
  int* out = chunks > 1 ? plan.lperm : plan.perm;
  constexpr int kU = 4;                // rows per thread loaded together
  int g4[kU];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s0 + u * kPlanThreads + tid;
      const int id = ids[s < hi ? s : lo];
      g4[u] = s >= hi ? E + 1 : id < 0 || id >= E ? E : id;
    }
  };
  load(lo);
  for (int g = tid; g <= E; g += kPlanThreads) start[g] = 0;
  __syncthreads();
  for (int s0 = lo; s0 < hi; s0 += kU * kPlanThreads) {
    if (s0 > lo) load(s0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (s0 + u * kPlanThreads >= hi) break;
      const uint64_t m = same_lanes(g4[u], bits);
      if (g4[u] <= E && lane == __builtin_ctzll(m)) atomicAdd(&start[g4[u]], __popcll(m));
    }
  }
  __syncthreads();
  if (chunks == 1)
    for (int g = tid; g <= E; g += kPlanThreads) tstart[g] = (start[g] + tile_rows - 1) / tile_rows;
  block_prefix(start, E + 1, wsum);
  if (chunks == 1) {
    if (tid == 0) start[E + 1] = S;
    group_tiles(start, tstart, E, tile_rows, plan, wsum, true);
  } else {
    int* ls = plan.lstart + (int64_t)c * (E + 2);
    for (int g = tid; g <= E; g += kPlanThreads) ls[g] = start[g];
    if (tid == 0) ls[E + 1] = hi - lo;
  }
  __syncthreads();
  for (int s0 = lo; s0 < hi; s0 += kU * kPlanThreads) {
    if (hi - lo > kU * kPlanThreads) load(s0);     // else still held from the counting
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (s0 + u * kPlanThreads >= hi) break;
      const uint64_t m = same_lanes(g4[u], bits);
      const int lead = __builtin_ctzll(m);
      int at = 0;
      if (g4[u] <= E && lane == lead) at = atomicAdd(&start[g4[u]], __popcll(m));
      at = __shfl(at, lead) + __popcll(m & ((1ull << lane) - 1));
      if (g4[u] <= E) out[lo + at] = s0 + u * kPlanThreads + tid;
    }
  }
}

// Many chunks: block c puts its chunk into the common order; block 0 lists
// the tiles.  group_plan_lds bytes at lds.
__device__ inline void group_place_block(const int32_t* __restrict__ ids, int S, int E, int c, int chunks, int tile_rows,
                                         const GroupPlan& plan, int* lds) {
  int* start = lds;                    // [E + 2] first rows of the groups, and the end
  int* tstart = lds + E + 2;           // [E + 2] first tiles, and the end
  int* move = lds + 2 * (E + 2);       // [E + 1] from a position in this chunk to the common one
  int* wsum = lds + 3 * (E + 2);
  const int tid = threadIdx.x;
  for (int g = tid; g <= E; g += kPlanThreads) {
    int n = 0, before = 0;
    for (int k0 = 0; k0 < chunks; k0 += 16) {      // 16 chunks' loads together
      int m[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int* ls = plan.lstart + (int64_t)(k0 + k < chunks ? k0 + k : 0) * (E + 2) + g;
        m[k] = ls[1] - ls[0];
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k0 + k < c) before += m[k];
        if (k0 + k < chunks) n += m[k];
      }
    }
    start[g] = n;
    tstart[g] = (n + tile_rows - 1) / tile_rows;
    move[g] = before - plan.lstart[(int64_t)c * (E + 2) + g];
  }
  __syncthreads();
  block_prefix(start, E + 1, wsum);
  if (tid == 0) start[E + 1] = S;
  group_tiles(start, tstart, E, tile_rows, plan, wsum, c == 0);
  const int lo = (int)((int64_t)c * S / chunks), hi = (int)((int64_t)(c + 1) * S / chunks);
  for (int i = lo + tid; i < hi; i += kPlanThreads) {
    const int s = plan.lperm[i], id = ids[s], g = id < 0 || id >= E ? E : id;
    plan.perm[start[g] + move[g] + (i - lo)] = s;
  }
}

}  // namespace awqk

namespace awq {

// The whole plan (LoRA), and its second launch alone (after the chunks were
// sorted inside another kernel's launch; nothing to do for one chunk).
hipError_t launch_group_plan(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const awqk::GroupPlan& plan,
                             hipStream_t st);
hipError_t launch_group_place(const int32_t* ids, int64_t S, int64_t E, int tile_rows, const awqk::GroupPlan& plan,
                              hipStream_t st);

}  // namespace awq
