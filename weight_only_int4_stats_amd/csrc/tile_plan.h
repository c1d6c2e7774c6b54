// Which tiles a product of k_tiles.h takes: heights, slices of the contraction,
// two heights in one launch.  Host code alone, so that it can be asked without
// a GPU.
#pragma once

#include <cstdint>

namespace awqk {

constexpr int kTileK = 64;                // contraction per stage
constexpr int kTileCols = 256;
constexpr int kTileXcds = 8;              // L2 slices (block i -> slice i mod 8)

// A tile's shape and its time per stage on a compute unit by itself and two at
// once (0: its LDS leaves room for one), in us.
struct TileShape {
  int mb, wm;
  double one, two;
};

struct TilePlan {
  int mb = 1, wm = 1, S = 1;
  double cost = 1e300;
};

// Time of `items` tiles of `stages` stages each: whole rounds of one tile (or
// two at once) per compute unit, and what a round costs beside its stages
// (start, first copies, stores).
inline double tile_time(const TileShape& h, int64_t items, int64_t stages, int64_t cus) {
  const int64_t load = (items + cus - 1) / cus;
  const double per = h.two > 0.0 ? (double)(load / 2) * h.two + (double)(load % 2) * h.one : (double)load * h.one;
  const double rounds = (double)(h.two > 0.0 ? (load + 1) / 2 : load);
  return per * (double)stages + 9.0 * rounds;
}

// Whether `tiles` tiles may be cut into S slices: up to two rounds of work, which
// bounds what the slices' sums take (four rounds: 0.1 % less time on average
// over 400 thousand sizes, 15 % at most, for twice the memory).
inline bool tile_splits(int64_t tiles, int S, int64_t stages, int64_t cus) {
  return S <= 16 && S * 2 <= stages && tiles * S <= 2 * cus;
}

// The shape and the number of slices of the contraction with the least
// estimated time.  Slices cost a second launch and their sums' way through
// memory (6.5 TB/s: they partly stay in the last cache).  Rows count in whole
// 16s, so that the choice is the same up to the next multiple.
template <int NSHAPES>
inline TilePlan tile_plan(const TileShape (&shapes)[NSHAPES], int64_t M, int64_t cols, int64_t stages, int64_t cus) {
  const int64_t ct = (cols + kTileCols - 1) / kTileCols, M16 = (M + 15) / 16 * 16;
  TilePlan best;
  for (const TileShape& h : shapes) {
    const int64_t tiles = (M + 16 * h.mb * h.wm - 1) / (16 * h.mb * h.wm) * ct;
    for (int S = 1; S == 1 || tile_splits(tiles, S, stages, cus); S *= 2) {
      const double cost = tile_time(h, tiles * S, (stages + S - 1) / S, cus) + (S > 1 ? 2.5 + (double)S * M16 * cols * 8 / 6.5e6 : 0.0);
      if (cost < best.cost) {
        best.mb = h.mb;
        best.wm = h.wm;
        best.S = S;
        best.cost = cost;
      }
    }
  }
  return best;
}

// What slices times rows may come to for any number of rows up to M.
template <int NSHAPES>
inline int64_t tile_parts(const TileShape (&shapes)[NSHAPES], int64_t M, int64_t cols, int64_t stages, int64_t cus) {
  const int64_t ct = (cols + kTileCols - 1) / kTileCols;
  int64_t most = 0;
  for (const TileShape& h : shapes)
    for (int S = 2; tile_splits(ct, S, stages, cus); S *= 2) {
      const int64_t rows = 2 * cus / (S * ct) * 16 * h.mb * h.wm, r = rows < M ? rows : M;
      most = S * r > most ? S * r : most;
    }
  return most;
}

inline int64_t tile_blocks(int64_t items) { return kTileXcds * ((items + kTileXcds - 1) / kTileXcds); }

// ---- dx (k_gemm_dx.hip): M rows of dz, contracted over N, K columns -----------------

// us per stage, fitted to the times of every shape and number of slices at 17
// sizes of 8 to 4096 rows, 1024 to 11008: the choice takes at most 2 % longer
// than the fastest there.  (128 rows by four waves never were: 147 to 145 us at
// 1500 rows of 5120 x 5120, 239 to 207 at 4096^3.)
constexpr TileShape kDxShapes[] = {{8, 2, 2.29, 0.0}, {4, 2, 1.45, 0.0}, {4, 1, 0.97, 1.51}, {2, 1, 0.64, 1.04}, {1, 1, 0.63, 0.89}};

inline TilePlan dx_plan(int64_t M, int64_t N, int64_t K, int64_t cus) {
  return tile_plan(kDxShapes, M, K, (N + kTileK - 1) / kTileK, cus);
}
// ---- the linear (k_linear.hip) --------------------------------------------------

// us per stage, fitted to the times of every shape and number of slices at 16
// sizes of 40 to 4096 rows, 1024 to 11008: the choice takes at most 3 % longer
// than the fastest there, 9 % at 4096 rows, 2048 -> 1027.
constexpr TileShape kLinearShapes[] = {{8, 2, 1.77, 0.0}, {4, 2, 1.06, 0.0}, {4, 1, 0.79, 1.35}, {2, 1, 0.58, 0.89}, {1, 1, 0.50, 0.87}};

struct LinearPlan {
  TilePlan t;
  int64_t wide = 0;       // > 0: column tiles 256 rows high of the mixed launch
  int64_t blocks = 0, wide_blocks = 0;
};

inline LinearPlan linear_plan(int64_t M, int64_t N, int64_t K, int64_t cus) {
  const int64_t stages = K / kTileK, ct = (N + kTileCols - 1) / kTileCols;
  LinearPlan p;
  p.t = tile_plan(kLinearShapes, M, N, stages, cus);
  const int64_t m256 = (M + 255) / 256, m128 = (M + 127) / 128;
  // only whole numbers of rounds of tall tiles are worth a cut
  for (int64_t r = 1; r * cus / m256 < ct && r <= 64; ++r) {
    const int64_t a = r * cus / m256;
    if (a < 1) continue;
    const double cost = tile_time(kLinearShapes[0], m256 * a, stages, cus) + tile_time(kLinearShapes[1], m128 * (ct - a), stages, cus);
    if (cost < p.t.cost) {
      p.t.cost = cost;
      p.t.S = 1;
      p.t.wm = 2;
      p.wide = a;
    }
  }
  const int rows = 16 * p.t.mb * p.t.wm;
  p.wide_blocks = tile_blocks(m256 * p.wide);
  p.blocks = p.wide ? p.wide_blocks + tile_blocks(m128 * (ct - p.wide)) : tile_blocks((M + rows - 1) / rows * ct * p.t.S);
  return p;
}

}  // namespace awqk
