// The loop that k_gemm_dx and k_linear_tiles share: fp16 rows (A) times packed
// 4-bit weights on the matrix cores, tiles of 16 MB WM rows x 256 columns per
// block of 4 WM waves (WM along the rows x 4 along the columns, each 16 MB x
// 64), 64 of the contraction per stage, NS stages in LDS.
//
//  * Every stage arrives by LDS DMA, NS stages ahead: as many as LDS holds (with
//    two blocks per compute unit for the small tiles), since few rows leave a
//    block little to do per stage.  Three cover the memory's latency already;
//    five and six measured the same.  The small tiles are bound by the
//    dequantization (0.5 to 1 us a stage), the tall ones by the matrix pipe and
//    the reads that feed it (1.8 us; 2.3 to 3 for dx, which has two products).
//  * One barrier per stage, ahead of its last sub-step's products: by then
//    every wave has read the stage's last operands into registers, so its slot
//    takes the copies of stage s + NS, and the next stage's first operands are
//    read while the last products run.
//  * A column block's operands are dequantized in place as soon as its last
//    product of a k32 step is issued, a few vector instructions after each
//    product.
#pragma once

#include "awq_device.h"
#include "k_epilogue.h"
#include "tile_plan.h"

namespace awqk {

// Position of an A row's 16-byte chunk c in LDS: c ^ ((r / 2) mod 8).
__device__ __forceinline__ int tile_swz(int r) { return (r >> 1) & 7; }

// The work item of this block: block i runs on L2 slice i mod 8, which takes the
// i-th eighth of the items, slices of the contraction slowest, then groups of GM
// row tiles, then columns, then the group's rows.  The 32 or 64 blocks that a
// slice runs at once so share few distinct stages of both operands.
template <int GM>
__device__ __forceinline__ bool tile_item(int64_t block, int64_t mtiles, int64_t ctiles, int S, int& slice, int64_t& mt,
                                          int64_t& ct) {
  const int64_t tiles = mtiles * ctiles, items = tiles * S, per = (items + kTileXcds - 1) / kTileXcds;
  const int64_t slot = block / kTileXcds, item = (block % kTileXcds) * per + slot;
  if (slot >= per || item >= items) return false;
  slice = (int)(item / tiles);
  const int64_t t = item - slice * tiles, g = t / (GM * ctiles), r = t - g * GM * ctiles;
  const int64_t gm = mtiles - g * GM < GM ? mtiles - g * GM : GM;
  mt = g * GM + r % gm;
  ct = r / gm;
  return true;
}

// OP, the packed operand: bytes of its part of a stage (OP::Bytes), the copies
// of this wave (op.copies, BW or one more), issue(s, lds, live), load(lds): a stage's
// words and constants into registers, begin(st) and column(st, c, hi, lo): the
// operand of column block c for k32 step st; chunk(st, b4): the A chunk that goes
// with it.  OP::Whole: the operand is hi + lo, and both meet A.  OP::Units: the sums
// of column block c are in a unit of their own, which unit() changes where
// fresh(s), by a factor ratio[c].
template <int MB, int WM, int NS, class OP>
struct Tile {
  static constexpr int Waves = 4 * WM;
  static constexpr int Threads = 64 * Waves;
  static constexpr int Rows = 16 * MB * WM;
  static constexpr int GM = Rows >= 128 ? 4 : 8;        // row tiles of a group
  static constexpr int A = Rows * kTileK * 2;
  static constexpr int Stage = A + OP::Bytes;
  static constexpr int Lds = NS * Stage;
  static constexpr int AW = MB >= 2 ? MB / 2 : 1;       // A copies of a wave that has any
  static constexpr int H = MB > 4 ? 2 : 1;              // sub-steps per k32 step
  static constexpr int MH = MB / H;                     // 16-row blocks per sub-step
  static constexpr int BW = 8 / Waves;                  // copies of packed words per wave
  static_assert((NS - 1) * (AW + BW + 1) <= 63, "copies in flight");

  // rows of xq from row m0 on (pitch Kp, a multiple of 64), stages [s0, s1)
  static __device__ __forceinline__ void run(uint8_t* lds, OP& op, const uint16_t* __restrict__ xq, int64_t m0,
                                             int rows, int64_t Kp, int64_t s0, int64_t s1, f32x4 (&acc)[MB][4]) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv >> 2, rl = lane & 15, b4 = lane >> 4;
    const bool has_a = MB >= 2 || wv < 2 * WM;
    uint32_t aoff[AW];
#pragma unroll
    for (int u = 0; u < AW; ++u) {
      // lane i of a copy: row 8 j + i / 8, chunk (i % 8) ^ swizzle
      const int r = 8 * (AW * wv + u) + (lane >> 3);
      aoff[u] = (uint32_t)(r * Kp * 2 + (((lane & 7) ^ tile_swz(r)) * 16));
    }
    auto issue = [&](int64_t s, uint32_t slot) {
      const bool live = s < s1;                          // past the end: copies of nothing, so that the counts stay
      const uint32_t lb = __builtin_amdgcn_readfirstlane(lds_addr(lds) + slot * Stage);
      if (has_a) {
        const i32x4 ars = rsrc4(xq + m0 * Kp, live ? (uint32_t)(rows * Kp * 2) : 0u);
#pragma unroll
        for (int u = 0; u < AW; ++u) dma16(ars, lb + (AW * wv + u) * 1024, aoff[u], live ? (uint32_t)(s * kTileK * 2) : 0u);
      }
      op.issue(s, lb + A, live);
    };
    // all but the newest n stages' copies landed, and this wave's LDS reads done
    auto wait = [&](auto n) {
      constexpr int k = decltype(n)::value;
      const int nops = (has_a ? AW : 0) + op.copies;
      if (nops == AW + BW + 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(k * (AW + BW + 1)));
      else if (nops == AW + BW) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(k * (AW + BW)));
      else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(k * BW));          // MB = 1: a wave without rows
    };
    // A fragments of sub-step q = H st + hh
    u32x4 a0[MH], a1[MH];
    const uint32_t alane = (uint32_t)((wm * 16 * MB + rl) * 128);
    const int sw = tile_swz(rl);                          // the same for rows 16 apart
    auto load_a = [&](const uint8_t* base, int q, u32x4 (&a)[MH]) {
      const int st = q / H, hh = q % H;
#pragma unroll
      for (int i = 0; i < MH; ++i)
        a[i] = *reinterpret_cast<const u32x4*>(base + alane + (hh * MH + i) * 2048 + ((OP::chunk(st, b4) ^ sw) * 16));
    };
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (s0 >= s1) return;
#pragma unroll
    for (int j = 0; j < NS; ++j) issue(s0 + j, j);
    wait(std::integral_constant<int, NS - 1>{});
    lds_barrier();
    u32x4 bq[4], bl[OP::Whole ? 4 : 1];
    load_a(lds, 0, a0);
    op.load(lds + A);
    op.begin(0);
#pragma unroll
    for (int c = 0; c < 4; ++c) op.column(0, c, bq[c], bl[OP::Whole ? c : 0]);
    uint32_t slot = 0;
    for (int64_t s = s0; s < s1; ++s) {
      const uint32_t nslot = slot + 1 == NS ? 0 : slot + 1;
      const uint8_t* cur = lds + slot * Stage;
      const uint8_t* nxt = lds + nslot * Stage;
      if constexpr (OP::Units) {
        // between the stages: among the products, in every stage, it took longer
        // (2048 x 4096 x 11008: 279 us against 252, groups of 64: the same)
        if (s == s0 || op.fresh(s)) {
          op.unit();
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[b][c][v] *= op.ratio[c];
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int q = 0; q < 2 * H; ++q) {
        u32x4 (&ac)[MH] = (q & 1) ? a1 : a0;
        u32x4 (&an)[MH] = (q & 1) ? a0 : a1;
        if (q < 2 * H - 1) {
          load_a(cur, q + 1, an);
        } else {
          wait(std::integral_constant<int, NS - 2>{});    // stage s + 1 landed, this wave done with s
          lds_barrier();
          issue(s + NS, slot);
          load_a(nxt, 0, an);
          op.load(nxt + A);
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool turn = q % H == H - 1;                 // the k32 step's last products
        const int st = q / H;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < MH; ++i) {
            const int b = (q % H) * MH + i;
            acc[b][c] = mfma16h(ac[i], bq[c], acc[b][c]);
            if constexpr (OP::Whole) acc[b][c] = mfma16h(ac[i], bl[c], acc[b][c]);
          }
          if (turn) {
            if (c == 0) op.begin(st ^ 1);
            op.column(st ^ 1, c, bq[c], bl[OP::Whole ? c : 0]);
          }
        }
        if (turn && MH >= 4) {
#pragma unroll
          for (int i = 0; i < 4 * MH; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                    // one matrix product
            if (i >= 2) __builtin_amdgcn_sched_group_barrier(0x002, OP::VAlu, 0);  // vector instructions
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      slot = nslot;
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));       // the copies past the end
    lds_barrier();                                        // LDS is free for what follows
  }
};

}  // namespace awqk
