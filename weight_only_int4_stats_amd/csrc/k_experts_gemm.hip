// Routed W4A16 products for many rows per expert (include/awq.h,
// awq_w4a16_experts_up / _down): prefills, whose floor is the matrix cores'.
//
//   z[slot][n] = sum_g D[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[row(slot)][k]
//
//  * k_experts_prep: the first block (many slots: blocks, put together by a
//    second launch) sorts the slots by expert and lists the row tiles; the
//    others convert the activation rows to fp16 (scaled by a power of two per
//    row, in the order the unpack yields), lay the steps and zero points out
//    group by group, and zero the output rows of slots without an expert.
//  * k_experts_gemm: tiles of BM = 16 MB rows of one expert x 256 weight rows, 4
//    waves of BM x 64, two blocks per compute unit.  64 channels per stage,
//    three LDS stages filled by LDS DMA two stages ahead; the rows of a tile are
//    gathered by the copies' addresses.  v_mfma_f32_16x16x32_f16 multiplies the
//    activations with the exact integers (q - z) 2^-9.  The accumulators hold
//    the sum in units of the current group's step: a new group multiplies them
//    by D[g - 1] / D[g] (fp32, one multiplication per value and group; the
//    quotient is within 1 unit of 2^-24 and 1 for equal steps: with the
//    reciprocal's product alone, up to 4 units, a row of one step drifted by a
//    unit a group) and the epilogue by the last step.  So no operand is
//    rounded, unlike step (q - z) in fp16 (1e-4 of every result), and no second
//    set of accumulators is needed.  Unpacking costs 9 vector instructions per eight codes; a wave's
//    tile is tall (128 rows) because they serve all of its rows: tiles of 64 rows
//    take twice as many per product (times at gemm_tile_rows).
//  * With SwiGLU a tile's columns alternate 16 gate rows and their 16 up rows,
//    so both meet in one lane.  down writes an fp32 row per slot; the weighted
//    sum over a token's slots is k_experts_combine's.  (fp16 rows, scaled by a
//    power of two per 64 columns, halve the bytes between the two, 218 instead
//    of 257 us a call for 4096 tokens, 8 of 64 experts, 1024 -> 2048, but they
//    round every term to 2^-11 of itself and more beside a large one.)
//  * 2048 tokens, 2 of 8 experts, 4096 -> 2 x 11008: 700 to 740 us a call (18 of
//    them the preparation), 0.94 to 0.99 PFLOP/s where a large library product
//    reaches 1.35.  Neither pipe is full: the matrix pipe is busy 48 % of the
//    cycles (33 % at K = 1024), with 3.6 other vector instructions per product.
//  * The tiles of one expert are ordered 8 row tiles at a time, rows fastest,
//    and each L2 slice takes a contiguous eighth of the order.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_experts.h"
#include "k_groups.h"
#include "k_rows_f16.h"

#include <type_traits>

namespace awqk {

constexpr int kGemmN = 256;                        // weight rows per tile
constexpr int kGemmK = 64;                         // channels per stage
constexpr int kGemmGroupM = 8;                     // row tiles taken together
constexpr int kXcd = 8;                            // L2 slices

struct GemmArgs {
  const uint16_t* x;
  int64_t K, ldx, N, ldy;
  const int32_t* ids;
  const uint32_t* qw;
  const uint16_t* scales;
  const uint8_t* zeros;
  void* y;
  int64_t xrows;
  int S, E, top_k, group, unit, ydt;          // unit: channels per constant (64 or 128, at most the group)
  // workspace
  uint16_t* xq;                                    // [xrows][K]
  int* pexp;                                       // [xrows]
  uint32_t* ctab;                                  // [E][K / unit][N]: D | -z 2^-9 << 16, both fp16
  GroupPlan plan;
  // first block of each part of the preparation
  int b_rows, b_consts, b_zero;
};

// One wave converts one row: fp16(x 2^p), p from the row's maximum, each
// 8-channel piece in the order (0,4 | 2,6 | 1,5 | 3,7).
template <int DT>
__device__ __forceinline__ void prep_row(const GemmArgs& p, int64_t row) {
  const int lane = threadIdx.x & 63;
  const uint16_t* src = p.x + row * p.ldx;
  uint16_t* dst = p.xq + row * p.K;
  const int n8 = (int)(p.K >> 3);
  constexpr int kKeep = 8;                         // pieces per lane held in registers (K up to 4096)
  u32x4 raw[kKeep];
  float am = 0.0f;
  auto piece_max = [&](const u32x4& w) {
#pragma unroll
    for (int c = 0; c < 4; ++c) am = fmaxf(am, fmaxf(fabsf(lo_f32<DT>(w[c])), fabsf(hi_f32<DT>(w[c]))));
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = lane + 64 * i;
    raw[i] = c < n8 ? ldg128(src + c * 8) : u32x4{0, 0, 0, 0};
    piece_max(raw[i]);
  }
  for (int c = lane + 64 * kKeep; c < n8; c += 64) piece_max(ldg128(src + c * 8));
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) am = fmaxf(am, __shfl_xor(am, off));
  if (am == __builtin_inff()) {                    // again, of the finite values
    am = 0.0f;
    for (int c = lane; c < n8; c += 64) {
      const u32x4 w = ldg128(src + c * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) am = fmaxf(am, fmaxf(finite_size(lo_f32<DT>(w[j])), finite_size(hi_f32<DT>(w[j]))));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) am = fmaxf(am, __shfl_xor(am, off));
  }
  const int pe = pow2_exp_for(am);
  if (lane == 0) p.pexp[row] = pe;
  auto convert = [&](int c, const u32x4& w) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[2 * j] = f32_to_f16_bits(ldexpf(lo_f32<DT>(w[j]), pe));
      h[2 * j + 1] = f32_to_f16_bits(ldexpf(hi_f32<DT>(w[j]), pe));
    }
    *reinterpret_cast<u32x4*>(dst + c * 8) = u32x4{h[0] | (h[4] << 16), h[2] | (h[6] << 16), h[1] | (h[5] << 16), h[3] | (h[7] << 16)};
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = lane + 64 * i;
    if (c < n8) convert(c, raw[i]);
  }
  for (int c = lane + 64 * kKeep; c < n8; c += 64) convert(c, ldg128(src + c * 8));
}

template <int DT>
__global__ __launch_bounds__(kPlanThreads) void k_experts_prep(const GemmArgs p, int tile_rows, int64_t cols) {
  extern __shared__ int prep_lds[];
  const int bid = blockIdx.x, tid = threadIdx.x;
  if (bid < p.b_rows) {
    group_sort_block(p.ids, p.S, p.E, bid, p.b_rows, tile_rows, p.plan, prep_lds);
  } else if (bid < p.b_consts) {
    const int64_t row = (int64_t)(bid - p.b_rows) * 16 + (tid >> 6);
    if (row < p.xrows) prep_row<DT>(p, row);
  } else if (bid < p.b_zero) {
    // a thread takes eight groups of one row of the [E N] stack
    const int G = (int)(p.K / p.group), U = (int)(p.K / p.unit), sh = p.group == 256 ? 1 : 0;
    const int64_t i = (int64_t)(bid - p.b_consts) * kPlanThreads + tid;
    const int64_t n = i / ((G + 7) / 8);
    const int g0 = (int)(i - n * ((G + 7) / 8)) * 8;
    if (n >= (int64_t)p.E * p.N) return;
    const int64_t e = n / p.N, r = n - e * p.N;
    const uint16_t* s = p.scales + n * G + g0;
    const uint8_t* z = p.zeros + n * G + g0;
    uint32_t sv[8], zv[8];
    if ((G & 7) == 0 && (uintptr_t)p.scales % 16 == 0 && (uintptr_t)p.zeros % 8 == 0) {
      const u32x4 s8 = ldg128(s);
      const uint2 z8 = *reinterpret_cast<const uint2*>(z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sv[j] = (s8[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
        zv[j] = ((j < 4 ? z8.x : z8.y) >> (8 * (j & 3))) & 0xFFu;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = g0 + j < G ? j : 0;
        sv[j] = s[k];
        zv[j] = z[k];
      }
    }
    uint32_t* c = p.ctab + (e * U + ((int64_t)g0 << sh)) * p.N + r;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (g0 + j < G) {
        const uint32_t v = sv[j] | (experts_nz(zv[j]) & 0xFFFF0000u);
        c[((int64_t)j << sh) * p.N] = v;
        if (sh) c[(((int64_t)j << sh) + 1) * p.N] = v;
      }
  } else {
    const int64_t slot = (int64_t)(bid - p.b_zero) * 16 + (tid >> 6);
    if (slot >= p.S) return;
    const int id = p.ids[slot];
    if (id >= 0 && id < p.E) return;
    const int es = p.ydt == DT_F32 ? 4 : 2, q = 16 / es;   // whole 16 bytes where the rows allow it
    uint8_t* y = reinterpret_cast<uint8_t*>(p.y) + slot * p.ldy * es;
    int64_t c = 0;
    if (p.ldy % q == 0 && (uintptr_t)p.y % 16 == 0) {
      c = cols / q * q;
      for (int64_t i = tid & 63; i < cols / q; i += 64) *reinterpret_cast<u32x4*>(y + i * 16) = u32x4{0, 0, 0, 0};
    }
    for (c += tid & 63; c < cols; c += 64) store_out(p.y, p.ydt, slot * p.ldy + c, 0.0f);
  }
}

template <int MODE, int MB, int SPG>
__global__ __launch_bounds__(256, 2) void k_experts_gemm(const GemmArgs p) {
  constexpr int BM = 16 * MB, HB = MB / 2;         // rows, 16-row blocks per sub-step
  constexpr int kA = BM * kGemmK * 2, kB = kGemmN * 32, kC = kGemmN * 4, kStage = kA + kB + kC;
  constexpr int kAc = BM / 32;                     // A copies per wave and stage
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;

  // ---- the tile
  const int64_t ncols = MODE == EXPERTS_SWIGLU ? p.N >> 1 : p.N;
  constexpr int kCols = MODE == EXPERTS_SWIGLU ? kGemmN / 2 : kGemmN;     // output columns per tile
  const int nt = (int)((ncols + kCols - 1) / kCols);
  const int64_t total = (int64_t)p.plan.ntile[1] * nt;
  const int64_t per = (total + kXcd - 1) / kXcd;
  const int64_t in = blockIdx.x / kXcd, at = (int64_t)(blockIdx.x % kXcd) * per + in;
  if (in >= per || at >= total) return;
  const GroupTile q0 = p.plan.tiles[at / nt];
  const int64_t rem = at - (int64_t)q0.before * nt;
  const int gi = (int)(rem / (kGemmGroupM * nt));
  const int gm = q0.tiles - gi * kGemmGroupM < kGemmGroupM ? q0.tiles - gi * kGemmGroupM : kGemmGroupM;
  const int in_group = (int)(rem - (int64_t)gi * kGemmGroupM * nt);
  const int64_t c0 = (int64_t)(in_group / gm) * kCols;
  const int r_tile = (gi * kGemmGroupM + in_group % gm) * BM;      // the tile's first row within the expert's
  const int e = __builtin_amdgcn_readfirstlane(q0.group);
  const int rows = __builtin_amdgcn_readfirstlane(q0.grows - r_tile < BM ? q0.grows - r_tile : BM);
  const int* perm = p.plan.perm + __builtin_amdgcn_readfirstlane(q0.gfirst + r_tile);
  auto xrow = [&](int slot) { return MODE == EXPERTS_DOWN ? slot : slot / p.top_k; };
  // weight row of tile column c, -1 past the last
  auto wrow = [&](int c) -> int64_t {
    if constexpr (MODE == EXPERTS_SWIGLU) {
      const int64_t n = c0 + (c >> 5) * 16 + (c & 15);
      return n < ncols ? n + ((c >> 4) & 1) * ncols : -1;
    } else {
      return c0 + c < ncols ? c0 + c : -1;
    }
  };

  // ---- copies: A rows of 128 bytes, 8 per copy, chunk c of row r at c ^ (r & 7);
  // B per 32 columns the first then the last 16 bytes of each; C four entries a lane
  const i32x4 ars = rsrc4(p.xq, (uint32_t)(p.xrows * p.K * 2));
  const i32x4 brs = rsrc4(reinterpret_cast<const uint8_t*>(p.qw) + (int64_t)e * p.N * (p.K >> 1), (uint32_t)(p.N * (p.K >> 1)));
  const int64_t U = p.K / p.unit;
  const i32x4 crs = rsrc4(p.ctab + (int64_t)e * U * p.N, (uint32_t)(U * p.N * 4));
  // the rows' slots and exponents wait in LDS for the epilogue: fetched there,
  // two dependent loads for every few rows, they took a tile 20 us
  int* slots = reinterpret_cast<int*>(lds + 3 * kStage);
  int* exps = slots + BM;
  if (tid < rows) {
    const int slot = perm[tid];
    slots[tid] = slot;
    exps[tid] = 9 - p.pexp[xrow(slot)];            // with the operands' 2^-9
  }
  uint32_t aoff[kAc];
#pragma unroll
  for (int u = 0; u < kAc; ++u) {
    const int r = 8 * (kAc * wv + u) + (lane >> 3);
    aoff[u] = r < rows ? (uint32_t)((int64_t)xrow(perm[r]) * p.K * 2) + (uint32_t)(((lane & 7) ^ (r & 7)) * 16) : kBufferOob;
  }
  uint32_t boff[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t n = wrow(64 * wv + 32 * u + (lane & 31));
    boff[u] = n < 0 ? kBufferOob : (uint32_t)(n * (p.K >> 1)) + (uint32_t)((lane >> 5) * 16);
  }
  const int64_t cn = wrow(4 * lane);
  const uint32_t coff = cn < 0 ? kBufferOob : (uint32_t)(cn * 4);
  const uint32_t lbase = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const int S = (int)(p.K / kGemmK);
  // part q of stage s's copies into buffer buf: the A copies q, q + 4, ..., and
  // the rest with the last
  auto copy = [&](int s, int buf, int q) {
    const uint32_t lb = lbase + (uint32_t)buf * kStage;
#pragma unroll
    for (int u = 0; u < kAc; ++u)
      if (u % 4 == q) dma16(ars, lb + (uint32_t)(kAc * wv + u) * 1024, aoff[u], (uint32_t)s * 128);
    if (q == 2) dma16(brs, lb + kA + (uint32_t)wv * 2048, boff[0], (uint32_t)s * 32);
    if (q == 3) {
      dma16(brs, lb + kA + (uint32_t)wv * 2048 + 1024, boff[1], (uint32_t)s * 32);
      if (wv == 0) dma16(crs, lb + kA + kB, coff, (uint32_t)(s / SPG) * (uint32_t)(p.N * 4));
    }
  };
  // every LDS access of this wave done, and all copies but the newest stage's
  auto wait_stage = [&](bool newest) {
    if (!newest) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    else if (wv == 0) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(kAc + 3));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(kAc + 2));
  };

  f32x4 acc[MB][4];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint2 w[4];                                      // a stage's words of the lane's columns
  uint32_t cz[4];                                  // and constants
  auto load_w = [&](const uint8_t* base) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int col = wv * 64 + n * 16 + rl;
      w[n] = *reinterpret_cast<const uint2*>(base + kA + (col >> 5) * 1024 + (b >> 1) * 512 + (col & 31) * 16 + (b & 1) * 8);
      cz[n] = *reinterpret_cast<const uint32_t*>(base + kA + kB + col * 4);
    }
  };
  // fragments of sub-step q = 2 st + hh: k32 step st, row blocks HB hh ..
  auto load_a = [&](const uint8_t* base, int q, u32x4 (&a)[HB]) {
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const int r = ((q & 1) * HB + i) * 16 + rl;
      a[i] = *reinterpret_cast<const u32x4*>(base + r * 128 + (((2 * b + (q >> 1)) ^ (r & 7)) * 16));
    }
  };
  u32x4 aE[HB], aO[HB], bq[4];
  float ratio[4], last[4] = {1.0f, 1.0f, 1.0f, 1.0f};   // D of the last unit / this unit's; the last unit's
  float any[4] = {0.0f, 0.0f, 0.0f, 0.0f};         // the largest |D|: 0 and the column is 0, or it is infinite
  auto nz = [&](int n) { return (cz[n] >> 16) * 0x10001u; };
#pragma unroll
  for (int q = 0; q < 4; ++q) copy(0, 0, q);
  if (S > 1)
#pragma unroll
    for (int q = 0; q < 4; ++q) copy(1, 1, q);
  wait_stage(S > 1);
  lds_barrier();
  load_a(lds, 0, aE);
  load_w(lds);
#pragma unroll
  for (int n = 0; n < 4; ++n) bq[n] = experts_unpack(w[n].x, nz(n));

  // A stage runs in four sub-steps.  In sub-step 1 a column's operands are
  // replaced by step 1's once its last product of step 0 is issued, in
  // sub-step 3 by the next stage's, whose words are read right after the
  // barrier: the unpacking runs between the products.
  int buf = 0;
  for (int s0 = 0; s0 < S; s0 += SPG) {             // SPG stages per unit
#pragma unroll
    for (int i = 0; i < SPG; ++i) {
      const int s = s0 + i;
      const bool cp = s + 2 < S;
      const int nxt = buf == 2 ? 0 : buf + 1, nxt2 = buf == 0 ? 2 : buf - 1;
      const uint8_t* cur = lds + buf * kStage;
      const uint8_t* ahead = lds + nxt * kStage;
      if (i == 0) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          // a step of 0 counts as 2^-60, which keeps the ratios finite and is
          // below the fp32 rounding of any other (2^-24 at least); an infinite
          // one as 2^60, above any other, until the epilogue
          const float f = f16_to_f32(cz[n] & 0xFFFFu), size = fabsf(f);
          const float d = size < 0x1p-60f ? 0x1p-60f : size == __builtin_inff() ? copysignf(0x1p60f, f) : f;
          any[n] = fmaxf(any[n], size);
          // the quotient, corrected by its remainder: equal steps give 1
          const float r = __builtin_amdgcn_rcpf(d), t = last[n] * r;
          ratio[n] = __builtin_fmaf(__builtin_fmaf(-t, d, last[n]), r, t);
          last[n] = d;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (cp) copy(s + 2, nxt2, q);
        if (q < 3) {
          load_a(cur, q + 1, (q & 1) ? aE : aO);
        } else {
          wait_stage(cp);
          lds_barrier();
          load_a(ahead, 0, aE);
          load_w(ahead);
        }
        __builtin_amdgcn_sched_barrier(0);
        const u32x4 (&a)[HB] = (q & 1) ? aO : aE;
        const int hh = q & 1;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int m = 0; m < HB; ++m) {
            f32x4& c = acc[hh * HB + m][n];
            if (i == 0 && q < 2) {
#pragma unroll
              for (int v = 0; v < 4; ++v) c[v] *= ratio[n];
            }
            c = mfma16h(a[m], bq[n], c);
          }
          if (q & 1) bq[n] = experts_unpack(q == 1 ? w[n].y : w[n].x, nz(n));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      buf = nxt;
    }
  }

  // ---- epilogue: the last group's step, then 16 rows at a time through the
  // wave's LDS area and out in whole row pieces.  Result lane: column l % 16,
  // rows 4 b + v.
  __syncthreads();                                 // every wave is done with the stages
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if (any[n] == 0.0f) last[n] *= 0.0f;
    if (any[n] == __builtin_inff()) last[n] *= any[n];
  }
  constexpr int kW = MODE == EXPERTS_SWIGLU ? 32 : 64;                    // outputs per row of the wave
  float* stg = reinterpret_cast<float*>(lds) + wv * 16 * (kW + 4);
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int r0 = m * 16;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = r0 + 4 * b + v;
      const int pe = r < rows ? exps[r] : 0;
      float* d = stg + (4 * b + v) * (kW + 4) + rl;
      if constexpr (MODE == EXPERTS_SWIGLU) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          d[16 * h] = swiglu(ldexpf(acc[m][2 * h][v] * last[2 * h], pe), ldexpf(acc[m][2 * h + 1][v] * last[2 * h + 1], pe));
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) d[16 * n] = ldexpf(acc[m][n][v] * last[n], pe);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0): the wave's writes landed
    __builtin_amdgcn_wave_barrier();
    if (MODE == EXPERTS_DOWN || p.ydt == DT_F32) {
      constexpr int kL = kW / 4;                   // lanes per row, four outputs each
#pragma unroll
      for (int i = 0; i < 16 * kL / 64; ++i) {
        const int r = i * (64 / kL) + lane / kL, c = (lane % kL) * 4;
        const f32x4 o = *reinterpret_cast<const f32x4*>(stg + r * (kW + 4) + c);
        if (r0 + r >= rows) continue;
        const int64_t col = c0 + wv * kW + c;
        float* y = reinterpret_cast<float*>(p.y) + (int64_t)slots[r0 + r] * p.ldy + col;
        if (col + 4 <= ncols) *reinterpret_cast<u32x4a4*>(y) = __builtin_bit_cast(u32x4, o);
        else
          for (int j = 0; j < 4; ++j)
            if (col + j < ncols) y[j] = o[j];
      }
    } else {
      constexpr int kL = kW / 8;                   // lanes per row, eight outputs each
#pragma unroll
      for (int i = 0; i < 16 * kL / 64; ++i) {
        const int r = i * (64 / kL) + lane / kL, c = (lane % kL) * 8;
        const f32x4 o0 = *reinterpret_cast<const f32x4*>(stg + r * (kW + 4) + c);
        const f32x4 o1 = *reinterpret_cast<const f32x4*>(stg + r * (kW + 4) + c + 4);
        const int64_t col = c0 + wv * kW + c;
        uint32_t h[8];
        if (r0 + r >= rows) continue;
        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + (int64_t)slots[r0 + r] * p.ldy + col;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = p.ydt == DT_F16 ? f32_to_f16_bits(o0[j]) : f32_to_bf16_bits(o0[j]);
          h[4 + j] = p.ydt == DT_F16 ? f32_to_f16_bits(o1[j]) : f32_to_bf16_bits(o1[j]);
        }
        if (col + 8 <= ncols)
          *reinterpret_cast<u32x4a2*>(y) = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
        else
          for (int j = 0; j < 8; ++j)
            if (col + j < ncols) y[j] = (uint16_t)h[j];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int MODE, int MB>
void gemm_launch(const GemmArgs& a, const dim3& grid, hipStream_t st) {
  constexpr size_t lds = 3 * (16 * MB * kGemmK * 2 + kGemmN * 36) + 16 * MB * 8;
  if (a.group == 64) hipLaunchKernelGGL((k_experts_gemm<MODE, MB, 1>), grid, dim3(256), lds, st, a);
  else hipLaunchKernelGGL((k_experts_gemm<MODE, MB, 2>), grid, dim3(256), lds, st, a);   // 256: a ratio of 1 between halves
}

}  // namespace awqk

namespace awq {
using namespace awqk;

// Rows per tile for S slots over E experts: tall tiles spend the fewest
// unpacks, but a tile walks all of K, so the card has to be full of them.
// 7188 rows on 19 experts (1408 -> 1076): 84 us with 128 rows (330 tiles), 77
// with 64 (600), 83 with 32 (1200).  25956 on 29 (1408 -> 2893): 325, 344, 407
// (2600 tiles of 128).  5734 on 6 (3136 -> 2 x 47, 45 tiles of 128): 92, 69, 57.
static int gemm_tile_rows(int64_t S, int64_t E, int64_t N) {
  const int64_t avg = S / E, cols = (N + kGemmN - 1) / kGemmN;
  return avg > 96 && S / 128 * cols >= 1536 ? 128 : avg > 40 && S / 64 * cols >= 512 ? 64 : 32;
}

struct GemmSpace {
  size_t xq, pexp, ctab, plan, total;
};
static GemmSpace gemm_space(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int64_t group) {
  const int64_t S = M * top_k, xrows = down ? S : M;
  GemmSpace g;
  g.xq = 0;
  g.pexp = g.xq + align_up((size_t)xrows * (size_t)K * 2, 256);
  g.ctab = g.pexp + align_up((size_t)xrows * 4, 256);
  g.plan = g.ctab + align_up((size_t)E * (size_t)N * (size_t)(K / (group == 64 ? 64 : 128)) * 4, 256);
  g.total = g.plan + group_plan_bytes(S, E, 32);   // the lowest tiles need the most: fewer slots may take lower ones
  return g;
}

size_t experts_gemm_ws_bytes(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k) {
  return gemm_space(down, M, N, K, E, top_k, 64).total;     // the smallest group needs the most
}

// Blocks of the preparation's parts: sort, rows, constants, zero rows.
struct PrepBlocks {
  int64_t sort, rows, consts, zero;
  int64_t all() const { return sort + rows + consts + zero; }
};
static PrepBlocks prep_blocks(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int group) {
  const int64_t S = M * top_k;
  return PrepBlocks{group_chunks(S), ((down ? S : M) + 15) / 16,
                    (E * N * ((K / group + 7) / 8) + kPlanThreads - 1) / kPlanThreads, down ? 0 : (S + 15) / 16};
}

static int64_t gemm_blocks(int mode, int64_t M, int64_t N, int64_t E, int64_t top_k) {
  const int64_t per = mode == EXPERTS_SWIGLU ? kGemmN / 2 : kGemmN, cols = mode == EXPERTS_SWIGLU ? N / 2 : N;
  const int64_t tiles = group_tiles_max(M * top_k, E, gemm_tile_rows(M * top_k, E, N)) * ((cols + per - 1) / per);
  return (tiles + kXcd - 1) / kXcd * kXcd;
}

int64_t experts_gemm_threads(int mode, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int group) {
  const int64_t prep = prep_blocks(mode == EXPERTS_DOWN, M, N, K, E, top_k, group).all() * kPlanThreads;
  const int64_t gemm = gemm_blocks(mode, M, N, E, top_k) * 256;
  return prep > gemm ? prep : gemm;
}

hipError_t launch_experts_gemm(const ExpertsCall& c, void* out, int64_t ldo, void* ws, hipStream_t st) {
  const bool down = c.mode == EXPERTS_DOWN;
  const int64_t S = c.M * c.top_k;
  const GemmSpace g = gemm_space(down, c.M, c.N, c.K, c.E, c.top_k, c.group);
  const int tile = gemm_tile_rows(S, c.E, c.N);
  char* w = reinterpret_cast<char*>(ws);
  GemmArgs a{};
  a.x = c.x;
  a.K = c.K;
  a.ldx = c.ldx;
  a.N = c.N;
  a.ldy = ldo;
  a.ids = c.ids;
  a.qw = c.qw;
  a.scales = c.scales;
  a.zeros = c.zeros;
  a.y = out;
  a.xrows = down ? S : c.M;
  a.S = (int)S;
  a.E = (int)c.E;
  a.top_k = c.top_k;
  a.group = c.group;
  a.unit = c.group == 64 ? 64 : 128;
  a.ydt = down ? DT_F32 : c.ydt;
  a.xq = reinterpret_cast<uint16_t*>(w + g.xq);
  a.pexp = reinterpret_cast<int*>(w + g.pexp);
  a.ctab = reinterpret_cast<uint32_t*>(w + g.ctab);
  a.plan = group_plan_at(w + g.plan, S, c.E, tile);
  const PrepBlocks blocks = prep_blocks(down, c.M, c.N, c.K, c.E, c.top_k, c.group);
  a.b_rows = (int)blocks.sort;
  a.b_consts = a.b_rows + (int)blocks.rows;
  a.b_zero = a.b_consts + (int)blocks.consts;
  const int64_t cols = c.mode == EXPERTS_SWIGLU ? c.N / 2 : c.N;
  const unsigned pb = (unsigned)blocks.all();
  if (c.xdt == DT_F16) hipLaunchKernelGGL((k_experts_prep<DT_F16>), dim3(pb), dim3(kPlanThreads), group_plan_lds(a.E), st, a, tile, cols);
  else hipLaunchKernelGGL((k_experts_prep<DT_BF16>), dim3(pb), dim3(kPlanThreads), group_plan_lds(a.E), st, a, tile, cols);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_group_place(c.ids, S, c.E, tile, a.plan, st);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)gemm_blocks(c.mode, c.M, c.N, c.E, c.top_k));
  auto go = [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    if (tile == 128) gemm_launch<MODE, 8>(a, grid, st);
    else if (tile == 64) gemm_launch<MODE, 4>(a, grid, st);
    else gemm_launch<MODE, 2>(a, grid, st);
  };
  if (c.mode == EXPERTS_UP) go(std::integral_constant<int, EXPERTS_UP>{});
  else if (c.mode == EXPERTS_SWIGLU) go(std::integral_constant<int, EXPERTS_SWIGLU>{});
  else go(std::integral_constant<int, EXPERTS_DOWN>{});
  return hipGetLastError();
}

}  // namespace awq
