// Routed W4A16 products for few rows per expert (include/awq.h,
// awq_w4a16_experts_up / _down): decode steps and small batches, where the
// product is bound by the chosen experts' packed words.
//
//   z[slot][n] = sum_g D[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[row(slot)][k]
//
//  * A block of 8 waves owns 64 weight rows of one expert (four 16-row tiles
//    of two waves each; a wave takes every other 256-channel pair of its
//    tile's rows) and finds the expert's slots itself by scanning the ids, 16
//    at a time, so a call needs no sorting launch and an expert without rows
//    costs one scan.
//  * With fewer slots than experts the grid has one block row per slot: every
//    16th slot of an expert takes 16 of its rows.  Otherwise one per expert,
//    its rows dealt to more blocks where there are many.
//  * v_mfma_f32_16x16x32_f16 with the tokens as the first operand (16 rows)
//    and 16 weight rows as the second: a result lane holds the weight row whose
//    words it read, so the group's step enters once, in fp32.
//  * The codes reach the matrix cores as (q - z) 2^-9, exact normal fp16 values:
//    the masked nibbles read as subnormals (q 2^-24 or q 2^-20), then one packed
//    fma per pair.  Feeding the subnormals themselves and taking z out with
//    the rows' sums saves those four of nine instructions per word, but the
//    matrix cores align a subnormal operand by its nominal exponent and drop
//    the low bits of its products: 2e-5 of a result against 2e-7.
//  * The packed words come through a per-wave LDS ring by LDS DMA, a pair of
//    128-channel units (16 rows x 128 bytes, whole lines) per step, two pairs
//    ahead.
//  * The rows' activations are staged in LDS a chunk of channels at a time (as
//    many channels as fit: 2048 for up to 8 rows, 1024 for 16), as fp16 scaled
//    by a power of two per (row, 128 channels), in the order the unpack yields;
//    beside them the chunk's steps and zero points.
//  * One token through 8 of 64 experts (2048 -> 2 x 1024, 17.6 MB of words): 8
//    us, launch and fill; 24 tokens (134 MB): 35 us, 3.8 TB/s, where a large copy
//    reaches 5.2.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_experts.h"
#include "k_rows_f16.h"

#include <type_traits>

namespace awqk {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * 64;
constexpr int kFewTiles = 4;                       // 16-row tiles per block
constexpr int kFewSlices = kFewWaves / kFewTiles;  // waves per tile
constexpr int kFewPairs = 2;                       // 256-channel pairs in flight per wave
constexpr int kFewX = 16 * (1024 + 8) * 2;         // staged activations, bytes
constexpr int kFewUnits = 16;                      // groups (of 64 or 128 channels) per chunk, at most
constexpr int kFewPitch = kFewUnits + 1;           // staged (step, zero) pairs per row
constexpr int kFewOPinv = kFewX;
constexpr int kFewOMeta = kFewOPinv + kFewUnits * 16 * 4;
constexpr int kFewORing = kFewOMeta + kFewTiles * 16 * kFewPitch * 8;
constexpr int kFewOList = kFewORing + kFewWaves * kFewPairs * 2048;
constexpr int kFewLds = kFewOList + 16 * 4 + 2 * kFewWaves * 4;   // two blocks per compute unit
static_assert(kFewLds <= 80 * 1024, "two blocks per compute unit");
static_assert(kFewORing % 16 == 0 && kFewOList % 16 == 0, "LDS regions");

struct FewArgs {
  const uint16_t* x;
  int64_t K, ldx, N, ldy;
  const int32_t* ids;
  const uint32_t* qw;
  const uint16_t* scales;
  const uint8_t* zeros;
  void* y;
  int S, E, top_k, glog, ydt, by_slot, groups;
};

// 16 bytes per lane into LDS (LDS DMA, non-temporal; an offset past the
// buffer's range writes 0).  Issued from asm, so the compiler adds no wait of
// its own before the LDS reads: the caller waits on the vector memory counter.
__device__ __forceinline__ void few_dma16(const i32x4& rs, uint32_t lds, uint32_t voff) {
  uint32_t keep;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen nt lds\n\ts_mov_b32 m0, %0"
               : "=&s"(keep) : "s"(lds), "v"(voff), "s"(rs) : "memory");
}

// MODE: EXPERTS_UP (y per slot), EXPERTS_SWIGLU (y per slot, silu(gate) * up),
// EXPERTS_DOWN (x per slot; y is the fp32 partial row of the slot).
template <int DT, int MODE, bool G64>
__global__ __launch_bounds__(kFewThreads) void k_experts_few(const FewArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  uint16_t* xs = reinterpret_cast<uint16_t*>(lds);
  float* red = reinterpret_cast<float*>(lds);                    // after the last chunk
  float* pinv = reinterpret_cast<float*>(lds + kFewOPinv);       // [128-channel unit][16 rows]
  uint2* meta = reinterpret_cast<uint2*>(lds + kFewOMeta);       // [weight row][kFewPitch]: step 2^9, -z 2^-9
  int* list = reinterpret_cast<int*>(lds + kFewOList);           // [16] slots
  int* wcount = list + 16;                                       // [2][kFewWaves]

  const int grp = blockIdx.y;
  const int64_t halfN = p.N >> 1;
  // ---- the expert
  int e;
  bool zero_rows = false;                                        // this block row zeroes the slots without an expert
  if (grp == p.groups) {
    e = -1;
    zero_rows = true;
  } else {
    e = p.by_slot ? p.ids[grp] : grp;
    if (e < 0 || e >= p.E) return;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  // ---- how many slots each wave's share of the ids holds
  const int s0 = (int)((int64_t)wv * p.S / kFewWaves), s1 = (int)((int64_t)(wv + 1) * p.S / kFewWaves);
  if (zero_rows) {
    const int64_t cols = MODE == EXPERTS_SWIGLU ? halfN : p.N;
    const int64_t per = MODE == EXPERTS_SWIGLU ? 8 * kFewTiles : 16 * kFewTiles;
    const int64_t c = (int64_t)blockIdx.x * per + (lane % per);
    for (int s = (int)blockIdx.z * kFewWaves + wv; s < p.S; s += (int)gridDim.z * kFewWaves) {
      const int id = p.ids[s];
      if ((id < 0 || id >= p.E) && lane < per && c < cols) store_out(p.y, p.ydt, (int64_t)s * p.ldy + c, 0.0f);
    }
    return;
  }
  // and, with a block row per slot, how many of them come before it
  int cnt = 0, ahead = 0;
  for (int s = s0; s < s1; s += 64) {
    const uint64_t m = __ballot(s + lane < s1 && p.ids[s + lane < s1 ? s + lane : s0] == e);
    cnt += __popcll(m);
    ahead += s >= grp ? 0 : __popcll(grp - s < 64 ? m & ((1ull << (grp - s)) - 1) : m);
  }
  if (lane == 0) {
    wcount[wv] = cnt;
    wcount[kFewWaves + wv] = ahead;
  }
  __syncthreads();
  int rows = 0, before = 0;
  ahead = 0;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    const int c = wcount[w];
    if (w < wv) before += c;
    rows += c;
    ahead += wcount[kFewWaves + w];
  }
  rows = __builtin_amdgcn_readfirstlane(rows);
  // The block's passes of 16 rows.  A block row per slot: 16 from its own on,
  // of every 16th slot; a block row per expert: dealt to gridDim.z blocks.
  const int r_first = p.by_slot ? __builtin_amdgcn_readfirstlane(ahead) : 16 * (int)blockIdx.z;
  if (p.by_slot && (r_first & 15)) return;
  const int r_step = 16 * (int)gridDim.z, r_end = p.by_slot && r_first + 16 < rows ? r_first + 16 : rows;
  if (r_first >= r_end) return;

  // ---- the block's weight rows: tile t holds rows tile_row(t) .. + 15 of the
  // expert, rows_in(t) of them; with SwiGLU tiles alternate gate, up
  const int64_t ncols = MODE == EXPERTS_SWIGLU ? halfN : p.N;
  const int tile = wv / kFewSlices, slice = wv % kFewSlices;
  auto tile_col = [&](int t) {
    return MODE == EXPERTS_SWIGLU ? ((int64_t)blockIdx.x * (kFewTiles / 2) + (t >> 1)) * 16
                                  : ((int64_t)blockIdx.x * kFewTiles + t) * 16;
  };
  auto rows_in = [&](int t) {
    const int64_t left = ncols - tile_col(t);
    return (int)(left < 0 ? 0 : left < 16 ? left : 16);
  };
  auto tile_row = [&](int t) {                     // within [0, N); for an empty tile any row
    const int64_t c = tile_col(t);
    return (c < ncols ? c : 0) + (MODE == EXPERTS_SWIGLU && (t & 1) ? halfN : 0);
  };
  const uint32_t rowb = (uint32_t)(p.K >> 1);      // bytes of a packed row
  const int GW = (int)(p.K >> p.glog);             // groups per row
  const int64_t wrow = (int64_t)e * p.N + tile_row(tile);
  const i32x4 wrs = rsrc4(reinterpret_cast<const uint8_t*>(p.qw) + wrow * rowb, (uint32_t)rows_in(tile) * rowb);
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_addr(lds) + kFewORing + (uint32_t)wv * kFewPairs * 2048);
  // A pair is two copies (rows 0..7 and 8..15, 128 bytes of each row) with
  // chunk c of row r' of half h at 16-byte slot 8 r' + (c ^ (r'/2 + 4 h)).
  const int dq = lane >> 3, ds = lane & 7;
  const uint32_t dv0 = (uint32_t)dq * rowb + (uint32_t)((ds ^ (dq >> 1)) * 16);
  const uint32_t dv1 = (uint32_t)(dq + 8) * rowb + (uint32_t)((ds ^ ((dq >> 1) | 4)) * 16);
  const int npair = (int)((p.K + 255) >> 8);       // the last may hold 64, 128 or 192 channels
  auto issue = [&](int slot, int q) {
    const uint32_t off = __builtin_amdgcn_readfirstlane(q < npair ? (uint32_t)q * 128 : kBufferOob);
    // past the row's end the copy takes the next row's words (or zeros): they
    // meet activations staged as zeros
    few_dma16(wrs, ring + (uint32_t)slot * 2048, dv0 + off);
    few_dma16(wrs, ring + (uint32_t)slot * 2048 + 1024, dv1 + off);
  };
  const uint8_t* wlds = lds + kFewORing + wv * kFewPairs * 2048 + (rl >> 3) * 1024 + (rl & 7) * 128;
  const int wsw = ((rl & 7) >> 1) | ((rl >> 3) << 2);

  for (int r0 = r_first; r0 < r_end; r0 += r_step) {
    const int nr = rows - r0 < 16 ? rows - r0 : 16;
    // ---- the pass's slots: ranks r0 .. r0 + nr - 1 among the expert's
    int run = before;
    for (int s = s0; s < s1; s += 64) {
      const bool hit = s + lane < s1 && p.ids[s + lane < s1 ? s + lane : s0] == e;
      const uint64_t m = __ballot(hit);
      const int rank = run + __popcll(m & ((1ull << lane) - 1));
      if (hit && rank >= r0 && rank < r0 + 16) list[rank - r0] = s + lane;
      run += __popcll(m);
    }
    __syncthreads();

    // channels per chunk: whole pairs, as many as fit the staged activations and the steps
    int kc = (kFewX / 2 / nr - 8) & ~255;
    constexpr int kcap = G64 ? kFewUnits * 64 : kFewUnits * 128;
    kc = kc < kcap ? kc : kcap;
    const int kall = (int)((p.K + 255) & ~(int64_t)255);
    kc = kc < kall ? kc : kall;
    const int pitch = kc + 8;

    int q = slice;                                 // this wave's next pair
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    int done = 0;                                  // pairs this wave has used: slot done % kFewPairs
    for (int c0 = 0; c0 < (int)p.K; c0 += kc) {
      if (c0) __syncthreads();                     // every wave has left the last chunk
      const int kn = (int)p.K - c0 < kc ? (int)p.K - c0 : kc;    // channels in this chunk
      // ---- the rows' activations: piece i = (row i / P, 8 channels i % P), P
      // pieces per row rounded up to whole pairs (the tail is zeros)
      const int P = ((kn + 255) & ~255) >> 3;
      for (int i = tid; i < nr * P; i += kFewThreads) {
        const int r = i / P, k8 = i - r * P;
        const int slot = list[r];
        const int64_t xrow = MODE == EXPERTS_DOWN ? slot : slot / p.top_k;
        u32x4 raw = {0, 0, 0, 0};
        if (k8 * 8 < kn) raw = ldg128(p.x + xrow * p.ldx + c0 + k8 * 8);
        float v[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[2 * c] = lo_f32<DT>(raw[c]);
          v[2 * c + 1] = hi_f32<DT>(raw[c]);
        }
        const int pe = pow2_exp_for(row16_finite_max(v));
        uint32_t h[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = f32_to_f16_bits(ldexpf(v[c], pe));
        const u32x4 o = {h[0] | (h[4] << 16), h[2] | (h[6] << 16), h[1] | (h[5] << 16), h[3] | (h[7] << 16)};
        *reinterpret_cast<u32x4*>(xs + r * pitch + k8 * 8) = o;
        if ((lane & 15) == 0) pinv[(k8 >> 4) * 16 + r] = ldexpf(1.0f, -pe);
      }
      // ---- the chunk's steps (times 2^9, undoing the operands' 2^-9) and zero
      // points, one (row, group) each; past the row's groups a step of 0
      const int ug = G64 ? 64 : 128;
      const int ng = ((kn + 255) & ~255) / ug;     // staged groups (of 64 or 128 channels)
      for (int i = tid; i < kFewTiles * 16 * kFewUnits; i += kFewThreads) {
        const int r = i / kFewUnits, u = i % kFewUnits;
        const int t = r >> 4, g = (c0 + u * ug) >> p.glog;
        uint2 m = make_uint2(0u, 0u);
        if (u < ng && g < GW && (r & 15) < rows_in(t)) {
          const int64_t at = ((int64_t)e * p.N + tile_row(t) + (r & 15)) * GW + g;
          m = make_uint2(__float_as_uint(f16_to_f32(p.scales[at]) * 512.0f), experts_nz(p.zeros[at]));
        }
        if (u < ng) meta[r * kFewPitch + u] = m;
      }
      if (c0 == 0) {
#pragma unroll
        for (int d = 0; d < kFewPairs; ++d) issue(d, q + d * kFewSlices);
      }
      __syncthreads();
      // ---- this wave's pairs of the chunk
      const int qend = (c0 + kc) >> 8;
      const uint16_t* xrow = xs + (rl < nr ? rl : nr - 1) * pitch;   // rows past nr repeat one; dropped
      const uint2* mrow = meta + (tile * 16 + rl) * kFewPitch;
      for (; q < npair && q < qend; q += kFewSlices) {
        const int slot = done & (kFewPairs - 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (kFewPairs - 1)) : "memory");
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int g = 2 * q + u - (c0 >> 7);     // unit within the chunk
          const f32x4 pv = *reinterpret_cast<const f32x4*>(pinv + g * 16 + 4 * b);
          if constexpr (!G64) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(wlds + slot * 2048 + (((4 * u + b) ^ wsw) * 16));
            const uint16_t* xp = xrow + 128 * g + 32 * b;
            const uint2 md = mrow[g];
            f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp + 8 * i), experts_unpack(w[i], md.y), part);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(__uint_as_float(md.x) * pv[v], part[v], acc[v]);
          } else {
            // words 2 b, 2 b + 1 of each 64-channel half: chunk (4 u + 2 h + b / 2), half b % 2
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 w = *reinterpret_cast<const uint2*>(
                  wlds + slot * 2048 + (((4 * u + 2 * h + (b >> 1)) ^ wsw) * 16) + (b & 1) * 8);
              const uint16_t* xp = xrow + 128 * g + 64 * h + 16 * b;
              const uint2 md = mrow[2 * g + h];
              f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp), experts_unpack(w.x, md.y), part);
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp + 8), experts_unpack(w.y, md.y), part);
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(__uint_as_float(md.x) * pv[v], part[v], acc[v]);
            }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // the slot's words are in registers
        issue(slot, q + kFewPairs * kFewSlices);
        ++done;
      }
    }
    // ---- a tile's waves meet in LDS, in slice order
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");             // the ring's last (empty) copies
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wv * 256 + (4 * b + v) * 16 + rl] = acc[v];
    __syncthreads();
    constexpr int kOut = MODE == EXPERTS_SWIGLU ? kFewTiles / 2 : kFewTiles;   // output tiles
    for (int i = tid; i < nr * kOut * 16; i += kFewThreads) {
      const int r = i / (kOut * 16), c = i % (kOut * 16);
      const int t = c >> 4, cl = c & 15;
      auto tile_sum = [&](int tl) {
        float s = red[tl * kFewSlices * 256 + r * 16 + cl];
#pragma unroll
        for (int k = 1; k < kFewSlices; ++k) s += red[(tl * kFewSlices + k) * 256 + r * 16 + cl];
        return s;
      };
      const int64_t col = (int64_t)blockIdx.x * kOut * 16 + c;
      if (col >= ncols) continue;
      float out;
      if constexpr (MODE == EXPERTS_SWIGLU) out = swiglu(tile_sum(2 * t), tile_sum(2 * t + 1));
      else out = tile_sum(t);
      const int64_t at = (int64_t)list[r] * p.ldy + col;
      if constexpr (MODE == EXPERTS_DOWN) reinterpret_cast<float*>(p.y)[at] = out;
      else store_out(p.y, p.ydt, at, out);
    }
    __syncthreads();                               // red and list are free again
  }
}

// down for single tokens: one block of 8 waves per (token, 16 weight rows)
// forms the whole weighted sum, so nothing meets in memory and there is one
// launch.  The waves share the token's slots and, with fewer slots than waves,
// a slot's channels; each takes chunks of four 256-channel pairs (16 rows x
// 1024 channels) whose words, constants and activations are all on their way
// together, and multiplies the one row with the matrix cores (every operand
// row repeats it).  8 of 64 experts, 1024 -> 2048: 6.7 us, where few-row blocks
// and the sum in a second launch take 7 + 4.7 us.
constexpr int kTokenPairs = 4;                     // pairs per chunk
constexpr int kTokenX = kTokenPairs * 256 * 2;     // a wave's staged activations, bytes
constexpr int kTokenMeta = 16 * 17 * 8;            // its steps and zero points
constexpr int kTokenWave = kTokenPairs * 2048 + kTokenX + kTokenPairs * 2 * 4 + kTokenMeta;
static_assert(kTokenWave % 16 == 0, "LDS regions");
constexpr int kTokenLds = kFewWaves * kTokenWave + kFewWaves * 16 * 4;

template <int DT, bool G64>
__global__ __launch_bounds__(kFewThreads) void k_experts_token(const FewArgs p, const float* __restrict__ weights,
                                                               int slices) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  uint8_t* mine = lds + wv * kTokenWave;                         // ring, activations, 2^-p per unit, constants
  uint16_t* xs = reinterpret_cast<uint16_t*>(mine + kTokenPairs * 2048);
  float* pinv = reinterpret_cast<float*>(mine + kTokenPairs * 2048 + kTokenX);
  uint2* meta = reinterpret_cast<uint2*>(mine + kTokenPairs * 2048 + kTokenX + kTokenPairs * 2 * 4);   // [row][17]
  float* red = reinterpret_cast<float*>(lds + kFewWaves * kTokenWave);
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_addr(mine));
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nrows = (int)(p.N - n0 < 16 ? p.N - n0 : 16);
  const int m = blockIdx.y;
  const uint32_t rowb = (uint32_t)(p.K >> 1);
  const int GW = (int)(p.K >> p.glog);
  const int npair = (int)((p.K + 255) >> 8);
  const int dq = lane >> 3, ds = lane & 7;
  const uint32_t dv0 = (uint32_t)dq * rowb + (uint32_t)((ds ^ (dq >> 1)) * 16);
  const uint32_t dv1 = (uint32_t)(dq + 8) * rowb + (uint32_t)((ds ^ ((dq >> 1) | 4)) * 16);
  const uint8_t* wlds = mine + (rl >> 3) * 1024 + (rl & 7) * 128;
  const int wsw = ((rl & 7) >> 1) | ((rl >> 3) << 2);
  const int sl = wv % slices;
  const int q0 = sl * npair / slices, q1 = (sl + 1) * npair / slices;
  constexpr int ug = G64 ? 64 : 128, kU = kTokenPairs * 256 / ug;  // channels per constant, constants per row and chunk

  float total = 0.0f;
  for (int j = wv / slices; j < p.top_k; j += kFewWaves / slices) {
    const int slot = m * p.top_k + j;
    const int e = __builtin_amdgcn_readfirstlane(p.ids[slot]);
    if (e < 0 || e >= p.E) continue;
    const float wt = weights[slot];
    const int64_t w0 = (int64_t)e * p.N + n0;
    const i32x4 wrs = rsrc4(reinterpret_cast<const uint8_t*>(p.qw) + w0 * rowb, (uint32_t)nrows * rowb);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int qc = q0; qc < q1; qc += kTokenPairs) {
      const int c0 = qc * 256;
      const int cend = (q1 * 256 < (int)p.K ? q1 * 256 : (int)p.K);   // the slice's channels end here
      // ---- everything the chunk needs, on its way together
      u32x4 raw[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = c0 + (lane + 64 * i) * 8;
        raw[i] = ldg128(p.x + (int64_t)slot * p.ldx + (k < cend ? k : 0));
        if (k >= cend) raw[i] = u32x4{0, 0, 0, 0};
      }
      uint32_t sv[kU / 4], zv[kU / 4];
#pragma unroll
      for (int i = 0; i < kU / 4; ++i) {           // entry (row, unit) = (i 4 + lane / 16, lane % 16) or halves of it
        const int at = lane + 64 * i, r = at / kU, g = (c0 + (at % kU) * ug) >> p.glog;
        const bool in = r < nrows && g < GW;
        const int64_t a = in ? (w0 + r) * GW + g : 0;
        sv[i] = in ? p.scales[a] : 0u;
        zv[i] = in ? p.zeros[a] : 0u;
      }
#pragma unroll
      for (int d = 0; d < kTokenPairs; ++d) {
        const uint32_t off = __builtin_amdgcn_readfirstlane(qc + d < q1 ? (uint32_t)(qc + d) * 128 : kBufferOob);
        few_dma16(wrs, ring + (uint32_t)d * 2048, dv0 + off);
        few_dma16(wrs, ring + (uint32_t)d * 2048 + 1024, dv1 + off);
      }
      // ---- activations: fp16 scaled by a power of two per 128 channels
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[2 * c] = lo_f32<DT>(raw[i][c]);
          v[2 * c + 1] = hi_f32<DT>(raw[i][c]);
        }
        const int pe = pow2_exp_for(row16_finite_max(v));
        uint32_t h[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = f32_to_f16_bits(ldexpf(v[c], pe));
        *reinterpret_cast<u32x4*>(xs + (lane + 64 * i) * 8) =
            u32x4{h[0] | (h[4] << 16), h[2] | (h[6] << 16), h[1] | (h[5] << 16), h[3] | (h[7] << 16)};
        if ((lane & 15) == 0) pinv[(lane >> 4) + 4 * i] = ldexpf(1.0f, -pe);
      }
#pragma unroll
      for (int i = 0; i < kU / 4; ++i) {
        const int at = lane + 64 * i;
        meta[at / kU * 17 + at % kU] = make_uint2(__float_as_uint(f16_to_f32(sv[i]) * 512.0f), experts_nz(zv[i]));
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int d = 0; d < kTokenPairs; ++d) {
        if (qc + d >= q1) break;                   // wave-uniform
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int g = 2 * d + u;
          const float pv = pinv[g];
          if constexpr (!G64) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(wlds + d * 2048 + (((4 * u + b) ^ wsw) * 16));
            const uint16_t* xp = xs + 128 * g + 32 * b;
            const uint2 md = meta[rl * 17 + g];
            f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp + 8 * i), experts_unpack(w[i], md.y), part);
            acc[0] = __builtin_fmaf(__uint_as_float(md.x) * pv, part[0], acc[0]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 w = *reinterpret_cast<const uint2*>(
                  wlds + d * 2048 + (((4 * u + 2 * h + (b >> 1)) ^ wsw) * 16) + (b & 1) * 8);
              const uint16_t* xp = xs + 128 * g + 64 * h + 16 * b;
              const uint2 md = meta[rl * 17 + 2 * g + h];
              f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp), experts_unpack(w.x, md.y), part);
              part = mfma16h(*reinterpret_cast<const u32x4*>(xp + 8), experts_unpack(w.y, md.y), part);
              acc[0] = __builtin_fmaf(__uint_as_float(md.x) * pv, part[0], acc[0]);
            }
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");         // the chunk is in registers: its LDS is free
      __builtin_amdgcn_wave_barrier();
    }
    total = __builtin_fmaf(wt, acc[0], total);
  }
  if (b == 0) red[wv * 16 + rl] = total;
  __syncthreads();
  if (tid < nrows) {
    float s = red[tid];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += red[w * 16 + tid];
    store_out(p.y, p.ydt, (int64_t)m * p.ldy + n0 + tid, s);
  }
}

// y[m] = sum_j w[m][j] P[m top_k + j] over the slots that have an expert, in
// slot order.  Four outputs per thread (P's rows are padded to a multiple of 4).
template <int YDT>
__global__ __launch_bounds__(256) void k_experts_combine(const float* __restrict__ P, int64_t ldp,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int top_k, int E,
                                                         int64_t M, int64_t N, void* __restrict__ y, int64_t ldy) {
  const int64_t n4 = (N + 3) >> 2;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * n4; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / n4, n = (i - m * n4) * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < top_k; ++j) {
      const int id = ids[m * top_k + j];
      if (id < 0 || id >= E) continue;
      const float w = weights[m * top_k + j];
      const f32x4 v = *reinterpret_cast<const f32x4*>(P + (m * top_k + j) * ldp + n);
  #pragma unroll
      for (int c = 0; c < 4; ++c) s[c] = __builtin_fmaf(w, v[c], s[c]);
    }
    if (n + 4 <= N) {
      if constexpr (YDT == DT_F32)
        *reinterpret_cast<u32x4a4*>(reinterpret_cast<float*>(y) + m * ldy + n) = __builtin_bit_cast(u32x4, s);
      else
        *reinterpret_cast<u32x2a2*>(reinterpret_cast<uint16_t*>(y) + m * ldy + n) =
            u32x2a2{from_f32<YDT>(s[0]) | (from_f32<YDT>(s[1]) << 16), from_f32<YDT>(s[2]) | (from_f32<YDT>(s[3]) << 16)};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < N) store_out(y, YDT, m * ldy + n + c, s[c]);
    }
  }
}

// Waves per slot of k_experts_token (0: the few-row kernel and a second
// launch).  Few enough slots that two seldom share an expert (whose words would be
// read twice), and at most two chunks per wave and slot.
int token_slices(int64_t S, int64_t E, int64_t K, int top_k) {
  int s = 1;
  while (s * 2 * top_k <= kFewWaves) s *= 2;
  const int64_t pairs = (K + 255) / 256;
  return 2 * S <= E && (pairs + s - 1) / s <= 2 * kTokenPairs ? s : 0;
}

template <int DT, int MODE>
void few_launch(const FewArgs& a, const dim3& grid, hipStream_t st) {
  if (a.glog == 6) hipLaunchKernelGGL((k_experts_few<DT, MODE, true>), grid, dim3(kFewThreads), kFewLds, st, a);
  else hipLaunchKernelGGL((k_experts_few<DT, MODE, false>), grid, dim3(kFewThreads), kFewLds, st, a);
}

}  // namespace awqk

namespace awq {
using namespace awqk;

static int64_t partial_ld(int64_t N) { return (N + 3) / 4 * 4; }

// Few rows per expert (this file) or tiles (k_experts_gemm.hip): few rows per
// expert, or 512 blocks (two per CU) do all 16-row passes at once while a
// tile's one block walks all of K.  64 experts: at 3 rows each (2048 -> 2 x
// 1024) 37 us against 43 us in tiles, at 12 rows (1024 -> 2049, 1650 blocks)
// 62 us against 45 us.  344 rows on each of 5 (3200 -> 2 x 10, 110 blocks) 27
// us against 45 us, 18 on each of 34 (2048 -> 231, 220 blocks) 24 us against 37
// us; 34 on each of 16 (256 -> 1524, 1000 blocks) 23 us against 20 us.
static bool few_rows(int64_t S, int64_t E, int64_t N) {
  return S <= 4096 && (S <= 6 * E || (S / 16 + E / 2 + 1) * ((N + 63) / 64) <= 512);
}

// Blocks that share an expert's rows, 16 at a time: twice the even share.
static unsigned few_deal(int64_t S, int64_t E) {
  if (S < E) return 1;                             // block rows per slot
  const int64_t z = (S / E + 7) / 8;
  return (unsigned)(z < 1 ? 1 : z > 256 ? 256 : z);
}

// The fp32 rows per slot that down adds up.
static size_t partial_bytes(bool down, int64_t S, int64_t N) {
  return down ? align_up((size_t)S * (size_t)partial_ld(N) * 4, 256) : 0;
}

size_t experts_ws_bytes(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k) {
  const int64_t S = M * top_k;
  if (down && token_slices(S, E, K, (int)top_k)) return 0;
  return partial_bytes(down, S, N) + (few_rows(S, E, N) ? 0 : experts_gemm_ws_bytes(down, M, N, K, E, top_k));
}

// (The few-row forms' grids are at most 32 N in any direction, and N K < 2^32.)
int64_t experts_threads(int mode, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int group) {
  const int64_t S = M * top_k;
  if (few_rows(S, E, N) || (mode == EXPERTS_DOWN && token_slices(S, E, K, (int)top_k))) return 0;
  return experts_gemm_threads(mode, M, N, K, E, top_k, group);
}

hipError_t launch_experts(const ExpertsCall& c, void* ws, hipStream_t st) {
  const int64_t S = c.M * c.top_k;
  const bool down = c.mode == EXPERTS_DOWN;
  void* out = down ? ws : c.y;                     // down: fp32 rows per slot first
  const int64_t ldo = down ? partial_ld(c.N) : c.ldy;
  hipError_t e;
  if (const int slices = down ? token_slices(S, c.E, c.K, c.top_k) : 0) {
    const FewArgs a{c.x, c.K, c.ldx, c.N, c.ldy, c.ids, c.qw, c.scales, c.zeros, c.y, (int)S, (int)c.E, c.top_k,
                    c.group == 64 ? 6 : c.group == 128 ? 7 : 8, c.ydt, 0, 0};
    const dim3 grid((unsigned)((c.N + 15) / 16), (unsigned)c.M), block(kFewThreads);
    const bool bf = c.xdt == DT_BF16, g64 = c.group == 64;
    if (bf && g64) hipLaunchKernelGGL((k_experts_token<DT_BF16, true>), grid, block, kTokenLds, st, a, c.weights, slices);
    else if (bf) hipLaunchKernelGGL((k_experts_token<DT_BF16, false>), grid, block, kTokenLds, st, a, c.weights, slices);
    else if (g64) hipLaunchKernelGGL((k_experts_token<DT_F16, true>), grid, block, kTokenLds, st, a, c.weights, slices);
    else hipLaunchKernelGGL((k_experts_token<DT_F16, false>), grid, block, kTokenLds, st, a, c.weights, slices);
    return hipGetLastError();
  }
  if (!few_rows(S, c.E, c.N)) {
    e = launch_experts_gemm(c, out, ldo, reinterpret_cast<char*>(ws) + partial_bytes(down, S, c.N), st);
  } else {
    const FewArgs a{c.x, c.K, c.ldx, c.N, ldo, c.ids, c.qw, c.scales, c.zeros, out, (int)S, (int)c.E, c.top_k,
                    c.group == 64 ? 6 : c.group == 128 ? 7 : 8, c.ydt, S < c.E, (int)(S < c.E ? S : c.E)};
    const int64_t cols = c.mode == EXPERTS_SWIGLU ? c.N / 2 : c.N;
    const int64_t per = c.mode == EXPERTS_SWIGLU ? 8 * kFewTiles : 16 * kFewTiles;
    const dim3 grid((unsigned)((cols + per - 1) / per), (unsigned)(a.groups + (down ? 0 : 1)), few_deal(S, c.E));
    const bool bf = c.xdt == DT_BF16;
    if (c.mode == EXPERTS_UP) bf ? few_launch<DT_BF16, EXPERTS_UP>(a, grid, st) : few_launch<DT_F16, EXPERTS_UP>(a, grid, st);
    else if (c.mode == EXPERTS_SWIGLU) bf ? few_launch<DT_BF16, EXPERTS_SWIGLU>(a, grid, st) : few_launch<DT_F16, EXPERTS_SWIGLU>(a, grid, st);
    else bf ? few_launch<DT_BF16, EXPERTS_DOWN>(a, grid, st) : few_launch<DT_F16, EXPERTS_DOWN>(a, grid, st);
    e = hipGetLastError();
  }
  if (e != hipSuccess || !down) return e;
  int64_t blocks = (c.M * ((c.N + 3) / 4) + 255) / 256;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  auto combine = [&](auto y) {
    hipLaunchKernelGGL((k_experts_combine<decltype(y)::value>), dim3((unsigned)blocks), dim3(256), 0, st, (const float*)ws,
                       ldo, c.ids, c.weights, c.top_k, (int)c.E, c.M, c.N, c.y, c.ldy);
  };
  if (c.ydt == DT_F32) combine(std::integral_constant<int, DT_F32>{});
  else if (c.ydt == DT_F16) combine(std::integral_constant<int, DT_F16>{});
  else combine(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError();
}

}  // namespace awq
