// The W4A16 product with an epilogue on the tiles of k_tiles.h
// (awq_w4a16_linear, more tokens than the memory-bound kernels take):
//   y[m][n] = act(sum_k step[n][g(k)] (q[n][k] - z[n][g(k)]) x[m][k] + bias[n]) + residual[m][n]
//   1. k_gemm_prep (the plain product's pre-pass): activation rows as fp16 under
//      an exact power of two per row, in the order the nibble unpack yields, and
//      steps and zero points group by group.
//   2. k_linear_tiles: tiles over slices of the contraction.  The matrix cores
//      multiply the activations with the exact integers (q - z) 2^-9; the sums are
//      held in units of the current group's step: a group's first stage
//      multiplies them by the last step over this one's (fp32), the end by the
//      last.  So no operand is rounded.  (Weights rounded to fp16, 13 instead of
//      9 vector instructions per eight: fp16 outputs off by 2.8e-4 of their size,
//      2.1e-4 this way; weights as two fp16 values in two products: 333 us
//      instead of 252 for 2048 tokens, 4096 -> 11008.)  Without slices the
//      sums pass LDS to lanes of eight adjacent columns and go through the
//      epilogue, with them they go to the workspace as fp32.
//   3. k_linear_reduce (slices): the slices' sums added in their order, then the
//      epilogue.
// 2048 tokens, 4096 -> 11008, bf16 with bias, gelu and pre: 252 us a call (274
// with groups of 64), bound by the matrix pipe and the vector instructions beside
// it; the plain product, which rounds the weights twice and stores one output,
// 190 to 205.  519 tokens, 4096 -> 1027, fp16 with bias and silu: 40, bound by the
// dequantization and by what surrounds the stages.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"

#include <type_traits>

#include "k_tiles.h"

namespace awqk {

// The packed weights as the tiles' operand.  Product c takes the columns
// 4 rl + c of its wave's 64, so that a lane ends with four adjacent outputs.  A
// stage holds 256 columns n of 32 bytes (64 k) in the order in which they are
// read, column 64 w + 4 r + c at place 64 w + 16 c + r (per 32 places the first
// 16 bytes of each, then the last 16), and the columns' constants (8 bytes each).
// Lane (rl, b4) reads the words 2 b4, 2 b4 + 1 of its four columns.
template <int WM>
struct LinearOp {
  static constexpr int BW = 2 / WM;
  static constexpr int WordBytes = kTileCols * kTileK / 2, Bytes = WordBytes + kTileCols * 4;
  static constexpr int VAlu = 4;
  static constexpr bool Whole = false, Units = true;
  static __device__ __forceinline__ int chunk(int st, int b4) { return 2 * b4 + st; }

  i32x4 brs, crs;
  int64_t N;
  int copies, wv, glog;
  uint32_t boff[BW], coff, wlane, clane;
  uint2 w[4];
  u32x4 c;
  uint32_t nz[4];                         // fp16(-z 2^-9) twice
  float ratio[4], last[4], any[4];        // the last unit / this one, this one, the largest step (0: the column is 0)

  __device__ __forceinline__ void init(const uint32_t* qw, int64_t n, int64_t K, int64_t n0, const uint32_t* ctab, int gl) {
    const int tid = threadIdx.x, lane = tid & 63;
    wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv & 3, rl = lane & 15, b4 = lane >> 4;
    N = n;
    glog = gl;
    const int cols = (int)(N - n0 < kTileCols ? N - n0 : kTileCols);
    brs = rsrc4(qw + n0 * (K >> 3), (uint32_t)(cols * (K >> 1)));
    crs = rsrc4(ctab + n0, (uint32_t)((((K >> glog) - 1) * N + cols) * 4));
    copies = wv == 0 ? BW + 1 : BW;
#pragma unroll
    for (int u = 0; u < BW; ++u) {
      // lane i of copy j: half i / 32 of the column at place 32 j + i % 32
      const int at = 32 * (BW * wv + u) + (lane & 31), col = (at & ~63) + 4 * (at & 15) + ((at >> 4) & 3);
      boff[u] = (uint32_t)(col * (K >> 1) + (lane >> 5) * 16);
    }
    coff = (uint32_t)(lane * 16);
    const int at = wn * 64 + rl;
    wlane = (uint32_t)((at >> 5) * 1024 + (b4 >> 1) * 512 + (at & 31) * 16 + (b4 & 1) * 8);
    clane = (uint32_t)(WordBytes + (wn * 64 + 4 * rl) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      last[i] = 1.0f;
      any[i] = 0.0f;
    }
  }
  __device__ __forceinline__ void issue(int64_t s, uint32_t lb, bool live) const {
    i32x4 b = brs, t = crs;
    b[2] = live ? b[2] : 0;
#pragma unroll
    for (int u = 0; u < BW; ++u) dma16(b, lb + (BW * wv + u) * 1024, boff[u], live ? (uint32_t)(s * 32) : 0u);
    if (wv == 0) {
      t[2] = live ? t[2] : 0;
      dma16(t, lb + WordBytes, coff, live ? (uint32_t)(((s * kTileK) >> glog) * N * 4) : 0u);
    }
  }
  __device__ __forceinline__ void load(const uint8_t* base) {
#pragma unroll
    for (int i = 0; i < 4; ++i)       // places 16 apart: halves of 256 bytes of blocks of 1 KB
      w[i] = *reinterpret_cast<const uint2*>(base + wlane + (i >> 1) * 1024 + (i & 1) * 256);
    c = *reinterpret_cast<const u32x4*>(base + clane);
#pragma unroll
    for (int i = 0; i < 4; ++i) nz[i] = __builtin_amdgcn_perm(c[i], c[i], 0x03020302u);
  }
  // whether stage s begins a group
  __device__ __forceinline__ bool fresh(int64_t s) const { return ((s * kTileK) & (((int64_t)1 << glog) - 1)) == 0; }
  // The sums' next unit: the loaded stage's steps.  A step of 0 counts as 2^-80
  // (codes masked to 0 instead: 264 us against 252 at 2048 x 4096 x 11008), which
  // keeps the ratios finite: a sum of 2^17 codes below 2^-5 times 2^14 in units of
  // 2^-80, scaled from a step of 2^16, is below 2^122.  An infinite one counts as
  // 2^60, until the end (steps()).  The quotient is corrected by its remainder:
  // equal steps give 1.
  __device__ __forceinline__ void unit() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = c[i];
      const float f = f16_to_f32(v & 0xFFFFu), size = fabsf(f);
      const float d = size == 0.0f ? 0x1p-80f : size == __builtin_inff() ? copysignf(0x1p60f, f) : f;
      any[i] = fmaxf(any[i], size);
      const float r = __builtin_amdgcn_rcpf(d), t = last[i] * r;
      ratio[i] = __builtin_fmaf(__builtin_fmaf(-t, d, last[i]), r, t);
      last[i] = d;
    }
  }
  // what the finished sums of the four columns are multiplied by
  __device__ __forceinline__ f32x4 steps() const {
    f32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = any[i] == 0.0f ? 0.0f : any[i] == __builtin_inff() ? last[i] * any[i] : last[i];
    return d;
  }
  __device__ __forceinline__ void begin(int) {}
  __device__ __forceinline__ void column(int st, int i, u32x4& codes, u32x4&) const {
    codes = once_codes(st ? w[i].y : w[i].x, nz[i]);
  }
};

template <int MB, int WM>
constexpr int kLinearStages = WM == 2 ? (MB == 8 ? 3 : 5) : (MB == 4 ? 4 : MB == 2 ? 5 : 6);

struct LinearArgs {
  const uint16_t* xq;
  const int* pm;
  const uint32_t* ctab;
  const uint32_t* qw;
  float* partial;        // [S][M][pitch]
  void* y;
  int64_t M, N, K, ldy, pitch;
  int glog, S;
};

// The tile of rows m0 on and columns n0 on, over slice bs of the contraction.
template <int MB, int WM, bool SPLIT>
__device__ __forceinline__ void linear_tile(uint8_t* tile_lds, const LinearArgs& a, const Epilogue& ep, int bs, int64_t m0,
                                            int64_t n0) {
  using Tl = Tile<MB, WM, kLinearStages<MB, WM>, LinearOp<WM>>;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv >> 2, wn = wv & 3, rl = lane & 15, b4 = lane >> 4;
  const int64_t stages = a.K / kTileK;
  const int rows = (int)(a.M - m0 < Tl::Rows ? a.M - m0 : Tl::Rows);
  LinearOp<WM> op;
  op.init(a.qw, a.N, a.K, n0, a.ctab, a.glog);
  f32x4 acc[MB][4];
  Tl::run(tile_lds, op, a.xq, m0, rows, a.K, bs * stages / a.S, (bs + 1) * stages / a.S, acc);
  const f32x4 steps = op.steps();

  // 16 x 16 layout: column 4 (lane % 16) + c, row 4 (lane / 16) + v
  const int64_t n = n0 + wn * 64 + 4 * rl, mw = m0 + wm * 16 * MB;
  const int cnt = a.N - n < 4 ? (int)(a.N > n ? a.N - n : 0) : 4;
  if constexpr (SPLIT) {
    if (cnt == 0) return;
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t m = mw + b * 16 + 4 * b4 + v;
        if (m < a.M)                                      // pitch a multiple of 8: whole fours
          *reinterpret_cast<f32x4*>(a.partial + ((int64_t)bs * a.M + m) * a.pitch + n) =
              f32x4{acc[b][0][v], acc[b][1][v], acc[b][2][v], acc[b][3][v]} * steps;
      }
  } else {
    // The sums pass the wave's own LDS area so that one copy of the epilogue's
    // code loops over them: inlined for each of the 32 rows a lane holds, its
    // fetch took longer than its work (25 of 160 us at 4096^3).
    constexpr int PB = MB * Tl::Waves * 4096 <= Tl::Lds ? MB : MB * Tl::Waves * 2048 <= Tl::Lds ? MB / 2 : MB / 4;
    static_assert(PB >= 1 && PB * Tl::Waves * 4096 <= Tl::Lds, "the waves' staging");
    f32x4* mine = reinterpret_cast<f32x4*>(tile_lds + wv * PB * 4096) + lane;
    const int c4 = cnt > 0 ? cnt : 0;
    float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ep.bias) load4_any(ep.bias, ep.bdt, n, c4, bias);
    float rn[4][4] = {};
    int pn[4] = {};
    auto fetch = [&](int64_t r) {                         // what rows r .. r + 3 of this lane need from memory
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const bool ok = r + v < a.M;
        pn[v] = ok ? a.pm[r + v] : 0;
        if (ep.res) load4_any(ep.res, ep.ydt, (r + v) * ep.ldr + n, ok ? c4 : 0, rn[v]);
      }
    };
    fetch(mw + 4 * b4);
#pragma unroll
    for (int ps = 0; ps < MB / PB; ++ps) {
#pragma unroll
      for (int b = 0; b < PB; ++b)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          mine[(b * 4 + v) * 64] = f32x4{acc[ps * PB + b][0][v], acc[ps * PB + b][1][v], acc[ps * PB + b][2][v], acc[ps * PB + b][3][v]};
#pragma unroll 1
      for (int b = 0; b < PB; ++b) {
        const int64_t m = mw + (ps * PB + b) * 16 + 4 * b4;
        float z[4][4], r[4][4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const f32x4 t = mine[(b * 4 + v) * 64];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            z[v][j] = ldexpf(t[j] * steps[j], kOnceUnit - pn[v]) + bias[j];
            r[v][j] = rn[v][j];
          }
        }
        fetch(m + 16);
        if (ep.pre) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (m + v < a.M) store4_any(ep.pre, ep.ydt, (m + v) * ep.ldp + n, c4, z[v]);
        }
        act_values(ep.act, z);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
#pragma unroll
          for (int j = 0; j < 4; ++j) z[v][j] += r[v][j];
          if (m + v < a.M) store4_any(a.y, ep.ydt, (m + v) * a.ldy + n, c4, z[v]);
        }
      }
    }
  }
}

template <int MB, int WM>
constexpr size_t kLinearLds = Tile<MB, WM, kLinearStages<MB, WM>, LinearOp<WM>>::Lds;

template <int MB, int WM, bool SPLIT>
__global__ __launch_bounds__(256 * WM) void k_linear_tiles(const LinearArgs a, const Epilogue ep) {
  using Tl = Tile<MB, WM, kLinearStages<MB, WM>, LinearOp<WM>>;
  extern __shared__ __attribute__((aligned(16))) uint8_t tile_lds[];
  int bs;
  int64_t mt, ct;
  if (!tile_item<Tl::GM>(blockIdx.x, (a.M + Tl::Rows - 1) / Tl::Rows, (a.N + kTileCols - 1) / kTileCols, a.S, bs, mt, ct)) return;
  linear_tile<MB, WM, SPLIT>(tile_lds, a, ep, bs, mt * Tl::Rows, ct * kTileCols);
}

// Two heights in one launch: the first `wide` column tiles 256 rows high, the
// others 128, so that a last round of tall tiles that would leave most compute
// units idle is spread over twice as many (2048 x 11008: 344 tall tiles on 256
// units take two rounds; 256 tall and 176 half ones 1.6).
__global__ __launch_bounds__(512) void k_linear_mixed(const LinearArgs a, const Epilogue ep, int64_t wide, int64_t wide_blocks) {
  extern __shared__ __attribute__((aligned(16))) uint8_t tile_lds[];
  int bs;
  int64_t mt, ct;
  if ((int64_t)blockIdx.x < wide_blocks) {
    if (!tile_item<4>(blockIdx.x, (a.M + 255) / 256, wide, 1, bs, mt, ct)) return;
    linear_tile<8, 2, false>(tile_lds, a, ep, 0, mt * 256, ct * kTileCols);
  } else {
    if (!tile_item<4>((int64_t)blockIdx.x - wide_blocks, (a.M + 127) / 128, (a.N + kTileCols - 1) / kTileCols - wide, 1, bs, mt, ct)) return;
    linear_tile<4, 2, false>(tile_lds, a, ep, 0, mt * 128, (wide + ct) * kTileCols);
  }
}

// Four columns per thread.
__global__ __launch_bounds__(256) void k_linear_reduce(const LinearArgs a, const Epilogue ep) {
  const int64_t per = (a.N + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * per) return;
  const int64_t m = i / per, n = (i - m * per) * 4;
  const int cnt = a.N - n < 4 ? (int)(a.N - n) : 4;
  const float* p = a.partial + m * a.pitch + n;
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.S; ++s) t += *reinterpret_cast<const f32x4*>(p + (int64_t)s * a.M * a.pitch);
  const int pw = a.pm[m];
  float z[4], b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (ep.bias) load4_any(ep.bias, ep.bdt, n, cnt, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = j < cnt ? ldexpf(t[j], kOnceUnit - pw) + b[j] : 0.0f;
  epi_store4(ep, a.y, a.ldy, m, n, cnt, z);
}

// Compute units of the current GPU.
inline int64_t linear_cus() { return awq::device_cus() > 0 ? awq::device_cus() : 256; }
inline LinearPlan linear_plan(int64_t M, int64_t N, int64_t K) { return linear_plan(M, N, K, linear_cus()); }

inline int64_t linear_pitch(int64_t N) { return (N + 7) / 8 * 8; }

template <int MB, int WM>
hipError_t linear_launch(const LinearArgs& a, const LinearPlan& p, const Epilogue& ep, hipStream_t st) {
  const dim3 grid((unsigned)p.blocks), block(256 * WM);
  if (a.S == 1) {
    hipLaunchKernelGGL((k_linear_tiles<MB, WM, false>), grid, block, (kLinearLds<MB, WM>), st, a, ep);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_linear_tiles<MB, WM, true>), grid, block, (kLinearLds<MB, WM>), st, a, ep);
  hipLaunchKernelGGL(k_linear_reduce, dim3((unsigned)((a.M * ((a.N + 3) / 4) + 255) / 256)), dim3(256), 0, st, a, ep);
  return hipGetLastError();
}

}  // namespace awqk

namespace awq {

int64_t linear_threads(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0) return 0;
  const awqk::LinearPlan p = awqk::linear_plan(M, N, K);
  const int64_t tiles = p.blocks * 256 * p.t.wm, prep = (M + (N + 15) / 16) * 256;
  return tiles > prep ? tiles : prep;
}

size_t linear_partial_bytes(int64_t M, int64_t N, int64_t K) {
  const awqk::LinearPlan p = awqk::linear_plan(M, N, K);
  return p.t.S > 1 ? align_up((size_t)p.t.S * M * awqk::linear_pitch(N) * 4, 256) : 0;
}

size_t linear_partial_bytes_upto(int64_t M, int64_t N, int64_t K) {
  const int64_t parts = awqk::tile_parts(awqk::kLinearShapes, M, N, K / awqk::kTileK, awqk::linear_cus());
  return align_up((size_t)parts * awqk::linear_pitch(N) * 4, 256);
}

hipError_t launch_linear_tiles(const uint16_t* xq, const int* pm, const uint32_t* ctab, const uint32_t* qw,
                               int64_t M, int64_t N, int64_t K, int group, float* partial, void* y, int64_t ldy,
                               const Epilogue& ep, hipStream_t st) {
  using namespace awqk;
  const LinearPlan p = linear_plan(M, N, K);
  const int glog = group == 64 ? 6 : group == 128 ? 7 : 8;
  const LinearArgs a{xq, pm, ctab, qw, partial, y, M, N, K, ldy, linear_pitch(N), glog, p.t.S};
  if (p.wide) {
    constexpr size_t lds = kLinearLds<8, 2> > kLinearLds<4, 2> ? kLinearLds<8, 2> : kLinearLds<4, 2>;
    hipLaunchKernelGGL(k_linear_mixed, dim3((unsigned)p.blocks), dim3(512), lds, st, a, ep, p.wide, p.wide_blocks);
    return hipGetLastError();
  }
#define AWQ_LT(MB, WM) return linear_launch<MB, WM>(a, p, ep, st)
  if (p.t.wm == 2) {
    if (p.t.mb == 8) AWQ_LT(8, 2);
    AWQ_LT(4, 2);
  }
  switch (p.t.mb) {
    case 4: AWQ_LT(4, 1);
    case 2: AWQ_LT(2, 1);
    default: AWQ_LT(1, 1);
  }
#undef AWQ_LT
}

}  // namespace awq
