// The gradient of the W4A16 product's input (awq_w4a16_gemm_dx):
//   dx[m][k] = sum_n dz[m][n] step[n][g(k)] (q[n][k] - z[n][g(k)])
// The same packed weights as the product, contracted over their rows.  A
// matrix-core operand wants eight consecutive values along the contraction in
// a lane, and a packed word holds eight along k: a lane reads the words of
// eight consecutive rows n at one place, takes the same half (four codes) of
// each, and a byte permutation puts the halves of rows n and n + 1 side by
// side, so that the masks which pull codes out of one word for the product
// (nibbles as fp16 subnormals) here give pairs along n.  Four columns k come
// out of it at once; a 16 x 16 x 32 product takes column 4 (lane % 16) + c for
// c = 0..3, so a lane ends with four adjacent outputs.
//
//   1. k_dx_consts: per row n an exact power of two e_n with
//      max_g |step| 2^e_n in [2^14, 2^15), the constants fp16(step 2^e_n) and
//      fp16(-z 2^-9) in pairs along n, and 2^-e_n (with the codes' 2^9).
//   2. k_dx_rows: dz[m][n] 2^-e_n as fp16 under one power of two per row m
//      (exact for what lies within 2^28 of the row's largest), padded with
//      zeros to a multiple of 64.
//   3. k_gemm_dx: the tiles of k_tiles.h, over slices of the contraction where
//      the tiles alone leave compute units without work.  A weight, up to 15
//      bits, is the sum of two fp16 values and meets dz in two products: with one,
//      rounded to 11 bits, an fp16 dx was off by 2.8e-4 of its size, 2.1e-4 with
//      all bits, and an fp32 dx showed all of it.
//   4. k_dx_reduce where the contraction is split: the slices' fp32 sums added
//      in their order.
// 2048 rows, 11008 -> 4096, bf16: 294 us a call (235 with one product), bound by
// the matrix pipe: 1.3 PFLOP/s of products, what a large library product
// reaches.  37 rows, 4096 -> 11008, fp16: 39 us (35) against 4.5 for the packed
// words alone: a stage costs 1 us whatever is in its rows, the dequantization and
// its products.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"
#include "k_rows_f16.h"

#include <type_traits>

#include "k_tiles.h"

namespace awqk {

constexpr int kDxCols = kTileCols;        // tile columns (k)
constexpr int kDxN = kTileK;              // contraction per stage
constexpr int kDxB = kDxN * kDxCols / 2;  // packed bytes per stage
constexpr int kDxC = 1024;                // constants per stage: up to 4 groups x 64 rows x 4 bytes

// Rows n in chunks of eight: ctab[g][n / 8] = the eight steps (four pairs),
// then the eight zero points.  A block takes 16 rows: their steps and zero
// points are read in whole lines into LDS (16 x kDxCh groups at a time), 16
// lanes find a row's largest step, and the table leaves in pieces of 64 bytes.
constexpr int kDxCh = 128;

__global__ __launch_bounds__(256) void k_dx_consts(const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                                                   int64_t N, int64_t Np, int64_t G, float* __restrict__ inv,
                                                   uint16_t* __restrict__ ctab) {
  __shared__ uint16_t sl[16][kDxCh + 2];
  __shared__ uint8_t zl[16][kDxCh + 4];
  __shared__ int es[16];
  const int tid = threadIdx.x;
  const int64_t n0 = (int64_t)blockIdx.x * 16;                   // < Np, a multiple of 64
  const int rows = (int)(N - n0 < 16 ? (N > n0 ? N - n0 : 0) : 16);
  auto load = [&](int64_t g0, int ng) {                          // groups g0 .. g0 + ng - 1 of the rows
    // a wave: four rows, all loads ahead of the LDS writes (rows and groups
    // past the end read the block's first ones)
    constexpr int H = kDxCh / 64;
    const int lane = tid & 63, wv = tid >> 6;
    uint16_t s[4][H];
    uint8_t z[4][H];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int r = 4 * wv + i, g = 64 * h + lane;
        const int64_t at = (n0 + (r < rows ? r : 0)) * G + g0 + (g < ng ? g : 0);
        s[i][h] = rows > 0 ? scales[at] : 0;
        z[i][h] = rows > 0 ? zeros[at] : 0;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        sl[4 * wv + i][64 * h + lane] = s[i][h];
        zl[4 * wv + i][64 * h + lane] = z[i][h];
      }
  };
  const int rr = tid >> 4, pp = tid & 15;
  float mx = 0.0f;
  for (int64_t g0 = 0; g0 < G; g0 += kDxCh) {
    const int ng = (int)(G - g0 < kDxCh ? G - g0 : kDxCh);
    if (g0 > 0) __syncthreads();
    load(g0, ng);
    __syncthreads();
    if (rr < rows)
      for (int g = pp; g < ng; g += 16) mx = fmaxf(mx, step_size<true>(sl[rr][g]));
  }
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 16));
  if (pp == 0) {
    const int e = step_pow<true>(mx);
    es[rr] = e;
    inv[n0 + rr] = rr < rows ? ldexpf(1.0f, -sum_pow<true>(e)) : 0.0f;
  }
  for (int64_t g0 = 0; g0 < G; g0 += kDxCh) {
    const int ng = (int)(G - g0 < kDxCh ? G - g0 : kDxCh);
    __syncthreads();
    if (G > kDxCh) {                                             // one chunk: still there
      load(g0, ng);
      __syncthreads();
    }
    // 16 words per group: of chunk c = w / 8, word w % 8 (0..3 steps, 4..7 zero points of a pair)
    for (int i = tid; i < ng * 16; i += 256) {
      const int g = i >> 4, w = i & 15, r = (w >> 3) * 8 + (w & 3) * 2;
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (r + j >= rows) continue;
        const uint32_t h = w & 4 ? once_zero(zl[r + j][g]) & 0xFFFFu : once_step(ldexpf(f16_to_f32(sl[r + j][g]), es[r + j]));
        v |= h << (16 * j);
      }
      reinterpret_cast<uint32_t*>(ctab)[(g0 + g) * Np + n0 + w] = v;
    }
  }
}

// One row of dz per block of 512 threads, in registers up to 512 KEEP chunks
// of eight values (KEEP = 0: longer, read twice).
template <int DT, int KEEP>
__global__ __launch_bounds__(512) void k_dx_rows(const uint16_t* __restrict__ dz, int64_t N, int64_t Np, int64_t ld,
                                                 const float* __restrict__ inv, uint16_t* __restrict__ out,
                                                 int* __restrict__ pexp) {
  __shared__ float wmax[8];
  const int64_t m = blockIdx.x, nch = Np >> 3;
  auto load = [&](int64_t c, float (&v)[8]) {
    const int64_t n = c * 8;
    load8_any(dz, DT, m * ld + n, N - n < 8 ? (int)(N > n ? N - n : 0) : 8, v);
    const f32x4 a = *reinterpret_cast<const f32x4*>(inv + n), b = *reinterpret_cast<const f32x4*>(inv + n + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] *= a[j];
      v[4 + j] *= b[j];
    }
  };
  auto size = [](const float (&v)[8], float am) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = fabsf(v[j]);
      am = s < __builtin_inff() ? fmaxf(am, s) : am;             // a row's power goes by its finite values
    }
    return am;
  };
  auto store = [&](int64_t c, const float (&v)[8], int p) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = f32_to_f16_bits(ldexpf(v[2 * j], p)) | (f32_to_f16_bits(ldexpf(v[2 * j + 1], p)) << 16);
    *reinterpret_cast<u32x4*>(out + m * Np + c * 8) = o;
  };
  auto row_exp = [&](float am) {
    am = wave_max(am);
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = am;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) am = fmaxf(am, wmax[w]);
    const int p = pow2_exp_for(am);
    if (threadIdx.x == 0) pexp[m] = p;
    return p;
  };
  float am = 0.0f;
  if constexpr (KEEP > 0) {
    float v[KEEP > 0 ? KEEP : 1][8];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int64_t c = threadIdx.x + 512 * i;
      if (c < nch) {
        load(c, v[i]);
        am = size(v[i], am);
      }
    }
    const int p = row_exp(am);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int64_t c = threadIdx.x + 512 * i;
      if (c < nch) store(c, v[i], p);
    }
  } else {
    for (int64_t c = threadIdx.x; c < nch; c += 512) {
      float v[8];
      load(c, v);
      am = size(v, am);
    }
    const int p = row_exp(am);
    for (int64_t c = threadIdx.x; c < nch; c += 512) {
      float v[8];
      load(c, v);
      store(c, v, p);
    }
  }
}

template <int DT>
void dx_rows(const void* dz, int64_t M, int64_t N, int64_t Np, int64_t ld, const float* inv, uint16_t* out, int* pexp,
             hipStream_t st) {
  const dim3 grid((unsigned)M), block(512);
  const uint16_t* d = (const uint16_t*)dz;
  if (Np <= 4096) hipLaunchKernelGGL((k_dx_rows<DT, 1>), grid, block, 0, st, d, N, Np, ld, inv, out, pexp);
  else if (Np <= 8192) hipLaunchKernelGGL((k_dx_rows<DT, 2>), grid, block, 0, st, d, N, Np, ld, inv, out, pexp);
  else if (Np <= 16384) hipLaunchKernelGGL((k_dx_rows<DT, 4>), grid, block, 0, st, d, N, Np, ld, inv, out, pexp);
  else hipLaunchKernelGGL((k_dx_rows<DT, 0>), grid, block, 0, st, d, N, Np, ld, inv, out, pexp);
}

// The packed weights as the tiles' operand.  A stage holds 64 rows n of 128
// bytes (256 k; row n's 16-byte chunk c at c ^ 2 (n / 8 mod 4), so that the four
// rows a read meets lie in different banks) and, per group of the tile, the 64
// rows' constants.  A lane (rl, b4) owns the columns 4 rl .. 4 rl + 3 of its
// wave's 64: half rl % 2 of word 8 wn + rl / 2.
template <int WM>
struct DxOp {
  static constexpr int BW = 2 / WM;       // copies of packed words per wave
  static constexpr int Bytes = kDxB + kDxC;
  static constexpr int VAlu = 4;
  static constexpr bool Whole = true, Units = false;
  static __device__ __forceinline__ int chunk(int st, int b4) { return 4 * st + b4; }

  const uint8_t* qw;
  int64_t N, KB;                          // rows, bytes of a packed row
  i32x4 crs;
  int copies, wv;
  uint32_t boff[BW], coff, wlane, clane, sel;
  uint32_t w[2][8];                       // the stage's words and constants
  u32x4 cm[2], cz[2];
  uint32_t p[4], p8[4], mh[4], ml[4];

  __device__ __forceinline__ void init(const uint32_t* words, int64_t n, int64_t K, int64_t k0, const uint16_t* ctab,
                                       int64_t Np, int glog) {
    const int tid = threadIdx.x, lane = tid & 63;
    wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv & 3, rl = lane & 15, b4 = lane >> 4;
    qw = reinterpret_cast<const uint8_t*>(words);
    N = n;
    KB = K >> 1;
    const int64_t G = K >> glog, g0 = k0 >> glog, left = G - g0;
    const int per = kDxCols >> glog, ng = (int)(left < per ? left : per);
    crs = rsrc4(ctab + g0 * Np * 2, (uint32_t)(ng * Np * 4));
    copies = wv == 0 ? BW + 1 : BW;
    // lane i of copy j = BW wv + u: row 8 j + i / 8; constants: group i / 16, piece i % 16
#pragma unroll
    for (int u = 0; u < BW; ++u) {
      const int j = BW * wv + u;
      boff[u] = (uint32_t)((8 * j + (lane >> 3)) * KB + k0 / 2 + (((lane & 7) ^ (2 * (j & 3))) * 16));
    }
    coff = (uint32_t)((lane >> 4) * Np * 4 + (lane & 15) * 16);
    const int word = wn * 8 + (rl >> 1);
    wlane = (uint32_t)(b4 * 1024 + (((word >> 2) ^ (2 * b4)) * 16) + (word & 3) * 4);
    clane = (uint32_t)(kDxB + ((wn * 64) >> glog) * 256 + b4 * 32);
    sel = (rl & 1) ? 0x07060302u : 0x05040100u;
  }
  __device__ __forceinline__ void issue(int64_t s, uint32_t lb, bool live) const {
    // the stage's rows of W: a descriptor of their own, so that no offset grows with N
    const int64_t left = N - s * kDxN;
    const i32x4 brs = rsrc4(qw + (live ? s * kDxN * KB : 0), live ? (uint32_t)((left < kDxN ? left : kDxN) * KB) : 0u);
#pragma unroll
    for (int u = 0; u < BW; ++u) dma16(brs, lb + (BW * wv + u) * 1024, boff[u], 0);
    if (wv == 0) {
      i32x4 c = crs;
      c[2] = live ? c[2] : 0;
      dma16(c, lb + kDxB, coff, live ? (uint32_t)(s * kDxN * 4) : 0u);
    }
  }
  __device__ __forceinline__ void load(const uint8_t* base) {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      cm[st] = *reinterpret_cast<const u32x4*>(base + clane + st * 128);
      cz[st] = *reinterpret_cast<const u32x4*>(base + clane + st * 128 + 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[st][j] = *reinterpret_cast<const uint32_t*>(base + wlane + st * 4096 + j * 128);
    }
  }
  // the lane's halves of rows n and n + 1 side by side
  __device__ __forceinline__ void begin(int st) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = __builtin_amdgcn_perm(w[st][2 * j + 1], w[st][2 * j], sel);
      p8[j] = p[j] >> 8;
      once_parts(cm[st][j], mh[j], ml[j]);
    }
  }
  __device__ __forceinline__ void column(int st, int c, u32x4& hi, u32x4& lo) const {
    const f16x2 scale = as_f16x2(c & 1 ? 0x68006800u : 0x78007800u);       // 2^11, 2^15
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = (c & 2 ? p8[j] : p[j]) & (c & 1 ? 0x00F000F0u : 0x000F000Fu), z = cz[st][j];
      const f16x2 code = __builtin_elementwise_fma(as_f16x2(v), scale, as_f16x2(z));
      hi[j] = __builtin_bit_cast(uint32_t, code * as_f16x2(mh[j]));
      lo[j] = __builtin_bit_cast(uint32_t, code * as_f16x2(ml[j]));
    }
  }
};

// Stages in LDS: what 160 KB hold with one block per compute unit for tall
// tiles, with two for the small ones.
template <int MB, int WM>
constexpr int kDxStages = WM == 2 ? (MB == 8 ? 3 : 6) : (MB == 4 ? 4 : MB == 2 ? 5 : 6);

// MB: 16-row blocks per wave, WM: waves along the rows.  S slices of the contraction; SPLIT: fp32 sums to
// partial [S][M][K] instead of dx.
template <int MB, int WM, bool SPLIT>
__global__ __launch_bounds__(256 * WM) void k_gemm_dx(const uint16_t* __restrict__ xq, const int* __restrict__ pm, int64_t M,
                                                 int64_t Np, const uint32_t* __restrict__ qw, int64_t N, int64_t K,
                                                 const uint16_t* __restrict__ ctab, int glog, int S,
                                                 float* __restrict__ partial, void* __restrict__ dx, int dxt,
                                                 int64_t lddx) {
  using Tl = Tile<MB, WM, kDxStages<MB, WM>, DxOp<WM>>;
  extern __shared__ __attribute__((aligned(16))) uint8_t tile_lds[];
  int bs;
  int64_t m0, k0;
  if (!tile_item<Tl::GM>(blockIdx.x, (M + Tl::Rows - 1) / Tl::Rows, (K + kDxCols - 1) / kDxCols, S, bs, m0, k0)) return;
  m0 *= Tl::Rows;
  k0 *= kDxCols;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv >> 2, wn = wv & 3, rl = lane & 15, b4 = lane >> 4;
  const int64_t stages = Np / kDxN;
  const int rows = (int)(M - m0 < Tl::Rows ? M - m0 : Tl::Rows);
  DxOp<WM> op;
  op.init(qw, N, K, k0, ctab, Np, glog);
  f32x4 acc[MB][4];
  Tl::run(tile_lds, op, xq, m0, rows, Np, bs * stages / S, (bs + 1) * stages / S, acc);

  // 16 x 16 layout: column lane % 16 of product c is k 4 (lane % 16) + c, row 4 (lane / 16) + v
  const int64_t k = k0 + wn * 64 + 4 * rl;
  if (k >= K) return;
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + wm * 16 * MB + a * 16 + 4 * b4 + v;
      if (m >= M) continue;
      const float o[4] = {acc[a][0][v], acc[a][1][v], acc[a][2][v], acc[a][3][v]};
      if constexpr (SPLIT) {
        *reinterpret_cast<f32x4*>(partial + ((int64_t)bs * M + m) * K + k) = f32x4{o[0], o[1], o[2], o[3]};
      } else {
        const int p = -pm[m];
        const float u[4] = {ldexpf(o[0], p), ldexpf(o[1], p), ldexpf(o[2], p), ldexpf(o[3], p)};
        store4_any(dx, dxt, m * lddx + k, 4, u);
      }
    }
}

__global__ __launch_bounds__(256) void k_dx_reduce(const float* __restrict__ partial, int S, int64_t M, int64_t K,
                                                   const int* __restrict__ pm, void* __restrict__ dx, int dxt,
                                                   int64_t lddx) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= M * K) return;
  const int64_t m = i / K, k = i - m * K;
  f32x4 s = *reinterpret_cast<const f32x4*>(partial + i);
  for (int j = 1; j < S; ++j) s += *reinterpret_cast<const f32x4*>(partial + (int64_t)j * M * K + i);
  const int p = -pm[m];
  const float u[4] = {ldexpf(s[0], p), ldexpf(s[1], p), ldexpf(s[2], p), ldexpf(s[3], p)};
  store4_any(dx, dxt, m * lddx + k, 4, u);
}

// dx = 0 (no rows to contract over).
__global__ __launch_bounds__(256) void k_dx_zero(int64_t M, int64_t K, void* __restrict__ dx, int dxt, int64_t lddx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < M * K) store_any(dx, dxt, i / K * lddx + i % K, 0.0f);
}

// Compute units of the current GPU.
inline int64_t dx_cus() { return awq::device_cus() > 0 ? awq::device_cus() : 256; }
inline TilePlan dx_plan(int64_t M, int64_t N, int64_t K) { return dx_plan(M, N, K, dx_cus()); }

inline int64_t dx_blocks(const TilePlan& p, int64_t M, int64_t K) {
  return tile_blocks((M + 16 * p.mb * p.wm - 1) / (16 * p.mb * p.wm) * ((K + kDxCols - 1) / kDxCols) * p.S);
}

struct DxWs {
  uint16_t* xq;
  int* pm;
  float* inv;
  uint16_t* ctab;
  float* partial;
  size_t bytes;
};

inline DxWs dx_ws(void* ws, int64_t M, int64_t N, int64_t K, int group, int S) {
  DxWs w{};
  char* base = (char*)ws;
  size_t off = 0;
  auto take = [&](size_t b) {
    char* q = base ? base + off : nullptr;
    off += awq::align_up(b, 256);
    return q;
  };
  const size_t Np = (size_t)((N + kDxN - 1) / kDxN * kDxN);
  w.inv = (float*)take(Np * 4);
  w.ctab = (uint16_t*)take(Np * (size_t)(K / group) * 4);
  w.pm = (int*)take((size_t)M * 4);
  w.xq = (uint16_t*)take((size_t)M * Np * 2);
  w.partial = S > 1 ? (float*)take((size_t)S * M * K * 4) : nullptr;
  w.bytes = off;
  return w;
}

template <int MB, int WM>
hipError_t dx_launch(const DxWs& w, const TilePlan& p, int64_t M, int64_t Np, const uint32_t* qw, int64_t N, int64_t K,
                     int glog, void* dx, int dxt, int64_t lddx, hipStream_t st) {
  const dim3 grid((unsigned)dx_blocks(p, M, K)), block(256 * WM);
  constexpr size_t lds = Tile<MB, WM, kDxStages<MB, WM>, DxOp<WM>>::Lds;
  if (p.S == 1) {
    hipLaunchKernelGGL((k_gemm_dx<MB, WM, false>), grid, block, lds, st, w.xq, w.pm, M, Np, qw, N, K, w.ctab, glog, p.S,
                       w.partial, dx, dxt, lddx);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_gemm_dx<MB, WM, true>), grid, block, lds, st, w.xq, w.pm, M, Np, qw, N, K, w.ctab, glog, p.S,
                     w.partial, dx, dxt, lddx);
  hipLaunchKernelGGL(k_dx_reduce, dim3((unsigned)((M * K / 4 + 255) / 256)), dim3(256), 0, st, w.partial, p.S, M, K,
                     w.pm, dx, dxt, lddx);
  return hipGetLastError();
}

}  // namespace awqk

namespace awq {

size_t gemm_dx_ws_bytes(int64_t M, int64_t N, int64_t K, int group) {
  using namespace awqk;
  if (M <= 0 || N <= 0 || K <= 0 || group <= 0) return 0;
  return dx_ws(nullptr, M, N, K, group, dx_plan(M, N, K).S).bytes;
}

// The most that any M' <= M may need: fewer rows may be split into more slices.
size_t gemm_dx_ws_bytes_upto(int64_t M, int64_t N, int64_t K) {
  using namespace awqk;
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const int64_t parts = tile_parts(kDxShapes, M, K, (N + kDxN - 1) / kDxN, dx_cus());
  return dx_ws(nullptr, M, N, K, 64, 1).bytes + align_up((size_t)parts * K * 4, 256);
}

int64_t gemm_dx_threads(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  const awqk::TilePlan p = awqk::dx_plan(M, N, K);
  const int64_t tiles = N > 0 ? awqk::dx_blocks(p, M, K) * 256 * p.wm : M * K;
  return tiles > M * 512 ? tiles : M * 512;
}

hipError_t launch_gemm_dx(const void* dz, int dzt, int64_t M, int64_t N, int64_t lddz, const uint32_t* qw,
                          const uint16_t* scales, const uint8_t* zeros, int64_t K, int group, void* dx, int dxt,
                          int64_t lddx, void* ws, hipStream_t st) {
  using namespace awqk;
  const int glog = group == 64 ? 6 : group == 128 ? 7 : group == 256 ? 8 : -1;
  if (glog < 0) return hipErrorInvalidValue;
  if (N == 0) {
    hipLaunchKernelGGL(k_dx_zero, dim3((unsigned)((M * K + 255) / 256)), dim3(256), 0, st, M, K, dx, dxt, lddx);
    return hipGetLastError();
  }
  const TilePlan p = dx_plan(M, N, K);
  const DxWs w = dx_ws(ws, M, N, K, group, p.S);
  const int64_t Np = (N + kDxN - 1) / kDxN * kDxN;
  hipLaunchKernelGGL(k_dx_consts, dim3((unsigned)(Np / 16)), dim3(256), 0, st, scales, zeros, N, Np, K >> glog, w.inv,
                     w.ctab);
  if (dzt == DT_F16) dx_rows<DT_F16>(dz, M, N, Np, lddz, w.inv, w.xq, w.pm, st);
  else dx_rows<DT_BF16>(dz, M, N, Np, lddz, w.inv, w.xq, w.pm, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
#define AWQ_DX(MB, WM) return dx_launch<MB, WM>(w, p, M, Np, qw, N, K, glog, dx, dxt, lddx, st)
  if (p.wm == 2) {
    if (p.mb == 8) AWQ_DX(8, 2);
    AWQ_DX(4, 2);
  }
  switch (p.mb) {
    case 4: AWQ_DX(4, 1);
    case 2: AWQ_DX(2, 1);
    default: AWQ_DX(1, 1);
  }
#undef AWQ_DX
}

}  // namespace awq
