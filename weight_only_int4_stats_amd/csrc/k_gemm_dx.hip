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
//   3. k_gemm_dx: tiles of 32 MB rows x 256 columns, 64 n per stage, three
//      stages in LDS filled by LDS DMA two ahead; wave (wm, wn) takes 16 MB
//      rows x 64 columns.  The weights are the product of two exact fp16
//      values, rounded once.
//   4. k_dx_reduce where the contraction is split: the slices' fp32 sums added
//      in their order.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"
#include "k_rows_f16.h"

namespace awqk {

constexpr int kDxCols = 256;              // tile columns (k)
constexpr int kDxN = 64;                  // contraction per stage
constexpr int kDxXcds = 8;                // L2 slices (block i -> slice i mod 8)
constexpr int kDxB = kDxN * kDxCols / 2;  // packed bytes per stage
constexpr int kDxC = 1024;                // constants per stage: up to 4 groups x 64 rows x 4 bytes

// Rows n in chunks of eight: ctab[g][n / 8] = the eight steps (four pairs),
// then the eight zero points.  One block of 256 threads per 16 rows, 16 lanes
// per row, as the product's constants.
__global__ __launch_bounds__(256) void k_dx_consts(const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                                                   int64_t N, int64_t Np, int64_t G, float* __restrict__ inv,
                                                   uint16_t* __restrict__ ctab) {
  const int rl = threadIdx.x >> 4, p = threadIdx.x & 15;
  const int64_t n = (int64_t)blockIdx.x * 16 + rl;               // < Np, a multiple of 64
  const bool ok = n < N;
  const int64_t g0 = p * G / 16, g1 = (p + 1) * G / 16;
  const uint16_t* sr = scales + (ok ? n : 0) * G;
  const uint8_t* zr = zeros + (ok ? n : 0) * G;
  float mx = 0.0f;
  if (ok)
    for (int64_t g = g0; g < g1; ++g) mx = fmaxf(mx, step_size<true>(sr[g]));
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  const int e = step_pow<true>(mx);
  if (p == 0) inv[n] = ok ? ldexpf(1.0f, -sum_pow<true>(e)) : 0.0f;
  const int64_t at = (n >> 3) * 16 + (n & 7);
  for (int64_t g = g0; g < g1; ++g) {
    uint16_t* c = ctab + g * Np * 2 + at;
    c[0] = (uint16_t)(ok ? f32_to_f16_bits(ldexpf(f16_to_f32(sr[g]), e)) : 0u);
    c[8] = (uint16_t)(ok ? once_zero(zr[g]) & 0xFFFFu : 0u);
  }
}

// One row of dz per block, read twice (the second time from the caches).
template <int DT>
__global__ __launch_bounds__(256) void k_dx_rows(const uint16_t* __restrict__ dz, int64_t N, int64_t Np, int64_t ld,
                                                 const float* __restrict__ inv, uint16_t* __restrict__ out,
                                                 int* __restrict__ pexp) {
  __shared__ float wmax[4];
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
  float am = 0.0f;
  for (int64_t c = threadIdx.x; c < nch; c += 256) {
    float v[8];
    load(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = fabsf(v[j]);
      am = s < __builtin_inff() ? fmaxf(am, s) : am;             // a row's power goes by its finite values
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) am = fmaxf(am, __shfl_xor(am, off));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = am;
  __syncthreads();
  const int p = pow2_exp_for(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])));
  if (threadIdx.x == 0) pexp[m] = p;
  for (int64_t c = threadIdx.x; c < nch; c += 256) {
    float v[8];
    load(c, v);
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = f32_to_f16_bits(ldexpf(v[2 * j], p)) | (f32_to_f16_bits(ldexpf(v[2 * j + 1], p)) << 16);
    *reinterpret_cast<u32x4*>(out + m * Np + c * 8) = o;
  }
}

// Position of a dz row's 16-byte chunk in LDS, as in the product's tiles.
__device__ __forceinline__ int dx_swz(int r) { return (r >> 1) & 7; }

// Four outputs of one row: columns k .. k + 3 (K is a multiple of 64).
__device__ __forceinline__ void dx_store4(void* dx, int dt, int64_t i, const float (&v)[4]) {
  if (dt == DT_F32) {
    u32x4a4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(v[j]);
    *reinterpret_cast<u32x4a4*>(reinterpret_cast<float*>(dx) + i) = o;
  } else {
    u32x2a2 o;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = dt == DT_F16 ? f32_to_f16_bits(v[2 * j]) | (f32_to_f16_bits(v[2 * j + 1]) << 16)
                          : f32_to_bf16_bits(v[2 * j]) | (f32_to_bf16_bits(v[2 * j + 1]) << 16);
    *reinterpret_cast<u32x2a2*>(reinterpret_cast<uint16_t*>(dx) + i) = o;
  }
}

template <int MB>
struct DxTile {
  static constexpr int Rows = 32 * MB;
  static constexpr int A = Rows * kDxN * 2;          // fp16 rows of dz
  static constexpr int Stage = A + kDxB + kDxC;
  static constexpr int ACopies = A / 1024;           // 4 MB copies of 1 KB, by wave: MB / 2 (waves 0..3 one each for MB = 1)
};

// MB: 16-row blocks per wave.  S slices of the contraction; SPLIT: fp32 sums to
// partial [S][M][K] instead of dx.
template <int MB, bool SPLIT>
__global__ __launch_bounds__(512) void k_gemm_dx(const uint16_t* __restrict__ xq, const int* __restrict__ pm, int64_t M,
                                                 int64_t Np, const uint32_t* __restrict__ qw, int64_t N, int64_t K,
                                                 const uint16_t* __restrict__ ctab, int glog, int S, int64_t tiles,
                                                 float* __restrict__ partial, void* __restrict__ dx, int dxt,
                                                 int64_t lddx) {
  using Tl = DxTile<MB>;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[Tl::Stage];
  __shared__ __attribute__((aligned(16))) uint8_t lds1[Tl::Stage];
  __shared__ __attribute__((aligned(16))) uint8_t lds2[Tl::Stage];
  // block i runs on L2 slice i mod 8, which takes the i-th eighth of the work
  // items (slice fastest, then rows, then columns: neighbours share dz or W)
  const int64_t items = tiles * S, per = (items + kDxXcds - 1) / kDxXcds;
  const int64_t slot = blockIdx.x / kDxXcds, item = (int64_t)(blockIdx.x % kDxXcds) * per + slot;
  if (slot >= per || item >= items) return;
  const int64_t mtiles = (M + Tl::Rows - 1) / Tl::Rows;
  const int bs = (int)(item % S);
  const int64_t t = item / S;
  const int64_t m0 = (t % mtiles) * Tl::Rows, k0 = (t / mtiles) * kDxCols;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 2, wn = wv & 3;
  const int rl = lane & 15, b4 = lane >> 4;
  const int64_t stages = Np / kDxN;
  const int64_t s0 = bs * stages / S, s1 = (bs + 1) * stages / S;
  const int rows = (int)(M - m0 < Tl::Rows ? M - m0 : Tl::Rows);
  const int64_t G = K >> glog, g0 = k0 >> glog;
  const int ng = (int)(G - g0 < (kDxCols >> glog) ? G - g0 : (kDxCols >> glog));
  const int64_t KB = K >> 1;                                     // bytes of a packed row
  const i32x4 ars = rsrc4(xq + m0 * Np, (uint32_t)(rows * Np * 2));
  const i32x4 crs = rsrc4(ctab + g0 * Np * 2, (uint32_t)(ng * Np * 4));

  // copies of 1 KB: A rows 8 j .. 8 j + 7 (lane i: row 8 j + i / 8, chunk
  // (i % 8) ^ swizzle), B rows 8 w .. 8 w + 7 of the stage (lane i: row i / 8,
  // 16-byte chunk (i % 8) ^ 2 (w % 4), so that the four rows a read meets lie
  // in different banks), C (wave 0: lane i group i / 16, piece i % 16)
  constexpr int AW = MB >= 2 ? MB / 2 : 1;                       // A copies of a wave that has any
  const bool has_a = MB >= 2 || wv < 4;
  const int nops = (has_a ? AW : 0) + 1 + (wv == 0 ? 1 : 0);
  uint32_t aoff[AW];
#pragma unroll
  for (int u = 0; u < AW; ++u) {
    const int r = 8 * (AW * wv + u) + (lane >> 3);
    aoff[u] = (uint32_t)(r * Np * 2 + (((lane & 7) ^ dx_swz(r)) * 16));
  }
  const uint32_t boff = (uint32_t)((8 * wv + (lane >> 3)) * KB + k0 / 2 + (((lane & 7) ^ (2 * (wv & 3))) * 16));
  const uint32_t coff = (uint32_t)((lane >> 4) * Np * 4 + (lane & 15) * 16);
  auto issue = [&](int64_t s, const uint8_t* base) {
    const uint32_t lb = __builtin_amdgcn_readfirstlane(lds_addr(base));
    if (has_a) {
#pragma unroll
      for (int u = 0; u < AW; ++u) dma16(ars, lb + (AW * wv + u) * 1024, aoff[u], (uint32_t)(s * kDxN * 2));
    }
    // the stage's rows of W: a descriptor of their own, so that no offset grows with N
    const int64_t left = N - s * kDxN;
    const i32x4 brs = rsrc4(reinterpret_cast<const uint8_t*>(qw) + s * kDxN * KB, (uint32_t)((left < kDxN ? left : kDxN) * KB));
    dma16(brs, lb + Tl::A + wv * 1024, boff, 0);
    if (wv == 0) dma16(crs, lb + Tl::A + kDxB, coff, (uint32_t)(s * kDxN * 4));
  };
  auto wait_newest = [&]() {                                     // all but the newest stage's copies landed
    if (nops == AW + 2) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(AW + 2));
    else if (nops == AW + 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(AW + 1));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(1));
  };

  f32x4 acc[MB][4];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // the lane's place in a packed row of the tile: word wn 8 + rl / 2, half
  // rl % 2; its group among the tile's (the same for the whole wave)
  const uint32_t sel = (rl & 1) ? 0x07060302u : 0x05040100u;
  const int word = wn * 8 + (rl >> 1);
  const int gl = (wn * 64) >> glog;
  const f16x2 c15 = as_f16x2(0x78007800u), c11 = as_f16x2(0x68006800u);   // 2^15, 2^11

  auto stage = [&](const uint8_t* base) {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int ch = 4 * st + b4;                                // rows n 8 ch .. 8 ch + 7 of the stage
      const u32x4 cm = *reinterpret_cast<const u32x4*>(base + Tl::A + kDxB + gl * 256 + ch * 32);
      const u32x4 cz = *reinterpret_cast<const u32x4*>(base + Tl::A + kDxB + gl * 256 + ch * 32 + 16);
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = *reinterpret_cast<const uint32_t*>(base + Tl::A + (8 * ch + j) * 128 +
                                                  (((word >> 2) ^ (2 * (ch & 3))) * 16) + (word & 3) * 4);
      u32x4 bq[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t p = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], sel), p8 = p >> 8;
        const uint32_t cmj = cm[j], czj = cz[j];
        const f16x2 d = as_f16x2(cmj), z = as_f16x2(czj);
        bq[0][j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(p & 0x000F000Fu), c15, z) * d);
        bq[1][j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(p & 0x00F000F0u), c11, z) * d);
        bq[2][j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(p8 & 0x000F000Fu), c15, z) * d);
        bq[3][j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(p8 & 0x00F000F0u), c11, z) * d);
      }
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        const int r = wm * 16 * MB + a * 16 + rl;
        const u32x4 af = *reinterpret_cast<const u32x4*>(base + r * 128 + ((ch ^ dx_swz(r)) * 16));
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][c] = mfma16h(af, bq[c], acc[a][c]);
      }
    }
  };

  // stage s is read from LDS array (s - s0) mod 3 while s + 1 and s + 2 arrive
  if (s0 < s1) issue(s0, lds0);
  if (s0 + 1 < s1) issue(s0 + 1, lds1);
  auto step = [&](int64_t s, const uint8_t* cur, const uint8_t* nxt2) {
    if (s + 1 < s1) wait_newest();
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    lds_barrier();                                               // stage s landed, and everyone is done with s - 1
    if (s + 2 < s1) issue(s + 2, nxt2);
    stage(cur);
  };
  for (int64_t s = s0; s < s1; s += 3) {
    step(s, lds0, lds2);
    if (s + 1 < s1) step(s + 1, lds1, lds0);
    if (s + 2 < s1) step(s + 2, lds2, lds1);
  }

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
        dx_store4(dx, dxt, m * lddx + k, u);
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
  dx_store4(dx, dxt, m * lddx + k, u);
}

// dx = 0 (no rows to contract over).
__global__ __launch_bounds__(256) void k_dx_zero(int64_t M, int64_t K, void* __restrict__ dx, int dxt, int64_t lddx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < M * K) store_any(dx, dxt, i / K * lddx + i % K, 0.0f);
}

struct DxPlan {
  int mb = 1, S = 1;
  int64_t tiles = 0, blocks = 0;
};

// Tile height and slices by the estimated time of the launch's rounds (one
// block per compute unit).  A stage of a wave takes 8 MB products of 16 cycles
// beside about 60 vector instructions of 4 cycles per k32 step.  Rows count in
// whole 32s, so that the choice is the same up to the next multiple.
inline DxPlan dx_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t cus = awq::device_cus() > 0 ? awq::device_cus() : 256;
  const int64_t stages = (N + kDxN - 1) / kDxN, ct = (K + kDxCols - 1) / kDxCols, M32 = (M + 31) / 32 * 32;
  DxPlan best;
  double best_cost = 1e300;
  for (int mb = 8; mb >= 1; mb >>= 1) {
    const int64_t tiles = (M + 32 * mb - 1) / (32 * mb) * ct;
    const double stage = 8.0 * mb * 16 * 2 > 1000 ? 8.0 * mb * 16 * 2 : 1000;      // cycles, two waves per SIMD
    for (int S = 1; S == 1 || (S <= 16 && S * 2 <= stages && tiles * S < 2 * cus); S *= 2) {
      const double rounds = (double)((tiles * S + cus - 1) / cus);
      const double cost = rounds * ((double)((stages + S - 1) / S) * stage + 6000.0) +
                          (S > 1 ? 5000.0 + (double)S * M32 * K * 8 / 1500.0 : 0.0);
      if (cost < best_cost) {
        best_cost = cost;
        best.mb = mb;
        best.S = S;
        best.tiles = tiles;
      }
    }
  }
  best.blocks = kDxXcds * ((best.tiles * best.S + kDxXcds - 1) / kDxXcds);
  return best;
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

template <int MB>
hipError_t dx_launch(const DxWs& w, const DxPlan& p, int64_t M, int64_t Np, const uint32_t* qw, int64_t N, int64_t K,
                     int glog, void* dx, int dxt, int64_t lddx, hipStream_t st) {
  const dim3 grid((unsigned)p.blocks), block(512);
  if (p.S == 1) {
    hipLaunchKernelGGL((k_gemm_dx<MB, false>), grid, block, 0, st, w.xq, w.pm, M, Np, qw, N, K, w.ctab, glog, p.S,
                       p.tiles, w.partial, dx, dxt, lddx);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_gemm_dx<MB, true>), grid, block, 0, st, w.xq, w.pm, M, Np, qw, N, K, w.ctab, glog, p.S,
                     p.tiles, w.partial, dx, dxt, lddx);
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

// The most that any M' <= M needs: fewer rows may be split into more slices.
// Past 512 compute units' worth of the tallest tiles nothing is split.
size_t gemm_dx_ws_bytes_upto(int64_t M, int64_t N, int64_t K) {
  using namespace awqk;
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  size_t most = gemm_dx_ws_bytes(M, N, K, 64);
  const int64_t split = 2 * (int64_t)device_cus() * 32 * 8;
  for (int64_t m = 32; m < M && m <= split; m += 32) {
    const size_t b = gemm_dx_ws_bytes(m, N, K, 64);
    most = b > most ? b : most;
  }
  return most;
}

int64_t gemm_dx_threads(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  const int64_t tiles = N > 0 ? awqk::dx_plan(M, N, K).blocks * 512 : M * K;
  return tiles > M * 256 ? tiles : M * 256;
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
  const DxPlan p = dx_plan(M, N, K);
  const DxWs w = dx_ws(ws, M, N, K, group, p.S);
  const int64_t Np = (N + kDxN - 1) / kDxN * kDxN;
  hipLaunchKernelGGL(k_dx_consts, dim3((unsigned)(Np / 16)), dim3(256), 0, st, scales, zeros, N, Np, K >> glog, w.inv,
                     w.ctab);
  if (dzt == DT_F16)
    hipLaunchKernelGGL((k_dx_rows<DT_F16>), dim3((unsigned)M), dim3(256), 0, st, (const uint16_t*)dz, N, Np, lddz, w.inv,
                       w.xq, w.pm);
  else
    hipLaunchKernelGGL((k_dx_rows<DT_BF16>), dim3((unsigned)M), dim3(256), 0, st, (const uint16_t*)dz, N, Np, lddz, w.inv,
                       w.xq, w.pm);
  switch (p.mb) {
    case 8: return dx_launch<8>(w, p, M, Np, qw, N, K, glog, dx, dxt, lddx, st);
    case 4: return dx_launch<4>(w, p, M, Np, qw, N, K, glog, dx, dxt, lddx, st);
    case 2: return dx_launch<2>(w, p, M, Np, qw, N, K, glog, dx, dxt, lddx, st);
    default: return dx_launch<1>(w, p, M, Np, qw, N, K, glog, dx, dxt, lddx, st);
  }
}

}  // namespace awq
