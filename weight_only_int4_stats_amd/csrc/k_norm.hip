// Layer norm and RMS norm of each row, and their backward pass
// (awq_layer_norm, awq_layer_norm_backward):
//   mu = mean x (RMS: 0),  r = 1 / sqrt(mean (x - mu)^2 + eps),  xh = (x - mu) r
//   y = xh w + b
//   a = dy w,  dx = r (a - mean a - xh mean(a xh))   (RMS: without mean a)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// Both are bound by memory (8192 x 4096: 32 us forward from 32 to 16 bits, 6.3
// TB/s; 37 + 5 us backward in bf16, 5.5 TB/s in the first): a row is read once
// and stays in registers (the variance is that of the centred values, and what
// the first sum's rounding left in their mean is taken off again: at a mean of
// 1e4 sigma it shifted every value by 1e-3 sigma), and the backward pass adds up dw and db in registers over
// all the rows a block takes, leaves one partial row per block and adds those in
// a second launch (k_col_reduce), in a fixed order.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"

namespace awqk {

// Sum over the T lanes of a row group (T = 64: one wave; more: the group's
// waves meet in LDS, red[2 waves of the block], the half turning with `turn`
// so that one barrier per sum is enough).
template <int T, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], float (*red)[16][NV], int turn) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (T > 64) {
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) red[turn][wv][i] = v[i];
    }
    __syncthreads();
    const int w0 = (int)(threadIdx.x / T) * (T / 64);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = red[turn][w0][i];
#pragma unroll
      for (int w = 1; w < T / 64; ++w) s += red[turn][w0 + w][i];
      v[i] = s;
    }
  }
}

// Of values with the mean square sq and the mean m; equal values may leave less
// than 0 by rounding.  (NaN stays.)
__device__ __forceinline__ float variance(float sq, float m) {
  const float v = __builtin_fmaf(-m, m, sq);
  return v < 0.0f ? 0.0f : v;
}

struct NormArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  int64_t M, K, ldx, ldy;
  float eps;
  int wdt, bdt, ydt;
};

// Lanes T of a row, KEEP chunks of eight values each in registers.
template <int XDT, int T, int KEEP, bool RMS>
__global__ __launch_bounds__(T > 256 ? T : 256) void k_norm(const NormArgs a) {
  __shared__ float red[1][16][1], red2[1][16][2];
  constexpr int RB = (T > 256 ? T : 256) / T;                    // rows per block
  const int t = threadIdx.x % T;
  const int64_t m = (int64_t)blockIdx.x * RB + threadIdx.x / T;
  const bool live = m < a.M;
  float v[KEEP][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int64_t c = (int64_t)(t + T * i) * 8;
    load8_any(a.x, XDT, m * a.ldx + c, live && c < a.K ? (a.K - c < 8 ? (int)(a.K - c) : 8) : 0, v[i]);
    if constexpr (!RMS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += v[i][j];
    }
  }
  float mu = 0.0f;
  if constexpr (!RMS) {
    group_sum<T, 1>(s, red, 0);
    mu = s[0] / (float)a.K;
  }
  float q[2] = {0.0f, 0.0f};                       // sums of the centred values' squares and of themselves
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int64_t c = (int64_t)(t + T * i) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = c + j < a.K ? v[i][j] - mu : 0.0f;
      q[0] = __builtin_fmaf(v[i][j], v[i][j], q[0]);
      if constexpr (!RMS) q[1] += v[i][j];
    }
  }
  float left = 0.0f;
  if constexpr (RMS) {
    s[0] = q[0];
    group_sum<T, 1>(s, red, 0);
    q[0] = s[0] / (float)a.K;
  } else {
    group_sum<T, 2>(q, red2, 0);
    left = q[1] / (float)a.K;
    q[0] = variance(q[0] / (float)a.K, left);
    mu += left;
  }
  const float r = 1.0f / sqrtf(q[0] + a.eps);
  if (!live) return;
  if (t == 0) {
    if (a.mean) a.mean[m] = mu;
    if (a.rstd) a.rstd[m] = r;
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int64_t c = (int64_t)(t + T * i) * 8;
    if (c >= a.K) continue;
    const int cnt = a.K - c < 8 ? (int)(a.K - c) : 8;
    float w[8], o[8];
    load8_any(a.w, a.wdt, c, cnt, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (v[i][j] - left) * r * w[j];
    if (a.b) {
      float b[8];
      load8_any(a.b, a.bdt, c, cnt, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += b[j];
    }
    store8_any(a.y, a.ydt, m * a.ldy + c, cnt, o);
  }
}

// Rows too long for registers: one block per row, read three times.
template <int XDT, bool RMS>
__global__ __launch_bounds__(1024) void k_norm_long(const NormArgs a) {
  __shared__ float red[1][16][1], red2[1][16][2];
  const int64_t m = blockIdx.x;
  auto cnt_at = [&](int64_t c) { return a.K - c < 8 ? (int)(a.K - c) : 8; };
  float mu = 0.0f;
  float s[1] = {0.0f};
  if constexpr (!RMS) {
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.K; c += 8192) {
      float v[8];
      load8_any(a.x, XDT, m * a.ldx + c, cnt_at(c), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += v[j];
    }
    group_sum<1024, 1>(s, red, 0);
    mu = s[0] / (float)a.K;
  }
  float q[2] = {0.0f, 0.0f};
  for (int64_t c = (int64_t)threadIdx.x * 8; c < a.K; c += 8192) {
    float v[8];
    load8_any(a.x, XDT, m * a.ldx + c, cnt_at(c), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = c + j < a.K ? v[j] - mu : 0.0f;
      q[0] = __builtin_fmaf(d, d, q[0]);
      q[1] += d;
    }
  }
  group_sum<1024, 2>(q, red2, 0);
  const float left = RMS ? 0.0f : q[1] / (float)a.K;
  const float r = 1.0f / sqrtf(variance(q[0] / (float)a.K, left) + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[m] = mu + left;
    if (a.rstd) a.rstd[m] = r;
  }
  for (int64_t c = (int64_t)threadIdx.x * 8; c < a.K; c += 8192) {
    const int cnt = cnt_at(c);
    float v[8], w[8], b[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    load8_any(a.x, XDT, m * a.ldx + c, cnt, v);
    load8_any(a.w, a.wdt, c, cnt, w);
    if (a.b) load8_any(a.b, a.bdt, c, cnt, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (v[j] - mu - left) * r * w[j] + b[j];
    store8_any(a.y, a.ydt, m * a.ldy + c, cnt, v);
  }
}

struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;        // [blocks][2 pitch]: dw, then db from pitch on (one block: not used)
  float* dw;             // the sums themselves; NULL: not formed
  float* db;
  int64_t M, K, lddy, ldx, lddx, pitch;
  int dyt, wdt;
};

// Sums over the W waves of a row group, as group_sum with W known at run time.
__device__ __forceinline__ void waves_sum(float (&v)[2], float (*red)[16][2], int turn, int w0, int W) {
  v[0] = wave_sum(v[0]);
  v[1] = wave_sum(v[1]);
  if (W == 1) return;                                            // block-uniform
  if ((threadIdx.x & 63) == 0) {
    red[turn][threadIdx.x >> 6][0] = v[0];
    red[turn][threadIdx.x >> 6][1] = v[1];
  }
  __syncthreads();
  // lane w of every 16 takes wave w's (one read instead of W in turn)
  const int w = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = row16_sum(w < W ? red[turn][w0 + w][i] : 0.0f);
}

// RB row groups of W waves each (W RB <= 16), KEEP chunks of eight values per
// lane.  Block b takes the rows b RB + i, (b + grid) RB + i, ...; W is just
// enough for a row, so that a width of 5120 leaves no lane idle.
// (dy's type is known at compile time: with loads of either kind the rows on
// their way went through scratch memory, 45 us instead of 37 at 8192 x 4096.  Rows of 8193
// to 16384 values with an fp32 x or dy still leave 3 to 8 registers there.)
template <int XDT, int DYT, int KEEP, bool RMS>
__global__ __launch_bounds__(1024) void k_norm_grad(const NormGradArgs a, int W, int RB) {
  __shared__ float red[2][16][2];
  extern __shared__ float meet[];                                // [RB - 1][KEEP 8][T], for the row groups to meet
  const int T = 64 * W, wv = threadIdx.x >> 6, rg = wv / W, w0 = rg * W;
  const int t = threadIdx.x - w0 * 64;
  int cnt[KEEP];
  float w[KEEP][8], dw[KEEP][8], db[KEEP][8];
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int64_t c = (int64_t)(t + T * i) * 8;
    cnt[i] = c < a.K ? (a.K - c < 8 ? (int)(a.K - c) : 8) : 0;
    load8_any(a.w, a.wdt, c, cnt[i], w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  }
  const float inv_k = 1.0f / (float)a.K;
  // the next two rows (one of 32-bit values) are on their way, as they lie in
  // memory, while this one's sums meet, so that a compute unit has some 48 KB in
  // flight (8192 x 4096 from cold caches: 60 us a call with none, 55 with two); a
  // lane with two chunks has no registers left for that
  constexpr bool AHEAD = KEEP == 1;
  constexpr int D = AHEAD && XDT != DT_F32 && DYT != DT_F32 ? 2 : 1;
  Raw8 nx[D][KEEP], ng[D][KEEP];
  float nmu[D], nr[D];
  auto fetch = [&](int64_t m, int d) {
    const bool live = m < a.M;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int64_t c = (int64_t)(t + T * i) * 8;
      nx[d][i] = raw8_load(a.x, XDT, m * a.ldx + c, live ? cnt[i] : 0);
      ng[d][i] = raw8_load(a.dy, DYT, m * a.lddy + c, live ? cnt[i] : 0);
    }
    nmu[d] = !RMS && live ? a.mean[m] : 0.0f;
    nr[d] = live ? a.rstd[m] : 0.0f;
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * RB;
  if constexpr (AHEAD) {
#pragma unroll
    for (int d = 0; d < D; ++d) fetch((int64_t)blockIdx.x * RB + rg + d * step, d);
  }
  for (int64_t mb = (int64_t)blockIdx.x * RB; mb < a.M; mb += step) {
    const int64_t m = mb + rg;
    const bool live = m < a.M;
    if constexpr (!AHEAD) fetch(m, 0);
    float xh[KEEP][8], g[KEEP][8];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      raw8_floats(nx[0][i], XDT, xh[i]);
      raw8_floats(ng[0][i], DYT, g[i]);
    }
    const float mu = nmu[0], r = nr[0];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i) {
        nx[0][i] = nx[D - 1][i];
        ng[0][i] = ng[D - 1][i];
      }
      nmu[0] = nmu[D - 1];
      nr[0] = nr[D - 1];
      fetch(m + D * step, D - 1);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = j < cnt[i] && live ? (xh[i][j] - mu) * r : 0.0f;
        dw[i][j] = __builtin_fmaf(g[i][j], xh[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= w[i][j];
        s[0] = __builtin_fmaf(g[i][j], xh[i][j], s[0]);
        s[1] += g[i][j];
      }
    waves_sum(s, red, turn, w0, W);
    turn ^= 1;
    const float mx = s[0] * inv_k, ma = RMS ? 0.0f : s[1] * inv_k;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      if (!live || cnt[i] == 0) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = r * (g[i][j] - ma - xh[i][j] * mx);
      store8_any(a.dx, XDT, m * a.lddx + (int64_t)(t + T * i) * 8, cnt[i], g[i]);
    }
  }
  // the row groups' sums meet in the first one's, in their order; one block's
  // are whole
  const bool whole = gridDim.x == 1;
  float* part = a.partial + (int64_t)blockIdx.x * 2 * a.pitch;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float (&d)[KEEP][8] = half ? db : dw;
    if (!(half ? a.db : a.dw)) continue;                         // grid-uniform
    if (RB > 1) {                                                // block-uniform
      __syncthreads();
      if (rg > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) meet[((rg - 1) * KEEP * 8 + i * 8 + j) * T + t] = d[i][j];
      }
      __syncthreads();
    }
    if (rg == 0) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i) {
        const int64_t c = (int64_t)(t + T * i) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          for (int q = 0; q < RB - 1; ++q) d[i][j] += meet[(q * KEEP * 8 + i * 8 + j) * T + t];
        if (whole) store8_any(half ? a.db : a.dw, DT_F32, c, cnt[i], d[i]);
        else if (c < a.pitch) store8_any(part, DT_F32, half * a.pitch + c, 8, d[i]);
      }
    }
  }
}

// Rows too long for registers: one block per row at a time, dw and db added up
// in the block's own partial row.
template <int XDT, bool RMS>
__global__ __launch_bounds__(1024) void k_norm_grad_long(const NormGradArgs a) {
  __shared__ float red[2][16][2];
  float* out = a.dw || a.db ? a.partial + (int64_t)blockIdx.x * 2 * a.pitch : nullptr;
  const float inv_k = 1.0f / (float)a.K;
  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const float mu = RMS ? 0.0f : a.mean[m], r = a.rstd[m];
    float s[2] = {0.0f, 0.0f};
    const bool first = m == blockIdx.x;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.K; c += 8192) {
      const int cnt = a.K - c < 8 ? (int)(a.K - c) : 8;
      float x[8], g[8], w[8];
      load8_any(a.x, XDT, m * a.ldx + c, cnt, x);
      load8_any(a.dy, a.dyt, m * a.lddy + c, cnt, g);
      load8_any(a.w, a.wdt, c, cnt, w);
      float dw[8], db[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = j < cnt ? (x[j] - mu) * r : 0.0f;
        dw[j] = g[j] * xh;
        db[j] = g[j];
        const float q = g[j] * w[j];
        s[0] = __builtin_fmaf(q, xh, s[0]);
        s[1] += q;
      }
      if (out) {                                                 // this thread's own columns (c + 7 < pitch)
        if (!first) {
          float o[8], p[8];
          load8_any(out, DT_F32, c, 8, o);
          load8_any(out, DT_F32, a.pitch + c, 8, p);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dw[j] += o[j];
            db[j] += p[j];
          }
        }
        store8_any(out, DT_F32, c, 8, dw);
        store8_any(out, DT_F32, a.pitch + c, 8, db);
      }
    }
    group_sum<1024, 2>(s, red, turn);
    turn ^= 1;
    const float mx = s[0] * inv_k, ma = RMS ? 0.0f : s[1] * inv_k;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.K; c += 8192) {
      const int cnt = a.K - c < 8 ? (int)(a.K - c) : 8;
      float x[8], g[8], w[8];
      load8_any(a.x, XDT, m * a.ldx + c, cnt, x);
      load8_any(a.dy, a.dyt, m * a.lddy + c, cnt, g);
      load8_any(a.w, a.wdt, c, cnt, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = r * (g[j] * w[j] - ma - (x[j] - mu) * r * mx);
      store8_any(a.dx, XDT, m * a.lddx + c, cnt, g);
    }
  }
}

template <int XDT, bool RMS>
hipError_t norm_dispatch(const NormArgs& a, hipStream_t st) {
#define AWQ_N(T, KEEP)                                                                                        \
  hipLaunchKernelGGL((k_norm<XDT, T, KEEP, RMS>), dim3((unsigned)((a.M + (T > 256 ? T : 256) / T - 1) / ((T > 256 ? T : 256) / T))), \
                     dim3(T > 256 ? T : 256), 0, st, a)
  if (a.K <= 512) AWQ_N(64, 1);
  else if (a.K <= 1024) AWQ_N(64, 2);
  else if (a.K <= 2048) AWQ_N(256, 1);
  else if (a.K <= 4096) AWQ_N(256, 2);
  else if (a.K <= 8192) AWQ_N(256, 4);
  else if (a.K <= 16384) AWQ_N(1024, 2);
  else if (a.K <= 32768) AWQ_N(1024, 4);
  else hipLaunchKernelGGL((k_norm_long<XDT, RMS>), dim3((unsigned)a.M), dim3(1024), 0, st, a);
#undef AWQ_N
  return hipGetLastError();
}

// Waves per row of the backward pass (0: rows too long for registers), chunks
// per lane and row groups per block.
struct NormGradPlan {
  int waves, keep, groups;
  int64_t blocks;
};
inline NormGradPlan norm_grad_plan(int64_t M, int64_t K) {
  NormGradPlan p{};
  const int64_t cus = awq::device_cus() > 0 ? awq::device_cus() : 256;
  if (K <= 16384) {
    p.keep = K <= 8192 ? 1 : 2;
    p.waves = (int)((K + 512 * p.keep - 1) / (512 * p.keep));
    p.groups = 16 / p.waves;
  } else {
    p.groups = 1;
  }
  // one block per compute unit, with as many rows each as make the whole, and
  // at least four: a block's partial sums cost as much as a row or two (519 x
  // 5120: 10 us with four rows a block, 11 with three, 14 with two and two
  // blocks per unit; 8192 x 4096 before rows came ahead: 43 us with one block per
  // unit, 49 with two).
  // Up to eight make one block, whose sums are whole: no second launch.
  const int64_t sets = (M + p.groups - 1) / p.groups;
  int64_t each = (sets + cus - 1) / cus;
  if (each < 4) each = 4;
  if (sets <= 8 && p.waves > 0) each = 8;
  p.blocks = (sets + each - 1) / each;
  return p;
}
// Whether one block forms the sums by itself.
inline bool norm_grad_whole(int64_t M, int64_t K) {
  const NormGradPlan p = norm_grad_plan(M, K);
  return p.waves > 0 && p.blocks == 1;
}
inline int64_t norm_pitch(int64_t K) { return (K + 63) / 64 * 64; }

template <int XDT, bool RMS>
hipError_t norm_grad_dispatch(const NormGradArgs& a, hipStream_t st) {
  const NormGradPlan p = norm_grad_plan(a.M, a.K);
  const dim3 grid((unsigned)p.blocks);
  if (p.waves == 0) {
    hipLaunchKernelGGL((k_norm_grad_long<XDT, RMS>), grid, dim3(1024), 0, st, a);
    return hipGetLastError();
  }
  const dim3 block((unsigned)(64 * p.waves * p.groups));
  const size_t lds = a.dw || a.db ? (size_t)(p.groups - 1) * 64 * p.waves * p.keep * 8 * 4 : 0;
#define AWQ_NG(DYT)                                                                                                  \
  if (p.keep == 1) hipLaunchKernelGGL((k_norm_grad<XDT, DYT, 1, RMS>), grid, block, lds, st, a, p.waves, p.groups); \
  else hipLaunchKernelGGL((k_norm_grad<XDT, DYT, 2, RMS>), grid, block, lds, st, a, p.waves, p.groups)
  if (a.dyt == DT_F16) {
    AWQ_NG(DT_F16);
  } else if (a.dyt == DT_BF16) {
    AWQ_NG(DT_BF16);
  } else {
    AWQ_NG(DT_F32);
  }
#undef AWQ_NG
  return hipGetLastError();
}

}  // namespace awqk

namespace awq {

int64_t norm_threads(int64_t M, int64_t K) { return M * (K > 8192 ? 1024 : 256); }

hipError_t launch_norm(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx, const void* w, int wdt,
                       const void* b, int bdt, float eps, int rms, void* y, int ydt, int64_t ldy, float* mean,
                       float* rstd, hipStream_t st) {
  using namespace awqk;
  const NormArgs a{x, w, b, y, mean, rstd, M, K, ldx, ldy, eps, wdt, bdt, ydt};
#define AWQ_ND(D) return rms ? norm_dispatch<D, true>(a, st) : norm_dispatch<D, false>(a, st)
  if (xdt == DT_F16) AWQ_ND(DT_F16);
  if (xdt == DT_BF16) AWQ_ND(DT_BF16);
  AWQ_ND(DT_F32);
#undef AWQ_ND
}

size_t norm_grad_ws_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || awqk::norm_grad_whole(M, K)) return 0;
  return (size_t)(awqk::norm_grad_plan(M, K).blocks * 2 * awqk::norm_pitch(K)) * 4;
}

// The most that any M' <= M needs: at most one block per compute unit.
size_t norm_grad_ws_bytes_upto(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return 0;
  const int64_t groups = awqk::norm_grad_plan(1, K).groups, sets = (M + groups - 1) / groups;
  const int64_t cus = device_cus() > 0 ? device_cus() : 256;
  return (size_t)((sets < cus ? sets : cus) * 2 * awqk::norm_pitch(K)) * 4;
}

hipError_t launch_norm_grad(const void* dy, int dyt, int64_t M, int64_t K, int64_t lddy, const void* x, int xdt,
                            int64_t ldx, const void* w, int wdt, const float* mean, const float* rstd, int rms,
                            void* dx, int64_t lddx, float* dw, float* db, void* ws, hipStream_t st) {
  using namespace awqk;
  const int64_t pitch = norm_pitch(K);
  const bool sums = dw || db;
  if (M > 0) {
    const NormGradArgs a{dy, x, w, mean, rstd, dx, (float*)ws, dw, db, M, K, lddy, ldx, lddx, pitch, dyt, wdt};
    hipError_t e;
    if (xdt == DT_F16) e = rms ? norm_grad_dispatch<DT_F16, true>(a, st) : norm_grad_dispatch<DT_F16, false>(a, st);
    else if (xdt == DT_BF16) e = rms ? norm_grad_dispatch<DT_BF16, true>(a, st) : norm_grad_dispatch<DT_BF16, false>(a, st);
    else e = rms ? norm_grad_dispatch<DT_F32, true>(a, st) : norm_grad_dispatch<DT_F32, false>(a, st);
    if (e != hipSuccess) return e;
  }
  if (!sums || (M > 0 && norm_grad_whole(M, K))) return hipSuccess;
  return launch_col_reduce((const float*)ws, M > 0 ? norm_grad_plan(M, K).blocks : 0, 2 * pitch, K, dw, pitch, db, st);
}

}  // namespace awq
