// The balance loss of a router's scores, its experts' slot counts, and the
// gradient of the logits (awq_balance_loss, awq_balance_loss_backward):
//   p_te   = exp(l_te) / sum_i exp(l_ti), or sigma(l_te) / sum_i sigma(l_ti)
//   c_e    = slots of the counted rows whose id is e,  n = sum_e c_e
//   slope_e = coef E c_e / (n T'),  loss = sum_e slope_e sum_t p_te
//   dl_te  = go p_te (slope_e - sum_i p_ti slope_i)       (sigmoid: times 1 - sigma(l_te))
// over the T' rows that are not masked out and have a usable logit.
//
//   1. k_balance: a wave per row, its logits in registers (lane l: experts
//      l, l + 64, ...); the p of a wave's rows add up in registers, the ids in
//      an integer histogram in LDS; a block leaves one partial row of both.
//   2. k_balance_finish: one block adds the partial rows in their order (the p
//      in double), and forms slopes and loss.
//   3. k_balance_grad: a wave per row again.
// Bound by reading the logits (and writing their gradient); nothing is added
// by floating-point atomics, so the results do not depend on an order.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"

namespace awqk {

constexpr int kBalWaves = 4;

// A row's scores in s (not yet divided by their sum, which is returned; 0: no
// usable logit) and, for the sigmoid, what is left of one in rest (1 - sigma).
// -inf and NaN are not usable; +inf counts as the largest float.  Sigmoid
// scores carry a common factor exp(-min(max l, 0)), so that a row of very low
// logits does not underflow.
template <int EPL, bool SIG, bool REST>
__device__ __forceinline__ float bal_scores(float (&s)[EPL], float (&rest)[EPL]) {
  float mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    s[i] = s[i] > -__builtin_inff() ? fminf(s[i], 3.4028234663852886e38f) : -__builtin_inff();   // NaN: not greater
    mx = fmaxf(mx, s[i]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  if (mx == -__builtin_inff()) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = rest[i] = 0.0f;
    return 0.0f;
  }
  float sum = 0.0f;
  const float c = SIG ? fminf(mx, 0.0f) : mx, ec = SIG ? expf(c) : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if constexpr (SIG) {
      // l >= 0 (then c = 0): 1 / (1 + e^-l);  l < 0: e^(l - c) / (1 + e^(l - c) e^c)
      const float l = s[i];
      const float a = expf(l >= 0.0f ? -l : l - c);
      const float d = 1.0f / (l >= 0.0f ? 1.0f + a : __builtin_fmaf(a, ec, 1.0f));
      s[i] = l >= 0.0f ? d : a * d;
      if constexpr (REST) rest[i] = l >= 0.0f ? a * d : d;
    } else {
      s[i] = expf(s[i] - c);
    }
    sum += s[i];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  return sum;
}

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  float* psum;           // [blocks][pitch]
  int32_t* count;        // [blocks][pitch], the number of counted rows at E
  int64_t T, ldl, pitch;
  int E, top_k, dt;
};

template <int EPL, bool SIG>
__global__ __launch_bounds__(64 * kBalWaves) void k_balance(const BalanceArgs a) {
  extern __shared__ int32_t bal_lds[];
  int32_t* hist = bal_lds;                                       // [E + 1]
  float* meet = reinterpret_cast<float*>(bal_lds + a.E + 1);     // [kBalWaves][64 EPL]
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int e = threadIdx.x; e <= a.E; e += 64 * kBalWaves) hist[e] = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kBalWaves + wv; t < a.T; t += (int64_t)gridDim.x * kBalWaves) {
    if (a.mask && a.mask[t] == 0) continue;                      // wave-uniform
    float s[EPL], rest[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      s[i] = e < a.E ? load_any(a.logits, a.dt, t * a.ldl + e) : -__builtin_inff();
    }
    const int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    const float sum = bal_scores<EPL, SIG, false>(s, rest);
    if (sum == 0.0f) continue;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = __builtin_fmaf(s[i], inv, acc[i]);
    if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
    if (lane == 0) atomicAdd(&hist[a.E], 1);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) meet[wv * 64 * EPL + 64 * i + lane] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += 64 * kBalWaves) {
    a.count[blockIdx.x * a.pitch + e] = hist[e];
    if (e < a.E) {
      float t = 0.0f;
      for (int w = 0; w < kBalWaves; ++w) t += meet[w * 64 * EPL + e];
      a.psum[blockIdx.x * a.pitch + e] = t;
    }
  }
}

// One block; thread e takes expert e.
__global__ __launch_bounds__(1024) void k_balance_finish(const float* __restrict__ psum, const int32_t* __restrict__ count,
                                                         int blocks, int64_t pitch, int E, double coef,
                                                         float* __restrict__ loss, int32_t* __restrict__ counts,
                                                         float* __restrict__ slope) {
  __shared__ double part[16];
  __shared__ long long total[16];
  const int e = threadIdx.x, lane = e & 63, wv = e >> 6;
  double p = 0.0;
  long long c = 0, rows = 0;
  if (e < E)
    for (int b = 0; b < blocks; ++b) {
      p += psum[b * pitch + e];
      c += count[b * pitch + e];
    }
  for (int b = 0; b < blocks; ++b) rows += count[b * pitch + E];
  long long n = c;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off);
  if (lane == 0) total[wv] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) n += total[w];
  const double sl = n > 0 && rows > 0 ? coef * (double)E * (double)c / ((double)n * (double)rows) : 0.0;
  double l = e < E ? sl * p : 0.0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off);
  if (lane == 0) part[wv] = l;
  __syncthreads();
  if (e < E) {
    counts[e] = (int32_t)c;
    slope[e] = (float)sl;
  }
  if (e == 0) {
    l = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) l += part[w];
    loss[0] = (float)l;
  }
}

struct BalanceGradArgs {
  const void* logits;
  const float* slope;
  const float* go;
  const uint8_t* mask;
  void* dl;
  int64_t T, ldl, ldd;
  int E, dt;
};

template <int EPL, bool SIG>
__global__ __launch_bounds__(64 * kBalWaves) void k_balance_grad(const BalanceGradArgs a) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  // the slopes about their mean, which the gradient does not see: what is left
  // cancels little in slope - sum p slope
  float d[EPL];
  float mean = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    d[i] = e < a.E ? a.slope[e] : 0.0f;
    mean += d[i];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mean += __shfl_xor(mean, off);
  mean /= (float)a.E;
  const float go = a.go ? a.go[0] : 1.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) d[i] -= mean;
  for (int64_t t = (int64_t)blockIdx.x * kBalWaves + wv; t < a.T; t += (int64_t)gridDim.x * kBalWaves) {
    float s[EPL], rest[EPL], o[EPL];
    const bool on = !a.mask || a.mask[t] != 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      s[i] = on && e < a.E ? load_any(a.logits, a.dt, t * a.ldl + e) : -__builtin_inff();
    }
    const float sum = bal_scores<EPL, SIG, SIG>(s, rest);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] *= inv;
      q = __builtin_fmaf(s[i], d[i], q);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) q += __shfl_xor(q, off);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // a score of 0 (masked, off, or far below) has no gradient, whatever go is
      o[i] = s[i] > 0.0f ? go * s[i] * (d[i] - q) : 0.0f;
      if constexpr (SIG) o[i] *= rest[i];
      const int e = lane + 64 * i;
      if (e < a.E) store_any(a.dl, a.dt, t * a.ldd + e, o[i]);
    }
  }
}

inline int64_t balance_blocks(int64_t T) {
  const int64_t want = (T + kBalWaves - 1) / kBalWaves;
  return want < 128 ? want : 128;
}
inline int64_t balance_pitch(int64_t E) { return (E + 1 + 63) / 64 * 64; }

}  // namespace awqk

namespace awq {

size_t balance_ws_bytes(int64_t T, int64_t E) {
  if (T <= 0 || E <= 0) return 0;
  return align_up((size_t)(awqk::balance_blocks(T) * awqk::balance_pitch(E)) * 8, 256);
}

hipError_t launch_balance(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const int32_t* ids, int top_k,
                          const uint8_t* mask, int sigmoid, double coef, float* loss, int32_t* counts, float* slope,
                          void* ws, hipStream_t st) {
  using namespace awqk;
  const int64_t blocks = T > 0 ? balance_blocks(T) : 0, pitch = balance_pitch(E);
  float* psum = (float*)ws;
  int32_t* count = (int32_t*)(psum + blocks * pitch);
  if (blocks > 0) {
    const BalanceArgs a{logits, ids, mask, psum, count, T, ldl, pitch, (int)E, top_k, dt};
#define AWQ_B(EPL)                                                                                              \
  {                                                                                                             \
    const size_t lds = (size_t)(E + 1 + kBalWaves * 64 * EPL) * 4;                                              \
    if (sigmoid) hipLaunchKernelGGL((k_balance<EPL, true>), dim3((unsigned)blocks), dim3(64 * kBalWaves), lds, st, a); \
    else hipLaunchKernelGGL((k_balance<EPL, false>), dim3((unsigned)blocks), dim3(64 * kBalWaves), lds, st, a); \
  }
    if (E <= 64) AWQ_B(1)
    else if (E <= 128) AWQ_B(2)
    else if (E <= 256) AWQ_B(4)
    else if (E <= 512) AWQ_B(8)
    else AWQ_B(16)
#undef AWQ_B
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_balance_finish, dim3(1), dim3((unsigned)((E + 63) / 64 * 64)), 0, st, psum, count, (int)blocks,
                     pitch, (int)E, coef, loss, counts, slope);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const float* slope,
                               const float* go, const uint8_t* mask, int sigmoid, void* dl, int64_t ldd, hipStream_t st) {
  using namespace awqk;
  const BalanceGradArgs a{logits, slope, go, mask, dl, T, ldl, ldd, (int)E, dt};
  const int64_t want = (T + kBalWaves - 1) / kBalWaves, blocks = want < 2048 ? want : 2048;
#define AWQ_BG(EPL)                                                                                             \
  {                                                                                                             \
    if (sigmoid) hipLaunchKernelGGL((k_balance_grad<EPL, true>), dim3((unsigned)blocks), dim3(64 * kBalWaves), 0, st, a); \
    else hipLaunchKernelGGL((k_balance_grad<EPL, false>), dim3((unsigned)blocks), dim3(64 * kBalWaves), 0, st, a); \
  }
  if (E <= 64) AWQ_BG(1)
  else if (E <= 128) AWQ_BG(2)
  else if (E <= 256) AWQ_BG(4)
  else if (E <= 512) AWQ_BG(8)
  else AWQ_BG(16)
#undef AWQ_BG
  return hipGetLastError();
}

}  // namespace awq
