// The balance loss of a router's scores, its experts' slot counts, and the
// gradient of the logits (awq_balance_loss, awq_balance_loss_backward):
//   p_te   = exp(l_te) / sum_i exp(l_ti), or sigma(l_te) / sum_i sigma(l_ti)
//   c_e    = slots of the counted rows whose id is e,  n = sum_e c_e
//   slope_e = coef E c_e / (n T'),  loss = sum_e slope_e sum_t p_te
//   dl_te  = go p_te (slope_e - sum_i p_ti slope_i)       (sigmoid: times 1 - sigma(l_te))
// over the T' rows that are not masked out and have a usable logit.
//
//   1. k_balance: a wave per row, its logits in registers (lane l: V adjacent
//      experts from V l on, one access; 2 x 8 above 512 experts), the next
//      row's on their way meanwhile; the p of a wave's rows add up in
//      registers, the ids in an integer histogram in LDS; the block's waves
//      meet in LDS in their order and leave one partial row.
//   2. k_balance_finish: a block per 64 experts adds the partial rows in their
//      order (the p in double) and forms slopes and loss.  (One block for all of
//      256 experts took 13 us to read half a megabyte.)
//   3. k_balance_grad: a wave per row again.
// Bound by reading the logits (and writing their gradient); nothing is added
// by floating-point atomics, so the results do not depend on an order.  16384 x
// 256 with sigmoid scores: 15 us and 11 for the gradient; 519 x 60: 8 and 3.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_epilogue.h"

namespace awqk {

constexpr int kBalWaves = 16;          // of k_balance's block
constexpr int kBalGradWaves = 4;       // of k_balance_grad's

// Experts of lane l: V adjacent ones from V l on, H times, 64 V apart.
template <int V, int H>
struct BalMap {
  static constexpr int N = V * H;
  static __device__ __forceinline__ int first(int lane, int h) { return (h * 64 + lane) * V; }
};

// V adjacent values of a row from e on; -inf past its end.
template <int DT, int V>
__device__ __forceinline__ void bal_load(const void* p, int64_t row, int e, int E, float* v) {
  constexpr float off = -__builtin_inff();
  if (e + V <= E) {
    if constexpr (DT == DT_F32) {
      const float* q = reinterpret_cast<const float*>(p) + row + e;
      if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const u32x4a4 a = *reinterpret_cast<const u32x4a4*>(q + j);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j + i] = __uint_as_float(a[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = q[j];
      }
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + row + e;
      uint32_t w[(V + 1) / 2];
      if constexpr (V == 8) {
        const u32x4a2 a = *reinterpret_cast<const u32x4a2*>(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = a[i];
      } else if constexpr (V == 4) {
        const u32x2a2 a = *reinterpret_cast<const u32x2a2*>(q);
        w[0] = a[0];
        w[1] = a[1];
      } else if constexpr (V == 2) {
        w[0] = (uint32_t)q[0] | ((uint32_t)q[1] << 16);
      } else {
        w[0] = q[0];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = j & 1 ? hi_f32<DT>(w[j / 2]) : lo_f32<DT>(w[j / 2]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = e + j < E ? load_any(p, DT, row + e + j) : off;
  }
}

template <int DT, int V>
__device__ __forceinline__ void bal_store(void* p, int64_t row, int e, int E, const float* v) {
  if constexpr (V >= 4) {
    if (e + V <= E) {
      if constexpr (DT == DT_F32) {
        float* q = reinterpret_cast<float*>(p) + row + e;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          u32x4a4 a;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(v[j + i]);
          *reinterpret_cast<u32x4a4*>(q + j) = a;
        }
      } else {
        uint16_t* q = reinterpret_cast<uint16_t*>(p) + row + e;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          u32x2a2 a;
#pragma unroll
          for (int i = 0; i < 2; ++i) a[i] = from_f32<DT>(v[j + 2 * i]) | (from_f32<DT>(v[j + 2 * i + 1]) << 16);
          *reinterpret_cast<u32x2a2*>(q + j) = a;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (e + j < E) store_any(p, DT, row + e + j, v[j]);
}

// exp(x) for x <= 0.  For logits in 32 bits 2^(x log2 e) with the product's
// rounding error (and what log2 e leaves of its fp32 value) put back in first
// order, so that far scores keep fp32's precision; for 16 bits without: |x|
// 2^-24 of the result, below what the logits themselves hold.  Past -126 in the
// exponent the result is 0.
template <bool WIDE>
__device__ __forceinline__ float bal_exp(float x) {
  constexpr float hi = kLog2E, lo = (float)(1.4426950408889634 - (double)kLog2E);
  if constexpr (!WIDE) return __builtin_amdgcn_exp2f(x * hi);
  x = x > -1000.0f ? x : -1000.0f;                 // (-inf: no inf - inf below)
  const float p = x * hi;
  const float r = __builtin_fmaf(x, hi, -p) + x * lo;
  const float e = __builtin_amdgcn_exp2f(p);
  return __builtin_fmaf(e, r * 0.69314718f, e);
}

// A row's scores in s (not yet divided by their sum, which is returned; 0: no
// usable logit) and, for the sigmoid, what is left of one in rest (1 - sigma).
// -inf and NaN are not usable; +inf counts as the largest float.  Sigmoid
// scores carry a common factor exp(-min(max l, 0)), so that a row of very low
// logits does not underflow.
template <int N, bool SIG, bool REST, bool WIDE>
__device__ __forceinline__ float bal_scores(float (&s)[N], float (&rest)[N]) {
  float mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = s[i] > -__builtin_inff() ? fminf(s[i], 3.4028234663852886e38f) : -__builtin_inff();   // NaN: not greater
    mx = fmaxf(mx, s[i]);
  }
  mx = wave_max(mx);
  if (mx == -__builtin_inff()) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = rest[i] = 0.0f;
    return 0.0f;
  }
  float sum = 0.0f;
  const float c = SIG ? fminf(mx, 0.0f) : mx, ec = SIG ? bal_exp<WIDE>(c) : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (SIG) {
      // l >= 0 (then c = 0): 1 / (1 + e^-l);  l < 0: e^(l - c) / (1 + e^(l - c) e^c)
      const float l = s[i];
      const float a = bal_exp<WIDE>(l >= 0.0f ? -l : l - c);
      const float d = quick_rcp(l >= 0.0f ? 1.0f + a : __builtin_fmaf(a, ec, 1.0f));
      s[i] = l >= 0.0f ? d : a * d;
      if constexpr (REST) rest[i] = l >= 0.0f ? a * d : d;
    } else {
      s[i] = bal_exp<WIDE>(s[i] - c);
    }
    sum += s[i];
  }
  return wave_sum(sum);
}

// What the blocks of k_balance_finish leave for the one that ends last.
struct BalanceEnd {
  double part[16];       // E <= 1024
  unsigned done;
};

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  float* loss;           // one block forms the results by itself
  int32_t* counts;
  float* slope;
  double coef;
  float2* partial;       // [blocks][pitch]: sum of p, slots (an integer's bits); at E (the bits of) all slots, rows
  BalanceEnd* last;
  int64_t T, ldl, pitch;
  int E, top_k;
};

// The loss's derivative by a p: coef E c / (n T').
__device__ __forceinline__ double bal_slope(double coef, int E, int c, double slots, double rows) {
  return slots > 0.0 && rows > 0.0 ? coef * (double)E * (double)c / (slots * rows) : 0.0;
}

template <int DT, int V, int H, bool SIG>
__global__ __launch_bounds__(64 * kBalWaves) void k_balance(const BalanceArgs a) {
  using Map = BalMap<V, H>;
  constexpr int N = Map::N;
  extern __shared__ int32_t bal_lds[];
  int32_t* hist = bal_lds;                                       // [E + 2]: slots of each expert, of all, rows
  float* meet = reinterpret_cast<float*>(bal_lds + a.E + 2);     // [kBalWaves][64 N]
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int e = threadIdx.x; e <= a.E + 1; e += 64 * kBalWaves) hist[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && gridDim.x > 1) a.last->done = 0;
  __syncthreads();
  float acc[N], next[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * kBalWaves;
  int64_t t = (int64_t)blockIdx.x * kBalWaves + wv;
  int next_id = -1;
  bool next_on = false;
  auto fetch = [&](int64_t r) {                                  // row r < T
#pragma unroll
    for (int h = 0; h < H; ++h) bal_load<DT, V>(a.logits, r * a.ldl, Map::first(lane, h), a.E, next + h * V);
    next_id = lane < a.top_k ? a.ids[r * a.top_k + lane] : -1;
    next_on = !a.mask || a.mask[r] != 0;
  };
  if (t < a.T) fetch(t);
  for (; t < a.T; t += step) {                                   // wave-uniform
    float s[N], rest[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = next[i];
    const int id = next_id;
    const bool on = next_on;
    if (t + step < a.T) fetch(t + step);
    if (!on) continue;
    const float sum = bal_scores<N, SIG, false, DT == DT_F32>(s, rest);
    if (sum == 0.0f) continue;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(s[i], inv, acc[i]);
    const bool named = id >= 0 && id < a.E;
    if (named) atomicAdd(&hist[id], 1);
    const int all = __popcll(__ballot(named));
    if (lane == 0) {
      atomicAdd(&hist[a.E], all);
      atomicAdd(&hist[a.E + 1], 1);
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < V; ++j) meet[wv * 64 * N + Map::first(lane, h) + j] = acc[h * V + j];
  __syncthreads();
  if (gridDim.x == 1) {
    __shared__ double part[kBalWaves];
    const double slots = hist[a.E], rows = hist[a.E + 1];
    double l = 0.0;
    for (int e = threadIdx.x; e < a.E; e += 64 * kBalWaves) {
      const double sl = bal_slope(a.coef, a.E, hist[e], slots, rows);
      double p = 0.0;
#pragma unroll
      for (int w = 0; w < kBalWaves; ++w) p += meet[w * 64 * N + e];
      l += sl * p;
      a.counts[e] = hist[e];
      a.slope[e] = (float)sl;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off);
    if (lane == 0) part[wv] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kBalWaves; ++w) l += part[w];
      a.loss[0] = (float)l;
    }
    return;
  }
  for (int e = threadIdx.x; e <= a.E; e += 64 * kBalWaves) {
    float2 v = make_float2(0.0f, __int_as_float(hist[e]));
    if (e < a.E) {
#pragma unroll
      for (int w = 0; w < kBalWaves; ++w) v.x += meet[w * 64 * N + e];
    } else {
      v = make_float2(__int_as_float(hist[a.E]), __int_as_float(hist[a.E + 1]));
    }
    a.partial[blockIdx.x * a.pitch + e] = v;
  }
}

// Block j adds the partial rows of experts 64 j .. 64 j + 63 in their order (16
// waves, every sixteenth row each, meeting in LDS in their order) and forms
// their counts and slopes; n and the number of rows come from the last column
// (slots, rows), which every block adds up for itself.  The parts of the loss
// meet in the block that ends last, again in their order: `last` holds the
// parts and a count of the blocks that are done, zeroed by k_balance.
__global__ __launch_bounds__(1024) void k_balance_finish(const float2* __restrict__ partial, int blocks, int64_t pitch,
                                                         int E, double coef, float* __restrict__ loss,
                                                         int32_t* __restrict__ counts, float* __restrict__ slope,
                                                         BalanceEnd* __restrict__ last) {
  __shared__ double p_s[16][64];
  __shared__ int32_t c_s[16][64];
  __shared__ long long tot[2][16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  const int ec = e < E ? e : 0;
  double p = 0.0;
  int32_t c = 0;
  long long slots = 0, rows = 0;
  constexpr int U = 16;                                          // partial rows in flight
  for (int b0 = wv; b0 < blocks; b0 += 16 * U) {
    float2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + 16 * u;                                 // past the end: the first row, not used
      v[u] = partial[(int64_t)(b < blocks ? b : 0) * pitch + ec];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = b0 + 16 * u < blocks;
      p += ok ? v[u].x : 0.0f;
      c += ok ? __float_as_int(v[u].y) : 0;
    }
  }
  for (int b = threadIdx.x; b < blocks; b += 1024) {
    const float2 v = partial[(int64_t)b * pitch + E];
    slots += __float_as_int(v.x);
    rows += __float_as_int(v.y);
  }
  p_s[wv][lane] = p;
  c_s[wv][lane] = c;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    slots += __shfl_xor(slots, off);
    rows += __shfl_xor(rows, off);
  }
  if (lane == 0) {
    tot[0][wv] = slots;
    tot[1][wv] = rows;
  }
  __syncthreads();
  if (wv > 0) return;
  for (int w = 1; w < 16; ++w) {
    p += p_s[w][lane];
    c += c_s[w][lane];
    slots += tot[0][w];
    rows += tot[1][w];
  }
  const double sl = bal_slope(coef, E, c, (double)slots, (double)rows);
  double l = e < E ? sl * p : 0.0;
  if (e < E) {
    counts[e] = c;
    slope[e] = (float)sl;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off);
  if (lane > 0) return;
  if (gridDim.x == 1) {
    loss[0] = (float)l;
    return;
  }
  __hip_atomic_store(&last->part[blockIdx.x], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__hip_atomic_fetch_add(&last->done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != gridDim.x - 1) return;
  l = 0.0;
  for (unsigned j = 0; j < gridDim.x; ++j) l += __hip_atomic_load(&last->part[j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  loss[0] = (float)l;
}

// No tokens: zeros.
__global__ __launch_bounds__(256) void k_balance_none(int E, float* __restrict__ loss, int32_t* __restrict__ counts,
                                                      float* __restrict__ slope) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e == 0) loss[0] = 0.0f;
  if (e < E) {
    counts[e] = 0;
    slope[e] = 0.0f;
  }
}

struct BalanceGradArgs {
  const void* logits;
  const float* slope;
  const float* go;
  const uint8_t* mask;
  void* dl;
  int64_t T, ldl, ldd;
  int E;
};

template <int DT, int V, int H, bool SIG>
__global__ __launch_bounds__(64 * kBalGradWaves) void k_balance_grad(const BalanceGradArgs a) {
  using Map = BalMap<V, H>;
  constexpr int N = Map::N;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t step = (int64_t)gridDim.x * kBalGradWaves;
  int64_t t = (int64_t)blockIdx.x * kBalGradWaves + wv;
  float next[N];
  auto fetch = [&](int64_t r) {
    const bool on = !a.mask || a.mask[r] != 0;                   // wave-uniform
#pragma unroll
    for (int h = 0; h < H; ++h) bal_load<DT, V>(a.logits, r * a.ldl, Map::first(lane, h), on ? a.E : 0, next + h * V);
  };
  if (t < a.T) fetch(t);
  // the slopes about their mean, which the gradient does not see: what is left
  // cancels little in slope - sum p slope.  In double, where the sum is exact and
  // equal slopes leave 0, as their gradient is.
  float d[N];
  double mean = 0.0;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = Map::first(lane, h) + j;
      d[h * V + j] = e < a.E ? a.slope[e] : 0.0f;
      mean += d[h * V + j];
    }
  const float go = a.go ? a.go[0] : 1.0f;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mean += __shfl_xor(mean, off);
  mean /= (double)a.E;
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = (float)((double)d[i] - mean);
  for (; t < a.T; t += step) {
    float s[N], rest[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = next[i];
    if (t + step < a.T) fetch(t + step);
    const float sum = bal_scores<N, SIG, SIG, DT == DT_F32>(s, rest);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] *= inv;
      q = __builtin_fmaf(s[i], d[i], q);
    }
    q = wave_sum(q);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // a score of 0 (masked, off, or far below) has no gradient, whatever go is
      const float o = s[i] > 0.0f ? go * s[i] * (d[i] - q) : 0.0f;
      s[i] = SIG ? o * rest[i] : o;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) bal_store<DT, V>(a.dl, t * a.ldd, Map::first(lane, h), a.E, s + h * V);
  }
}

inline int64_t balance_blocks(int64_t T) {
  // a row per wave up to 256 blocks; up to eight rows per wave make one block,
  // which forms the results by itself
  const int64_t want = (T + kBalWaves - 1) / kBalWaves;
  return want <= 8 ? 1 : want < 256 ? want : 256;
}
inline int64_t balance_pitch(int64_t E) { return (E + 1 + 63) / 64 * 64; }

template <int DT, int V, int H>
hipError_t balance_launch(const BalanceArgs& a, bool sigmoid, int64_t blocks, hipStream_t st) {
  const size_t lds = (size_t)(a.E + 2 + kBalWaves * 64 * V * H) * 4;
  const dim3 grid((unsigned)blocks), block(64 * kBalWaves);
  if (sigmoid) hipLaunchKernelGGL((k_balance<DT, V, H, true>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((k_balance<DT, V, H, false>), grid, block, lds, st, a);
  return hipGetLastError();
}
template <int DT, int V, int H>
hipError_t balance_launch(const BalanceGradArgs& a, bool sigmoid, int64_t blocks, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(64 * kBalGradWaves);
  if (sigmoid) hipLaunchKernelGGL((k_balance_grad<DT, V, H, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_balance_grad<DT, V, H, false>), grid, block, 0, st, a);
  return hipGetLastError();
}
template <int DT, class A>
hipError_t balance_dispatch(const A& a, bool sigmoid, int64_t blocks, hipStream_t st) {
  if (a.E <= 64) return balance_launch<DT, 1, 1>(a, sigmoid, blocks, st);
  if (a.E <= 128) return balance_launch<DT, 2, 1>(a, sigmoid, blocks, st);
  if (a.E <= 256) return balance_launch<DT, 4, 1>(a, sigmoid, blocks, st);
  if (a.E <= 512) return balance_launch<DT, 8, 1>(a, sigmoid, blocks, st);
  return balance_launch<DT, 8, 2>(a, sigmoid, blocks, st);
}
template <class A>
hipError_t balance_typed(const A& a, int dt, bool sigmoid, int64_t blocks, hipStream_t st) {
  if (dt == DT_F16) return balance_dispatch<DT_F16>(a, sigmoid, blocks, st);
  if (dt == DT_BF16) return balance_dispatch<DT_BF16>(a, sigmoid, blocks, st);
  return balance_dispatch<DT_F32>(a, sigmoid, blocks, st);
}

}  // namespace awqk

namespace awq {

size_t balance_ws_bytes(int64_t T, int64_t E) {
  if (T <= 0 || E <= 0 || awqk::balance_blocks(T) == 1) return 0;
  return align_up((size_t)(awqk::balance_blocks(T) * awqk::balance_pitch(E)) * 8, 256) + 256;   // and a BalanceEnd
}

hipError_t launch_balance(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const int32_t* ids, int top_k,
                          const uint8_t* mask, int sigmoid, double coef, float* loss, int32_t* counts, float* slope,
                          void* ws, hipStream_t st) {
  using namespace awqk;
  const int64_t blocks = T > 0 ? balance_blocks(T) : 0, pitch = balance_pitch(E);
  if (blocks == 0) {
    hipLaunchKernelGGL(k_balance_none, dim3((unsigned)((E + 255) / 256)), dim3(256), 0, st, (int)E, loss, counts, slope);
    return hipGetLastError();
  }
  BalanceEnd* last = (BalanceEnd*)ws;
  static_assert(sizeof(BalanceEnd) <= 256, "ahead of the partial rows");
  float2* partial = ws ? (float2*)((char*)ws + 256) : nullptr;
  const hipError_t e = balance_typed(BalanceArgs{logits, ids, mask, loss, counts, slope, coef, partial, last, T, ldl, pitch, (int)E, top_k}, dt,
                                     sigmoid != 0, blocks, st);
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(k_balance_finish, dim3((unsigned)((E + 63) / 64)), dim3(1024), 0, st, partial, (int)blocks, pitch,
                     (int)E, coef, loss, counts, slope, last);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const float* slope,
                               const float* go, const uint8_t* mask, int sigmoid, void* dl, int64_t ldd, hipStream_t st) {
  using namespace awqk;
  const int64_t want = (T + kBalGradWaves - 1) / kBalGradWaves, blocks = want < 2048 ? want : 2048;
  return balance_typed(BalanceGradArgs{logits, slope, go, mask, dl, T, ldl, ldd, (int)E}, dt, sigmoid != 0, blocks, st);
}

}  // namespace awq
