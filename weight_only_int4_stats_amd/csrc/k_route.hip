// Expert routing: scores of a token's logits, a bias and groups that choose,
// the top k and their weights (include/awq.h, awq_route_experts).
//
// One wave per token, V = ceil(E / 64) consecutive experts per lane.  The row
// is read once and never leaves registers: the softmax's maximum and sum are
// wave reductions, a group's two largest choices are merged over the lanes
// that hold it, and the k winners are taken one after another.  Choices are
// doubles (a choice between close scores must not depend on rounding), but a
// winner is found on their float roundings, which keep the order: one float
// maximum over the wave and one ballot, and only a tie of the roundings is
// settled on the doubles.  Equal choices leave the lowest lane, and the lane's
// lowest expert, first.
#include "awq_device.h"
#include "awq_internal.h"

#include <type_traits>

namespace awqk {

// Maximum over the wave, in every lane (row exchanges, then the two swaps
// across the 16-lane rows; no LDS traffic).
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, quad_xor1(v));
  v = fmaxf(v, quad_xor2(v));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

template <int DT>
__device__ __forceinline__ float route_load(const void* p, int64_t i) {
  float f;
  if constexpr (DT == DT_F32) f = reinterpret_cast<const float*>(p)[i];
  else f = to_f32<DT>(reinterpret_cast<const uint16_t*>(p)[i]);
  return fminf(f, 3.402823466e+38f);   // +inf counts as the largest float; NaN is handled by the caller
}

// (a1, a2) and (b1, b2), each the two largest of a set: the two largest of both.
__device__ __forceinline__ void merge_top2(double& a1, double& a2, double b1, double b2) {
  const double lo = fmin(a1, b1);
  a1 = fmax(a1, b1);
  a2 = fmax(lo, fmax(a2, b2));
}

struct RouteArgs {
  const void* logits;
  int64_t T, ldl;
  int E;
  const float* bias;
  int sigmoid, n_group, topk_group, group_top, top_k, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

template <int DT, int V>
__global__ __launch_bounds__(256) void k_route(const RouteArgs p) {
  constexpr double kNone = -__builtin_inf();
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= p.T) return;
  const char* row = reinterpret_cast<const char*>(p.logits) + t * p.ldl * (DT == DT_F32 ? 4 : 2);

  float l[V];
  bool ok[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    float f = -__builtin_inff();
    if (e < p.E) {
      if constexpr (DT == DT_F32) f = reinterpret_cast<const float*>(row)[e];
      else f = to_f32<DT>(reinterpret_cast<const uint16_t*>(row)[e]);
    }
    ok[i] = f > -__builtin_inff();                 // false for NaN too
    l[i] = ok[i] ? fminf(f, 3.402823466e+38f) : -__builtin_inff();
  }

  // ---- scores and choices
  double c[V];
  double mx = 0.0, sum = 0.0;
  if (!p.sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    mx = (double)wave_max(m);                      // -inf: no expert is usable, every choice below is -inf
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = ok[i] ? exp((double)l[i] - mx) : 0.0;
      sum += c[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = c[i] / sum;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    if (p.bias && e < p.E) c[i] += (double)p.bias[e];
    if (!ok[i]) c[i] = kNone;
  }

  // ---- groups
  if (p.n_group > 1) {
    const int gs = p.E / p.n_group;
    const bool two = p.group_top == 2 && gs > 1;
    const int lg = gs / V;                         // lanes per group
    double gv = kNone;                             // lane g: what group g is worth
    if (gs % V == 0 && (lg & (lg - 1)) == 0) {
      double a1 = c[0], a2 = kNone;
#pragma unroll
      for (int i = 1; i < V; ++i) merge_top2(a1, a2, c[i], kNone);
      for (int off = 1; off < lg; off <<= 1) {
        const double b1 = __shfl_xor(a1, off), b2 = __shfl_xor(a2, off);
        merge_top2(a1, a2, b1, b2);
      }
      gv = __shfl(two ? a1 + a2 : a1, (lane * lg) & 63);
    } else {
      for (int g = 0; g < p.n_group; ++g) {
        double a1 = kNone, a2 = kNone;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = lane * V + i;
          if (e >= g * gs && e < (g + 1) * gs) merge_top2(a1, a2, c[i], kNone);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const double b1 = __shfl_xor(a1, off), b2 = __shfl_xor(a2, off);
          merge_top2(a1, a2, b1, b2);
        }
        if (lane == g) gv = two ? a1 + a2 : a1;
      }
    }
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const double v = __shfl(gv, g);
      rank += (v > gv || (v == gv && g < lane)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(lane < p.n_group && rank < p.topk_group);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < p.E && !((keep >> (e / gs)) & 1)) c[i] = kNone;
    }
  }

  // ---- the top k: lane j keeps winner j
  int mine = -1;
  double cb;
  int ib;
  auto best = [&]() {
    cb = c[0];
    ib = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (c[i] > cb) {
        cb = c[i];
        ib = i;
      }
  };
  best();
  for (int j = 0; j < p.top_k; ++j) {
    const float kb = (float)cb;
    const float m = wave_max(kb);
    if (!(m > -__builtin_inff())) break;           // nothing usable left (wave-uniform)
    uint64_t at = __ballot(kb == m);
    if (at & (at - 1)) {                           // a tie of the roundings: the doubles decide
      const double d = wave_max(kb == m ? cb : kNone);
      at = __ballot(kb == m && cb == d);
    }
    const int w = __builtin_ctzll(at);
    const int wi = __builtin_amdgcn_readlane(ib, w);
    if (lane == j) mine = w * V + wi;
    if (lane == w) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == wi) c[i] = kNone;
    }
    best();
  }

  // ---- weights: the winners' scores again, from their logits
  double s = 0.0;
  if (mine >= 0) {
    const float f = route_load<DT>(row, mine);
    s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)f)) : exp((double)f - mx) / sum;
  }
  if (p.renorm) {
    const double total = wave_sum(s);
    if (total > 0.0) s /= total;
  }
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = mine;
    p.weights[t * p.top_k + lane] = (float)(s * (double)p.scale);
  }
}

}  // namespace awqk

namespace awq {

hipError_t launch_route(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const float* bias,
                        int sigmoid, int n_group, int topk_group, int group_top, int top_k, int renorm,
                        float scale, int32_t* ids, float* weights, hipStream_t st) {
  using namespace awqk;
  const RouteArgs p{logits, T, ldl, (int)E, bias, sigmoid, n_group, topk_group, group_top, top_k, renorm,
                    scale, ids, weights};
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  auto go = [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    if (E <= 64) hipLaunchKernelGGL((k_route<DT, 1>), grid, block, 0, st, p);
    else if (E <= 128) hipLaunchKernelGGL((k_route<DT, 2>), grid, block, 0, st, p);
    else if (E <= 256) hipLaunchKernelGGL((k_route<DT, 4>), grid, block, 0, st, p);
    else if (E <= 512) hipLaunchKernelGGL((k_route<DT, 8>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_route<DT, 16>), grid, block, 0, st, p);
  };
  if (dt == DT_F16) go(std::integral_constant<int, DT_F16>{});
  else if (dt == DT_BF16) go(std::integral_constant<int, DT_BF16>{});
  else go(std::integral_constant<int, DT_F32>{});
  return hipGetLastError();
}

}  // namespace awq
