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
//
// The choosing runs in float first (route_float) wherever float can prove the
// order: without a bias the logits themselves are the keys, with one the
// choice's float error is far below the distance that two neighbours in the
// order must have.  A row with a closer call (about one in a hundred) repeats it in
// doubles.  16384 tokens, 256 experts in 8 groups, top 8 with a bias: 29 us
// in doubles alone, 23 to 25 us with both: a winner takes some thirty
// instructions, six of them steps across the lanes, for the wave's one token.
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
  int sigmoid, n_group, gsize, topk_group, group_top, top_k, renorm;   // gsize: experts per group
  float scale;
  int32_t* ids;
  float* weights;
};

// Floats as unsigned integers in the same order (-inf: kNoKey; 0 is below all).
constexpr uint32_t kNoKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t to_key(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return v > o ? v : o;
}
// Maximum over the wave, as a scalar: shifts inside the 16-lane rows, the rows'
// last lanes broadcast onwards, the last lane read.
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max_dpp<0x111, 0xF>(v);
  v = max_dpp<0x112, 0xF>(v);
  v = max_dpp<0x114, 0xF>(v);
  v = max_dpp<0x118, 0xF>(v);
  v = max_dpp<0x142, 0xA>(v);
  v = max_dpp<0x143, 0xC>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// (a1, a2) and another lane's pair: the two largest of both.
__device__ __forceinline__ void merge_keys(uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
  const uint32_t lo = a1 < b1 ? a1 : b1, hi2 = a2 > b2 ? a2 : b2;
  a1 = a1 > b1 ? a1 : b1;
  a2 = lo > hi2 ? lo : hi2;
}
template <int CTRL>
__device__ __forceinline__ void merge_keys_dpp(uint32_t& a1, uint32_t& a2) {
  merge_keys(a1, a2, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a1, CTRL, 0xF, 0xF, false),
             (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a2, CTRL, 0xF, 0xF, false));
}

// exp(d + dl) within 2^-21 of the value (dl: the rounding error of d), and
// within 2^-100 of it where d was held to -100 .. 80: 2^(d log2 e), the product
// in two floats.  log2 e = kL + kLl (1 / ln 2 = 1.44269504088896340736,
// its nearest float and the nearest float to the rest, 1.92596299e-8: the
// splitting of a constant in two parts of Cody and Waite, Software Manual for
// the Elementary Functions, 1980).
__device__ __forceinline__ float exp_f32(float d, float dl) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kL = (float)kLog2e, kLl = (float)(kLog2e - (double)kL);
  const bool in = d > -100.0f && d < 80.0f;
  d = in ? d : d > 0.0f ? 80.0f : -100.0f;
  dl = in ? dl : 0.0f;
  const float t = d * kL;
  const float lo = __builtin_fmaf(dl, kL, __builtin_fmaf(d, kLl, __builtin_fmaf(d, kL, -t)));
  const float r = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(r * 0x1.62e43p-1f, lo, r);
}

// The choosing in float: lane j gets winner j's expert (-1: none left).
// Returns false where the order is not certain.  l: -inf where not usable, mx
// the largest; bias: the lane's.
template <int V>
__device__ __forceinline__ bool route_float(const RouteArgs& p, const float (&l)[V], const float (&bias)[V], float mx,
                                            int& mine) {
  constexpr float kNone = -__builtin_inff();
  const int lane = threadIdx.x & 63;
  const int gs = p.gsize;
  const bool two = p.n_group > 1 && p.group_top == 2 && gs > 1;
  const bool scores = p.bias || two;               // else the logits decide
  uint32_t c[V];
  float margin = 0.0f;                             // what choices must differ by, but for 2^-21 of themselves
  if (scores) {
    float s[V];
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + exp_f32(-l[i], 0.0f));
      margin = 0x1p-18f;
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = l[i] - mx, b = d - l[i];   // the difference and its rounding error
        const float x = exp_f32(d, (l[i] - (d - b)) - (mx + b));
        s[i] = l[i] > kNone ? x : 0.0f;
        sum += s[i];
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
      const float r = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= r;
      margin = r * 0x1p-18f;                       // no score exceeds r
    }
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] > kNone ? to_key(s[i] + bias[i]) : kNoKey;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = to_key(l[i]);
  }

  // ---- groups: their values, and whether the cut between the kept and the
  // others is clear
  if (p.n_group > 1) {
    const int lg = gs / V;
    const bool whole = gs % V == 0 && (lg & (lg - 1)) == 0;   // a group is a power of two of whole lanes
    uint32_t a1, a2, gv = 0;
    // the size of the largest finite choice of the pairs that this lane sums:
    // where a pair cancels, its rounding is what the sum is off by
    float term = 0.0f;
    auto pair = [&]() {
      const float x = from_key(a1), y = from_key(a2);
      if (fabsf(x) < __builtin_inff()) term = fmaxf(term, fabsf(x));
      if (fabsf(y) < __builtin_inff()) term = fmaxf(term, fabsf(y));
      a1 = to_key(x + y);
    };
    if (whole) {
      a1 = c[0];
      a2 = kNoKey;
#pragma unroll
      for (int i = 1; i < V; ++i) merge_keys(a1, a2, c[i], kNoKey);
      if (lg > 1) merge_keys_dpp<0xB1>(a1, a2);    // lane ^ 1, ^ 2, then mirrors of equal halves
      if (lg > 2) merge_keys_dpp<0x4E>(a1, a2);
      if (lg > 4) merge_keys_dpp<0x141>(a1, a2);
      if (lg > 8) merge_keys_dpp<0x140>(a1, a2);
      if (lg > 16) merge_keys(a1, a2, (uint32_t)__shfl_xor((int)a1, 16), (uint32_t)__shfl_xor((int)a2, 16));
      if (lg > 32) merge_keys(a1, a2, (uint32_t)__shfl_xor((int)a1, 32), (uint32_t)__shfl_xor((int)a2, 32));
      if (two) pair();
      gv = (uint32_t)__shfl((int)a1, (lane * lg) & 63);
    } else {
      for (int g = 0; g < p.n_group; ++g) {
        a1 = a2 = kNoKey;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = lane * V + i;
          if (e >= g * gs && e < (g + 1) * gs) merge_keys(a1, a2, c[i], kNoKey);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
          merge_keys(a1, a2, (uint32_t)__shfl_xor((int)a1, off), (uint32_t)__shfl_xor((int)a2, off));
        if (two) pair();
        if (lane == g) gv = a1;
      }
    }
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)gv, g);
      rank += (v > gv || (v == gv && g < lane)) ? 1 : 0;
    }
    const bool in = lane < p.n_group;
    const uint64_t keep = __ballot(in && rank < p.topk_group);
    if (p.topk_group < p.n_group) {
      const float least = from_key(~wave_max_key(in && rank < p.topk_group ? ~gv : 0u));
      const float most = from_key(wave_max_key(in && rank >= p.topk_group ? gv : 0u));
      // a group is off by a margin and a float rounding (2^-24) of its choices and of their sum
      const float far = scores ? 2.0f * margin + 0x1p-20f * (fabsf(least) + fabsf(most) + term)
                               : 0x1p-18f * (1.0f + fabsf(least) + fabsf(most));
      if (__any(!(least - most > far))) return false;   // also where both are -inf
    }
    if (whole) {
      const bool out = !((keep >> (lane >> (31 - __builtin_clz((unsigned)lg)))) & 1);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = out ? kNoKey : c[i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = (lane * V + i) / gs;
        if (g < 64 && !((keep >> g) & 1)) c[i] = kNoKey;
      }
    }
  }
  const bool keys = !p.bias;                       // the logits order the experts
  if (two && keys) {                               // the scores were for the groups alone
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = c[i] > kNoKey ? to_key(l[i]) : kNoKey;
  }

  // ---- the top k and the next, lane j keeping number j.  Up to four experts
  // per lane in descending order (stable: equal keys keep the lower expert
  // first), more searched for their largest.
  constexpr bool kSorted = V <= 4;
  uint32_t order = 0;                              // sorted: the lane's experts left, two bits each
  if constexpr (kSorted) {
    uint32_t id[V];
#pragma unroll
    for (int i = 0; i < V; ++i) id[i] = (uint32_t)i;
#pragma unroll
    for (int n = V - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool s = c[i + 1] > c[i];
        const uint32_t hi = s ? c[i + 1] : c[i], lo = s ? c[i] : c[i + 1];
        const uint32_t ih = s ? id[i + 1] : id[i], il = s ? id[i] : id[i + 1];
        c[i] = hi;
        c[i + 1] = lo;
        id[i] = ih;
        id[i + 1] = il;
      }
#pragma unroll
    for (int i = 0; i < V; ++i) order |= id[i] << (2 * i);
  }
  uint32_t mykey = 0;
  mine = -1;
  for (int j = 0; j <= p.top_k; ++j) {
    uint32_t cb = c[0], ib = order;
    if constexpr (!kSorted) {
      ib = 0;
#pragma unroll
      for (int i = 1; i < V; ++i) {
        const bool g = c[i] > cb;
        cb = g ? c[i] : cb;
        ib = g ? (uint32_t)i : ib;
      }
    }
    const uint32_t m = wave_max_key(cb);
    const int w = __builtin_ctzll(__ballot(cb == m));
    uint32_t wi = (uint32_t)__builtin_amdgcn_readlane((int)ib, w);
    if constexpr (kSorted) wi &= 3;
    mykey = lane == j ? m : mykey;
    mine = lane == j ? w * V + (int)wi : mine;
    const bool won = lane == w;
    if constexpr (kSorted) {
      order = won ? order >> 2 : order;
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) c[i] = won ? c[i + 1] : c[i];
      c[V - 1] = won ? kNoKey : c[V - 1];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = (won && (uint32_t)i == wi) ? kNoKey : c[i];
    }
  }
  // ---- was it certain?  Each winner's distance from the next; equal logits
  // are ties.  Logits whose scores could meet in double, far down (softmax) or
  // saturated, are not: the sigmoids of f and f - gap are exp(-f) gap apart, at
  // 24 and the least gap still thirty steps of the doubles below 1 (2^-53), at
  // 28 less than one.  (A cut between groups up there shows in the first winner.)
  const uint32_t nextkey = (uint32_t)__shfl((int)mykey, lane + 1);
  const float f = from_key(mykey), n = from_key(nextkey), gap = f - n;
  bool sure;
  const float low = p.sigmoid ? -30.0f : mx - 600.0f, high = p.sigmoid ? 24.0f : __builtin_inff();
  if (keys) {
    sure = f > low && f < high && (gap == 0.0f || gap > 0x1p-18f * (1.0f + fabsf(f)));
  } else {
    sure = gap > margin + 0x1p-21f * (fabsf(f) + fabsf(n));
  }
  const bool there = mykey > kNoKey, last = nextkey <= kNoKey;   // last: nothing usable after it
  sure = sure || (last && (!keys || (f > low && f < high)));
  if (__any(lane < p.top_k && there && !sure)) return false;
  mine = lane < p.top_k && there ? mine : -1;
  return true;
}

// The choosing in double; also gives the softmax's sum.
template <int V>
__device__ __forceinline__ void route_double(const RouteArgs& p, const float (&l)[V], double mx, double& sum, int& mine) {
  constexpr double kNone = -__builtin_inf();
  const int lane = threadIdx.x & 63;
  double c[V];
  if (!p.sigmoid) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i] > -__builtin_inff() ? exp((double)l[i] - mx) : 0.0;
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
    if (!(l[i] > -__builtin_inff())) c[i] = kNone;
  }

  // ---- groups
  if (p.n_group > 1) {
    const int gs = p.gsize;
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
  mine = -1;
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

}

template <int DT, int V>
__global__ __launch_bounds__(256) void k_route(const RouteArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= p.T) return;
  const char* row = reinterpret_cast<const char*>(p.logits) + t * p.ldl * (DT == DT_F32 ? 4 : 2);

  // a logit of -inf or NaN switches its expert off; +inf counts as the largest float
  float l[V], bias[V];
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i, at = e < p.E ? e : 0;
    if constexpr (DT == DT_F32) l[i] = reinterpret_cast<const float*>(row)[at];
    else l[i] = to_f32<DT>(reinterpret_cast<const uint16_t*>(row)[at]);
    bias[i] = 0.0f;
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = p.bias[lane * V + i < p.E ? lane * V + i : 0];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = fminf(l[i], 3.402823466e+38f);
    const bool in = (lane * V + i < p.E) & (l[i] > -__builtin_inff());
    l[i] = in ? x + 0.0f : -__builtin_inff();      // -0 and 0 are one key
    m = fmaxf(m, l[i]);
  }
  m = wave_max(m);                                 // -inf: no expert is usable

  // the softmax's sum is left out where it cancels
  const bool no_sum = p.sigmoid || p.renorm;
  double sum = 1.0;
  int mine;
  if (!no_sum || !route_float<V>(p, l, bias, m, mine)) route_double<V>(p, l, (double)m, sum, mine);

  // ---- weights: the winners' scores again, from their logits
  double s = 0.0;
  if (mine >= 0) {
    const float f = route_load<DT>(row, mine);
    s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)f)) : exp((double)f - (double)m) / sum;
  }
  if (p.renorm) {
    double total = s;                              // lanes past the winners hold 0
    if (p.top_k > 16) {
      total = wave_sum(s);
    } else {
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) total += __shfl_xor(total, off);
    }
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
  const RouteArgs p{logits, T, ldl, (int)E, bias, sigmoid, n_group, (int)E / n_group, topk_group, group_top, top_k,
                    renorm, scale, ids, weights};
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
