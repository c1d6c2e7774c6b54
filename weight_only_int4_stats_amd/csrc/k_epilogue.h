// The epilogue of the W4A16 product (awq_w4a16_linear): bias, activation and
// residual applied in fp32 to a finished sum, and the activations' slopes.
#pragma once

#include <type_traits>

#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

using awq::Epilogue;

// A kernel's epilogue argument: NoEpi is the plain product (the sum is stored
// as it is), Epilogue the one above.
struct NoEpi {};
template <class EP>
constexpr bool kHasEpi = false;
template <>
inline constexpr bool kHasEpi<Epilogue> = true;

// Sum and maximum over a wave, in every lane: four exchanges within the 16-lane
// rows and two swaps between them, no LDS traffic (a shuffle each would be six
// round trips through LDS).
__device__ __forceinline__ float wave_sum(float v) {
  v += quad_xor1(v);
  v += quad_xor2(v);
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));   // row_half_mirror
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));   // row_mirror
  v = pair_sum16(v, v);
  return pair_sum32(v, v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, quad_xor1(v));
  v = fmaxf(v, quad_xor2(v));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));
  const auto r16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r16[0]), __uint_as_float(r16[1]));
  const auto r32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r32[0]), __uint_as_float(r32[1]));
}

// Element i of an array of type dt.
__device__ __forceinline__ float load_any(const void* p, int dt, int64_t i) {
  if (dt == DT_F32) return reinterpret_cast<const float*>(p)[i];
  const uint32_t h = reinterpret_cast<const uint16_t*>(p)[i];
  return dt == DT_F16 ? f16_to_f32(h) : bf16_to_f32(h);
}
__device__ __forceinline__ void store_any(void* p, int dt, int64_t i, float v) {
  if (dt == DT_F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(dt == DT_F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v));
}

// Elements i .. i + cnt - 1 (cnt <= 8; the others read as 0) at any alignment
// of the element: one or two 128-bit accesses where all eight are there.
__device__ __forceinline__ void load8_any(const void* p, int dt, int64_t i, int cnt, float (&v)[8]) {
  if (cnt >= 8) {
    if (dt == DT_F32) {
      const u32x4a4* q = reinterpret_cast<const u32x4a4*>(reinterpret_cast<const float*>(p) + i);
      const u32x4a4 a = q[0], b = q[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = __uint_as_float(a[j]);
        v[4 + j] = __uint_as_float(b[j]);
      }
    } else {
      const u32x4a2 a = *reinterpret_cast<const u32x4a2*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = a[j];
        v[2 * j] = dt == DT_F16 ? f16_to_f32(w & 0xFFFFu) : __uint_as_float(w << 16);
        v[2 * j + 1] = dt == DT_F16 ? f16_to_f32(w >> 16) : __uint_as_float(w & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < cnt ? load_any(p, dt, i + j) : 0.0f;
  }
}
// The same in two steps: eight values as they lie in memory (16-bit types: lo
// alone), so that a load may be on its way while other work runs, and their
// conversion.
struct Raw8 {
  u32x4 lo, hi;
};
__device__ __forceinline__ Raw8 raw8_load(const void* p, int dt, int64_t i, int cnt) {
  const u32x4 none{0u, 0u, 0u, 0u};
  if (cnt >= 8) {
    if (dt == DT_F32) {
      const u32x4a4* q = reinterpret_cast<const u32x4a4*>(reinterpret_cast<const float*>(p) + i);
      return Raw8{q[0], q[1]};
    }
    return Raw8{*reinterpret_cast<const u32x4a2*>(reinterpret_cast<const uint16_t*>(p) + i), none};
  }
  // whole values first: parts of a vector set one by one end in scratch memory
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    e[j] = 0;
    if (j < cnt) e[j] = dt == DT_F32 ? reinterpret_cast<const uint32_t*>(p)[i + j] : reinterpret_cast<const uint16_t*>(p)[i + j];
  }
  if (dt == DT_F32) return Raw8{u32x4{e[0], e[1], e[2], e[3]}, u32x4{e[4], e[5], e[6], e[7]}};
  return Raw8{u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16}, none};
}
__device__ __forceinline__ void raw8_floats(const Raw8& r, int dt, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = r.lo[j], b = r.hi[j];
    if (dt == DT_F32) {
      v[j] = __uint_as_float(a);
      v[4 + j] = __uint_as_float(b);
    } else {
      v[2 * j] = dt == DT_F16 ? f16_to_f32(a & 0xFFFFu) : __uint_as_float(a << 16);
      v[2 * j + 1] = dt == DT_F16 ? f16_to_f32(a >> 16) : __uint_as_float(a & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void store8_any(void* p, int dt, int64_t i, int cnt, const float (&v)[8]) {
  if (cnt >= 8) {
    if (dt == DT_F32) {
      u32x4a4* q = reinterpret_cast<u32x4a4*>(reinterpret_cast<float*>(p) + i);
      u32x4a4 a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = __float_as_uint(v[j]);
        b[j] = __float_as_uint(v[4 + j]);
      }
      q[0] = a;
      q[1] = b;
    } else {
      u32x4a2 a;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = dt == DT_F16 ? f32_to_f16_bits(v[2 * j]) | (f32_to_f16_bits(v[2 * j + 1]) << 16)
                            : f32_to_bf16_bits(v[2 * j]) | (f32_to_bf16_bits(v[2 * j + 1]) << 16);
      *reinterpret_cast<u32x4a2*>(reinterpret_cast<uint16_t*>(p) + i) = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) store_any(p, dt, i + j, v[j]);
  }
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;
constexpr float kPhi0 = 0.3989422804014327f;      // 1 / sqrt(2 pi)

// 1 / d for d in [1, 2^20]: the hardware's estimate and one Newton step.  (The
// IEEE division and expf, erfcf of the device library take 2.5 times as long:
// the epilogue's backward pass over 2048 x 11008 values was bound by them.)
__device__ __forceinline__ float quick_rcp(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

// s = 1 / (1 + exp(-z)) and t = 1 - s, both without cancellation.  The
// exponential's argument is rounded: |z| 2^-24 of the smaller of the two.
__device__ __forceinline__ void logistic(float z, float& s, float& t) {
  const float a = __builtin_amdgcn_exp2f(-kLog2E * fabsf(z));
  const float r = quick_rcp(1.0f + a), q = a * r;
  s = z < 0.0f ? q : r;
  t = z < 0.0f ? r : q;
}

// e = exp(-z^2 / 2) and the normal distribution's Phi(z).  Its tail is
// Phi(-|z|) = e P(t) with t = 1 / (1 + 0.3 |z| / sqrt 2): erfc(x) exp(x^2) / 2 as
// a polynomial of degree 9 in t, fitted over x in [0, 13] for the least
// largest relative error (2.1e-8; 5e-7 as evaluated in fp32).
__device__ __forceinline__ void normal_tail(float z, float& e, float& phi) {
  const float t = quick_rcp(__builtin_fmaf(0.21213203f, fminf(fabsf(z), 1e4f), 1.0f));
  float p = -0.06526048481464386f;
  p = __builtin_fmaf(p, t, 0.24551217257976532f);
  p = __builtin_fmaf(p, t, -0.26261571049690247f);
  p = __builtin_fmaf(p, t, 0.2825837731361389f);
  p = __builtin_fmaf(p, t, -0.05466487631201744f);
  p = __builtin_fmaf(p, t, 0.11145494133234024f);
  p = __builtin_fmaf(p, t, 0.0727686658501625f);
  p = __builtin_fmaf(p, t, 0.08566296100616455f);
  p = __builtin_fmaf(p, t, 0.08455654978752136f);
  p = __builtin_fmaf(p, t, 2.01171861e-06f);
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2E * z * z);
  p *= e;
  phi = z < 0.0f ? p : 1.0f - p;
}

// act(z).  Below -1e4 every one of them is 0 in fp32; said here, -inf gives its
// limit and not -inf 0.
__device__ __forceinline__ float act_value(int act, float z) {
  if (act == awq::LINEAR_NONE) return z;
  if (act == awq::LINEAR_RELU) return z <= 0.0f ? 0.0f : z;
  float s, t;
  if (act == awq::LINEAR_GELU) {
    normal_tail(z, t, s);
  } else {
    // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)),  u = sqrt(2 / pi) (z + 0.044715 z^3)
    const float u = act == awq::LINEAR_GELU_TANH ? 2.0f * kGeluC * z * __builtin_fmaf(kGeluK * z, z, 1.0f) : z;
    logistic(u, s, t);
  }
  return z < -1e4f ? -0.0f : z * s;
}

// act of sixteen values, the choice made once.
__device__ __forceinline__ void act_values(int act, float (&z)[4][4]) {
  auto all = [&](auto kind) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[v][j] = act_value(decltype(kind)::value, z[v][j]);
  };
  if (act == awq::LINEAR_RELU) all(std::integral_constant<int, awq::LINEAR_RELU>{});
  else if (act == awq::LINEAR_GELU) all(std::integral_constant<int, awq::LINEAR_GELU>{});
  else if (act == awq::LINEAR_GELU_TANH) all(std::integral_constant<int, awq::LINEAR_GELU_TANH>{});
  else if (act == awq::LINEAR_SILU) all(std::integral_constant<int, awq::LINEAR_SILU>{});
}

// act'(z).  Past 1e4 they are 0 and 1 in fp32; held there, infinities give
// their limits.
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == awq::LINEAR_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);   // NaN stays
  z = z > 1e4f ? 1e4f : z < -1e4f ? -1e4f : z;
  float s, t;
  if (act == awq::LINEAR_GELU) {
    normal_tail(z, t, s);
    return __builtin_fmaf(z * kPhi0, t, s);
  }
  float u = z, du = 1.0f;
  if (act == awq::LINEAR_GELU_TANH) {
    u = 2.0f * kGeluC * z * __builtin_fmaf(kGeluK * z, z, 1.0f);
    du = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluK * z, z, 1.0f);
  }
  logistic(u, s, t);
  return __builtin_fmaf(z * du, s * t, s);
}

// act' of eight values, the choice made once: their chains of dependent
// instructions run side by side.
__device__ __forceinline__ void act_slopes(int act, float (&z)[8]) {
  auto all = [&](auto kind) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = act_slope(decltype(kind)::value, z[j]);
  };
  if (act == awq::LINEAR_RELU) all(std::integral_constant<int, awq::LINEAR_RELU>{});
  else if (act == awq::LINEAR_GELU) all(std::integral_constant<int, awq::LINEAR_GELU>{});
  else if (act == awq::LINEAR_GELU_TANH) all(std::integral_constant<int, awq::LINEAR_GELU_TANH>{});
  else all(std::integral_constant<int, awq::LINEAR_SILU>{});
}

// One output (row m, column n) in two steps: what it needs from memory, asked
// for ahead of the work that ends in its sum (a load behind an earlier output's
// store would wait for it: the batch-1 product of 4096 -> 11008 takes 7.9 us,
// 8.1 with both at the store, 6.7 without an epilogue), and the finished sum z
// through the epilogue.
struct EpiIn {
  float bias, res;
};
template <class EP>
__device__ __forceinline__ EpiIn epi_fetch(const EP& ep, bool live, int64_t m, int64_t n) {
  EpiIn f{0.0f, 0.0f};
  if constexpr (kHasEpi<EP>) {
    if (ep.bias && live) f.bias = load_any(ep.bias, ep.bdt, n);
    if (ep.res && live) f.res = load_any(ep.res, ep.ydt, m * ep.ldr + n);
  }
  return f;
}
__device__ __forceinline__ void epi_store(const Epilogue& ep, void* y, int64_t ldy, int64_t m, int64_t n, float z,
                                          const EpiIn& f) {
  z += f.bias;
  if (ep.pre) store_any(ep.pre, ep.ydt, m * ep.ldp + n, z);
  store_any(y, ep.ydt, m * ldy + n, act_value(ep.act, z) + f.res);
}

// Elements i .. i + cnt - 1 (cnt <= 4; the others read as 0).
__device__ __forceinline__ void load4_any(const void* p, int dt, int64_t i, int cnt, float (&v)[4]) {
  if (cnt >= 4) {
    if (dt == DT_F32) {
      const u32x4a4 a = *reinterpret_cast<const u32x4a4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(a[j]);
    } else {
      const u32x2a2 a = *reinterpret_cast<const u32x2a2*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w = a[j];
        v[2 * j] = dt == DT_F16 ? f16_to_f32(w & 0xFFFFu) : __uint_as_float(w << 16);
        v[2 * j + 1] = dt == DT_F16 ? f16_to_f32(w >> 16) : __uint_as_float(w & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < cnt ? load_any(p, dt, i + j) : 0.0f;
  }
}
__device__ __forceinline__ void store4_any(void* p, int dt, int64_t i, int cnt, const float (&v)[4]) {
  if (cnt >= 4) {
    if (dt == DT_F32) {
      u32x4a4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = __float_as_uint(v[j]);
      *reinterpret_cast<u32x4a4*>(reinterpret_cast<float*>(p) + i) = a;
    } else {
      u32x2a2 a;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        a[j] = dt == DT_F16 ? f32_to_f16_bits(v[2 * j]) | (f32_to_f16_bits(v[2 * j + 1]) << 16)
                            : f32_to_bf16_bits(v[2 * j]) | (f32_to_bf16_bits(v[2 * j + 1]) << 16);
      *reinterpret_cast<u32x2a2*>(reinterpret_cast<uint16_t*>(p) + i) = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cnt) store_any(p, dt, i + j, v[j]);
  }
}

// Columns n .. n + cnt - 1 of row m; z with its bias.
__device__ __forceinline__ void epi_store4(const Epilogue& ep, void* y, int64_t ldy, int64_t m, int64_t n, int cnt,
                                           float (&z)[4]) {
  float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (ep.res) load4_any(ep.res, ep.ydt, m * ep.ldr + n, cnt, r);
  if (ep.pre) store4_any(ep.pre, ep.ydt, m * ep.ldp + n, cnt, z);
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = act_value(ep.act, z[j]) + r[j];
  store4_any(y, ep.ydt, m * ldy + n, cnt, z);
}

// ---- weights of all their bits ---------------------------------------------------
// step (q - z) has up to 15 bits, an fp16 operand 11.  The matrix cores take it
// under an epilogue, and for dx, as two: the code (q - z) 2^-9, exact, times
// either part of step 2^e, with the row's largest one in [2^14, 2^15).  (The plain
// product's D' q - D' z rounds twice, which an fp16 output would show beside its
// own rounding: 2.8e-4 of an output's size, 2.1e-4 with weights in fp32.)
constexpr int kOncePow = 15;          // max step 2^e < 2^15
constexpr int kOnceUnit = 9;          // the codes carry 2^-9

// -z 2^-9 as fp16, twice.
__device__ __forceinline__ uint32_t once_zero(uint32_t z) {
  return f32_to_f16_bits(-(float)z * 0x1p-9f) * 0x10001u;
}

// step 2^e as fp16; 0 has no sign.
__device__ __forceinline__ uint32_t once_step(float d) {
  const uint32_t b = f32_to_f16_bits(d);
  return b & 0x7FFFu ? b : 0u;
}

// Two of them as hi + lo, exactly: hi has the upper 7 bits of one unit less, so
// that lo has at most 5 and neither is 0 or of the other sign.  (Times a code's
// 4 bits both stay exact.  With a rest of 0 or of the other sign, an infinity
// that meets both would end as 0 inf or inf - inf, where the weight's product
// with it is an infinity.)  A step below 2^-19 of the row's largest loses its last bits.
__device__ __forceinline__ void once_parts(uint32_t d, uint32_t& hi, uint32_t& lo) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 less = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, d), u16x2{1, 1});
  hi = __builtin_bit_cast(uint32_t, less) & 0xFFF0FFF0u;
  lo = __builtin_bit_cast(uint32_t, as_f16x2(d) - as_f16x2(hi));
}

// The codes (q - z) 2^-9 of one packed word, in the order (0,4 | 2,6 | 1,5 | 3,7).
__device__ __forceinline__ u32x4 once_codes(uint32_t w, uint32_t nz) {
  const f16x2 c15 = as_f16x2(0x78007800u), c11 = as_f16x2(0x68006800u);   // 2^15, 2^11
  const f16x2 n = as_f16x2(nz);
  const uint32_t w8 = w >> 8;
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x000F000Fu), c15, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x000F000Fu), c15, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x00F000F0u), c11, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x00F000F0u), c11, n))};
}

// Pairs of fp16 values times the two of `mult`.
__device__ __forceinline__ u32x4 once_times(const u32x4& c, uint32_t mult) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = c[j];
    o[j] = __builtin_bit_cast(uint32_t, as_f16x2(v) * as_f16x2(mult));
  }
  return o;
}

// A step's size for the row's power of two: under an epilogue of any sign, and
// 0 where it is not finite, so that it takes nothing from the row's others.
template <bool ONCE>
__device__ __forceinline__ float step_size(uint32_t bits) {
  const float v = f16_to_f32(bits);
  if constexpr (!ONCE) return v;
  return fabsf(v) < __builtin_inff() ? fabsf(v) : 0.0f;
}

// The power of two of a row whose largest step is mx (0: none), as the
// constants carry it, for the plain product and under an epilogue; and what
// the finished sums carry of it.
template <bool ONCE>
__device__ __forceinline__ int step_pow(float mx) {
  if (!(mx > 0.0f)) return ONCE ? kOnceUnit : 0;
  int ex;
  frexpf(mx, &ex);                   // mx < 2^ex
  return (ONCE ? kOncePow : -9) - ex;
}
template <bool ONCE>
__device__ __forceinline__ int sum_pow(int e) {
  return ONCE ? e - kOnceUnit : e;
}

}  // namespace awqk
