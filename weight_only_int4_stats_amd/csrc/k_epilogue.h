// The epilogue of the W4A16 product (awq_w4a16_linear): bias, activation and
// residual applied in fp32 to a finished sum, and the activations' slopes.
#pragma once

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

// 1 / (1 + exp(-z))
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + expf(-z)); }

constexpr float kGeluC = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kPhi0 = 0.3989422804014327f;      // 1 / sqrt(2 pi)

// act(z).  Below -1e4 every one of them is 0 in fp32; said here, -inf gives its
// limit and not -inf 0.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case awq::LINEAR_RELU: return z <= 0.0f ? 0.0f : z;
    case awq::LINEAR_GELU: return z < -1e4f ? -0.0f : 0.5f * z * erfcf(-z * kSqrtHalf);
    // 0.5 z (1 + tanh u) = z / (1 + exp(-2 u)),  u = sqrt(2 / pi) (z + 0.044715 z^3)
    case awq::LINEAR_GELU_TANH:
      return z < -1e4f ? -0.0f : z * logistic(2.0f * kGeluC * z * __builtin_fmaf(kGeluK * z, z, 1.0f));
    case awq::LINEAR_SILU: return z < -1e4f ? -0.0f : z * logistic(z);
    default: return z;
  }
}

// act'(z).  Past 1e4 they are 0 and 1 in fp32; held there, infinities give
// their limits.
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == awq::LINEAR_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);   // NaN stays
  z = z > 1e4f ? 1e4f : z < -1e4f ? -1e4f : z;
  if (act == awq::LINEAR_GELU) {
    const float d = kPhi0 * expf(-0.5f * z * z);
    return __builtin_fmaf(z, d, 0.5f * erfcf(-z * kSqrtHalf));
  }
  if (act == awq::LINEAR_GELU_TANH) {
    const float u2 = 2.0f * kGeluC * z * __builtin_fmaf(kGeluK * z, z, 1.0f);
    const float s = logistic(u2), t = logistic(-u2);        // t = 1 - s without its cancellation
    const float du2 = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluK * z, z, 1.0f);
    return __builtin_fmaf(z * du2, s * t, s);
  }
  const float s = logistic(z), t = logistic(-z);
  return s * __builtin_fmaf(z, t, 1.0f);
}

// One output: z the finished sum of (row m, column n).
__device__ __forceinline__ void epi_store(const Epilogue& ep, void* y, int64_t ldy, int64_t m, int64_t n, float z) {
  if (ep.bias) z += load_any(ep.bias, ep.bdt, n);
  if (ep.pre) store_any(ep.pre, ep.ydt, m * ep.ldp + n, z);
  float o = act_value(ep.act, z);
  if (ep.res) o += load_any(ep.res, ep.ydt, m * ep.ldr + n);
  store_any(y, ep.ydt, m * ldy + n, o);
}

// Columns n .. n + cnt - 1 of row m, their bias in b.
__device__ __forceinline__ void epi_store8(const Epilogue& ep, void* y, int64_t ldy, int64_t m, int64_t n, int cnt,
                                           float (&z)[8], const float (&b)[8]) {
  float r[8];
  if (ep.res) load8_any(ep.res, ep.ydt, m * ep.ldr + n, cnt, r);
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] += b[j];
  if (ep.pre) store8_any(ep.pre, ep.ydt, m * ep.ldp + n, cnt, z);
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = act_value(ep.act, z[j]);
  if (ep.res) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += r[j];
  }
  store8_any(y, ep.ydt, m * ldy + n, cnt, z);
}

// ---- weights rounded once -------------------------------------------------------
// The kernels that feed step (q - z) to the matrix cores in fp16 form it under
// an epilogue as the product of two exact fp16 values, (q - z) 2^-9 and
// step 2^e with the row's largest one in [2^14, 2^15): one rounding, where the
// plain product's D' q - D' z rounds its constant too.  On 16-bit outputs the
// second rounding shows (fp16: 4.1e-4 of an output's size against 2.7e-4).
// Four more vector instructions per packed word.
constexpr int kOncePow = 15;          // max step 2^e < 2^15
constexpr int kOnceUnit = 9;          // the codes carry 2^-9

// -z 2^-9 as fp16, twice.
__device__ __forceinline__ uint32_t once_zero(uint32_t z) {
  return f32_to_f16_bits(-(float)z * 0x1p-9f) * 0x10001u;
}

// One packed word -> 8 operands in the order (0,4 | 2,6 | 1,5 | 3,7), each
// times the two fp16 values of `mult`.
__device__ __forceinline__ u32x4 once_dequant(uint32_t w, uint32_t mult, uint32_t nz) {
  const f16x2 c15 = as_f16x2(0x78007800u), c11 = as_f16x2(0x68006800u);   // 2^15, 2^11
  const f16x2 n = as_f16x2(nz), d = as_f16x2(mult);
  const uint32_t w8 = w >> 8;
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x000F000Fu), c15, n) * d),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x000F000Fu), c15, n) * d),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x00F000F0u), c11, n) * d),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x00F000F0u), c11, n) * d)};
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
