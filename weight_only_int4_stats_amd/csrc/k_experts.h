// What the routed W4A16 products' kernels share.
#pragma once

#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

using awq::EXPERTS_DOWN;
using awq::EXPERTS_SWIGLU;
using awq::EXPERTS_UP;

// Maximum over each 16-lane row, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, quad_xor1(v));
  v = fmaxf(v, quad_xor2(v));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false)));
}

// |v|, 0 for what is not finite.  A row's power of two goes by its finite
// values, so that an infinite activation does not push the others past fp16's
// range: where the maximum turns out infinite it is formed again of these.
__device__ __forceinline__ float finite_size(float v) { return fabsf(v) < __builtin_inff() ? fabsf(v) : 0.0f; }

// The maximum of |v[0 .. 7]| over each 16-lane row, of the finite values.
__device__ __forceinline__ float row16_finite_max(const float (&v)[8]) {
  float am = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) am = fmaxf(am, fabsf(v[c]));
  am = row16_max(am);
  if (am == __builtin_inff()) {                    // whole 16-lane rows branch
    am = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) am = fmaxf(am, finite_size(v[c]));
    am = row16_max(am);
  }
  return am;
}

// -z 2^-9 as fp16, twice.
__device__ __forceinline__ uint32_t experts_nz(uint32_t z) {
  return f32_to_f16_bits(-(float)z * 0x1p-9f) * 0x10001u;
}

// One packed word -> 8 operands (q - z) 2^-9 in fp16, exact, in the order
// (0,4 | 2,6 | 1,5 | 3,7).  The masked nibbles are fp16 subnormals, q 2^-24 or
// (odd nibbles) q 2^-20; a packed fma scales and subtracts.
__device__ __forceinline__ u32x4 experts_unpack(uint32_t w, uint32_t nz) {
  const f16x2 c15 = as_f16x2(0x78007800u), c11 = as_f16x2(0x68006800u), n = as_f16x2(nz);   // 2^15, 2^11
  const uint32_t w8 = w >> 8;
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x000F000Fu), c15, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x000F000Fu), c15, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w & 0x00F000F0u), c11, n)),
               __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_f16x2(w8 & 0x00F000F0u), c11, n))};
}

__device__ __forceinline__ void store_out(void* y, int ydt, int64_t i, float v) {
  if (ydt == DT_F32) reinterpret_cast<float*>(y)[i] = v;
  else if (ydt == DT_F16) reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)f32_to_f16_bits(v);
  else reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)f32_to_bf16_bits(v);
}

// silu(gate) * up in fp32; a gate of -inf gives -0 up, the limit.
__device__ __forceinline__ float swiglu(float gate, float up) {
  const float s = gate / (1.0f + expf(-gate));
  return (gate == -__builtin_inff() ? -0.0f : s) * up;
}

}  // namespace awqk

namespace awq {

// The tiled form (k_experts_gemm.hip), into out [slots][ldo] (down: fp32).
size_t experts_gemm_ws_bytes(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k);
int64_t experts_gemm_threads(int mode, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int group);
hipError_t launch_experts_gemm(const ExpertsCall& c, void* out, int64_t ldo, void* ws, hipStream_t st);

}  // namespace awq
