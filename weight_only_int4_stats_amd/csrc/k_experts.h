// What the routed W4A16 products' kernels share.
#pragma once

#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

using awq::EXPERTS_DOWN;
using awq::EXPERTS_SWIGLU;
using awq::EXPERTS_UP;

// silu(gate) * up in fp32; a gate of -inf gives -0 up, the limit.
__device__ __forceinline__ float swiglu(float gate, float up) {
  const float s = gate / (1.0f + expf(-gate));
  return (gate == -__builtin_inff() ? -0.0f : s) * up;
}

}  // namespace awqk
