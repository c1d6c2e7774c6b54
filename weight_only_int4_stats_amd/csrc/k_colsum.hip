// Column sums of fp32 partial rows: the second stage of the gradients that sum
// over the rows of a batch (a norm's weight and bias, a linear's bias).  The
// first stage leaves one partial row per block; here a block of 256 threads
// takes 64 columns, 16 groups of 16 lanes (four columns each) walk the rows
// g, g + 16, ..., and the groups meet in LDS in their order, so the result does
// not depend on when a block ran.  (Atomics would: their order changes a sum's
// bits.)  Bound by reading the partials, which the first stage has just
// written to the caches.
#include "awq_device.h"
#include "awq_internal.h"

namespace awqk {

__global__ __launch_bounds__(256) void k_col_reduce(const float* __restrict__ partial, int64_t rows, int64_t pitch,
                                                    int64_t cols, float* __restrict__ out0, int64_t at1,
                                                    float* __restrict__ out1) {
  __shared__ f32x4 part[16][16];
  const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane * 4;          // pitch is a multiple of 64
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* p = partial + c;
#pragma unroll 4
  for (int64_t g = grp; g < rows; g += 16) s += *reinterpret_cast<const f32x4*>(p + g * pitch);
  part[grp][lane] = s;
  __syncthreads();
  if (grp == 0) {
    for (int g = 1; g < 16; ++g) s += part[g][lane];
    // columns [0, cols) go to out0, [at1, at1 + cols) to out1
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + j < cols) {
        if (out0) out0[c + j] = s[j];
      } else if (out1 && c + j >= at1 && c + j < at1 + cols) {
        out1[c + j - at1] = s[j];
      }
    }
  }
}

}  // namespace awqk

namespace awq {

hipError_t launch_col_reduce(const float* partial, int64_t rows, int64_t pitch, int64_t cols, float* out0,
                             int64_t at1, float* out1, hipStream_t st) {
  const int64_t end = out1 ? at1 + cols : cols;
  if (cols <= 0 || (!out0 && !out1)) return hipSuccess;
  hipLaunchKernelGGL(awqk::k_col_reduce, dim3((unsigned)((end + 63) / 64)), dim3(256), 0, st, partial, rows, pitch,
                     cols, out0, at1, out1);
  return hipGetLastError();
}

}  // namespace awq
