// The backward pass of the product's epilogue (awq_bias_act_backward):
//   dz[m][n] = dy[m][n] act'(pre[m][n]),  dbias[n] = sum_m dz[m][n]
// One pass over dy and pre: a wave takes 512 columns (8 per lane, one 128-bit
// access of 16-bit values each), the block's four waves every fourth row of its
// chunk of rows; the sums stay in registers, meet in LDS and leave the block
// as one partial row, which k_col_reduce adds.  The sum takes the fp32 values
// before their rounding to dz's type.  2048 x 11008 with gelu: 32 us, 4.2 TB/s
// (33 with the activation chosen per value, 54 with the device library's erfcf
// and expf: bound by the vector instructions as much as by memory).
#include "k_epilogue.h"

namespace awqk {

template <int DT>
__global__ __launch_bounds__(256) void k_act_bias(const void* __restrict__ dy, int64_t M, int64_t N, int64_t lddy,
                                                  const void* __restrict__ pre, int64_t ldp, int act,
                                                  void* __restrict__ dz, int64_t lddz, float* __restrict__ partial,
                                                  int64_t pitch, int64_t rows) {
  __shared__ float red[3][512];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t n = ((int64_t)blockIdx.x * 64 + lane) * 8;
  const int cnt = N - n < 8 ? (int)(N > n ? N - n : 0) : 8;
  const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < M ? m0 + rows : M;
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (cnt > 0) {
#pragma unroll 2
    for (int64_t m = m0 + wv; m < m1; m += 4) {
      float g[8];
      load8_any(dy, DT, m * lddy + n, cnt, g);
      if (pre) {
        float z[8];
        load8_any(pre, DT, m * ldp + n, cnt, z);
        act_slopes(act, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= z[j];
        store8_any(dz, DT, m * lddz + n, cnt, g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
    }
  }
  if (!partial) return;
  if (wv > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wv - 1][j * 64 + lane] = sum[j];
  }
  __syncthreads();
  if (wv == 0 && n < pitch) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = ((sum[j] + red[0][j * 64 + lane]) + red[1][j * 64 + lane]) + red[2][j * 64 + lane];
      if (gridDim.y == 1) {                                      // one chunk: the sums are whole
        if (j < cnt) partial[n + j] = t;
      } else {
        partial[(int64_t)blockIdx.y * pitch + n + j] = j < cnt ? t : 0.0f;
      }
    }
  }
}

// Chunks of rows: enough blocks to fill the chip, at least 16 rows each; one
// chunk's sums go to dbias itself.
inline int64_t act_bias_chunks(int64_t M, int64_t N) {
  const int64_t tiles = (N + 511) / 512;
  int64_t c = (4 * (int64_t)awq::device_cus() + tiles - 1) / tiles;
  if (M <= 64) return 1;                 // one launch: 37 rows of 4096 in 4.2 us instead of 4.2 + 2.9
  const int64_t most = (M + 15) / 16;
  if (c > most) c = most;
  return c < 1 ? 1 : c > 1024 ? 1024 : c;
}
inline int64_t act_bias_pitch(int64_t N) { return (N + 63) / 64 * 64; }

}  // namespace awqk

namespace awq {

size_t act_bias_ws_bytes(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || awqk::act_bias_chunks(M, N) == 1) return 0;
  return align_up((size_t)(awqk::act_bias_chunks(M, N) * awqk::act_bias_pitch(N)) * 4, 256);
}

hipError_t launch_act_bias(const void* dy, int dt, int64_t M, int64_t N, int64_t lddy, const void* pre, int64_t ldp,
                           int act, void* dz, int64_t lddz, float* dbias, void* ws, hipStream_t st) {
  using namespace awqk;
  const int64_t want = act_bias_chunks(M, N), rows = M > 0 ? (M + want - 1) / want : 1, chunks = (M + rows - 1) / rows;
  const int64_t pitch = act_bias_pitch(N);
  float* partial = chunks == 1 ? dbias : dbias ? (float*)ws : nullptr;
  if (M > 0 && (pre || dbias)) {
    const dim3 grid((unsigned)((N + 511) / 512), (unsigned)chunks), block(256);
#define AWQ_AB(D) \
  hipLaunchKernelGGL((k_act_bias<D>), grid, block, 0, st, dy, M, N, lddy, pre, ldp, act, dz, lddz, partial, pitch, rows)
    if (dt == DT_F16) AWQ_AB(DT_F16);
    else if (dt == DT_BF16) AWQ_AB(DT_BF16);
    else AWQ_AB(DT_F32);
#undef AWQ_AB
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!dbias || chunks == 1) return hipSuccess;
  return launch_col_reduce(partial, M > 0 ? chunks : 0, pitch, N, dbias, 0, nullptr, st);
}

}  // namespace awq
