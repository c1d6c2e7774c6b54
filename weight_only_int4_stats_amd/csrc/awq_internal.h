// Host-side launchers of the gfx950 kernels (one translation unit each).
// Every launcher enqueues on `st` and returns hipGetLastError() of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

// Quantizer variant: input channels per group (64, 128, 256), bits per code,
// and the grid (asymmetric with a zero point, or symmetric max|w| / 2^(N-1)).
struct QuantVariant {
  int group = 128;
  int bits = 4;
  bool sym = false;
};

// ---- calibration statistic (mean |x|) -------------------------------------
size_t act_stats_ws_bytes(int64_t K);
hipError_t launch_act_stats(const void* x, int dt, int64_t T, int64_t K, int64_t ldx,
                            float* mean_abs, void* ws, hipStream_t st);

// ---- quantize + pack --------------------------------------------------------
hipError_t launch_quantize_pack(const void* w, int dt, int64_t N, int64_t K, const float* s, int group,
                                uint32_t* qw, uint16_t* scales, uint8_t* zeros, float* dbg,
                                hipStream_t st);
hipError_t launch_quantize_codes(const void* w, int dt, int64_t N, int64_t K, const float* s,
                                 QuantVariant qv, uint8_t* codes, uint16_t* scales, uint8_t* zeros,
                                 hipStream_t st);

// ---- scale search -----------------------------------------------------------
size_t search_ws_bytes(int dt, int64_t N, int64_t K, int64_t T, int n_alpha);
hipError_t launch_search(const void* w, int dt, int64_t N, int64_t K, const void* x, int64_t T,
                         int64_t ldx, const float* mean_abs, const double* alphas, int n_alpha,
                         QuantVariant qv, const uint8_t* kept, float* s_out, float* inv_s_out,
                         double* loss_out, int32_t* best_out, void* ws, hipStream_t st);

// ---- mixed-precision baseline: the n most salient channels (k_salient.hip) ---
hipError_t launch_salient_channels(const float* mean_abs, int64_t K, int64_t n_keep, uint8_t* kept,
                                   hipStream_t st);

// Gram form of the search loss (k_gram.hip): Xt [K][Tp] 16-bit, fp32 partial
// tiles of G (gram_partial_floats), G [K][K] fp64, P [K][2 Kp] fp16 (Kp = K
// rounded up to 256; per 256-wide block the high then the low parts of each
// row of G scaled by 2^-sk[k]).
int64_t gram_tokens_padded(int64_t T);
int64_t gram_loss_tiles(int64_t N, int64_t K);
int64_t gram_partial_floats(int64_t T, int64_t K);
hipError_t launch_gram_prepare(const void* x, int dt, int64_t T, int64_t K, int64_t ldx,
                               uint16_t* Xt, float* Gp, double* G, uint16_t* P, int* sk,
                               hipStream_t st);
hipError_t launch_gram_loss(const uint16_t* E, int64_t N, int64_t K, const int* pexp,
                            const uint16_t* P, const int* sk, double* partial, int nc,
                            hipStream_t st);

// ---- folding 1/s into the producer of x (k_fold.hip) ---------------------------
hipError_t launch_fold_scales(void* v, int dt, int64_t rows, int64_t cols, int64_t ld, const float* s,
                              int axis, hipStream_t st);

// ---- epilogue of the W4A16 product (k_epilogue.h) -----------------------------
enum : int { LINEAR_NONE = 0, LINEAR_RELU = 2, LINEAR_GELU = 3, LINEAR_GELU_TANH = 4, LINEAR_SILU = 5 };

// y = act(z + bias) + res, and z + bias itself into pre; NULL members are left
// out.  res and pre are rows of y's type.
struct Epilogue {
  const void* bias;
  const void* res;
  void* pre;
  int64_t ldr, ldp;
  int bdt, ydt, act;
};

// ---- W4A16 product ----------------------------------------------------------
// ep (optional, for awq_w4a16_linear): the epilogue; then inv_s is NULL and the
// weights keep all their bits (k_epilogue.h)
// group: input channels per step / zero point (64, 128 or 256)
bool gemv1_supported(int64_t K, int64_t N);   // batch-1 GEMV kernels cover this shape
hipError_t launch_gemv1(const void* x, int xdt, int64_t K, const uint32_t* qw,
                        const uint16_t* scales, const uint8_t* zeros, int64_t N, int group,
                        const float* r, void* y, int ydt, hipStream_t st, const Epilogue* ep = nullptr);
size_t gemm_ws_bytes(int64_t M, int64_t N, int64_t K, int group);
hipError_t launch_w4a16(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx,
                        const uint32_t* qw, const uint16_t* scales, const uint8_t* zeros,
                        int64_t N, int group, const float* inv_s, void* y, int ydt, int64_t ldy,
                        void* ws, hipStream_t st);

// 2 <= M <= 64 (k_mid.hip): the memory-bound small-batch product
bool mid_supported(int64_t M, int64_t N, int64_t K);
size_t mid_ws_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_mid(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx, const uint32_t* qw,
                      const uint16_t* scales, const uint8_t* zeros, int64_t N, int group,
                      const float* inv_s, void* y, int ydt, int64_t ldy, void* ws, hipStream_t st,
                      const Epilogue* ep = nullptr);

// 2 <= M <= 16 (k_skinny.hip): one block per compute unit with the
// activations, steps and zero points staged in LDS; blocks (0: shape not
// covered) and launch.  No workspace.
int skinny_st_blocks(int64_t M, int64_t N, int64_t K, int group);
hipError_t launch_skinny_st(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx,
                            const uint32_t* qw, const uint16_t* scales, const uint8_t* zeros,
                            int64_t N, int group, const float* inv_s, void* y, int ydt, int64_t ldy,
                            hipStream_t st, const Epilogue* ep = nullptr);
// Layers whose rows exceed one launch's steps and zero points: the kernel on
// row chunks, one launch each (chunks: 1 = one launch, 0 = not covered).
int skinny_st_chunks(int64_t M, int64_t N, int64_t K, int group);
hipError_t launch_skinny_st_chunked(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx,
                                    const uint32_t* qw, const uint16_t* scales, const uint8_t* zeros,
                                    int64_t N, int group, const float* inv_s, void* y, int ydt, int64_t ldy,
                                    hipStream_t st, const Epilogue* ep = nullptr);

// ---- limits of the operators whose weight depends on the row -------------------
constexpr int64_t kMaxRows = (int64_t)1 << 24;       // slots, or rows with adapters
constexpr int64_t kMaxAdapters = 8192;               // the sort's three tables in LDS: 96 KB

// ---- expert routing (k_route.hip) --------------------------------------------
hipError_t launch_route(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const float* bias,
                        int sigmoid, int n_group, int topk_group, int group_top, int top_k, int renorm,
                        float scale, int32_t* ids, float* weights, hipStream_t st);

// ---- routed W4A16 products (k_experts.hip) ------------------------------------
enum : int { EXPERTS_UP = 0, EXPERTS_SWIGLU = 1, EXPERTS_DOWN = 2 };

// One call of awq_w4a16_experts_up / _down with checked arguments.
struct ExpertsCall {
  int mode;                    // EXPERTS_*
  const uint16_t* x;
  int xdt;
  int64_t M, K, ldx;
  const int32_t* ids;
  const float* weights;        // down
  int top_k;
  const uint32_t* qw;
  const uint16_t* scales;
  const uint8_t* zeros;
  int64_t E, N;
  int group;
  void* y;
  int ydt;
  int64_t ldy;
};
// of the sizes alone (M, K, top_k, E, N; every group size)
size_t experts_ws_bytes(bool down, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k);
// threads of the largest of its launches (which have 32-bit sizes)
int64_t experts_threads(int mode, int64_t M, int64_t N, int64_t K, int64_t E, int64_t top_k, int group);
hipError_t launch_experts(const ExpertsCall& c, void* ws, hipStream_t st);

// ---- per-row low-rank adapters (k_lora.hip) -----------------------------------
struct LoraCall {
  const uint16_t* x;
  int xdt;
  int64_t M, K, ldx;
  const int32_t* adapter;
  const uint16_t* a;
  const uint16_t* b;
  int64_t n_adapters, R;
  const int32_t* ranks;
  const float* scaling;
  const void* base;
  int64_t ldb, N;
  void* y;
  int ydt;
  int64_t ldy;
};
size_t lora_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R);
int64_t lora_threads(int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R);
hipError_t launch_lora(const LoraCall& c, void* ws, hipStream_t st);

// ---- operators of a block around the packed linears -----------------------------
size_t block_ws_bytes(int op, int64_t M, int64_t N, int64_t K, int64_t T);        // for any M' <= M
size_t block_ws_bytes_exact(int op, int64_t M, int64_t N, int64_t K, int64_t T);

// The product with an epilogue (k_w4a16.hip chooses, k_linear.hip: the tiles)
bool linear_mid(int64_t M, int64_t N, int64_t K);    // the 17 .. 64 token kernel serves this shape
size_t linear_ws_bytes(int64_t M, int64_t N, int64_t K, int group);
size_t linear_ws_bytes_upto(int64_t M, int64_t N, int64_t K);      // of any M' <= M, whatever the group
size_t linear_partial_bytes(int64_t M, int64_t N, int64_t K);
size_t linear_partial_bytes_upto(int64_t M, int64_t N, int64_t K);
int64_t linear_threads(int64_t M, int64_t N, int64_t K);   // of the largest of its launches
hipError_t launch_linear(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx, const uint32_t* qw,
                         const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y, int64_t ldy,
                         const Epilogue& ep, void* ws, hipStream_t st);
hipError_t launch_linear_tiles(const uint16_t* xq, const int* pm, const uint32_t* ctab, const uint32_t* qw,
                               int64_t M, int64_t N, int64_t K, int group, float* partial, void* y, int64_t ldy,
                               const Epilogue& ep, hipStream_t st);

// Column sums of partial rows (k_colsum.hip): columns [0, cols) to out0 and
// [at1, at1 + cols) to out1 (either may be NULL); pitch a multiple of 64.
hipError_t launch_col_reduce(const float* partial, int64_t rows, int64_t pitch, int64_t cols, float* out0,
                             int64_t at1, float* out1, hipStream_t st);

// The epilogue's backward pass (k_act_bias.hip); pre NULL: the bias's gradient
// alone, dbias NULL: dz alone.
size_t act_bias_ws_bytes(int64_t M, int64_t N);
hipError_t launch_act_bias(const void* dy, int dt, int64_t M, int64_t N, int64_t lddy, const void* pre, int64_t ldp,
                           int act, void* dz, int64_t lddz, float* dbias, void* ws, hipStream_t st);

// The gradient of the product's input (k_gemm_dx.hip)
size_t gemm_dx_ws_bytes(int64_t M, int64_t N, int64_t K, int group);
size_t gemm_dx_ws_bytes_upto(int64_t M, int64_t N, int64_t K);
int64_t gemm_dx_threads(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_dx(const void* dz, int dzt, int64_t M, int64_t N, int64_t lddz, const uint32_t* qw,
                          const uint16_t* scales, const uint8_t* zeros, int64_t K, int group, void* dx, int dxt,
                          int64_t lddx, void* ws, hipStream_t st);

// Layer and RMS norm, forward and backward (k_norm.hip)
int64_t norm_threads(int64_t M, int64_t K);
hipError_t launch_norm(const void* x, int xdt, int64_t M, int64_t K, int64_t ldx, const void* w, int wdt,
                       const void* b, int bdt, float eps, int rms, void* y, int ydt, int64_t ldy, float* mean,
                       float* rstd, hipStream_t st);
size_t norm_grad_ws_bytes(int64_t M, int64_t K);
size_t norm_grad_ws_bytes_upto(int64_t M, int64_t K);
hipError_t launch_norm_grad(const void* dy, int dyt, int64_t M, int64_t K, int64_t lddy, const void* x, int xdt,
                            int64_t ldx, const void* w, int wdt, const float* mean, const float* rstd, int rms,
                            void* dx, int64_t lddx, float* dw, float* db, void* ws, hipStream_t st);

// Balance loss of a router and its gradient (k_balance.hip)
size_t balance_ws_bytes(int64_t T, int64_t E);
hipError_t launch_balance(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const int32_t* ids, int top_k,
                          const uint8_t* mask, int sigmoid, double coef, float* loss, int32_t* counts, float* slope,
                          void* ws, hipStream_t st);
hipError_t launch_balance_grad(const void* logits, int dt, int64_t T, int64_t E, int64_t ldl, const float* slope,
                               const float* go, const uint8_t* mask, int sigmoid, void* dl, int64_t ldd, hipStream_t st);

// ---- plain streaming read (k_stream.hip): bytes a multiple of 1024, blocks
// of 1024 threads, unroll 1, 2, 4 or 8 units in flight per wave
hipError_t launch_read_stream(const void* p, int64_t bytes, int blocks, int unroll, uint32_t* block_xor,
                              hipStream_t st);

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Compute units of the current device (cached per device).
int device_cus();

}  // namespace awq
