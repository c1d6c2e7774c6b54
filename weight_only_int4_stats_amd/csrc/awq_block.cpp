// C ABI of the operators of a block around the packed linears: argument
// validation on the host, then the kernel launchers.  Nothing here allocates
// device memory or keeps state.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/awq.h"
#include "awq_checks.h"
#include "awq_internal.h"

namespace {

using awq::aligned;
using awq::bytes_of;
using awq::from_hip;
using awq::group_ok;
using awq::is_act_dtype;
using awq::is_any_dtype;
using awq::kMaxRows;
using awq::kMaxThreads;
using awq::overlap;

bool act_ok(awq_act a) {
  return a == AWQ_ACT_NONE || a == AWQ_ACT_RELU || a == AWQ_ACT_GELU || a == AWQ_ACT_GELU_TANH || a == AWQ_ACT_SILU;
}

// Rows of an array: for the checks of what may share memory.
struct Rows {
  const void* p;
  int64_t n, bytes, pitch;
};
Rows rows_of(const void* p, int64_t n, int64_t cols, int64_t ld, awq_dtype dt) {
  const int64_t b = (int64_t)bytes_of(dt);
  return {p, n, cols * b, ld * b};
}
bool meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1 || a.bytes < 1 || b.bytes < 1) return false;
  return overlap(a.p, a.n, a.bytes, a.pitch, b.p, b.n, b.bytes, b.pitch);
}
// The same elements, one by one (an operation in place).
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.bytes == b.bytes && (a.pitch == b.pitch || a.n == 1); }
bool meet_apart(const Rows& a, const Rows& b) { return !same(a, b) && meet(a, b); }
bool ws_ok(const void* ws, size_t bytes, size_t need) { return need == 0 || (ws && bytes >= need && aligned(ws, 256)); }

// Sizes of one packed linear that the products' 32-bit offsets and launches take.
bool linear_sizes(int64_t M, int64_t N, int64_t K) {
  return M <= kMaxRows && N <= AWQ_MAX_LINEAR_N && K <= AWQ_MAX_K && N <= ((int64_t)1 << 33) / K;
}

}  // namespace

namespace awq {

size_t block_ws_bytes(int op, int64_t M, int64_t N, int64_t K, int64_t T) {
  switch (op) {
    case AWQ_OP_LINEAR:
      return M < 1 || N < 1 || K < 1 || !linear_sizes(M, N, K) ? 0 : linear_ws_bytes_upto(M, N, K);
    case AWQ_OP_BIAS_ACT_BACKWARD:
      return M < 1 || N < 1 || M > kMaxRows || N > AWQ_MAX_LINEAR_N ? 0 : act_bias_ws_bytes(M, N);
    case AWQ_OP_GEMM_DX:
      return M < 1 || N < 1 || K < 1 || !linear_sizes(M, N, K) ? 0 : gemm_dx_ws_bytes_upto(M, N, K);
    case AWQ_OP_LAYER_NORM_BACKWARD:
      return M < 1 || K < 1 || M > kMaxRows || K > AWQ_MAX_K ? 0 : norm_grad_ws_bytes_upto(M, K);
    case AWQ_OP_BALANCE_LOSS:
      return M < 1 || T < 1 || M > kMaxRows || T > AWQ_MAX_EXPERTS ? 0 : balance_ws_bytes(M, T);
  }
  return 0;
}

size_t block_ws_bytes_exact(int op, int64_t M, int64_t N, int64_t K, int64_t T) {
  if ((op != AWQ_OP_LINEAR && op != AWQ_OP_GEMM_DX) || M < 1 || N < 1 || K < 1 || !linear_sizes(M, N, K))
    return block_ws_bytes(op, M, N, K, T);
  size_t most = 0;
  for (int g = 64; g <= 256; g *= 2) {              // which kernel serves a shape depends on it
    if (K % g != 0) continue;
    const size_t b = op == AWQ_OP_LINEAR ? linear_ws_bytes(M, N, K, g) : gemm_dx_ws_bytes(M, N, K, g);
    most = b > most ? b : most;
  }
  return most;
}

}  // namespace awq

extern "C" {

awq_status awq_w4a16_linear(const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx, const int32_t* qweight,
                            const uint16_t* scales, const uint8_t* zeros, int64_t N, int group_size, const void* bias,
                            awq_dtype bdt, awq_act act, const void* residual, int64_t ldr, void* pre, int64_t ldp,
                            void* y, awq_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (!group_ok(group_size) || !act_ok(act)) return AWQ_ERR_UNSUPPORTED;
  if (!is_act_dtype(xdt) || !is_any_dtype(ydt) || (bias && !is_any_dtype(bdt))) return AWQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0 || K % group_size != 0 || ldx < K || ldy < N || (residual && ldr < N) || (pre && ldp < N))
    return AWQ_ERR_SHAPE;
  if (K > AWQ_MAX_K) return AWQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return AWQ_OK;
  if (!x || !qweight || !scales || !zeros || !y) return AWQ_ERR_NULL;
  if (!linear_sizes(M, N, K) || awq::linear_threads(M, N, K) > kMaxThreads) return AWQ_ERR_UNSUPPORTED;
  const uintptr_t yb = bytes_of(ydt);
  if (ldx % 8 != 0 || !aligned(x, 16) || !aligned(qweight, 16) || !aligned(scales, 2) || !aligned(y, yb) ||
      (bias && !aligned(bias, bytes_of(bdt))) || (residual && !aligned(residual, yb)) || (pre && !aligned(pre, yb)))
    return AWQ_ERR_ALIGN;
  if (!ws_ok(ws, ws_bytes, awq::linear_ws_bytes(M, N, K, group_size))) return AWQ_ERR_WORKSPACE;
  const Rows rx = rows_of(x, M, K, ldx, xdt), ry = rows_of(y, M, N, ldy, ydt), rr = rows_of(residual, M, N, ldr, ydt),
             rp = rows_of(pre, M, N, ldp, ydt);
  if (meet(rx, ry) || meet(rx, rp) || meet(ry, rp) || meet(rr, rp) || meet_apart(rr, ry)) return AWQ_ERR_UNSUPPORTED;
  const awq::Epilogue ep{bias, residual, pre, ldr, ldp, (int)bdt, (int)ydt, (int)act};
  return from_hip(awq::launch_linear(x, (int)xdt, M, K, ldx, (const uint32_t*)qweight, scales, zeros, N, group_size, y,
                                     ldy, ep, ws, (hipStream_t)stream));
}

awq_status awq_bias_act_backward(const void* dy, awq_dtype dt, int64_t M, int64_t N, int64_t lddy, const void* pre,
                                 int64_t ldp, awq_act act, void* dz, int64_t lddz, float* dbias, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (!act_ok(act)) return AWQ_ERR_UNSUPPORTED;
  if (!is_any_dtype(dt)) return AWQ_ERR_DTYPE;
  const bool has_act = act != AWQ_ACT_NONE;
  if (M < 0 || N < 0 || lddy < N || (has_act && (ldp < N || lddz < N))) return AWQ_ERR_SHAPE;
  if (N == 0) return AWQ_OK;
  if (M > 0 && (!dy || (has_act && (!pre || !dz)))) return AWQ_ERR_NULL;
  if (M > kMaxRows || N > AWQ_MAX_LINEAR_N) return AWQ_ERR_UNSUPPORTED;
  const uintptr_t b = bytes_of(dt);
  if (!aligned(dy, b) || (has_act && (!aligned(pre, b) || !aligned(dz, b))) || !aligned(dbias, 4)) return AWQ_ERR_ALIGN;
  if (dbias && !ws_ok(ws, ws_bytes, awq::act_bias_ws_bytes(M, N))) return AWQ_ERR_WORKSPACE;
  if (has_act) {
    const Rows rdy = rows_of(dy, M, N, lddy, dt), rp = rows_of(pre, M, N, ldp, dt), rdz = rows_of(dz, M, N, lddz, dt);
    if (meet_apart(rdy, rdz) || meet_apart(rp, rdz)) return AWQ_ERR_UNSUPPORTED;
  }
  return from_hip(awq::launch_act_bias(dy, (int)dt, M, N, lddy, has_act ? pre : nullptr, ldp, (int)act, dz, lddz, dbias,
                                       ws, (hipStream_t)stream));
}

awq_status awq_w4a16_gemm_dx(const void* dz, awq_dtype dzt, int64_t M, int64_t N, int64_t lddz, const int32_t* qweight,
                             const uint16_t* scales, const uint8_t* zeros, int64_t K, int group_size, void* dx,
                             awq_dtype dxt, int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
  if (!group_ok(group_size)) return AWQ_ERR_UNSUPPORTED;
  if (!is_act_dtype(dzt) || !is_any_dtype(dxt)) return AWQ_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0 || K % group_size != 0 || lddz < N || lddx < K) return AWQ_ERR_SHAPE;
  if (K > AWQ_MAX_K) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  if (!dx || (N > 0 && (!dz || !qweight || !scales || !zeros))) return AWQ_ERR_NULL;
  if (!linear_sizes(M, N, K) || awq::gemm_dx_threads(M, N, K) > kMaxThreads) return AWQ_ERR_UNSUPPORTED;
  if (!aligned(dx, bytes_of(dxt)) || (N > 0 && (!aligned(dz, 2) || !aligned(qweight, 16) || !aligned(scales, 2))))
    return AWQ_ERR_ALIGN;
  if (!ws_ok(ws, ws_bytes, awq::gemm_dx_ws_bytes(M, N, K, group_size))) return AWQ_ERR_WORKSPACE;
  if (meet(rows_of(dz, M, N, lddz, dzt), rows_of(dx, M, K, lddx, dxt))) return AWQ_ERR_UNSUPPORTED;
  return from_hip(awq::launch_gemm_dx(dz, (int)dzt, M, N, lddz, (const uint32_t*)qweight, scales, zeros, K, group_size,
                                      dx, (int)dxt, lddx, ws, (hipStream_t)stream));
}

awq_status awq_layer_norm(const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx, const void* weight,
                          awq_dtype wdt, const void* bias, awq_dtype bdt, float eps, int rms, void* y, awq_dtype ydt,
                          int64_t ldy, float* mean, float* rstd, void* stream) {
  if (!is_any_dtype(xdt) || !is_any_dtype(wdt) || !is_any_dtype(ydt) || (bias && !is_any_dtype(bdt))) return AWQ_ERR_DTYPE;
  if (M < 0 || K <= 0 || ldx < K || ldy < K) return AWQ_ERR_SHAPE;
  if (K > AWQ_MAX_K || !(eps >= 0.0f) || std::isinf(eps)) return AWQ_ERR_UNSUPPORTED;
  if (M == 0) return AWQ_OK;
  if (!x || !weight || !y) return AWQ_ERR_NULL;
  if (M > kMaxRows || awq::norm_threads(M, K) > kMaxThreads) return AWQ_ERR_UNSUPPORTED;
  if (!aligned(x, bytes_of(xdt)) || !aligned(weight, bytes_of(wdt)) || (bias && !aligned(bias, bytes_of(bdt))) ||
      !aligned(y, bytes_of(ydt)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return AWQ_ERR_ALIGN;
  if (meet_apart(rows_of(x, M, K, ldx, xdt), rows_of(y, M, K, ldy, ydt))) return AWQ_ERR_UNSUPPORTED;
  return from_hip(awq::launch_norm(x, (int)xdt, M, K, ldx, weight, (int)wdt, bias, (int)bdt, eps, rms != 0, y, (int)ydt,
                                   ldy, mean, rstd, (hipStream_t)stream));
}

awq_status awq_layer_norm_backward(const void* dy, awq_dtype dyt, int64_t M, int64_t K, int64_t lddy, const void* x,
                                   awq_dtype xdt, int64_t ldx, const void* weight, awq_dtype wdt, const float* mean,
                                   const float* rstd, int rms, void* dx, int64_t lddx, float* dweight, float* dbias,
                                   void* ws, size_t ws_bytes, void* stream) {
  if (!is_any_dtype(dyt) || !is_any_dtype(xdt) || !is_any_dtype(wdt)) return AWQ_ERR_DTYPE;
  if (M < 0 || K <= 0 || lddy < K || ldx < K || lddx < K) return AWQ_ERR_SHAPE;
  if (K > AWQ_MAX_K) return AWQ_ERR_UNSUPPORTED;
  if (M > 0 && (!dy || !x || !weight || !rstd || (!rms && !mean) || !dx)) return AWQ_ERR_NULL;
  if (M > kMaxRows) return AWQ_ERR_UNSUPPORTED;
  if (!aligned(dy, bytes_of(dyt)) || !aligned(x, bytes_of(xdt)) || !aligned(weight, bytes_of(wdt)) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dx, bytes_of(xdt)) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return AWQ_ERR_ALIGN;
  if ((dweight || dbias) && !ws_ok(ws, ws_bytes, awq::norm_grad_ws_bytes(M, K))) return AWQ_ERR_WORKSPACE;
  const Rows rdx = rows_of(dx, M, K, lddx, xdt);
  if (meet_apart(rows_of(dy, M, K, lddy, dyt), rdx) || meet_apart(rows_of(x, M, K, ldx, xdt), rdx)) return AWQ_ERR_UNSUPPORTED;
  return from_hip(awq::launch_norm_grad(dy, (int)dyt, M, K, lddy, x, (int)xdt, ldx, weight, (int)wdt, mean, rstd,
                                        rms != 0, dx, lddx, dweight, dbias, ws, (hipStream_t)stream));
}

awq_status awq_balance_loss(const void* logits, awq_dtype ldt, int64_t T, int64_t E, int64_t ldl, const int32_t* ids,
                            int top_k, const uint8_t* mask, awq_score score, double coef, float* loss, int32_t* counts,
                            float* slope, void* ws, size_t ws_bytes, void* stream) {
  if (!is_any_dtype(ldt)) return AWQ_ERR_DTYPE;
  if (score != AWQ_SCORE_SOFTMAX && score != AWQ_SCORE_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (T < 0 || E < 1 || ldl < E || top_k < 1) return AWQ_ERR_SHAPE;
  if (E > AWQ_MAX_EXPERTS || top_k > AWQ_MAX_TOP_K || T > kMaxRows) return AWQ_ERR_UNSUPPORTED;
  if (!loss || !counts || !slope || (T > 0 && (!logits || !ids))) return AWQ_ERR_NULL;
  if (!aligned(logits, bytes_of(ldt)) || !aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(slope, 4))
    return AWQ_ERR_ALIGN;
  if (!ws_ok(ws, ws_bytes, awq::balance_ws_bytes(T, E))) return AWQ_ERR_WORKSPACE;
  return from_hip(awq::launch_balance(logits, (int)ldt, T, E, ldl, ids, top_k, mask, score == AWQ_SCORE_SIGMOID, coef,
                                      loss, counts, slope, ws, (hipStream_t)stream));
}

awq_status awq_balance_loss_backward(const void* logits, awq_dtype ldt, int64_t T, int64_t E, int64_t ldl,
                                     const float* slope, const float* grad, const uint8_t* mask, awq_score score,
                                     void* dlogits, int64_t ldd, void* stream) {
  if (!is_any_dtype(ldt)) return AWQ_ERR_DTYPE;
  if (score != AWQ_SCORE_SOFTMAX && score != AWQ_SCORE_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (T < 0 || E < 1 || ldl < E || ldd < E) return AWQ_ERR_SHAPE;
  if (E > AWQ_MAX_EXPERTS || T > kMaxRows) return AWQ_ERR_UNSUPPORTED;
  if (T == 0) return AWQ_OK;
  if (!logits || !slope || !dlogits) return AWQ_ERR_NULL;
  if (!aligned(logits, bytes_of(ldt)) || !aligned(slope, 4) || !aligned(grad, 4) || !aligned(dlogits, bytes_of(ldt)))
    return AWQ_ERR_ALIGN;
  if (meet_apart(rows_of(logits, T, E, ldl, ldt), rows_of(dlogits, T, E, ldd, ldt))) return AWQ_ERR_UNSUPPORTED;
  return from_hip(awq::launch_balance_grad(logits, (int)ldt, T, E, ldl, slope, grad, mask, score == AWQ_SCORE_SIGMOID,
                                           dlogits, ldd, (hipStream_t)stream));
}

}  // extern "C"
