// C ABI of the operators whose weight depends on the row: argument validation
// on the host, then the kernel launchers.  Nothing here allocates device
// memory or keeps state.
#include <hip/hip_runtime.h>

#include "../../include/awq.h"
#include "awq_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool is_act_dtype(awq_dtype d) { return d == AWQ_F16 || d == AWQ_BF16; }
bool is_any_dtype(awq_dtype d) { return d == AWQ_F16 || d == AWQ_BF16 || d == AWQ_F32; }
uintptr_t bytes_of(awq_dtype d) { return d == AWQ_F32 ? 4 : 2; }
bool group_ok(int g) { return g == 64 || g == 128 || g == 256; }
awq_status from_hip(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

using awq::kMaxAdapters;
using awq::kMaxRows;
constexpr int64_t kMaxThreads = 0xFFFFFFFF;          // of a launch

// Whether na rows of wa bytes, pa apart, from a and nb rows of wb, pb apart, from
// b share a byte; rows of different distances: whether their extents meet.
bool overlap(const void* a, int64_t na, int64_t wa, int64_t pa, const void* b, int64_t nb, int64_t wb, int64_t pb) {
  const int64_t d = (int64_t)((intptr_t)b - (intptr_t)a);
  if (d >= (__int128)(na - 1) * pa + wa || -d >= (__int128)(nb - 1) * pb + wb) return false;
  if (na == 1) pa = pb;
  if (nb == 1) pb = pa;
  if (pa != pb || pa < wa || pa < wb) return true;
  // b's row j starts r bytes into a's row j + q
  const int64_t q = (d >= 0 ? d : d - (pa - 1)) / pa, r = d - q * pa;
  auto rows_meet = [&](int64_t by) { return by < na && by + nb > 0; };
  return (r < wa && rows_meet(q)) || (r + wb > pa && rows_meet(q + 1));
}

awq_status experts(int mode, const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx, const int32_t* ids,
                   const float* weights, int top_k, const int32_t* qweight, const uint16_t* scales,
                   const uint8_t* zeros, int64_t E, int64_t N, int group_size, void* y, awq_dtype ydt,
                   int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (!group_ok(group_size)) return AWQ_ERR_UNSUPPORTED;
  if (!is_act_dtype(xdt) || !is_any_dtype(ydt)) return AWQ_ERR_DTYPE;
  const bool down = mode == awq::EXPERTS_DOWN;
  const int64_t cols = mode == awq::EXPERTS_SWIGLU ? N / 2 : N;
  if (M < 0 || N < 0 || E < 1 || top_k < 1 || K <= 0 || K % group_size != 0 || ldx < K || ldy < cols) return AWQ_ERR_SHAPE;
  if (mode == awq::EXPERTS_SWIGLU && N % 2 != 0) return AWQ_ERR_SHAPE;
  if (E > AWQ_MAX_EXPERTS || top_k > AWQ_MAX_TOP_K || K > AWQ_MAX_K) return AWQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return AWQ_OK;
  if (!x || !ids || !qweight || !scales || !zeros || !y || (down && !weights)) return AWQ_ERR_NULL;
  if (M > kMaxRows / top_k || N > ((int64_t)1 << 32) / K - 1) return AWQ_ERR_UNSUPPORTED;
  if ((down ? M * top_k : M) * K * 2 >= (int64_t)1 << 31) return AWQ_ERR_UNSUPPORTED;
  if (awq::experts_threads(mode, M, N, K, E, top_k, group_size) > kMaxThreads) return AWQ_ERR_UNSUPPORTED;
  if (ldx % 8 != 0 || !aligned(x, 16) || !aligned(qweight, 16) || !aligned(scales, 2) || !aligned(ids, 4) ||
      !aligned(y, bytes_of(ydt)) || (down && !aligned(weights, 4)))
    return AWQ_ERR_ALIGN;
  const size_t need = awq::experts_ws_bytes(down, M, N, K, E, top_k);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return AWQ_ERR_WORKSPACE;
  const int64_t slots = M * top_k, ob = (int64_t)bytes_of(ydt);
  if (overlap(x, down ? slots : M, K * 2, ldx * 2, y, down ? M : slots, cols * ob, ldy * ob)) return AWQ_ERR_UNSUPPORTED;
  const awq::ExpertsCall c{mode, (const uint16_t*)x, (int)xdt, M, K, ldx, ids, weights, top_k,
                           (const uint32_t*)qweight, scales, zeros, E, N, group_size, y, (int)ydt, ldy};
  return from_hip(awq::launch_experts(c, ws, (hipStream_t)stream));
}

}  // namespace

extern "C" {

awq_status awq_route_experts(const void* logits, awq_dtype ldt, int64_t T, int64_t E, int64_t ldl,
                             const float* bias, awq_score score, int n_group, int topk_group,
                             int group_top, int top_k, int renormalize, float scale, int32_t* ids,
                             float* weights, void* stream) {
  if (!is_any_dtype(ldt)) return AWQ_ERR_DTYPE;
  if (score != AWQ_SCORE_SOFTMAX && score != AWQ_SCORE_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (T < 0 || E < 1 || ldl < E || n_group < 1 || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
      group_top < 1 || group_top > 2 || top_k < 1 || top_k > E / n_group * topk_group)
    return AWQ_ERR_SHAPE;
  if (E > AWQ_MAX_EXPERTS || n_group > 64 || top_k > AWQ_MAX_TOP_K || T > kMaxThreads / 64 - 3) return AWQ_ERR_UNSUPPORTED;
  if (T == 0) return AWQ_OK;
  if (!logits || !ids || !weights) return AWQ_ERR_NULL;
  if (!aligned(logits, bytes_of(ldt)) || !aligned(ids, 4) || !aligned(weights, 4) || (bias && !aligned(bias, 4)))
    return AWQ_ERR_ALIGN;
  return from_hip(awq::launch_route(logits, (int)ldt, T, E, ldl, bias, score == AWQ_SCORE_SIGMOID, n_group,
                                    topk_group, group_top, top_k, renormalize != 0, scale, ids, weights,
                                    (hipStream_t)stream));
}

awq_status awq_w4a16_experts_up(const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* ids, int top_k, const int32_t* qweight,
                                const uint16_t* scales, const uint8_t* zeros, int64_t E, int64_t N,
                                int group_size, awq_act act, void* y, awq_dtype ydt, int64_t ldy,
                                void* ws, size_t ws_bytes, void* stream) {
  if (act != AWQ_ACT_NONE && act != AWQ_ACT_SWIGLU) return AWQ_ERR_UNSUPPORTED;
  return experts(act == AWQ_ACT_SWIGLU ? awq::EXPERTS_SWIGLU : awq::EXPERTS_UP, x, xdt, M, K, ldx, ids, nullptr,
                 top_k, qweight, scales, zeros, E, N, group_size, y, ydt, ldy, ws, ws_bytes, stream);
}

awq_status awq_w4a16_experts_down(const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx,
                                  const int32_t* ids, const float* weights, int top_k,
                                  const int32_t* qweight, const uint16_t* scales,
                                  const uint8_t* zeros, int64_t E, int64_t N, int group_size,
                                  void* y, awq_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes,
                                  void* stream) {
  return experts(awq::EXPERTS_DOWN, x, xdt, M, K, ldx, ids, weights, top_k, qweight, scales, zeros, E, N,
                 group_size, y, ydt, ldy, ws, ws_bytes, stream);
}

awq_status awq_lora_add(const void* x, awq_dtype xdt, int64_t M, int64_t K, int64_t ldx,
                        const int32_t* adapter, const void* a, const void* b, int64_t n_adapters,
                        int64_t R, const int32_t* ranks, const float* scaling, const void* base,
                        int64_t ldb, int64_t N, void* y, awq_dtype ydt, int64_t ldy, void* ws,
                        size_t ws_bytes, void* stream) {
  if (!is_act_dtype(xdt) || !is_any_dtype(ydt)) return AWQ_ERR_DTYPE;
  if (M < 0 || N < 0 || n_adapters < 0 || K <= 0 || R < 8 || ldx < K || ldy < N || (base && ldb < N)) return AWQ_ERR_SHAPE;
  if (R > AWQ_MAX_RANK || K > AWQ_MAX_K || M > kMaxRows || n_adapters > kMaxAdapters) return AWQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return AWQ_OK;
  if (!adapter || !y || (n_adapters > 0 && (!x || !a || !b))) return AWQ_ERR_NULL;
  if (K % 8 != 0 || R % 8 != 0 || ldx % 8 != 0 || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(adapter, 4) || (ranks && !aligned(ranks, 4)) || (scaling && !aligned(scaling, 4)) ||
      (base && !aligned(base, bytes_of(ydt))) || !aligned(y, bytes_of(ydt)))
    return AWQ_ERR_ALIGN;
  if (N > kMaxThreads || awq::lora_threads(M, N, K, n_adapters, R) > kMaxThreads) return AWQ_ERR_UNSUPPORTED;
  const size_t need = awq::lora_ws_bytes(M, N, K, n_adapters, R);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return AWQ_ERR_WORKSPACE;
  const int64_t ob = (int64_t)bytes_of(ydt);
  const bool in_place = base == y && (ldb == ldy || M == 1);
  if ((n_adapters > 0 && overlap(x, M, K * 2, ldx * 2, y, M, N * ob, ldy * ob)) ||
      (base && !in_place && overlap(base, M, N * ob, ldb * ob, y, M, N * ob, ldy * ob)))
    return AWQ_ERR_UNSUPPORTED;
  const awq::LoraCall c{(const uint16_t*)x, (int)xdt, M, K, ldx, adapter, (const uint16_t*)a, (const uint16_t*)b,
                        n_adapters, R, ranks, scaling, base, ldb, N, y, (int)ydt, ldy};
  return from_hip(awq::launch_lora(c, ws, (hipStream_t)stream));
}

}  // extern "C"
