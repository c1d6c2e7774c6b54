// Argument checks that the C entry points share (host only).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/awq.h"

namespace awq {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool is_act_dtype(awq_dtype d) { return d == AWQ_F16 || d == AWQ_BF16; }
inline bool is_any_dtype(awq_dtype d) { return d == AWQ_F16 || d == AWQ_BF16 || d == AWQ_F32; }
inline uintptr_t bytes_of(awq_dtype d) { return d == AWQ_F32 ? 4 : 2; }
inline bool group_ok(int g) { return g == 64 || g == 128 || g == 256; }
inline awq_status from_hip(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }
constexpr int64_t kMaxThreads = 0xFFFFFFFF;          // of a launch

// Whether na rows of wa bytes, pa apart, from a and nb rows of wb, pb apart, from
// b share a byte; rows of different distances: whether their extents meet.
inline bool overlap(const void* a, int64_t na, int64_t wa, int64_t pa, const void* b, int64_t nb, int64_t wb, int64_t pb) {
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

}  // namespace awq
