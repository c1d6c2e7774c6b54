// Low-rank adapters of many requests beside a shared projection
// (include/awq.h, awq_lora_add):
//   h[m]  = A_a[:r_a] x[m]                     (k_lora_shrink, fp32)
//   y[m]  = base[m] + scaling_a B_a[:, :r_a] h[m]   (k_lora_expand)
//
// Both products run on the matrix cores over 16 rows of one adapter.  Up to
// kLoraScan rows, a block finds its adapter's rows by scanning the index (as
// many block rows as rows or adapters, whichever is fewer); beyond that a plan
// sorts the rows by adapter and a block takes 16 (shrink) or 64 (expand) of
// one adapter's.  The shrink splits K over blocks and waves; the expand sums
// the blocks' parts in their order.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_groups.h"
#include "k_rows_f16.h"

#include <type_traits>

namespace awqk {

constexpr int kLoraScan = 512;       // rows up to which the blocks find their rows themselves
constexpr int kLoraTile = 64;        // rows per tile of the plan
constexpr int kLoraMaxSplit = 32;    // K splits of the shrink

struct LoraArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* adapter;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* ranks;
  const float* scaling;
  const void* base;
  int64_t ldb;
  void* y;
  int64_t ldy, N;
  float* h;                          // [ksplit][M][R]
  GroupPlan plan;
  int M, K, R, n_adapters, ksplit, planned, by_row, nx;   // nx: blocks per block row
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (DT == DT_F16) return mfma16h(a, b, c);
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The rows a block works on: its adapter (-1: none), and rows [0, n) of it.
struct LoraRows {
  int a, n;
  const int* perm;                   // planned: the rows; else they are listed 16 at a time
};

// Finds the block's adapter and counts its rows; `first` by-row blocks leave
// when another row's block has the adapter (n = 0).  count_lds: 8 ints.
__device__ __forceinline__ LoraRows lora_rows(const LoraArgs& p, int grp, int* count_lds, int& before) {
  LoraRows r{-1, 0, nullptr};
  before = 0;
  if (p.planned) {
    const int t = grp;
    if (t >= p.plan.ntile[0]) return r;
    const GroupTile q = p.plan.tiles[t];
    r.a = q.group < p.n_adapters ? q.group : -1;
    r.n = q.rows;
    r.perm = p.plan.perm + q.first;
    return r;
  }
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
  auto norm = [&](int id) { return id < 0 || id >= p.n_adapters ? -1 : id; };
  const int a = p.by_row ? norm(p.adapter[grp]) : grp < p.n_adapters ? grp : -1;
  const int s0 = wv * p.M / nw, s1 = (wv + 1) * p.M / nw;
  int cnt = 0, first = 0x7FFFFFFF;
  for (int s = s0; s < s1; s += 64) {
    const uint64_t m = __ballot(s + lane < s1 && norm(p.adapter[s + lane < s1 ? s + lane : s0]) == a);
    if (m && first == 0x7FFFFFFF) first = s + __builtin_ctzll(m);
    cnt += __popcll(m);
  }
  if (lane == 0) {
    count_lds[wv] = cnt;
    count_lds[4 + wv] = first;
  }
  __syncthreads();
  int n = 0, f = 0x7FFFFFFF;
  for (int w = 0; w < nw; ++w) {
    if (w < wv) before += count_lds[w];
    n += count_lds[w];
    f = count_lds[4 + w] < f ? count_lds[4 + w] : f;
  }
  r.a = a;
  r.n = p.by_row && f != grp ? 0 : n;
  return r;
}

// Rows r0 .. r0 + 15 of the block's into list[16]; the caller synchronises.
__device__ __forceinline__ void lora_list(const LoraArgs& p, const LoraRows& r, int before, int r0, int* list) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
  if (r.perm) {
    if (threadIdx.x < 16 && r0 + (int)threadIdx.x < r.n) list[threadIdx.x] = r.perm[r0 + threadIdx.x];
    return;
  }
  const int s0 = wv * p.M / nw, s1 = (wv + 1) * p.M / nw;
  int run = before;
  for (int s = s0; s < s1; s += 64) {
    const int id = p.adapter[s + lane < s1 ? s + lane : s0];
    const bool hit = s + lane < s1 && (id < 0 || id >= p.n_adapters ? -1 : id) == r.a;
    const uint64_t m = __ballot(hit);
    const int rank = run + __popcll(m & ((1ull << lane) - 1));
    if (hit && rank >= r0 && rank < r0 + 16) list[rank - r0] = s + lane;
    run += __popcll(m);
  }
}

__device__ __forceinline__ int lora_rank(const LoraArgs& p, int a) {
  if (!p.ranks) return p.R;
  const int r = p.ranks[a];
  return r < 0 ? 0 : r > p.R ? p.R : r;
}

// h[part][m][r] for 16 rows of an adapter at a time.  Four waves share the
// block's K range, 64 channels a step: lane (row or rank l % 16, b = l / 16)
// holds channels 16 b .. 16 b + 15 of the step, so a row's 64 channels are one
// 128-byte line.  RB: 16-rank blocks.
template <int DT, int RB>
__global__ __launch_bounds__(256) void k_lora_shrink(const LoraArgs p) {
  __shared__ int list[16];
  __shared__ int count[8];
  __shared__ float red[4][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  int before;
  const int bx = (int)(blockIdx.x % (unsigned)p.ksplit), by = (int)(blockIdx.x / (unsigned)p.ksplit);
  const LoraRows r = lora_rows(p, p.planned ? by >> 2 : by, count, before);
  if (r.a < 0 || r.n == 0) return;
  const int rank = lora_rank(p, r.a);
  const int steps = (p.K + 63) >> 6;
  const int part = bx * 4 + wv, parts = p.ksplit * 4;
  const int k0 = (int)((int64_t)part * steps / parts), k1 = (int)((int64_t)(part + 1) * steps / parts);
  const int rb = (rank + 15) >> 4;               // rank blocks in use
  const uint16_t* A = p.a + (int64_t)r.a * p.R * p.K;
  const int rstart = p.planned ? (by & 3) * 16 : 0;
  const int rend = p.planned && rstart + 16 < r.n ? rstart + 16 : r.n;
  for (int r0 = rstart; r0 < rend; r0 += 16) {
    lora_list(p, r, before, r0, list);
    __syncthreads();
    const int nr = rend - r0 < 16 ? rend - r0 : 16;
    const uint16_t* xr = p.x + (int64_t)list[rl < nr ? rl : 0] * p.ldx;
    f32x4 acc[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = k0; s < k1; ++s) {
      const int k = s * 64 + b * 16;
      u32x4 xv[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) xv[c] = k + 8 * c < p.K ? ldg128(xr + k + 8 * c) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (i < rb) {
          const int rr = i * 16 + rl;
          const uint16_t* ar = A + (int64_t)(rr < rank ? rr : 0) * p.K;   // ranks past the adapter's: dropped
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const u32x4 av = k + 8 * c < p.K ? ldg128(ar + k + 8 * c) : u32x4{0, 0, 0, 0};
            acc[i] = mfma16<DT>(xv[c], av, acc[i]);
          }
        }
      }
    }
    // result lane: rank l % 16, rows 4 b + v; the waves' parts in wave order
    float* h = p.h + (int64_t)bx * p.M * p.R;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (i < rb) {
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wv][(4 * b + v) * 16 + rl] = acc[i][v];
        __syncthreads();
        const int row = tid >> 4, rr = i * 16 + (tid & 15);
        if (row < nr && rr < p.R)
          h[(int64_t)list[row] * p.R + rr] = rr < rank ? ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid] : 0.0f;
        __syncthreads();
      }
    }
    __syncthreads();                               // list is free again (also with rank 0)
  }
}

template <int YDT>
__device__ __forceinline__ float lora_base(const LoraArgs& p, int64_t m, int64_t n) {
  if (!p.base) return 0.0f;
  if constexpr (YDT == DT_F32) return reinterpret_cast<const float*>(p.base)[m * p.ldb + n];
  else return to_f32<YDT>(reinterpret_cast<const uint16_t*>(p.base)[m * p.ldb + n]);
}
template <int YDT>
__device__ __forceinline__ void lora_store(const LoraArgs& p, int64_t m, int64_t n, float v) {
  if constexpr (YDT == DT_F32) reinterpret_cast<float*>(p.y)[m * p.ldy + n] = v;
  else reinterpret_cast<uint16_t*>(p.y)[m * p.ldy + n] = (uint16_t)from_f32<YDT>(v);
}

constexpr int kLoraCols = 64;                      // columns per wave of the expand
constexpr int kLoraHPitch = 256 + 8;               // staged h, 16-bit values per row

// y = base + scaling B h for 16 rows of an adapter at a time, 64 columns per
// wave.  B is the first operand (16 columns of y per product) and h the
// second, so a result lane holds four values of one row; lane group b's
// columns are 16 b .. 16 b + 15 over the four products, contiguous.  h, scaled
// by a power of two per row, enters as the sum of two 16-bit values.
template <int DT, int YDT>
__global__ __launch_bounds__(256) void k_lora_expand(const LoraArgs p) {
  __shared__ int list[16];
  __shared__ int count[8];
  __shared__ __attribute__((aligned(16))) uint16_t hs[2][16][kLoraHPitch];
  __shared__ float back[16];                       // scaling / the row's power of two
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  int before;
  const int bx = (int)(blockIdx.x % (unsigned)p.nx), by = (int)(blockIdx.x / (unsigned)p.nx);
  const LoraRows r = lora_rows(p, by, count, before);
  if (r.n == 0) return;
  const int rank = r.a < 0 ? 0 : lora_rank(p, r.a);
  const int rk = (rank + 31) >> 5;                 // 32-rank steps
  const uint16_t* B = p.b + (r.a < 0 ? 0 : (int64_t)r.a * p.N * p.R);
  const float sc = r.a < 0 ? 0.0f : p.scaling ? p.scaling[r.a] : 1.0f;
  const int64_t c0 = ((int64_t)bx * 4 + wv) * kLoraCols;
  for (int r0 = 0; r0 < r.n; r0 += 16) {
    __syncthreads();
    lora_list(p, r, before, r0, list);
    __syncthreads();
    const int nr = r.n - r0 < 16 ? r.n - r0 : 16;
    if (rank > 0) {
      // 16 threads per row, ranks j, j + 16, ...
      const int row = tid >> 4, j = tid & 15;
      const float* h = p.h + (int64_t)list[row < nr ? row : 0] * p.R;
      float v[16];
      float am = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = 0.0f;
        const int rr = i * 16 + j;
        if (i * 16 < rank) {
          if (rr < rank)
            for (int s = 0; s < p.ksplit; ++s) v[i] += h[(int64_t)s * p.M * p.R + rr];
          am = fmaxf(am, fabsf(v[i]));
        }
      }
      am = fmaxf(am, quad_xor1(am));
      am = fmaxf(am, quad_xor2(am));
      am = fmaxf(am, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(am), 0x141, 0xF, 0xF, false)));
      am = fmaxf(am, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(am), 0x140, 0xF, 0xF, false)));
      const int pe = pow2_exp_for(am);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i * 16 < rk * 32) {
          const float f = ldexpf(v[i], pe);
          const uint32_t hi = from_f32<DT>(f);
          hs[0][row][i * 16 + j] = (uint16_t)hi;
          hs[1][row][i * 16 + j] = (uint16_t)from_f32<DT>(f - to_f32<DT>(hi));
        }
      }
      if (j == 0) back[row] = ldexpf(sc, -pe);
    }
    __syncthreads();
    f32x4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < rk; ++s) {
      const int k = s * 32 + 8 * b;
      const u32x4 hi = *reinterpret_cast<const u32x4*>(&hs[0][rl][k]);
      const u32x4 lo = *reinterpret_cast<const u32x4*>(&hs[1][rl][k]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // operand row i of product q is column c0 + 16 (i / 4) + 4 q + i % 4
        const int64_t n = c0 + 16 * (rl >> 2) + 4 * q + (rl & 3);
        u32x4 w = {0, 0, 0, 0};
        if (n < p.N && k < rank) {
          w = ldg128(B + n * p.R + k);
          if (k + 8 > rank) {                      // what B holds past the rank is not used
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (k + 2 * c >= rank) w[c] = 0;
              else if (k + 2 * c + 1 >= rank) w[c] &= 0xFFFFu;
            }
          }
        }
        acc[q] = mfma16<DT>(w, hi, acc[q]);
        acc[q] = mfma16<DT>(w, lo, acc[q]);
      }
    }
    if (rl < nr) {
      const int64_t m = list[rl];
      const float f = rank > 0 ? back[rl] : 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t n = c0 + 16 * b + 4 * q + v;
          if (n < p.N) {
            const float base = lora_base<YDT>(p, m, n);
            lora_store<YDT>(p, m, n, rank > 0 ? __builtin_fmaf(f, acc[q][v], base) : base);
          }
        }
    }
  }
}

}  // namespace awqk

namespace awq {
using namespace awqk;

static bool lora_planned(int64_t M) { return M > kLoraScan; }

// Block rows of the scan: one per row, or one per adapter and one for none.
static int lora_groups(int64_t M, int64_t n_adapters) { return (int)(M < n_adapters + 1 ? M : n_adapters + 1); }

static int lora_ksplit(int64_t M, int64_t K, int64_t n_adapters) {
  const int64_t blocks = lora_planned(M) ? (M + 15) / 16 : lora_groups(M, n_adapters);
  const int64_t steps = (K + 63) / 64;
  int64_t want = 512 / blocks;                     // about two blocks per compute unit
  if (want > steps / 4) want = steps / 4;          // a step per wave at least
  if (want > kLoraMaxSplit) want = kLoraMaxSplit;
  return want < 1 ? 1 : (int)want;
}

size_t lora_ws_bytes(int64_t M, int64_t K, int64_t n_adapters, int64_t R) {
  if (M <= 0 || K <= 0 || n_adapters < 0 || R <= 0) return 0;
  size_t b = n_adapters ? align_up((size_t)lora_ksplit(M, K, n_adapters) * (size_t)M * (size_t)R * 4, 256) : 0;
  if (lora_planned(M)) b += group_plan_bytes(M, n_adapters, kLoraTile);
  return b;
}

hipError_t launch_lora(const LoraCall& c, void* ws, hipStream_t st) {
  LoraArgs p{};
  p.x = c.x;
  p.ldx = c.ldx;
  p.adapter = c.adapter;
  p.a = c.a;
  p.b = c.b;
  p.ranks = c.ranks;
  p.scaling = c.scaling;
  p.base = c.base;
  p.ldb = c.ldb;
  p.y = c.y;
  p.ldy = c.ldy;
  p.N = c.N;
  p.M = (int)c.M;
  p.K = (int)c.K;
  p.R = (int)c.R;
  p.n_adapters = (int)c.n_adapters;
  p.ksplit = lora_ksplit(c.M, c.K, c.n_adapters);
  p.planned = lora_planned(c.M);
  p.nx = (int)((c.N + 4 * kLoraCols - 1) / (4 * kLoraCols));
  p.h = reinterpret_cast<float*>(ws);
  p.by_row = c.M < c.n_adapters + 1;
  unsigned gy = (unsigned)lora_groups(c.M, c.n_adapters);
  if (p.planned) {
    const size_t hb = lora_ws_bytes(c.M, c.K, c.n_adapters, c.R) - group_plan_bytes(c.M, c.n_adapters, kLoraTile);
    p.plan = group_plan_at(reinterpret_cast<char*>(ws) + hb, c.M, c.n_adapters, kLoraTile);
    const hipError_t e = launch_group_plan(c.adapter, c.M, c.n_adapters, kLoraTile, p.plan, st);
    if (e != hipSuccess) return e;
    gy = (unsigned)group_tiles_max(c.M, c.n_adapters, kLoraTile);
  }
  auto go = [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    if (c.n_adapters > 0) {
      const dim3 grid((unsigned)p.ksplit * (p.planned ? gy * 4 : gy)), block(256);
      const int64_t rb = (c.R + 15) / 16;
      if (rb <= 1) hipLaunchKernelGGL((k_lora_shrink<DT, 1>), grid, block, 0, st, p);
      else if (rb <= 2) hipLaunchKernelGGL((k_lora_shrink<DT, 2>), grid, block, 0, st, p);
      else if (rb <= 4) hipLaunchKernelGGL((k_lora_shrink<DT, 4>), grid, block, 0, st, p);
      else if (rb <= 8) hipLaunchKernelGGL((k_lora_shrink<DT, 8>), grid, block, 0, st, p);
      else hipLaunchKernelGGL((k_lora_shrink<DT, 16>), grid, block, 0, st, p);
    }
    const dim3 grid((unsigned)p.nx * gy), block(256);
    if (c.ydt == DT_F32) hipLaunchKernelGGL((k_lora_expand<DT, DT_F32>), grid, block, 0, st, p);
    else if (c.ydt == DT_F16) hipLaunchKernelGGL((k_lora_expand<DT, DT_F16>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_lora_expand<DT, DT_BF16>), grid, block, 0, st, p);
  };
  if (c.xdt == DT_F16) go(std::integral_constant<int, DT_F16>{});
  else go(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError();
}

}  // namespace awq
