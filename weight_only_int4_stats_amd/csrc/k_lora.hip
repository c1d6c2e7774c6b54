// Low-rank adapters of many requests beside a shared projection
// (include/awq.h, awq_lora_add):
//   h[m]  = A_a[:r_a] x[m]                     (k_lora_shrink, fp32)
//   y[m]  = base[m] + scaling_a B_a[:, :r_a] h[m]   (k_lora_expand)
//
// Both products run on the matrix cores over 16 rows of one adapter.  Up to
// kLoraScan rows, a block finds its adapter's rows by scanning the index (as
// many block rows as rows or adapters, whichever is fewer; many rows of few
// adapters are dealt to more blocks, 16 at a time); beyond that a plan
// sorts the rows by adapter and a block takes 16 (shrink) or 64 (expand) of
// one adapter's.  The shrink splits K over blocks and waves; the expand sums
// the blocks' parts in their order.
//
// 4096 rows of 6 adapters (rank 32, 4096 -> 4096, 16-bit base and output): plan
// 7.5, shrink 12, expand 22 us, which a plain copy of base would take 17.5 of;
// 64 rows of 32 adapters (rank up to 64, 4096 -> 11008): shrink 8, expand 15
// us, a chain of dependent loads (index, rank, h, base) at 2 TB/s of B.
#include "awq_device.h"
#include "awq_internal.h"
#include "k_groups.h"
#include "k_rows_f16.h"

#include <type_traits>

namespace awqk {

// Rows up to which the blocks find their rows themselves: at 1462 rows of 8
// adapters (424 -> 4502) a call takes 98 us so, 30 us with a plan.
constexpr int kLoraScan = 512;
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
  int M, K, R, n_adapters, ksplit, planned, by_row, nx, deal;   // nx: blocks per block row; deal below
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (DT == DT_F16) return mfma16h(a, b, c);
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The rows a block works on: its adapter (-1: none) and how many.
struct LoraRows {
  int a, n;
  int first, end;                    // the block's passes start at ranks first, first + step, ... < end
  const int* perm;                   // planned: the rows
  uint64_t mask;                     // up to 64 rows in all: which
  int before;                        // else: rows before this wave's share of the index
};

// Finds the block's adapter, counts its rows and says which of them are the
// block's (n = 0: none).  With a block per row, every 16th of an adapter's rows
// is the first of 16; with a block row per adapter, p.deal blocks share it and
// this is the part-th.  count_lds: two ints per wave.
__device__ __forceinline__ LoraRows lora_rows(const LoraArgs& p, int grp, int part, int* count_lds) {
  LoraRows r{-1, 0, 0, 0, nullptr, 0, 0};
  auto mine16 = [&](int n, int ahead) {
    r.first = p.by_row ? ahead : 16 * part;
    r.end = p.by_row && ahead + 16 < n ? ahead + 16 : n;
    r.n = (p.by_row && (ahead & 15)) || r.first >= n ? 0 : n;
  };
  if (p.planned) {
    if (grp >= p.plan.ntile[0]) return r;
    const GroupTile q = p.plan.tiles[grp];
    r.a = q.group < p.n_adapters ? q.group : -1;
    r.n = r.end = q.rows;
    r.perm = p.plan.perm + q.first;
    return r;
  }
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
  auto norm = [&](int id) { return id < 0 || id >= p.n_adapters ? -1 : id; };
  if (p.M <= 64) {                   // every wave sees the whole index
    const int mine = norm(p.adapter[lane < p.M ? lane : 0]);
    r.a = p.by_row ? __builtin_amdgcn_readlane(mine, grp) : grp < p.n_adapters ? grp : -1;
    r.mask = __ballot(lane < p.M && mine == r.a);
    mine16(__popcll(r.mask), __popcll(r.mask & ((1ull << (grp & 63)) - 1)));
    return r;
  }
  r.a = p.by_row ? norm(p.adapter[grp]) : grp < p.n_adapters ? grp : -1;
  const int s0 = wv * p.M / nw, s1 = (wv + 1) * p.M / nw;
  int cnt = 0, ahead = 0;            // of the wave's share; of them before row grp
  for (int s = s0; s < s1; s += 64) {
    const uint64_t m = __ballot(s + lane < s1 && norm(p.adapter[s + lane < s1 ? s + lane : s0]) == r.a);
    ahead += s >= grp ? 0 : __popcll(grp - s < 64 ? m & ((1ull << (grp - s)) - 1) : m);
    cnt += __popcll(m);
  }
  if (lane == 0) {
    count_lds[wv] = cnt;
    count_lds[nw + wv] = ahead;
  }
  __syncthreads();
  int n = 0;
  ahead = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < wv) r.before += count_lds[w];
    n += count_lds[w];
    ahead += count_lds[nw + w];
  }
  mine16(n, ahead);
  return r;
}

// Rows r0 .. r0 + 15 of the block's into list[16]; the caller synchronises.
__device__ __forceinline__ void lora_list(const LoraArgs& p, const LoraRows& r, int r0, int* list) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
  if (r.perm) {
    if (threadIdx.x < 16 && r0 + (int)threadIdx.x < r.n) list[threadIdx.x] = r.perm[r0 + threadIdx.x];
    return;
  }
  if (p.M <= 64) {                   // every wave writes the same
    const int rank = __popcll(r.mask & ((1ull << lane) - 1));
    if (((r.mask >> lane) & 1) && rank >= r0 && rank < r0 + 16) list[rank - r0] = lane;
    return;
  }
  const int s0 = wv * p.M / nw, s1 = (wv + 1) * p.M / nw;
  int run = r.before;
  for (int s = s0; s < s1; s += 64) {
    const int id = p.adapter[s + lane < s1 ? s + lane : s0];
    const bool hit = s + lane < s1 && (id < 0 || id >= p.n_adapters ? -1 : id) == r.a;
    const uint64_t m = __ballot(hit);
    const int rank = run + __popcll(m & ((1ull << lane) - 1));
    if (hit && rank >= r0 && rank < r0 + 16) list[rank - r0] = s + lane;
    run += __popcll(m);
  }
}

// The adapter's rank and scaling (0 for none).
struct LoraAdapter {
  int rank;
  float scaling;
};
__device__ __forceinline__ LoraAdapter lora_adapter(const LoraArgs& p, int a) {
  const int at = a < 0 ? 0 : a;
  LoraAdapter d{p.R, 1.0f};
  if (p.n_adapters == 0) return LoraAdapter{0, 0.0f};
  if (p.ranks) d.rank = p.ranks[at];
  if (p.scaling) d.scaling = p.scaling[at];
  d.rank = a < 0 || d.rank < 0 ? 0 : d.rank > p.R ? p.R : d.rank;
  return d;
}
// Block row grp's adapter where it is known without the rows, so that its rank
// is on its way while they are looked for.
__device__ __forceinline__ bool lora_known(const LoraArgs& p, int grp, int& a) {
  a = grp < p.n_adapters ? grp : -1;
  return !p.planned && !p.by_row;
}

// Steps of 64 channels whose loads are in flight together in a wave of the
// shrink, for MT 16-row and RB 16-rank blocks (registers).
template <int MT, int RB>
constexpr int lora_unroll() { return MT + RB <= 2 ? 8 : MT + RB <= 3 ? 4 : MT + RB <= 6 ? 2 : 1; }

// acc[t][i] += 16 rows (xr[t]: this lane's row) x ranks 16 i .. 16 i + 15 over
// the steps k0, k0 + stride, ... < k1 of 64 channels: lane (row or rank l % 16,
// b = l / 16) holds channels 16 b .. 16 b + 15 of a step, so a row's 64
// channels are one 128-byte line.
template <int DT, int MT, int RB>
__device__ __forceinline__ void lora_shrink_steps(const LoraArgs& p, const uint16_t* const (&xr)[MT], const uint16_t* A,
                                                  int rank, int k0, int k1, int stride, f32x4 (&acc)[MT][RB]) {
  constexpr int U = lora_unroll<MT, RB>();
  const int lane = threadIdx.x & 63, rl = lane & 15, b = lane >> 4;
  // rows past the rank repeat the first (from the cache); their results are dropped
  const uint16_t* ar[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) ar[i] = A + (int64_t)(i * 16 + rl < rank ? i * 16 + rl : 0) * p.K;
  // whole: every step lies inside the range and inside K, so no load is guarded
  constexpr int CH = RB > 8 ? 1 : 2;               // halves of a step loaded together
  auto steps = [&](int s, auto whole) {
#pragma unroll
    for (int c0 = 0; c0 < 2; c0 += CH) {
      u32x4 xv[U][MT][CH], av[U][RB][CH];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int k = (s + u * stride) * 64 + b * 16 + 8 * (c0 + c);
          const bool in = decltype(whole)::value || (s + u * stride < k1 && k < p.K);
#pragma unroll
          for (int t = 0; t < MT; ++t) xv[u][t][c] = in ? ldg128(xr[t] + k) : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < RB; ++i) av[u][i][c] = in ? ldg128(ar[i] + k) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[t][i] = mfma16<DT>(xv[u][t][c], av[u][i][c], acc[t][i]);
    }
  };
  for (int s = k0; s < k1; s += U * stride) {
    if (s + (U - 1) * stride < k1 && (s + (U - 1) * stride + 1) * 64 <= p.K) steps(s, std::true_type{});
    else steps(s, std::false_type{});
  }
}

// h[part][m][r] for 16 MT rows of an adapter at a time; the block's eight
// waves share its K range.  Planned, a block takes a whole tile with MT = 4,
// so that A is read once per 64 rows, or a quarter of one with MT = 1.
constexpr int kShrinkWaves = 8;
template <int DT, int MT, int RB>
__global__ __launch_bounds__(kShrinkWaves * 64) void k_lora_shrink(const LoraArgs p) {
  constexpr int W = kShrinkWaves, RG = RB < 4 ? RB : 4;   // rank blocks that meet in LDS together
  __shared__ int list[16 * MT];
  __shared__ int count[2 * W];
  __shared__ float red[RG][W][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  const int bx = (int)(blockIdx.x % (unsigned)p.ksplit), byd = (int)(blockIdx.x / (unsigned)p.ksplit);
  const int by = byd / p.deal, dealt = byd % p.deal;
  constexpr int kSub = kLoraTile / (16 * MT);      // blocks per tile of the plan
  int known;
  LoraAdapter ad{0, 0.0f};
  const bool early = lora_known(p, by, known);
  if (early) ad = lora_adapter(p, known);
  const LoraRows r = lora_rows(p, p.planned ? by / kSub : by, dealt, count);
  if (r.a < 0 || r.n == 0) return;
  if (!early) ad = lora_adapter(p, r.a);
  const int rank = ad.rank;
  const int steps = (p.K + 63) >> 6;
  const int part = bx * W + wv, parts = p.ksplit * W;
  const int k0 = (int)((int64_t)part * steps / parts), k1 = (int)((int64_t)(part + 1) * steps / parts);
  const uint16_t* A = p.a + (int64_t)r.a * p.R * p.K;
  const int rstart = p.planned ? by % kSub * 16 * MT : r.first;
  const int rend = p.planned && rstart + 16 * MT < r.n ? rstart + 16 * MT : r.end;
  for (int r0 = rstart; r0 < rend; r0 += 16 * MT * p.deal) {
#pragma unroll
    for (int t = 0; t < MT; ++t) lora_list(p, r, r0 + 16 * t, list + 16 * t);
    __syncthreads();
    const int nr = rend - r0 < 16 * MT ? rend - r0 : 16 * MT;
    const uint16_t* xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xr[t] = p.x + (int64_t)list[16 * t + rl < nr ? 16 * t + rl : 0] * p.ldx;
    f32x4 acc[MT][RB];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < RB; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    lora_shrink_steps<DT, MT, RB>(p, xr, A, rank, k0, k1, 1, acc);
    // result lane: rank l % 16, rows 4 b + v; the waves' parts in wave order
    float* h = p.h + (int64_t)bx * p.M * p.R;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i0 = 0; i0 < RB; i0 += RG) {
        if (i0 * 16 < rank && 16 * t < nr) {
#pragma unroll
          for (int i = 0; i < RG; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[i][wv][(4 * b + v) * 16 + rl] = acc[t][i0 + i][v];
          __syncthreads();
          for (int j = tid; j < RG * 256; j += W * 64) {
            const int i = j >> 8, row = 16 * t + ((j >> 4) & 15), rr = (i0 + i) * 16 + (j & 15);
            if (row < nr && rr < rank) {
              float o = red[i][0][j & 255];
#pragma unroll
              for (int k = 1; k < W; ++k) o += red[i][k][j & 255];
              h[(int64_t)list[row] * p.R + rr] = o;
            }
          }
          __syncthreads();
        }
      }
    __syncthreads();                               // list is free again (also with rank 0)
  }
}

// One row of h as the sum of NP 16-bit values, scaled by a power of two: 16
// threads per row, thread j of them holding ranks j, j + 16, ... in v (zeros
// past the rank).  Writes ranks 0 .. pad - 1 of each part (stride apart) and
// scaling / the power of two.  Two fp16 or three bf16 parts hold h to 2^-23 of
// itself, whatever the output's type: a base that cancels most of B h leaves
// the low bits of h in a 16-bit output too.  (Two bf16 parts hold 2^-17 and
// save next to nothing: 4096 rows of 6 adapters, rank 32, 45.0 us a call
// instead of 45.2.)
template <int DT>
constexpr int lora_parts() { return DT == DT_BF16 ? 3 : 2; }
template <int DT, int NP, int NI>
__device__ __forceinline__ void lora_split_row(int j, int pad, float sc, uint16_t* part, int stride, float* back, const float (&v)[NI]) {
  // the power of two goes by the finite values: an infinite one stays infinite
  // and the others what they are
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) am = fmaxf(am, fabsf(v[i]) < __builtin_inff() ? fabsf(v[i]) : 0.0f);
  am = fmaxf(am, quad_xor1(am));
  am = fmaxf(am, quad_xor2(am));
  am = fmaxf(am, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(am), 0x141, 0xF, 0xF, false)));
  am = fmaxf(am, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(am), 0x140, 0xF, 0xF, false)));
  const int pe = pow2_exp_for(am);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * 16 + j;
    if (r < pad) {
      float f = ldexpf(v[i], pe);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const uint32_t h = from_f32<DT>(f);
        part[k * stride + r] = (uint16_t)h;
        f = fabsf(f) < __builtin_inff() ? f - to_f32<DT>(h) : 0.0f;   // the first part says it all
      }
    }
  }
  if (j == 0) *back = ldexpf(sc, -pe);
}

// 8 ranks k .. k + 7 of column n of B, and what of them the product may see:
// nothing past the last column or the rank, whatever B holds there.  The load
// is unconditional so that nothing waits for it here.
__device__ __forceinline__ u32x4 lora_b(const LoraArgs& p, const uint16_t* B, int64_t n, int k, int rank) {
  return ldg128(B + (n < p.N && k < rank ? n * p.R + k : 0));
}
__device__ __forceinline__ u32x4 lora_b_mask(u32x4 w, const LoraArgs& p, int64_t n, int k, int rank) {
  const int left = n < p.N ? rank - k : 0;         // ranks of the eight that are there
#pragma unroll
  for (int c = 0; c < 4; ++c) w[c] &= left > 2 * c + 1 ? 0xFFFFFFFFu : left > 2 * c ? 0xFFFFu : 0u;
  return w;
}

// 4 NQ consecutive outputs of row m from column n: y = base + f acc.  Accesses
// of 16 bytes (NQ = 1 and 16-bit outputs: 8) wherever the rows start: 3358 rows
// of 3785 columns took 75 us one column at a time.
template <int YDT, int NQ>
struct LoraOut {
  static constexpr int NW = YDT == DT_F32 ? 4 * NQ : 2 * NQ;   // 32-bit words
  uint32_t w[NW];
  __device__ __forceinline__ void load(const LoraArgs& p, int64_t m, int64_t n) {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
    if (!p.base) return;
    if constexpr (YDT == DT_F32) {
      const uint32_t* b = reinterpret_cast<const uint32_t*>(p.base) + m * p.ldb + n;
      if (n + 4 * NQ <= p.N) {
#pragma unroll
        for (int i = 0; i < NW; i += 4) {
          const u32x4 t = *reinterpret_cast<const u32x4a4*>(b + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[i + j] = t[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < NW; ++i)
          if (n + i < p.N) w[i] = b[i];
      }
    } else {
      const uint16_t* b = reinterpret_cast<const uint16_t*>(p.base) + m * p.ldb + n;
      if (n + 4 * NQ <= p.N) {
        if constexpr (NQ == 1) {
          const u32x2a2 t = *reinterpret_cast<const u32x2a2*>(b);
          w[0] = t[0];
          w[1] = t[1];
        } else {
#pragma unroll
          for (int i = 0; i < NW; i += 4) {
            const u32x4 t = *reinterpret_cast<const u32x4a2*>(b + 2 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i + j] = t[j];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i)
          if (n + i < p.N) w[i >> 1] |= (uint32_t)b[i] << (16 * (i & 1));
      }
    }
  }
  __device__ __forceinline__ void store(const LoraArgs& p, int64_t m, int64_t n, float f, const f32x4* acc, bool add) {
    uint32_t o[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = 0;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) {
      if constexpr (YDT == DT_F32) {
        const float base = __uint_as_float(w[i]);
        o[i] = __float_as_uint(add ? __builtin_fmaf(f, acc[i >> 2][i & 3], base) : base);
      } else {
        const float base = i & 1 ? hi_f32<YDT>(w[i >> 1]) : lo_f32<YDT>(w[i >> 1]);
        o[i >> 1] |= from_f32<YDT>(add ? __builtin_fmaf(f, acc[i >> 2][i & 3], base) : base) << (16 * (i & 1));
      }
    }
    if constexpr (YDT == DT_F32) {
      uint32_t* y = reinterpret_cast<uint32_t*>(p.y) + m * p.ldy + n;
      if (n + 4 * NQ <= p.N) {
#pragma unroll
        for (int i = 0; i < NW; i += 4) *reinterpret_cast<u32x4a4*>(y + i) = u32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < NW; ++i)
          if (n + i < p.N) y[i] = o[i];
      }
    } else {
      uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + m * p.ldy + n;
      if (n + 4 * NQ <= p.N) {
        if constexpr (NQ == 1) {
          *reinterpret_cast<u32x2a2*>(y) = u32x2a2{o[0], o[1]};
        } else {
#pragma unroll
          for (int i = 0; i < NW; i += 4) *reinterpret_cast<u32x4a2*>(y + 2 * i) = u32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i)
          if (n + i < p.N) y[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
};

constexpr int kLoraCols = 64;                      // columns per wave of the expand

// y = base + scaling B h, PR rows of an adapter at a time, 64 columns per
// wave.  B is the first operand (16 columns of y per product) and h the
// second, so a result lane holds four values of one row.  The products' rows
// are dealt so that lane group b's values of NQ products are 4 NQ consecutive
// columns (16 bytes) and the four groups' pieces lie side by side: an access
// covers 64 bytes of each of 16 rows.  A wave's part of B stays in registers
// for all of the block's rows.  RK: 32-rank steps.
template <int DT, int YDT, int RK, int PR>
__global__ __launch_bounds__(256) void k_lora_expand(const LoraArgs p) {
  constexpr int kPitch = RK * 32 + 8, NP = lora_parts<DT>();
  constexpr int NQ = YDT == DT_F32 ? 1 : 2, NC = 4 / NQ;   // products per piece, pieces per row
  __shared__ int list[PR];
  __shared__ int count[8];
  __shared__ __attribute__((aligned(16))) uint16_t hs[NP][PR][kPitch];
  __shared__ float back[PR];                       // scaling / the row's power of two
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  const int bx = (int)(blockIdx.x % (unsigned)p.nx), byd = (int)(blockIdx.x / (unsigned)p.nx);
  const int by = byd / p.deal, dealt = byd % p.deal;
  int known;
  LoraAdapter ad{0, 0.0f};
  const bool early = lora_known(p, by, known);
  if (early) ad = lora_adapter(p, known);
  const LoraRows r = lora_rows(p, by, dealt, count);
  if (r.n == 0) return;
  if (!early) ad = lora_adapter(p, r.a);
  const int rank = ad.rank;
  const float sc = ad.scaling;
  const int rk = (rank + 31) >> 5;
  const uint16_t* B = p.b + (r.a < 0 ? 0 : (int64_t)r.a * p.N * p.R);
  const int64_t c0 = ((int64_t)bx * 4 + wv) * kLoraCols;
  const int64_t cl = c0 + 4 * NQ * b;              // this lane's first piece; the others 16 NQ columns on
  auto bcol = [&](int q) { return c0 + q / NQ * 16 * NQ + 4 * NQ * (rl >> 2) + 4 * (q % NQ) + (rl & 3); };
  u32x4 w[RK][4];
  if (rank > 0) {
#pragma unroll
    for (int s = 0; s < RK; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q) w[s][q] = lora_b(p, B, bcol(q), s * 32 + 8 * b, rank);
  }
  for (int r0 = r.first; r0 < r.end; r0 += PR * p.deal) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PR; i += 16) lora_list(p, r, r0 + i, list + i);
    __syncthreads();
    const int nr = r.end - r0 < PR ? r.end - r0 : PR;
    if (rank > 0) {
      // 16 threads per row; the K parts, four at a time, are added in their order
      const int64_t pitch = (int64_t)p.M * p.R;
      for (int row = tid >> 4; row < (nr + 15) / 16 * 16; row += 16) {
        const float* h = p.h + (int64_t)list[row < nr ? row : 0] * p.R;
        float v[RK * 2];
#pragma unroll
        for (int i = 0; i < RK * 2; ++i) v[i] = 0.0f;
        for (int s0 = 0; s0 < p.ksplit; s0 += 4) {
          float g[4][RK * 2];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < RK * 2; ++i) {
              const int rr = i * 16 + (tid & 15);
              const bool in = s0 + s < p.ksplit && rr < rank;
              const float f = h[in ? (s0 + s) * pitch + rr : 0];
              g[s][i] = in ? f : 0.0f;
            }
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < RK * 2; ++i) v[i] += g[s][i];
        }
        lora_split_row<DT, NP>(tid & 15, rk * 32, sc, hs[0][row], PR * kPitch, back + row, v);
      }
    }
    __syncthreads();
    if (r0 == r.first && rank > 0) {
#pragma unroll
      for (int s = 0; s < RK; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[s][q] = lora_b_mask(w[s][q], p, bcol(q), s * 32 + 8 * b, rank);
    }
#pragma unroll
    for (int t = 0; t < PR; t += 16) {
      if (t >= nr) break;
      const int row = t + rl;
      // base 16 rows at a time: for all of the block's rows ahead of the staging
      // it cost registers and time (26 us instead of 21 us for 4096 rows)
      LoraOut<YDT, NQ> out[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (row < nr) out[c].load(p, list[row], cl + 16 * NQ * c);
      f32x4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < RK; ++s) {
        if (s < rk) {
          u32x4 h[NP];
#pragma unroll
          for (int k = 0; k < NP; ++k) h[k] = *reinterpret_cast<const u32x4*>(&hs[k][row][s * 32 + 8 * b]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < NP; ++k) acc[q] = mfma16<DT>(w[s][q], h[k], acc[q]);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (row < nr) out[c].store(p, list[row], cl + 16 * NQ * c, rank > 0 ? back[row] : 0.0f, acc + NQ * c, rank > 0);
    }
  }
}

// Few rows and a small A: one launch in which every block forms its rows' h
// itself (8 waves share K) and expands it to 128 columns, 16 per wave.
constexpr int kLoraOneCols = 128;
template <int DT, int YDT, int RB>
__global__ __launch_bounds__(512) void k_lora_one(const LoraArgs p) {
  constexpr int RK = (RB + 1) / 2, kPitch = RK * 32 + 8, NP = lora_parts<DT>();
  __shared__ int list[16];
  __shared__ int count[16];
  __shared__ float red[8][256];
  __shared__ float hv[16][RB * 16 + 1];
  __shared__ __attribute__((aligned(16))) uint16_t hs[NP][16][kPitch];
  __shared__ float back[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rl = lane & 15, b = lane >> 4;
  const int bx = (int)(blockIdx.x % (unsigned)p.nx), byd = (int)(blockIdx.x / (unsigned)p.nx);
  const int by = byd / p.deal, dealt = byd % p.deal;
  int known;
  LoraAdapter ad{0, 0.0f};
  const bool early = lora_known(p, by, known);
  if (early) ad = lora_adapter(p, known);
  const LoraRows r = lora_rows(p, by, dealt, count);
  if (r.n == 0) return;
  if (!early) ad = lora_adapter(p, r.a);
  const int rank = ad.rank;
  const float sc = ad.scaling;
  const int rk = (rank + 31) >> 5;
  const uint16_t* A = p.a + (r.a < 0 ? 0 : (int64_t)r.a * p.R * p.K);
  const uint16_t* B = p.b + (r.a < 0 ? 0 : (int64_t)r.a * p.N * p.R);
  const int64_t c0 = (int64_t)bx * kLoraOneCols + wv * 16;
  u32x4 w[RK];
  if (rank > 0) {
#pragma unroll
    for (int s = 0; s < RK; ++s) w[s] = lora_b(p, B, c0 + rl, s * 32 + 8 * b, rank);
  }
  for (int r0 = r.first; r0 < r.end; r0 += 16 * p.deal) {
    __syncthreads();
    lora_list(p, r, r0, list);
    __syncthreads();
    const int nr = r.end - r0 < 16 ? r.end - r0 : 16;
    LoraOut<YDT, 1> out;
    const int64_t m = list[rl < nr ? rl : 0];
    if (rl < nr) out.load(p, m, c0 + 4 * b);
    if (rank > 0) {
      f32x4 acc[1][RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) acc[0][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const uint16_t* const xr[1] = {p.x + m * p.ldx};
      lora_shrink_steps<DT, 1, RB>(p, xr, A, rank, wv, (p.K + 63) >> 6, 8, acc);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (i * 16 < rank) {
          __syncthreads();
#pragma unroll
          for (int v = 0; v < 4; ++v) red[wv][(4 * b + v) * 16 + rl] = acc[0][i][v];
          __syncthreads();
          if (tid < 256) {
            float t = red[0][tid];
#pragma unroll
            for (int k = 1; k < 8; ++k) t += red[k][tid];
            hv[tid >> 4][i * 16 + (tid & 15)] = t;
          }
        }
      }
      __syncthreads();
      if (tid < 256) {
        const int row = tid >> 4, j = tid & 15;
        float v[RK * 2];
#pragma unroll
        for (int i = 0; i < RK * 2; ++i) v[i] = i * 16 + j < rank ? hv[row][i * 16 + j] : 0.0f;
        lora_split_row<DT, NP>(j, rk * 32, sc, hs[0][row], 16 * kPitch, back + row, v);
      }
      __syncthreads();
    }
    if (r0 == r.first && rank > 0) {
#pragma unroll
      for (int s = 0; s < RK; ++s) w[s] = lora_b_mask(w[s], p, c0 + rl, s * 32 + 8 * b, rank);
    }
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < RK; ++s) {
      if (s < rk) {
#pragma unroll
        for (int k = 0; k < NP; ++k) acc = mfma16<DT>(w[s], *reinterpret_cast<const u32x4*>(&hs[k][rl][s * 32 + 8 * b]), acc);
      }
    }
    if (rl < nr) out.store(p, m, c0 + 4 * b, rank > 0 ? back[rl] : 0.0f, &acc, rank > 0);
  }
}

}  // namespace awqk

namespace awq {
using namespace awqk;

static bool lora_planned(int64_t M) { return M > kLoraScan; }

// Block rows of the scan: one per row, or one per adapter and one for none.
static int lora_groups(int64_t M, int64_t n_adapters) { return (int)(M < n_adapters + 1 ? M : n_adapters + 1); }

// Blocks of a block row, which take its rows 16 at a time in turn: twice the
// even share (calls of 123 rows of one adapter, 1488 -> 3181: 31 us with one
// block row, 13 us with 8; 289 rows of two, 168 -> 244: 34 us and 13 us).
static int lora_deal(int64_t M, int64_t n_adapters) {
  const int64_t deal = (M / (n_adapters + 1) + 7) / 8;
  return lora_planned(M) || deal < 1 ? 1 : (int)deal;
}

// One launch (k_lora_one) while forming h again costs less than a second
// launch: every pass of 16 rows reads A and its rows of x in every block of
// 128 columns, from the caches.  At most 256 KB of A per pass and 48 MB in all:
// over 672 sizes (K 1024 and 4096, 1024 to 16384 columns, ranks 8 to 64, 1 to
// 32 adapters, 1 to 512 rows, bf16) the calls take 1.4 % more than with the
// better form at each, 1.8 % with 64 MB and 2.3 % with 32.  512 rows of one
// adapter, rank 16, 4096 -> 16384 (1 GB): 191 us in one launch, 24 in two; 8
// rows of 8 adapters, rank 16, 4096 -> 1024 (16 MB): 8.6 and 9.2.
static bool lora_one(int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R) {
  const int64_t a = R * K * 2, passes = lora_groups(M, n_adapters) + M / 16;
  return !lora_planned(M) && R <= 64 && a <= (256 << 10) &&
         (N + kLoraOneCols - 1) / kLoraOneCols * passes * (a + 16 * K * 2) <= (48 << 20);
}

// Block rows of the expand, and of the one launch.
static int64_t lora_block_rows(int64_t M, int64_t n_adapters) {
  return lora_planned(M) ? group_tiles_max(M, n_adapters, kLoraTile) : lora_groups(M, n_adapters) * lora_deal(M, n_adapters);
}

// Parts that K may be split into: a step per wave at least.
static int64_t lora_max_split(int64_t K) {
  const int64_t want = (K + 63) / 64 / kShrinkWaves;
  return want < 1 ? 1 : want > kLoraMaxSplit ? kLoraMaxSplit : want;
}

static int lora_ksplit(int64_t M, int64_t K, int64_t n_adapters) {
  const int64_t blocks = lora_planned(M) ? (M + kLoraTile - 1) / kLoraTile : lora_block_rows(M, n_adapters);
  const int64_t want = 256 / blocks, most = lora_max_split(K);   // about a block per compute unit
  return want < 1 ? 1 : (int)(want < most ? want : most);
}

// The K parts of h, for M rows or any fewer (the split falls as the rows grow):
// from 512 rows on 256 / (M / 64) parts of M rows, 16384 rows in all, or one.
static size_t lora_h_bytes(int64_t M, int64_t K, int64_t n_adapters, int64_t R) {
  if (!n_adapters) return 0;
  int64_t rows = M * lora_max_split(K);
  const int64_t all = 256 * kLoraTile;
  if (lora_planned(M) && rows > all) rows = M > all ? M : all;
  return align_up((size_t)rows * (size_t)R * 4, 256);
}

size_t lora_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R) {
  if (M <= 0 || N <= 0 || K <= 0 || n_adapters < 0 || R <= 0 || lora_one(M, N, K, n_adapters, R)) return 0;
  return lora_h_bytes(M, K, n_adapters, R) + (lora_planned(M) ? group_plan_bytes(M, n_adapters, kLoraTile) : 0);
}

// Of the launch over all columns: the shrink has at most 4 blocks of 512 per
// block row and K split, far from 2^32 at the most rows there may be.
int64_t lora_threads(int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R) {
  const bool one = lora_one(M, N, K, n_adapters, R);
  const int64_t cols = one ? kLoraOneCols : 4 * kLoraCols;
  return (N + cols - 1) / cols * lora_block_rows(M, n_adapters) * (one ? 512 : 256);
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
  p.h = reinterpret_cast<float*>(ws);
  p.by_row = c.M < c.n_adapters + 1;
  p.deal = lora_deal(c.M, c.n_adapters);
  const unsigned gy = (unsigned)lora_block_rows(c.M, c.n_adapters);
  const bool one = lora_one(c.M, c.N, c.K, c.n_adapters, c.R);
  const int64_t cols = one ? kLoraOneCols : 4 * kLoraCols;
  p.nx = (int)((c.N + cols - 1) / cols);
  if (p.planned) {
    p.plan = group_plan_at(reinterpret_cast<char*>(ws) + lora_h_bytes(c.M, c.K, c.n_adapters, c.R), c.M, c.n_adapters, kLoraTile);
    const hipError_t e = launch_group_plan(c.adapter, c.M, c.n_adapters, kLoraTile, p.plan, st);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)p.nx * gy);
  auto typed = [&](auto dtc, auto ydc) {
    constexpr int DT = decltype(dtc)::value, YDT = decltype(ydc)::value;
    if (one) {
      if (c.R <= 16) hipLaunchKernelGGL((k_lora_one<DT, YDT, 1>), grid, dim3(512), 0, st, p);
      else if (c.R <= 32) hipLaunchKernelGGL((k_lora_one<DT, YDT, 2>), grid, dim3(512), 0, st, p);
      else hipLaunchKernelGGL((k_lora_one<DT, YDT, 4>), grid, dim3(512), 0, st, p);
      return;
    }
    if (c.n_adapters > 0) {
      auto shrink = [&](auto mt, auto rb) {
        constexpr int MT = decltype(mt)::value, RB = decltype(rb)::value;
        const dim3 sg((unsigned)p.ksplit * (p.planned ? gy * (kLoraTile / (16 * MT)) : gy));
        hipLaunchKernelGGL((k_lora_shrink<DT, MT, RB>), sg, dim3(kShrinkWaves * 64), 0, st, p);
      };
      auto ranked = [&](auto mt) {
        if (c.R <= 16) shrink(mt, std::integral_constant<int, 1>{});
        else if (c.R <= 32) shrink(mt, std::integral_constant<int, 2>{});
        else shrink(mt, std::integral_constant<int, 4>{});
      };
      if (c.R > 128) shrink(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
      else if (c.R > 64) shrink(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
      else if (p.planned) ranked(std::integral_constant<int, 4>{});
      else ranked(std::integral_constant<int, 1>{});
    }
    auto expand = [&](auto pr) {
      constexpr int PR = decltype(pr)::value;
      if (c.R <= 32) hipLaunchKernelGGL((k_lora_expand<DT, YDT, 1, PR>), grid, dim3(256), 0, st, p);
      else if (c.R <= 64) hipLaunchKernelGGL((k_lora_expand<DT, YDT, 2, PR>), grid, dim3(256), 0, st, p);
      else if (c.R <= 128) hipLaunchKernelGGL((k_lora_expand<DT, YDT, 4, 16>), grid, dim3(256), 0, st, p);
      else hipLaunchKernelGGL((k_lora_expand<DT, YDT, 8, 16>), grid, dim3(256), 0, st, p);
    };
    if (p.planned) expand(std::integral_constant<int, kLoraTile>{});
    else expand(std::integral_constant<int, 16>{});
  };
  auto go = [&](auto dtc) {
    if (c.ydt == DT_F32) typed(dtc, std::integral_constant<int, DT_F32>{});
    else if (c.ydt == DT_F16) typed(dtc, std::integral_constant<int, DT_F16>{});
    else typed(dtc, std::integral_constant<int, DT_BF16>{});
  };
  if (c.xdt == DT_F16) go(std::integral_constant<int, DT_F16>{});
  else go(std::integral_constant<int, DT_BF16>{});
  return hipGetLastError();
}

}  // namespace awq
