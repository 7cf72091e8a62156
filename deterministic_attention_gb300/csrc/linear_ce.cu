// Softmax cross entropy of the output projection without its logits, forward
// and backward, for sm_103a (oxide-train README: the output projection of a
// vocabulary of 50,257, padded to 50,432, on bf16 tensor cores):
//
//   z = x w^T,  lse_n = ln sum_v exp z_nv,  loss_n = lse_n - z_n,target
//   dz_nv = (g_n + e_n) exp(z_nv - lse_n) - g_n [v = target_n]
//   dx = dz w,  dw = dz^T x
//
// Forward: one product (product.cuh) whose epilogue leaves, for every row and
// 128 columns, the largest logit and the sum of exponentials below it, and a
// second kernel that merges them.  Backward, one piece of the vocabulary after
// another: the piece's dz as bf16 into the workspace (the logits computed
// again), then its share of dx, and its rows of dw.  Rounding dz to bf16, which
// the tensor core's second products need, is the one rounding between the
// inputs and the results (half a step is 2^-8 of a dz at most); the sums over the
// vocabulary and over the tokens are in fp32.  dz is held over the largest
// |dloss| (ce_unit_kernel): where all rows weigh the same, as with a mean, a
// target's dz is then next to -1, which is a bf16 number, and not next to -dloss,
// whose rounding would be the same in every row and so in dx and dw as a whole
// (dloss = 1/240: 3.4e-3).
//
// Measured (device): 32,768 rows, d = 1536, V = 50,432: forward 2.5 ms in short runs
// (2.0 PFLOP/s; the measured bf16 peak, 1.90, is a library product's), 2.83 for
// seconds (1.79 PFLOP/s at 1,500 MHz, under the power limit); backward 8.9 ms (1.71
// PFLOP/s, under the power limit; 7.7 at best, 9.3 for seconds): a piece of 12,800
// words takes 0.69 (dz), 0.69 (dx) and 0.67 ms (dw), 0.68 at the measured peak.  1,187
// rows, d = 768: backward 176 us (with fp32 dw 202), the tensor pipe busy 81 to 84 %
// of the time; forward of 128 rows 21 us, 11.4 of them what the weights' 77 MB take at
// the copy rate.  What mattered: tiles in bands (dx and dz had read dz and x from
// DRAM once per column tile: 573 -> 407 and 484 -> 408 us), 32-byte stores, a
// tile's row data loaded while the tile before it is taken (a tile of d = 768 takes
// 4.8 us of products and took 5.3 of epilogue; now 3.3), all loads of a sum to add to
// before the sums (dx of a middle piece 575 -> 450 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "exp2_poly.cuh"
#include "product.cuh"

namespace detattn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSumThreads = 256;

// ------------------------------------------------------------ forward
struct StatsEpi {
  static constexpr int kCols = 128;
  static constexpr bool kOwnInputs = true;
  using Args = CeStatsArgs;
  const Args* args;
  int row, col, target;
  __device__ __forceinline__ StatsEpi(const Args& a, const product::Unit&, int r, int c)
      : args(&a), row(r), col(c), target(row < a.N ? a.targets[row] : -1) {}
  __device__ __forceinline__ void prepare() {
    if (target >= args->V && col == 0) atomicOr(&g_product_status, 2u);
  }
  __device__ __forceinline__ void take(uint32_t taddr) {
    const Args& a = *args;
    float m = -INFINITY, s = 0.0f, held = 0.0f;  // s is held over 2^held
    each32<kCols>(taddr, [&](int c, uint32_t (&v)[32]) {
      const int c0 = col + c;
      // Columns past the vocabulary, in its last tile.
      if (c0 + 32 > a.V) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c0 + i >= a.V) v[i] = 0xFF800000u;
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < 32; i += 2) top = fmax3(top, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
      // (Rounded by itself: base - held is 0, and s stays, where the largest does.)
      const float base = top == -INFINITY ? 0.0f : __fmul_rn(top, kLog2e);
      const uint64_t nb = f2_make(-base, -base), l2 = f2_make(kLog2e, kLog2e);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float p, q;
        f2_split(f2_fma(f2_make(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), l2, nb), p, q);
        sum[i / 2 & 1] = f2_add(sum[i / 2 & 1], f2_make(ex2_approx(p), ex2_approx(q)));
      }
      float s0, s1;
      f2_split(f2_add(sum[0], sum[1]), s0, s1);
      s = s * ex2_approx(m == -INFINITY ? -INFINITY : held - base) + (s0 + s1);
      m = top;
      held = base;
      const unsigned at = static_cast<unsigned>(target - c0);
      if (at < 32u && target < a.V) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) z = at == static_cast<unsigned>(i) ? __uint_as_float(v[i]) : z;
        a.z_target[row] = z;
      }
    });
    if (row < a.N) a.part[static_cast<size_t>(col / kCols) * a.N + row] = make_float2(m, s);
  }
};

// A block merges kFinishRows rows; the threads that share a row take its parts
// eight at a time.  A part's sum is 2^r times what its largest logit asks for, r
// the rounding of m log2e: it is taken back here, so that loss does not lose what
// lse does.
constexpr int kFinishRows = 8, kFinishWarps = 16, kFinishGroups = kFinishWarps * 32 / kFinishRows;
struct Merged {
  float m = -INFINITY, s = 0.0f;
  __device__ __forceinline__ void add(float m1, float s1) {
    const float top = fmaxf(m, m1), base = top == -INFINITY ? 0.0f : top;
    s = s * exp2f((m - base) * kLog2e) + s1 * exp2f((m1 - base) * kLog2e);
    m = top;
  }
};
__global__ void __launch_bounds__(kFinishWarps * 32) ce_finish_kernel(const CeFinishArgs a) {
  __shared__ float2 sh[kFinishWarps][kFinishRows];
  griddep_launch_dependents();
  const int lane = threadIdx.x % kFinishRows, group = threadIdx.x / kFinishRows;
  const int row = min(blockIdx.x * kFinishRows + lane, a.N - 1);
  const int t = a.targets[row];
  griddep_wait();
  const float2* p = a.part + row;
  Merged all;
  for (int i0 = group; i0 < a.parts; i0 += 8 * kFinishGroups) {
    float2 x[8];
    float m = all.m;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kFinishGroups;
      x[k] = i < a.parts ? p[static_cast<size_t>(i) * a.N] : make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, x[k].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float s = all.s * exp2f((all.m - base) * kLog2e);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float r = x[k].x == -INFINITY ? 0.0f : fmaf(x[k].x, kLog2e, -__fmul_rn(x[k].x, kLog2e));
      s += x[k].y * exp2f((x[k].x - base) * kLog2e - r);
    }
    all.m = m;
    all.s = s;
  }
#pragma unroll
  for (int o = kFinishRows; o < 32; o <<= 1) {
    const float m1 = __shfl_xor_sync(0xFFFFFFFFu, all.m, o), s1 = __shfl_xor_sync(0xFFFFFFFFu, all.s, o);
    all.add(m1, s1);
  }
  if ((threadIdx.x & 31) < kFinishRows) sh[threadIdx.x >> 5][lane] = make_float2(all.m, all.s);
  __syncthreads();
  if (threadIdx.x >= kFinishRows) return;
  all = Merged();
#pragma unroll
  for (int i = 0; i < kFinishWarps; ++i) all.m = fmaxf(all.m, sh[i][lane].x);
  const float base = all.m == -INFINITY ? 0.0f : all.m;
#pragma unroll
  for (int i = 0; i < kFinishWarps; ++i) all.s += sh[i][lane].y * exp2f((sh[i][lane].x - base) * kLog2e);
  if (blockIdx.x * kFinishRows + lane >= static_cast<unsigned>(a.N)) return;
  // The largest logit's own exponential is 1: what is below is rounding.
  const float ln = logf(all.s < 1.0f ? 1.0f : all.s);
  a.lse[row] = all.m + ln;
  a.loss[row] = t >= 0 && t < a.V ? (all.m - a.z_target[row]) + ln : 0.0f;
}

// ------------------------------------------------------------ backward: dz of a piece
// The unit of dz: the largest |dloss| of the rows that have a target (1 where that is
// zero or not finite).  Where a row's gradient over it would near an end of fp32's
// range, above 2^32 (sums over 2^24 rows and words still fit) or below 2^-100 (times
// the smaller exponentials), its mantissa alone: bf16 holds what fp32 does, so dz then
// neither overflows nor vanishes before dx and dw do.
__global__ void __launch_bounds__(1024) ce_unit_kernel(const int* __restrict__ targets,
                                                       const float* __restrict__ dloss,
                                                       const float* __restrict__ dlse, float* __restrict__ unit,
                                                       int N, int V) {
  __shared__ float sh[3][32];
  griddep_launch_dependents();
  float m = 0.0f, most = 0.0f, least = INFINITY;  // of |dloss|; of a row's dloss and dloss + dlse
  auto row = [&](float x) {
    x = fabsf(x);
    if (x < INFINITY) most = fmaxf(most, x);  // (a row that is not finite is by itself)
    if (x > 0.0f) least = fminf(least, x);
  };
#pragma unroll 4
  for (int i = threadIdx.x; i < N; i += 1024) {
    const int t = targets[i];
    const float g = t >= 0 && t < V ? dloss[i] : 0.0f;
    m = fmaxf(m, fabsf(g));
    row(g);
    if (dlse != nullptr) row(g + dlse[i]);
  }
  auto warp = [&]() {
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    }
  };
  warp();
  if ((threadIdx.x & 31) == 0) {
    sh[0][threadIdx.x >> 5] = m;
    sh[1][threadIdx.x >> 5] = most;
    sh[2][threadIdx.x >> 5] = least;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  m = sh[0][threadIdx.x];
  most = sh[1][threadIdx.x];
  least = sh[2][threadIdx.x];
  warp();
  if (threadIdx.x == 0) {
    const bool near = most <= m * 0x1p32f && least >= m * 0x1p-100f;
    int e;
    *unit = !(m > 0.0f && m < INFINITY) ? 1.0f : near ? m : 2.0f * frexpf(m, &e);
  }
}

struct GradEpi {
  static constexpr int kCols = 128;
  static constexpr bool kOwnInputs = true;
  using Args = CeGradArgs;
  const Args* args;
  int row, col, target;
  float lse2, g, gp;   // dloss and dloss + dlse, then over the unit
  uint32_t live, sign; // masks of a pair
  __device__ __forceinline__ GradEpi(const Args& a, const product::Unit&, int r, int c)
      : args(&a), row(r), col(c), target(-1), lse2(0.0f), g(0.0f), gp(0.0f), live(0u), sign(0u) {
    if (row < a.N) {
      target = a.targets[row];
      lse2 = a.lse[row];
      g = a.dloss[row];
      if (a.dlse != nullptr) gp = a.dlse[row];
    }
  }
  __device__ __forceinline__ void prepare() {
    const Args& a = *args;
    const float unit = *a.unit;
    if (target >= a.V && col == 0 && a.v0 == 0) atomicOr(&g_product_status, 2u);
    if (target >= a.V) target = -1;
    if (target < 0) g = 0.0f;
    gp = (g + gp) / unit;
    g /= unit;
    // gp exp(z - lse) = +-2^(z log2e - (lse log2e - log2 |gp|)); a row that takes
    // no gradient is zero whatever its logits are.
    live = row < a.N && (gp != 0.0f || g != 0.0f) ? 0xFFFFFFFFu : 0u;
    lse2 = lse2 * kLog2e - log2f(fabsf(gp));
    if (gp < 0.0f) sign = 0x80008000u;
    target -= a.v0;  // column of the piece (none: negative)
  }
  __device__ __forceinline__ void take(uint32_t taddr) {
    const Args& a = *args;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dz) + static_cast<size_t>(row) * a.ld + col;
    const uint64_t nb = f2_make(-lse2, -lse2), l2 = f2_make(kLog2e, kLog2e);
    each32<kCols>(taddr, [&](int c, uint32_t (&v)[32]) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float p, q;
        f2_split(f2_fma(f2_make(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), l2, nb), p, q);
        v[i] = __float_as_uint(ex2_approx(p));
        v[i + 1] = __float_as_uint(ex2_approx(q));
      }
      const unsigned at = static_cast<unsigned>(target - (col + c));
      if (at < 32u) {
        const float s = sign ? -g : g;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = __float_as_uint(__uint_as_float(v[i]) - (at == static_cast<unsigned>(i) ? s : 0.0f));
      }
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = (pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])) ^ sign) & live;
      // (Rows of the workspace are whole sectors; what lies behind the piece is never read.)
      if (row < a.N) {
        if (col + c < a.width) store32(dst + c, w);
        if (col + c + 16 < a.width) store32(dst + c + 16, w + 8);
      }
    });
  }
};

// ------------------------------------------------------------ backward: dx and dw
// Four neighbouring columns of a finished sum.
__device__ __forceinline__ void store4(const CeStoreArgs& a, int row, int col, float4 s, float unit) {
  const size_t at = static_cast<size_t>(row) * a.cols + col;
  s = make_float4(s.x * unit, s.y * unit, s.z * unit, s.w * unit);
  if (a.add) {
    const float4 o = *reinterpret_cast<const float4*>(a.acc + at);
    s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w);
  }
  if (a.out == nullptr)
    *reinterpret_cast<float4*>(a.acc + at) = s;
  else if (a.out_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = s;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

struct StoreEpi {
  static constexpr int kCols = 128;
  static constexpr bool kOwnInputs = false;
  using Args = CeStoreArgs;
  const Args* args;
  int row, col, part, tile_row, tile_col;
  float unit;
  __device__ __forceinline__ StoreEpi(const Args& a, const product::Unit& w, int r, int c)
      : args(&a), row(r), col(c), part(w.part), tile_row(r - w.mt * kCeTile), tile_col(c - w.nt * kCeTile),
        unit(*a.unit) {}
  __device__ __forceinline__ void prepare() {}
  __device__ __forceinline__ void take(uint32_t taddr) {
    const Args& a = *args;
    each32<kCols>(taddr, [&](int c, uint32_t (&v)[32]) {
      if (part >= 0) {
        float* dst = a.partial + (static_cast<size_t>(part) * kCeTile + tile_row) * kCeTile + tile_col + c;
#pragma unroll
        for (int i = 0; i < 32; i += 8) store32(dst + i, v + i);
        return;
      }
      if (row >= a.rows) return;
      const size_t at = static_cast<size_t>(row) * a.cols + col + c;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * unit);
      if (a.add) {
        // All of the loads, then the sums: one latency for 32 columns.
        float4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = col + c + 4 * i < a.cols ? *reinterpret_cast<const float4*>(a.acc + at + 4 * i)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + o[i].x);
          v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + o[i].y);
          v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + o[i].z);
          v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + o[i].w);
        }
      }
      const bool whole = col + c + 32 <= a.cols;
      if (a.out == nullptr || a.out_fp32) {
        float* dst = (a.out == nullptr ? a.acc : static_cast<float*>(a.out)) + at;
        if (whole && a.wide) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) store32(dst + i, v + i);
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (col + c + i < a.cols) *reinterpret_cast<uint4*>(dst + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        if (whole && a.wide) {
          store32(dst, w);
          store32(dst + 16, w + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + c + 8 * i < a.cols)
              *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
    });
  }
};

// Tiles that were cut along K: their ranges added in ascending order, four
// columns per thread.
__global__ void __launch_bounds__(kSumThreads) ce_sum_kernel(const CeStoreArgs a, const ProductPlan p) {
  constexpr int kVecs = kCeTile * kCeTile / 4;
  griddep_launch_dependents();
  griddep_wait();
  const int idx = blockIdx.x * kSumThreads + threadIdx.x;
  const int cut = idx / kVecs, at = idx % kVecs;
  int mt, nt;
  product::tile_at(p, p.whole + cut, &mt, &nt);
  const int row = mt * kCeTile + at / (kCeTile / 4), col = nt * kCeTile + (at % (kCeTile / 4)) * 4;
  if (row >= a.rows || col >= a.cols) return;
  const float4* src = reinterpret_cast<const float4*>(a.partial) + static_cast<size_t>(cut) * p.splits * kVecs + at;
  float4 s = src[0];
#pragma unroll 4
  for (int z = 1; z < p.splits; ++z) {
    const float4 x = src[static_cast<size_t>(z) * kVecs];
    s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
  }
  store4(a, row, col, s, *a.unit);
}

cudaError_t launch_sum(const CeStoreArgs& a, const ProductPlan& p, cudaStream_t st) {
  if (p.splits == 1) return cudaSuccess;
  const int cut = p.tiles_m * p.tiles_n - p.whole;
  return launch_dependent(ce_sum_kernel, dim3(static_cast<unsigned>(cut * (kCeTile * kCeTile / 4 / kSumThreads))),
                          kSumThreads, st, true, a, p);
}

}  // namespace

ProductPlan product_plan(long M, long N, long K, bool cut) {
  ProductPlan p{};
  p.band = 8;
  p.tiles_m = static_cast<int>((M + kCeTile - 1) / kCeTile);
  p.tiles_n = static_cast<int>((N + kCeTile - 1) / kCeTile);
  p.n_k = static_cast<int>((K + product::kBK - 1) / product::kBK);
  const long tiles = static_cast<long>(p.tiles_m) * p.tiles_n;
  const int teams = product_teams(2);
  p.splits = 1;
  p.whole = static_cast<int>(tiles);
  const int rem = static_cast<int>(tiles % teams);
  if (cut && rem != 0) {
    // The cut of the last round's tiles that leaves the busiest team the
    // fewest steps; cutting at all costs about twelve (partial tiles written
    // and added up, a second launch).
    double best = 0.0;
    for (int s = 1; s <= 32 && s <= p.n_k; ++s) {
      const int rounds = (rem * s + teams - 1) / teams;
      const double cost = rounds * (static_cast<double>((p.n_k + s - 1) / s) + (s > 1 ? 12.0 : 0.0));
      if (s == 1 || cost < best) {
        best = cost;
        p.splits = s;
      }
    }
    if (p.splits > 1) p.whole = static_cast<int>(tiles - rem);
  }
  const long units = p.whole + (tiles - p.whole) * p.splits;
  p.units = static_cast<int>(units);
  p.teams = static_cast<int>(units < teams ? units : teams);
  return p;
}

cudaError_t launch_ce_stats(const CUtensorMap& mx, const CUtensorMap& mw, const ProductPlan& p,
                            const CeStatsArgs& a, cudaStream_t st) {
  return product::launch<false, false, StatsEpi>(mx, mw, p, a, false, st);
}

cudaError_t launch_ce_finish(const CeFinishArgs& a, cudaStream_t st) {
  return launch_dependent(ce_finish_kernel, dim3(static_cast<unsigned>((a.N + kFinishRows - 1) / kFinishRows)),
                          kFinishWarps * 32, st, true, a);
}

cudaError_t launch_ce_unit(const int* targets, const float* dloss, const float* dlse, float* unit, int N,
                           int V, cudaStream_t st) {
  return launch_dependent(ce_unit_kernel, dim3(1), 1024, st, false, targets, dloss, dlse, unit, N, V);
}

cudaError_t launch_ce_dz(const CUtensorMap& mx, const CUtensorMap& mw, const ProductPlan& p,
                         const CeGradArgs& a, cudaStream_t st) {
  return product::launch<false, false, GradEpi>(mx, mw, p, a, true, st);
}

cudaError_t launch_ce_dx(const CUtensorMap& mdz, const CUtensorMap& mw, const ProductPlan& p,
                         const CeStoreArgs& a, cudaStream_t st) {
  cudaError_t e = product::launch<false, true, StoreEpi>(mdz, mw, p, a, true, st);
  return e != cudaSuccess ? e : launch_sum(a, p, st);
}

cudaError_t launch_ce_dw(const CUtensorMap& mdz, const CUtensorMap& mx, const ProductPlan& p,
                         const CeStoreArgs& a, cudaStream_t st) {
  cudaError_t e = product::launch<true, true, StoreEpi>(mdz, mx, p, a, true, st);
  return e != cudaSuccess ? e : launch_sum(a, p, st);
}

cudaError_t take_ce_status(cudaStream_t st, unsigned* out) { return product::take_status(st, out); }

cudaError_t launch_ce_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  product::wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

}  // namespace detattn
