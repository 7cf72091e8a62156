// Orthogonalised update of a weight matrix for sm_103a: momentum, division by
// the Frobenius norm, and Newton-Schulz steps
//
//   X <- a X + b (X X^T) X + c (X X^T)^2 X
//
// by three products each (oxide-train README and RustingBrain page end a step
// in AdamW; neither describes this update):
//
//   A = X X^T,   P = a I + b A + c A A,   X <- P X       (m <= n; X <- X P by columns else)
//
// A and P are symmetric: their tiles on and below the diagonal are computed, and
// what lies above is read as the transpose of what lies below.  Between the
// products the matrices are fp16, scaled by powers of two (kMuonX, kMuonA, kMuonP):
// the singular values stay below about 1.2 (15.9 fit), so fp16's eleven bits cost a step 2^-12 of a value where bf16 costs 2^-9, at the same
// rate; five steps leave 1.2e-3 of the result's norm (768 x 768 of normal
// numbers; bf16 9.8e-3).  Sums are fp32 throughout, the norm's in double.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "product.cuh"

namespace detattn {
namespace {

constexpr int kInThreads = 256;

// ------------------------------------------------------------ momentum, norm, scaling
__device__ __forceinline__ void load8(const MuonInArgs& a, size_t at, float (&f)[8]) {
  if (a.g_fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.g) + at);
    const float4 x = p[0], y = p[1];
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.g) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load_momentum(const MuonInArgs& a, size_t at, float (&m)[8]) {
  const float4* p = reinterpret_cast<const float4*>(a.momentum + at);
  const float4 x = p[0], y = p[1];
  m[0] = x.x, m[1] = x.y, m[2] = x.z, m[3] = x.w;
  m[4] = y.x, m[5] = y.y, m[6] = y.z, m[7] = y.w;
}

// A square in one of three ranges, so that the sum neither overflows nor loses
// small gradients: below 2^-40 scaled by 2^80, above 2^40 by 2^-80.
struct Squares {
  float small = 0.0f, mid = 0.0f, big = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float m = fabsf(x);
    if (m < 9.094947e-13f) {
      const float y = x * 1.2089258e24f;
      small = fmaf(y, y, small);
    } else if (m > 1.0995116e12f) {
      const float y = x * 8.271806e-25f;
      big = fmaf(y, y, big);
    } else {
      mid = fmaf(x, x, mid);  // (a NaN too)
    }
  }
  __device__ __forceinline__ double total() const {
    return static_cast<double>(big) * 1.461501637330903e48 + static_cast<double>(mid) +
           static_cast<double>(small) * 6.842277657836021e-49;
  }
};

// momentum <- beta momentum + g (where there is one), and each block's sum of
// the squares of the update.  Grid (blocks, batch).
__global__ void __launch_bounds__(kInThreads) muon_momentum_kernel(const MuonInArgs a) {
  __shared__ double sh[kInThreads / 32];
  griddep_launch_dependents();
  const int block = blockIdx.y * a.blocks + blockIdx.x;
  for (int i = block * kInThreads + threadIdx.x; i < a.n_counts; i += a.batch * a.blocks * kInThreads)
    a.counts[i] = 0u;
  const size_t base = static_cast<size_t>(blockIdx.y) * a.count;
  const long vecs = a.count / 8;
  double total = 0.0;
  Squares sq;
  int n = 0;
  const long step = static_cast<long>(a.blocks) * kInThreads;
  // Two vectors at a time: the loads of both, then the rest.
  for (long i = static_cast<long>(blockIdx.x) * kInThreads + threadIdx.x; i < vecs; i += 2 * step) {
    float g[2][8], m[2][8];
    const size_t at[2] = {base + static_cast<size_t>(i) * 8, base + static_cast<size_t>(i + step) * 8};
    const bool both = i + step < vecs;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k == 0 || both) {
        load8(a, at[k], g[k]);
        if (a.momentum != nullptr) load_momentum(a, at[k], m[k]);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !both) continue;
      if (a.momentum != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[k][j] = fmaf(a.beta, m[k][j], g[k][j]);
          g[k][j] = a.nesterov ? fmaf(a.beta, m[k][j], g[k][j]) : m[k][j];
        }
        float4* p = reinterpret_cast<float4*>(a.momentum + at[k]);
        p[0] = make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
        p[1] = make_float4(m[k][4], m[k][5], m[k][6], m[k][7]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq.add(g[k][j]);
    }
    // In fp32 for 256 squares at most, then in double (whose rate is 1/64 of fp32's).
    if (++n == 16) {
      total += sq.total();
      sq = Squares();
      n = 0;
    }
  }
  total += sq.total();
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kInThreads / 32; ++i) s += sh[i];
    a.sums[static_cast<size_t>(blockIdx.y) * a.blocks + blockIdx.x] = s;
  }
}

// X = kMuonX u / (|u| + eps) in fp16.
__global__ void __launch_bounds__(kInThreads) muon_scale_kernel(const MuonInArgs a) {
  __shared__ double sh[kInThreads / 32];
  __shared__ float factors[2];
  griddep_launch_dependents();
  griddep_wait();
  double total = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += kInThreads)
    total += a.sums[static_cast<size_t>(blockIdx.y) * a.blocks + i];
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    total = 0.0;
    for (int i = 0; i < kInThreads / 32; ++i) total += sh[i];
    // In two factors: neither the norm's inverse nor the values overflow.
    const double norm = sqrt(total) + static_cast<double>(a.eps);
    int e = 0;
    const double part = frexp(norm, &e);  // norm = part 2^e
    const int e0 = -e / 2, e1 = -e - e0;
    factors[0] = exp2f(static_cast<float>(e0));
    factors[1] = exp2f(static_cast<float>(e1)) * static_cast<float>(static_cast<double>(kMuonX) / part);
  }
  __syncthreads();
  const float s0 = factors[0], s1 = factors[1];
  const size_t base = static_cast<size_t>(blockIdx.y) * a.count;
  const long vecs = a.count / 8;
  const long step = static_cast<long>(a.blocks) * kInThreads;
  for (long i = static_cast<long>(blockIdx.x) * kInThreads + threadIdx.x; i < vecs; i += 2 * step) {
    const size_t at[2] = {base + static_cast<size_t>(i) * 8, base + static_cast<size_t>(i + step) * 8};
    const bool both = i + step < vecs;
    float g[2][8], m[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k == 0 || both) {
        if (a.momentum == nullptr || a.nesterov) load8(a, at[k], g[k]);
        if (a.momentum != nullptr) load_momentum(a, at[k], m[k]);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !both) continue;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float u[2];
#pragma unroll
        for (int l = 0; l < 2; ++l)
          u[l] = a.momentum == nullptr ? g[k][j + l] : a.nesterov ? fmaf(a.beta, m[k][j + l], g[k][j + l]) : m[k][j + l];
        const __half2 h = __floats2half2_rn(u[0] * s0 * s1, u[1] * s0 * s1);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(static_cast<__half*>(a.x) + at[k]) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------ products
// All products of all steps in one launch: tiles in one order (step by step; in a
// step the tiles of A, of P, of the next X, matrix by matrix), dealt to teams in
// turn.  What a tile needs is counted: a finished tile of A or P adds to the
// counts of its row block and its column block, a finished tile of X to that of
// its block along the shorter side, and a tile starts when the counts of the
// blocks it reads are complete.  That one X is complete follows from any complete
// block of P (all blocks of A, so all blocks of X, went into it), and so does that
// nobody still reads what a tile overwrites: A(i, j) of the next step is written
// after blocks i and j of the next X, so after blocks i and j of P, which every
// reader of blocks i and j of A has added to.  The launch is cooperative: all
// blocks are resident, each takes its tiles in order, and a tile waits only for
// tiles before it, so every wait ends (they are bounded all the same).
//
// Against a launch for each product this fills rounds (4096 x 6144 has 136, 136 and
// 384 tiles a step for 76 teams) and starts a tile as soon as its own inputs are
// there: 12 x 768 x 1280 took 226 us and did 331 (214 now, with less double arithmetic
// before it), 4096 x 6144 1,190 and 1,258, 768 x 768 109 and 115.  A tile is ready 3 to 4 us after its last product (the queue of
// products 0.3 to 1.3, its stores 1 to 3, the fence before the count 0.7) and seen
// 1.2 us later: with at most a dozen matrices that chain, not the rate of the
// products, is the time.  Measured and not kept: a warp that looks at the counts ahead
// of the producer (768 x 768: 122 us); all tiles of a symmetric result computed
// where the teams are idle anyway (768 x 768: 109.4 us against 110.4); two groups of
// matrices by turns (12 x 768 x 1280: 250 us); the tiles above the diagonal written
// too (a tile's epilogue 6 us in the place of 2); how an operand lies in memory chosen
// step by step and not in runs (258 us: the issue of a product then takes longer than
// the product); sixteen
// epilogue warps (107.8, 219 and 1,174 us where eight took 109.6, 215 and 1,179); one
// count per block and tile in the place of its warps' (106.7, 217 and 1,200 against
// 109.4, 216 and 1,200).
enum : int { kGram = 0, kPoly = 1, kNext = 2 };

struct MuonUnit {
  int batch, mt, nt, kind, step, n_k;
};
__device__ __forceinline__ MuonUnit muon_unit(const MuonChainArgs& a, int u) {
  MuonUnit w;
  const int sym = a.batch * a.sym_tiles, full = a.tiles_s * a.tiles_o, per = 2 * sym + a.batch * full;
  w.step = u / per;
  int r = u - w.step * per;
  w.kind = r < sym ? kGram : r < 2 * sym ? kPoly : kNext;
  r -= w.kind * sym;
  if (w.kind == kNext) {
    w.batch = r / full;
    r -= w.batch * full;
    // Along the shorter side first: few columns (rows) of X at a time.
    const int s = r % a.tiles_s, o = r / a.tiles_s;
    w.mt = a.wide ? s : o;
    w.nt = a.wide ? o : s;
    w.n_k = (a.side + product::kBK - 1) / product::kBK;
  } else {
    w.batch = r / a.sym_tiles;
    r -= w.batch * a.sym_tiles;
    // Tiles (i, j), j <= i, in order of i: i (i + 1) / 2 + j = r.
    int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > r) --i;
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    w.mt = i;
    w.nt = r - i * (i + 1) / 2;
    w.n_k = ((w.kind == kPoly ? a.side : a.wide ? a.n : a.m) + product::kBK - 1) / product::kBK;
  }
  return w;
}
__device__ __forceinline__ unsigned* muon_count(const MuonChainArgs& a, int batch, int kind, int block) {
  return a.counts + ((static_cast<size_t>(batch) * 3 + kind) * a.tiles_s + block) * kMuonCountStride;
}
// Waits (bounded) until both counts have reached `target`; what was counted is then visible.
__device__ __forceinline__ bool wait_counts(const unsigned* p, const unsigned* q, unsigned target,
                                            uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    unsigned v, x;
    asm volatile(
        "ld.relaxed.gpu.global.u32 %0, [%2];\n\t"
        "ld.relaxed.gpu.global.u32 %1, [%3];"
        : "=r"(v), "=r"(x)
        : "l"(p), "l"(q)
        : "memory");
    if (v >= target && x >= target) {
      asm volatile("fence.acq_rel.gpu;" ::: "memory");
      return true;
    }
    if ((it & 15u) == 0u) {
      const uint64_t t = globaltimer_ns();
      if (it == 0) t0 = t;
      if (t - t0 > limit_ns) return false;
    }
    __nanosleep(20);
  }
  return false;
}
// Waits (bounded) until this block's producer has seen the inputs of `n` tiles.
__device__ __forceinline__ bool wait_ready(uint32_t ready, int n, uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 31); ++it) {  // (2^26 looks take a few seconds, less than limits may be)
    int v;
    asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(ready) : "memory");
    if (v >= n) return true;
    if ((it & 63u) == 0u) {
      const uint64_t t = globaltimer_ns();
      if (it == 0) t0 = t;
      if (t - t0 > limit_ns) return false;
    }
    __nanosleep(40);
  }
  return false;
}
// Until everything that tile `w` reads is there.
template <int CTAS>
__device__ __forceinline__ bool wait_inputs(const MuonChainArgs& a, const MuonUnit& w) {
  constexpr unsigned kArrivals = CTAS * product::kEpiWarps;
  if (w.kind == kGram && w.step == 0) return true;  // X is the kernel before's
  const unsigned target = kArrivals * (w.kind == kGram ? a.tiles_o * w.step
                                                       : a.tiles_s * (w.step + 1));
  const int kind = w.kind == kGram ? kNext : w.kind - 1;
  const int s = w.kind == kNext ? (a.wide ? w.mt : w.nt) : w.mt;
  const bool ok = wait_counts(muon_count(a, w.batch, kind, s),
                              muon_count(a, w.batch, kind, w.kind == kNext ? s : w.nt), target, a.wait_ns);
  // The tiles were written by ordinary stores and are read by TMA.
  asm volatile("fence.proxy.async;" ::: "memory");
  return ok;
}
// The steps of a tile in runs whose operands lie alike in memory: f(first step,
// end, A with K along its rows, the same of B).  Of a symmetric matrix whose
// tiles above the diagonal are not written, block i's part beyond the diagonal
// is read as the transpose of what is written.
template <int CTAS, class F>
__device__ __forceinline__ void muon_runs(const MuonChainArgs& a, const MuonUnit& w, F&& f) {
  constexpr std::bool_constant<false> rows;
  constexpr std::bool_constant<true> cols;
  constexpr int kPer = 128 * CTAS / product::kBK;  // steps of a tile's width
  if (w.kind == kGram) {
    if (a.wide)
      f(0, w.n_k, rows, rows);
    else
      f(0, w.n_k, cols, cols);
    return;
  }
  // Steps up to the end of A's and of B's tile on the diagonal.
  const int past_m = min((w.mt + 1) * kPer, w.n_k), past_n = min((w.nt + 1) * kPer, w.n_k);
  if (w.kind == kPoly) {  // (nt <= mt)
    f(0, past_n, rows, rows);
    f(past_n, past_m, rows, cols);
    f(past_m, w.n_k, cols, cols);
  } else if (a.wide) {
    f(0, past_m, rows, cols);
    f(past_m, w.n_k, cols, cols);
  } else {
    f(0, past_n, rows, rows);
    f(past_n, w.n_k, rows, cols);
  }
}

// A thread's part of a tile: row `row`, kCols columns from `col`.
template <int CTAS>
struct MuonTile {
  static constexpr int kCols = 64 * CTAS;
  const MuonChainArgs& a;
  const int kind, row, col;
  const bool last, diagonal;
  int rows, cols;
  long ld;
  size_t at;
  float alpha, beta, diag;
  uint4 add[kCols / 8];
  __device__ __forceinline__ MuonTile(const MuonChainArgs& args, const MuonUnit& w, int r, int c)
      : a(args), kind(w.kind), row(r), col(c), last(w.kind == kNext && w.step == args.steps - 1),
        diagonal(w.kind == kPoly && w.mt == w.nt) {
    rows = kind == kNext ? a.m : a.side;
    cols = kind == kNext ? a.n : a.side;
    ld = kind == kNext ? a.n : a.ld;
    at = (static_cast<size_t>(w.batch) * rows + row) * ld + col;
    const float* k = a.coeffs[w.step];
    alpha = kind == kGram ? kMuonA / (kMuonX * kMuonX) : kind == kPoly ? k[2] * (kMuonP / (kMuonA * kMuonA))
            : last        ? 1.0f / (kMuonX * kMuonP)
                          : 1.0f / kMuonP;
    beta = k[1] * (kMuonP / kMuonA);
    diag = k[0] * kMuonP;
  }
  // What is added to A A: from L2, where other blocks' stores are.
  __device__ __forceinline__ void fetch() {
    const __half* p = static_cast<const __half*>(a.gram_out) + at;
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i)
      add[i] = row < rows && col + 8 * i < cols ? __ldcg(reinterpret_cast<const uint4*>(p + 8 * i))
                                                : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void take(uint32_t taddr, int next) {
    void* out = kind == kGram ? a.gram_out : kind == kPoly ? a.poly_out : last ? a.o : a.x_out[next];
    const bool on32 = ld % 16 == 0 && (!last || a.o_on32);
    each32<kCols>(taddr, [&](int c, uint32_t (&v)[32]) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = alpha * __uint_as_float(v[2 * i]), y = alpha * __uint_as_float(v[2 * i + 1]);
        if (kind == kPoly) {
          const uint4 q = add[c / 8 + i / 4];
          const uint32_t s = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s));
          x = fmaf(beta, f.x, x);
          y = fmaf(beta, f.y, y);
          if (diagonal) {
            if (row == col + c + 2 * i) x += diag;
            if (row == col + c + 2 * i + 1) y += diag;
          }
        }
        if (last) {
          w[i] = pack_bf16x2(x, y);
        } else {
          const __half2 h = __floats2half2_rn(x, y);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      if (row < rows) {
        __half* dst = static_cast<__half*>(out) + at + c;
        if (on32 && col + c + 32 <= cols) {
          store32(dst, w);
          store32(dst + 16, w + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + c + 8 * i < cols)
              *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
    });
  }
};

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(product::kThreads, 1)
    muon_chain_kernel(const __grid_constant__ MuonChainArgs a) {
  using namespace product;
  constexpr int kTile = 128 * CTAS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int ready;  // this block's tiles whose inputs are there
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CTAS == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int team = blockIdx.x / CTAS, teams = gridDim.x / CTAS;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto lead_bar = [&](int i) {
    return CTAS == 2 ? map_shared_rank(smem_u32(&bars[i]), 0) : smem_u32(&bars[i]);
  };
  if (warp == 1) {
    if constexpr (CTAS == 2) {
      tmem_alloc_pair(smem_u32(&tmem_slot), 2 * kTile);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_slot), 2 * kTile);
      tmem_relinquish();
    }
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    ready = 0;
    init_barriers<CTAS>(bars);
    fence_barrier_init();
  }
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int units = a.steps * a.batch * (2 * a.sym_tiles + a.tiles_s * a.tiles_o);
  bool ok = true;
  int steps = 0;  // warp 1: products issued (even block), or to be issued (odd block)

  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      int it = 0, tile = 0;
      for (int u = team; u < units && ok; u += teams) {
        const MuonUnit w = muon_unit(a, u);
        if (!(ok = wait_inputs<CTAS>(a, w))) break;
        asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(&ready)), "r"(++tile) : "memory");
        const int cur = w.step & 1;
        // Each operand's matrix: [K contiguous, K along the rows].
        const CUtensorMap* ma = w.kind == kPoly ? a.gram : w.kind == kNext && a.wide ? a.poly : a.x[cur];
        const CUtensorMap* mb = w.kind == kPoly ? a.gram : w.kind == kNext && !a.wide ? a.poly : a.x[cur];
        const int m = w.mt * kTile + rank * 128, n = w.nt * kTile + rank * 128;
        muon_runs<CTAS>(a, w, [&](int kb0, int kb1, auto a_mn, auto b_mn) {
          for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
            if (it >= kStages && !(ok = mbar_wait_hint(bar(kBarEmpty + r.s), r.parity ^ 1u, a.wait_ns))) break;
            if (rank == 0) mbar_arrive_expect_tx(bar(kBarFull + r.s), CTAS * kStageBytes);
            const uint32_t to = lead_bar(kBarFull + r.s), da = s0 + r.s * kStageBytes, db = da + kOperandBytes;
            const int k = kb * kBK;
            auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
              if constexpr (CTAS == 2)
                tma_load_3d_pair(dst, map, to, c0, c1, w.batch);
              else
                tma_load_3d(dst, map, to, c0, c1, w.batch);
            };
            if constexpr (a_mn.value) {
              load(da, ma + 1, m, k);
              load(da + 8192, ma + 1, m + 64, k);
            } else {
              load(da, ma, k, m);
            }
            if constexpr (b_mn.value) {
              load(db, mb + 1, n, k);
              load(db + 8192, mb + 1, n + 64, k);
            } else {
              load(db, mb, k, n);
            }
            r.next();
          }
        });
      }
      bool landed = true;
      if (rank == 0)
        for (int k = it > kStages ? it - kStages : 0; k < it && landed; ++k)
          landed = mbar_wait_hint(bar(kBarFull + k % kStages), (k / kStages) & 1, a.wait_ns);
      if (!ok || !landed) atomicOr(&g_product_status, 1u);
    }
    __syncwarp();
  } else if (warp == 1 && rank != 0) {
    for (int u = team; u < units; u += teams) steps += muon_unit(a, u).n_k;
  } else if (warp == 1) {
    Ring r;
    int n = 0;
    for (int u = team; u < units && ok; u += teams, ++n) {
      const MuonUnit w = muon_unit(a, u);
      const int acc = n & 1;
      if (n >= 2 &&
          !(ok = warp_all(mbar_wait_hint<CTAS == 2>(bar(kBarAccFree + acc), ((n >> 1) & 1) ^ 1, a.wait_ns))))
        break;
      tc_fence_after();
      muon_runs<CTAS>(a, w, [&](int kb0, int kb1, auto a_mn, auto b_mn) {
        constexpr uint32_t kId = idesc(kTile, kTile, a_mn.value, b_mn.value, true);
        constexpr uint32_t kStepA = a_mn.value ? 2048u : 32u, kStepB = b_mn.value ? 2048u : 32u;
        const uint64_t dA0 = sdesc_sw128(s0, a_mn.value ? 8192 : 16, 1024);
        const uint64_t dB0 = sdesc_sw128(s0 + kOperandBytes, b_mn.value ? 8192 : 16, 1024);
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
          // A tile's first operands wait for other blocks' tiles, as long as their
          // copies' producer does and a little longer.
          if (!(ok = warp_all(mbar_wait_hint(bar(kBarFull + r.s), r.parity, kb == 0 ? 3 * a.wait_ns : a.wait_ns)))) break;
          tc_fence_after();
          const uint64_t da = desc_add(dA0, r.s * kStageBytes), db = desc_add(dB0, r.s * kStageBytes);
          if constexpr (CTAS == 2) {
            mma_ss_x4_pair(tmem + acc * kTile, da, desc_add(da, kStepA), desc_add(da, 2 * kStepA),
                           desc_add(da, 3 * kStepA), db, desc_add(db, kStepB), desc_add(db, 2 * kStepB),
                           desc_add(db, 3 * kStepB), kId, kb > 0 ? 1u : 0u);
            mma_commit_pair(bar(kBarEmpty + r.s));
          } else {
            mma_ss_x4(tmem + acc * kTile, da, desc_add(da, kStepA), desc_add(da, 2 * kStepA),
                      desc_add(da, 3 * kStepA), db, desc_add(db, kStepB), desc_add(db, 2 * kStepB),
                      desc_add(db, 3 * kStepB), kId, kb > 0 ? 1u : 0u);
            mma_commit(bar(kBarEmpty + r.s));
          }
          r.next();
          ++steps;
        }
      });
      if (ok) {
        if constexpr (CTAS == 2)
          mma_commit_pair(bar(kBarAcc + acc));
        else
          mma_commit(bar(kBarAcc + acc));
      }
    }
    if constexpr (CTAS == 2)
      mma_commit_pair(bar(kBarDrain));
    else
      mma_commit(bar(kBarDrain));
  } else if (warp >= kFirstEpiWarp) {
    const int quarter = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
    const uint32_t tl = tmem + half * MuonTile<CTAS>::kCols + (static_cast<uint32_t>(quarter * 32) << 16);
    int n = 0;
    for (int u = team; u < units; u += teams, ++n) {
      const MuonUnit w = muon_unit(a, u);
      const int acc = n & 1;
      MuonTile<CTAS> t(a, w, w.mt * kTile + rank * 128 + quarter * 32 + lane,
                       w.nt * kTile + half * MuonTile<CTAS>::kCols);
      if (w.kind == kPoly) {
        // The producer has seen what this tile reads, and says so here.
        if (!(ok = warp_all(wait_ready(smem_u32(&ready), n + 1, 3 * a.wait_ns)))) break;
        t.fetch();
      }
      if (!(ok = warp_all(mbar_wait_hint(bar(kBarAcc + acc), (n >> 1) & 1, 4 * a.wait_ns)))) break;
      tc_fence_after();
      t.take(tl + acc * kTile, (w.step & 1) ^ 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CTAS == 2)
          mbar_arrive_pair(lead_bar(kBarAccFree + acc));
        else
          mbar_arrive(bar(kBarAccFree + acc));
      }
      if (t.last) continue;
      // Once this warp's part is there for all blocks, it counts.
      if (lane == 0) {
        __threadfence();
        auto count = [&](int block) {
          asm volatile("red.relaxed.gpu.global.add.u32 [%0], 1;" ::"l"(muon_count(a, w.batch, w.kind, block))
                       : "memory");
        };
        if (w.kind == kNext) {
          count(a.wide ? w.mt : w.nt);
        } else {
          count(w.mt);
          if (w.mt != w.nt) count(w.nt);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_product_status, 1u);
  }
  tc_fence_before();
  __syncthreads();
  // As in product_kernel: each block waits for its own copies of the last commits.
  if (warp == 1) {
    for (int k = steps > kStages ? steps - kStages : 0; k < steps && ok; ++k)
      ok = warp_all(mbar_wait_hint(bar(kBarEmpty + k % kStages), (k / kStages) & 1, a.wait_ns));
    if (!warp_all(mbar_wait_hint(bar(kBarDrain), 0, a.wait_ns)) || !ok) {
      if (lane == 0) atomicOr(&g_product_status, 1u);
    }
    __syncwarp();
  }
  if constexpr (CTAS == 2) cluster_sync();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    if constexpr (CTAS == 2)
      tmem_dealloc_pair(tmem_slot, 2 * kTile);
    else
      tmem_dealloc(tmem_slot, 2 * kTile);
  }
}

// Failure-detection self-test: the waits for other blocks' tiles, on a count that
// nothing adds to, and for this block's producer.
__device__ unsigned g_no_count = 0;
__global__ void muon_wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ int ready;
  if (threadIdx.x == 0) ready = 0;
  __syncwarp();
  const bool counts = product::warp_all(wait_counts(&g_no_count, &g_no_count, 1u, limit_ns));
  const bool seen = product::warp_all(wait_ready(smem_u32(&ready), 1, limit_ns));
  if (threadIdx.x == 0 && !counts && !seen) atomicOr(&g_product_status, 1u);
}

template <int CTAS>
cudaError_t launch_chain_t(const MuonChainArgs& a, long units, cudaStream_t st) {
  // Teams that are resident at once, by device (0: not asked yet).  Their number
  // changes no bit: a tile's sum is one team's whatever the team.
  static int resident[64] = {};
  static unsigned long long attr_ctx[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = current_context_id();
  auto* kernel = muon_chain_kernel<CTAS>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = product::kThreads;
  cfg.dynamicSmemBytes = product::kSmemBytes;
  cfg.stream = st;
  int teams = dev < 64 && ctx != 0 && attr_ctx[dev] == ctx ? resident[dev] : 0;
  if (teams == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, product::kSmemBytes);
    if (e != cudaSuccess) return e;
    if constexpr (CTAS == 1) {
      int per_sm = 0, sms = 0;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, product::kThreads, product::kSmemBytes);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      teams = per_sm * sms;
    } else {
      cfg.gridDim = dim3(kProductSms);
      e = cudaOccupancyMaxActiveClusters(&teams, kernel, &cfg);
    }
    if (e != cudaSuccess) return e;
    if (teams < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) {
      resident[dev] = teams;
      attr_ctx[dev] = ctx;
    }
  }
  if (teams > product_teams(CTAS)) teams = product_teams(CTAS);
  if (teams > units) teams = static_cast<int>(units);
  cfg.gridDim = dim3(static_cast<unsigned>(CTAS * teams));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

int muon_sum_blocks(int batch, long count) {
  // About four vectors a thread, no more than eight blocks per SM over all matrices.
  long b = (count / 8 + 4 * kInThreads - 1) / (4 * kInThreads);
  const long most = 8l * kProductSms / batch;
  if (b > most) b = most;
  return static_cast<int>(b < 1 ? 1 : b);
}

cudaError_t launch_muon_momentum(const MuonInArgs& a, cudaStream_t st) {
  return launch_dependent(muon_momentum_kernel, dim3(a.blocks, a.batch), kInThreads, st, false, a);
}
cudaError_t launch_muon_scale(const MuonInArgs& a, cudaStream_t st) {
  return launch_dependent(muon_scale_kernel, dim3(a.blocks, a.batch), kInThreads, st, true, a);
}
MuonPlan muon_plan(int batch, int m, int n) {
  const long side = m < n ? m : n, other = m < n ? n : m;
  MuonPlan best{};
  double least = 0.0;
  for (int ctas = 1; ctas <= 2; ++ctas) {
    MuonPlan p{};
    p.ctas = ctas;
    const long tile = 128 * p.ctas, teams = product_teams(p.ctas);
    p.tiles_s = static_cast<int>((side + tile - 1) / tile);
    p.tiles_o = static_cast<int>((other + tile - 1) / tile);
    p.sym_tiles = p.tiles_s * (p.tiles_s + 1) / 2;
    p.units = static_cast<long>(batch) * (2l * p.sym_tiles + static_cast<long>(p.tiles_s) * p.tiles_o);
    // Clocks of a step: a product takes its share of the teams' time and at least
    // one tile's; a pair's step of 64 along K takes about 600, a block's 400
    // (what L2 delivers to all of them), and a tile's start and end
    // 2000 for each.  (768 x 768: 110 us with single blocks, 138 with pairs; 12 x 768 x
    // 1280 276 and 226; 4096 x 6144 1,745 and 1,190.  Their transposes take the same.)
    auto product_clocks = [&](long tiles, long k) {
      const double t = static_cast<double>((k + 63) / 64) * (p.ctas == 2 ? 600.0 : 400.0) + p.ctas * 2000.0;
      const double all = t * static_cast<double>(tiles) * batch / static_cast<double>(teams);
      return all > t ? all : t;
    };
    const double cost = product_clocks(p.sym_tiles, other) + product_clocks(p.sym_tiles, side) +
                        product_clocks(static_cast<long>(p.tiles_s) * p.tiles_o, side);
    if (ctas == 1 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}
cudaError_t launch_muon_chain(const MuonChainArgs& a, int ctas, long units, cudaStream_t st) {
  return ctas == 2 ? launch_chain_t<2>(a, units, st) : launch_chain_t<1>(a, units, st);
}
cudaError_t take_muon_status(cudaStream_t st, unsigned* out) { return product::take_status(st, out); }
cudaError_t launch_muon_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  product::wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  muon_wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

}  // namespace detattn
