// Products on the tensor cores for the ends of a training step, sm_103a:
//
//   C[m, n] = sum_k A[m, k] B[n, k]      (bf16 operands, fp32 sums)
//
// with what becomes of a tile's sums given by an epilogue class.  An operand
// lies in memory either with K contiguous or with its own index contiguous
// (A_MN, B_MN); both are what the tensor core reads from a 128-byte swizzled
// tile.  One persistent block per SM; two blocks of a cluster work on one
// tile of 256 x 256 (cta_group::2: each loads half of the rows of A and half of
// the rows of B, 32 KB a step of 64 along K, for 512 clocks of MMA):
//   warp 0       TMA producer, a ring of 7 stages
//   warp 1       (even block) tcgen05.mma issuer
//   warps 4-11   epilogue: warp w has rows 32 (w % 4) .. + 31 of its block's 128
//                and one half of the tile's columns
// Two accumulators in TMEM take turns, so a tile's epilogue runs beside the
// next tile's products.  Units of work (tiles, or ranges along K of a tile) go
// to teams in a fixed order: every element is summed in one order.
//
// The update's chain of products (muon.cu) has the same parts, with CTAS = 1 or 2
// blocks on a tile (one block: 128 x 128, the same 32 KB for 256 clocks) and fp16.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "block_ptx.cuh"
#include "step_launch.h"

namespace detattn {

namespace {
// Set by waits that run out (bit 0); one word for each translation unit.
__device__ unsigned int g_product_status;
}  // namespace

namespace product {

constexpr int kThreads = 384, kEpiWarps = 8, kFirstEpiWarp = 4;
constexpr int kBK = 64;
constexpr int kOperandBytes = 128 * kBK * 2;      // 16 KB: a block's half of A or B
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 7;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
static_assert(kSmemBytes <= 226 * 1024, "shared memory");

enum : int {
  kBarFull = 0,                     // both blocks' tiles are there (the even block's)
  kBarEmpty = kBarFull + kStages,   // their products are done (each block's)
  kBarAcc = kBarEmpty + kStages,    // an accumulator is complete (each block's)
  kBarAccFree = kBarAcc + 2,        // it has been read by the team (the even block's)
  kBarDrain = kBarAccFree + 2,
  kNumBars
};

struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Completes on a barrier of either block of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// kind::f16 with fp16 operands: idesc_bf16 with zero operand formats.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn, bool f16) {
  return f16 ? (idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10))) : idesc_bf16(M, N, a_mn, b_mn);
}

template <int CTAS>
__device__ __forceinline__ void init_barriers(uint64_t* bars) {
  auto init = [&](int i, uint32_t count) { mbar_init(smem_u32(&bars[i]), count); };
  for (int s = 0; s < kStages; ++s) {
    init(kBarFull + s, 1);
    init(kBarEmpty + s, 1);
  }
  for (int i = 0; i < 2; ++i) {
    init(kBarAcc + i, 1);
    init(kBarAccFree + i, CTAS * kEpiWarps);
  }
  init(kBarDrain, 1);
}

// ---------------------------------------------------------------- units of work
struct Unit {
  int mt, nt;          // tile
  int kb0, kb1;        // steps [kb0, kb1)
  int part;            // partial slot, -1: a whole tile
};
// Row and column tile of tile `t`.  Bands of p.band tile rows, and
// in a band column by column: the teams at work at one time share few
// rows of either operand.
__device__ __forceinline__ void tile_at(const ProductPlan& p, int t, int* mt, int* nt) {
  const int band = t / (p.band * p.tiles_n), m0 = band * p.band, rows = min(p.band, p.tiles_m - m0);
  const int r = t - m0 * p.tiles_n;
  *mt = m0 + r % rows;
  *nt = r / rows;
}
__device__ __forceinline__ Unit unit_at(const ProductPlan& p, int u) {
  Unit w;
  int tile = u;
  w.kb0 = 0;
  w.kb1 = p.n_k;
  w.part = -1;
  if (u >= p.whole) {
    const int r = u - p.whole, z = r % p.splits;
    tile = p.whole + r / p.splits;
    if (p.splits > 1) {
      w.kb0 = static_cast<int>(static_cast<long>(p.n_k) * z / p.splits);
      w.kb1 = static_cast<int>(static_cast<long>(p.n_k) * (z + 1) / p.splits);
      w.part = r;
    }
  }
  tile_at(p, tile, &w.mt, &w.nt);
  return w;
}

// Epi: a class with
//   static constexpr int kCols: columns of a thread's part of the tile (128)
//   static constexpr bool kOwnInputs: the operands are what the call got, not what
//       the kernel before wrote: their copies need not wait for it
//   struct Args
//   __device__ Epi(const Args&, const Unit&, int row, int col)
//       row: this thread's row of C; col: its first column; starts loads (it runs
//       before the tile before it is taken)
//   __device__ void prepare()
//       what follows from them
//   __device__ void take(uint32_t taddr)
//       reads kCols columns of TMEM at taddr and stores them
template <bool A_MN, bool B_MN, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const ProductPlan p, const typename Epi::Args ea) {
  constexpr int kTile = 256;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int team = blockIdx.x / 2, teams = gridDim.x / 2;
  // The same offsets in both blocks (the products read both at one address).
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto lead_bar = [&](int i) { return map_shared_rank(smem_u32(&bars[i]), 0); };
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 2 * kTile);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    init_barriers<2>(bars);
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  int steps = 0;  // warp 1: products issued (even block), or to be issued (odd block)

  if (warp == 0) {
    if (lane == 0) {
      if constexpr (!Epi::kOwnInputs) griddep_wait();
      Ring r;
      int it = 0;  // steps so far, over all units
      for (int u = team; u < p.units && ok; u += teams) {
        const Unit w = unit_at(p, u);
        const int m = w.mt * kTile + rank * 128, n = w.nt * kTile + rank * 128;
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
          if (it >= kStages && !(ok = mbar_wait_hint(bar(kBarEmpty + r.s), r.parity ^ 1u, p.wait_ns)))
            break;
          if (rank == 0) mbar_arrive_expect_tx(bar(kBarFull + r.s), 2 * kStageBytes);
          const uint32_t to = lead_bar(kBarFull + r.s), da = s0 + r.s * kStageBytes;
          const uint32_t db = da + kOperandBytes;
          const int k = kb * kBK;
          auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
            tma_load_3d_pair(dst, map, to, c0, c1, 0);
          };
          if constexpr (A_MN) {
            load(da, &ma, m, k);
            load(da + 8192, &ma, m + 64, k);
          } else {
            load(da, &ma, k, m);
          }
          if constexpr (B_MN) {
            load(db, &mb, n, k);
            load(db + 8192, &mb, n + 64, k);
          } else {
            load(db, &mb, k, n);
          }
          r.next();
        }
      }
      // The copies in flight, before the block ends (the odd block's complete
      // on the even one's barriers; it leaves no earlier).
      bool landed = true;
      if (rank == 0)
        for (int k = it > kStages ? it - kStages : 0; k < it && landed; ++k)
          landed = mbar_wait_hint(bar(kBarFull + k % kStages), (k / kStages) & 1, p.wait_ns);
      if (!ok || !landed) atomicOr(&g_product_status, 1u);
    }
    __syncwarp();
  } else if (warp == 1 && rank != 0) {
    for (int u = team; u < p.units; u += teams) {
      const Unit w = unit_at(p, u);
      steps += w.kb1 - w.kb0;
    }
  } else if (warp == 1) {
    constexpr uint32_t kId = idesc(kTile, kTile, A_MN, B_MN, false);
    // K contiguous: 16 of K are 32 bytes of the swizzled row.  K along the rows:
    // 16 rows of 128 bytes, atoms of 64 columns 8 KB apart.
    constexpr uint32_t kStepA = A_MN ? 2048u : 32u, kStepB = B_MN ? 2048u : 32u;
    const uint64_t dA0 = sdesc_sw128(s0, A_MN ? 8192 : 16, 1024);
    const uint64_t dB0 = sdesc_sw128(s0 + kOperandBytes, B_MN ? 8192 : 16, 1024);
    Ring r;
    int n = 0;  // accumulators filled
    for (int u = team; u < p.units && ok; u += teams, ++n) {
      const Unit w = unit_at(p, u);
      const int acc = n & 1;
      if (n >= 2 &&
          !(ok = warp_all(mbar_wait_hint<true>(bar(kBarAccFree + acc), ((n >> 1) & 1) ^ 1, p.wait_ns))))
        break;
      tc_fence_after();
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (!(ok = warp_all(mbar_wait_hint(bar(kBarFull + r.s), r.parity, p.wait_ns)))) break;
        tc_fence_after();
        const uint64_t a = desc_add(dA0, r.s * kStageBytes), b = desc_add(dB0, r.s * kStageBytes);
        mma_ss_x4_pair(tmem + acc * kTile, a, desc_add(a, kStepA), desc_add(a, 2 * kStepA),
                       desc_add(a, 3 * kStepA), b, desc_add(b, kStepB), desc_add(b, 2 * kStepB),
                       desc_add(b, 3 * kStepB), kId, kb > w.kb0 ? 1u : 0u);
        mma_commit_pair(bar(kBarEmpty + r.s));
        r.next();
        ++steps;
      }
      if (ok) mma_commit_pair(bar(kBarAcc + acc));
    }
    mma_commit_pair(bar(kBarDrain));
  } else if (warp >= kFirstEpiWarp) {
    static_assert(Epi::kCols == kTile / 2, "half of the tile's columns");
    const int quarter = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
    const uint32_t tl = tmem + half * Epi::kCols + (static_cast<uint32_t>(quarter * 32) << 16);
    griddep_wait();
    auto part = [&](int u) {
      const Unit w = unit_at(p, u);
      return Epi(ea, w, w.mt * kTile + rank * 128 + quarter * 32 + lane, w.nt * kTile + half * Epi::kCols);
    };
    int n = 0;
    Epi next = part(team < p.units ? team : 0);
    for (int u = team; u < p.units; u += teams, ++n) {
      const int acc = n & 1;
      Epi e = next;
      e.prepare();
      if (u + teams < p.units) next = part(u + teams);
      if (!(ok = warp_all(mbar_wait_hint(bar(kBarAcc + acc), (n >> 1) & 1, p.wait_ns)))) break;
      tc_fence_after();
      e.take(tl + acc * kTile);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(lead_bar(kBarAccFree + acc));
    }
    if (!ok && lane == 0) atomicOr(&g_product_status, 1u);
  }
  tc_fence_before();
  __syncthreads();
  // A commit arrives in both blocks on its own time: each block waits for its
  // own copy of every commit that nobody here has waited for (the last round
  // of the ring, and the last commit of all) before the team leaves.
  if (warp == 1) {
    for (int k = steps > kStages ? steps - kStages : 0; k < steps && ok; ++k)
      ok = warp_all(mbar_wait_hint(bar(kBarEmpty + k % kStages), (k / kStages) & 1, p.wait_ns));
    if (!warp_all(mbar_wait_hint(bar(kBarDrain), 0, p.wait_ns)) || !ok) {
      if (lane == 0) atomicOr(&g_product_status, 1u);
    }
    __syncwarp();
  }
  cluster_sync();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_slot, 2 * kTile);
  }
}

// dependent: starts while the kernel before it on the stream still runs and
// waits for it before it reads or writes memory.
template <bool A_MN, bool B_MN, class Epi>
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const ProductPlan& p,
                   const typename Epi::Args& a, bool dependent, cudaStream_t st) {
  static unsigned long long attr_ctx[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = current_context_id();
  auto* kernel = product_kernel<A_MN, B_MN, Epi>;
  if (dev >= 64 || ctx == 0 || attr_ctx[dev] != ctx) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_ctx[dev] = ctx;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.teams));
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, p, a);
}

// Failure-detection self-test: the kernel's waits on a barrier that nothing
// arrives on.
static __global__ void wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_barrier_init();
  }
  __syncwarp();
  const bool own = warp_all(mbar_wait_hint(smem_u32(&bar), 0, limit_ns));
  const bool pair = warp_all(mbar_wait_hint<true>(smem_u32(&bar), 0, limit_ns));
  if (threadIdx.x == 0 && !own && !pair) atomicOr(&g_product_status, 1u);
}

// Read-and-clear of this translation unit's status word; synchronous on `st`.
static cudaError_t take_status(cudaStream_t st, unsigned* out) {
  unsigned val = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&val, g_product_status, sizeof(val), 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && val)
    e = cudaMemcpyToSymbolAsync(g_product_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  *out = val;
  return e;
}

}  // namespace product

// 32 bytes in one store: a whole sector of a row by one thread.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// COLS columns of TMEM, 32 at a time: f(c, v) with the next ones under way.
template <int COLS, class F>
__device__ __forceinline__ void each32(uint32_t taddr, F&& f) {
  uint32_t v[2][32];
  tmem_ld32_nowait(taddr, v[0]);
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    uint32_t(&now)[32] = v[c / 32 & 1];
    __syncwarp();
    tmem_wait_ld();
    reg_fence32(now);
    if (c + 32 < COLS) tmem_ld32_nowait(taddr + c + 32, v[c / 32 + 1 & 1]);
    f(c, now);
  }
}

// A small kernel after the products that waits for the kernel before it.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, bool dependent,
                             A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = static_cast<unsigned>(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace detattn
