// Weight gradient from an 8-bit checkpoint, for sm_103a:
//
//   dw[m, n] = row_scale[m] * sum_t X[t, m] dY[t, n],   X[t, m] = q[t, m] 2^(e[t, m / 32] - 127)
//
// (RustingBrain vs PyTorch/TensorFlow page, "Where the time goes now": GEMMs
// are most of a step.)  X is the layer input that the forward kept; where the
// forward kept the normed input before its weight, row_scale is that weight.
//
// Every checkpointed value is a bf16 number, so the product runs on the bf16
// tensor cores with no further rounding of X: TMA brings the int8 tile and
// the dY tile, eight warps turn the int8 tile into the swizzled bf16 operand
// next to it, and one warp issues tcgen05.mma.  Tokens are the K dimension of
// both operands, which are read MN-major as they lie in memory.
//
// What bounds it is shared memory: for a step of 64 tokens a block alone on a
// 128 x 256 tile would move 112 KB (int8 in and out 16, bf16 in and out 32,
// dY in and out 64), 875 clocks at 128 bytes a clock for 512 clocks of MMA.  A
// pair of blocks (cta_group::2) on a 256 x 256 tile shares dY: 80 KB each, 625
// clocks.  So blocks work in pairs, one persistent block per SM:
//   warp 0       TMA producer: int8 and dY tiles of 64 tokens, five stages
//   warp 1       (even block) tcgen05.mma issuer, M = 256, N = 256, K = 16
//   warps 2, 3   (odd block) tell the issuer what that block has ready
//   warps 4-11   int8 -> bf16
//   warps 12-19  epilogue: accumulators -> fp32 sums in registers -> dw
// Two accumulators in TMEM take turns: one is added to the tile's sum in
// registers after every 1024 tokens while the other fills.
// Tiles left over when all pairs have taken an equal number of whole ones
// are cut along the tokens, one range per pair, and a second kernel adds the
// ranges in ascending order.  Every element's sum has one fixed order.
#include <cuda_runtime.h>

#include <cstdint>

#include "act8.cuh"
#include "block_launch.h"

namespace detattn {

__device__ unsigned int g_wgrad_status;

namespace {

constexpr int kStages = 5;
constexpr int kHalfM = kWgradBM / 2, kHalfN = kWgradBN / 2;
constexpr int kRawBytes = kWgradBK * kHalfM;         // 8 KB
constexpr int kABytes = kWgradBK * kHalfM * 2;       // 16 KB: two atoms of 64 columns
constexpr int kBBytes = kWgradBK * kHalfN * 2;       // 16 KB: two atoms
constexpr int kStageBytes = kRawBytes + kABytes + kBBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
static_assert(kSmemBytes <= 226 * 1024, "shared memory");
static_assert(kRawBytes % 1024 == 0 && kABytes % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
constexpr int kCtrlWarps = 4, kConvWarps = 8, kEpiWarps = 8;
constexpr int kThreads = 32 * (kCtrlWarps + kConvWarps + kEpiWarps);
// Registers per thread after reallocation: an epilogue thread holds 128 sums.
constexpr int kCtrlRegs = 48, kConvRegs = 64, kEpiRegs = 152;
constexpr int kRegBudget = 32 * (kCtrlWarps * kCtrlRegs + kConvWarps * kConvRegs + kEpiWarps * kEpiRegs);

enum : int {
  kBarRaw = 0,               // int8 tile here (each block's own)
  kBarB = kStages,           // both dY halves (the even block's)
  kBarConv = 2 * kStages,    // bf16 operand written here (each block's own)
  kBarPeer = 3 * kStages,    // ... and in the odd block (the even block's)
  kBarEmpty = 4 * kStages,   // the stage's products are done (each block's)
  kBarAcc = 5 * kStages,     // an accumulator is complete (each block's)
  kBarAccFree = kBarAcc + 2, // it has been read here (each block's own)
  kBarPeerFree = kBarAcc + 4,  // ... and in the odd block (the even block's)
  kBarDrain = kBarAcc + 6,
  kNumBars = kBarAcc + 7
};

__device__ __forceinline__ void gave_up() { atomicOr(&g_wgrad_status, 1u); }
__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

// Work of one pair, in order: whole tiles pair, pair + pairs, ..., then
// token ranges of the remaining tiles.
struct Unit {
  int tile, kb0, kb1;  // token steps [kb0, kb1)
  int part;            // partial slot, -1: a whole tile
};
__device__ __forceinline__ int unit_count(const Act8WgradArgs& a) {
  return a.whole_tiles + (a.tiles_m * a.tiles_n - a.whole_tiles) * a.splits;
}
__device__ __forceinline__ Unit unit_at(const Act8WgradArgs& a, int u) {
  const int n_k = (a.rows + kWgradBK - 1) / kWgradBK;
  Unit w;
  if (u < a.whole_tiles) {
    w = {u, 0, n_k, -1};
  } else {
    const int r = u - a.whole_tiles, z = r % a.splits;
    w.tile = a.whole_tiles + r / a.splits;
    w.kb0 = static_cast<int>(static_cast<long>(n_k) * z / a.splits);
    w.kb1 = static_cast<int>(static_cast<long>(n_k) * (z + 1) / a.splits);
    w.part = a.splits > 1 ? r : -1;
  }
  return w;
}
__device__ __forceinline__ int unit_chunks(const Act8WgradArgs& a, int u) {
  const Unit w = unit_at(a, u);
  return (w.kb1 - w.kb0 + kWgradChunk - 1) / kWgradChunk;
}
// Steps of all units of a pair.
__device__ __forceinline__ int total_steps(const Act8WgradArgs& a, int pair, int pairs) {
  int total = 0;
  for (int u = pair; u < unit_count(a); u += pairs) {
    const Unit w = unit_at(a, u);
    total += w.kb1 - w.kb0;
  }
  return total;
}
// Tiles run down the checkpoint's columns first: the pairs at work at one
// time share few column panels of dY.
__device__ __forceinline__ void tile_origin(const Act8WgradArgs& a, int tile, int* m0, int* n0) {
  *m0 = (tile % a.tiles_m) * kWgradBM;
  *n0 = (tile / a.tiles_m) * kWgradBN;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    act8_wgrad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdy,
                      const Act8WgradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  // The same offsets in both blocks (the products read both at one address).
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto sRaw = [&](int s) { return s0 + s * kStageBytes; };
  auto sA = [&](int s) { return s0 + s * kStageBytes + kRawBytes; };
  auto sB = [&](int s) { return s0 + s * kStageBytes + kRawBytes + kABytes; };
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto lead_bar = [&](int i) { return map_shared_rank(smem_u32(&bars[i]), 0); };
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarRaw + s), 1);
      mbar_init(bar(kBarB + s), 1);
      mbar_init(bar(kBarConv + s), kConvWarps);
      mbar_init(bar(kBarPeer + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarAcc + i), 1);
      mbar_init(bar(kBarAccFree + i), kEpiWarps);
      mbar_init(bar(kBarPeerFree + i), 1);
    }
    mbar_init(bar(kBarDrain), 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mdy);
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const int n_units = unit_count(a);
  bool ok = true;

  if (warp < kCtrlWarps) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      if (lane == 0) {
        int s = 0, it = 0;  // stage; steps so far, over all units
        uint32_t parity = 1;
        for (int u = pair; u < n_units && ok; u += pairs) {
          const Unit w = unit_at(a, u);
          int m0, n0;
          tile_origin(a, w.tile, &m0, &n0);
          m0 += rank * kHalfM;
          n0 += rank * kHalfN;
          for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
            if (it >= kStages && !(ok = mbar_wait(bar(kBarEmpty + s), parity, a.wait_ns))) break;
            mbar_arrive_expect_tx(bar(kBarRaw + s), kRawBytes);
            tma_load_2d(sRaw(s), &mq, bar(kBarRaw + s), m0, kb * kWgradBK);
            if (rank == 0) mbar_arrive_expect_tx(bar(kBarB + s), 2 * kBBytes);
            const uint32_t to = lead_bar(kBarB + s);
            tma_load_2d_pair(sB(s), &mdy, to, n0, kb * kWgradBK);
            tma_load_2d_pair(sB(s) + 8192, &mdy, to, n0 + 64, kb * kWgradBK);
            if (++s == kStages) {
              s = 0;
              parity ^= 1u;
            }
          }
        }
        // After a wait that ran out: the copies in flight, before the block ends.
        if (!ok)
          for (int k = it > kStages ? it - kStages : 0; k < it; ++k) {
            mbar_wait(bar(kBarRaw + k % kStages), (k / kStages) & 1, a.wait_ns);
            if (rank == 0) mbar_wait(bar(kBarB + k % kStages), (k / kStages) & 1, a.wait_ns);
          }
      }
      if (!ok) gave_up();
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      constexpr uint32_t kId = idesc_bf16(kWgradBM, kWgradBN, true, true);
      // MN-major tiles: 16 tokens are 16 rows of 128 bytes; atoms lie 8 KB apart.
      const uint64_t dA0 = sdesc_sw128(sA(0), 8192, 1024);
      const uint64_t dB0 = sdesc_sw128(sB(0), 8192, 1024);
      int s = 0, n = 0;  // n: accumulators filled
      uint32_t parity = 0;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const Unit w = unit_at(a, u);
        for (int c = w.kb0; c < w.kb1 && ok; c += kWgradChunk, ++n) {
          const int acc = n & 1, end = min(c + kWgradChunk, w.kb1);
          if (n >= 2) {
            const uint32_t p = ((n >> 1) & 1) ^ 1;
            if (!(ok = warp_all(mbar_wait(bar(kBarAccFree + acc), p, a.wait_ns)))) break;
            if (!(ok = warp_all(mbar_wait_cluster(bar(kBarPeerFree + acc), p, a.wait_ns)))) break;
          }
          tc_fence_after();
          for (int kb = c; kb < end; ++kb) {
            if (!(ok = warp_all(mbar_wait(bar(kBarB + s), parity, a.wait_ns)))) break;
            if (!(ok = warp_all(mbar_wait(bar(kBarConv + s), parity, a.wait_ns)))) break;
            if (!(ok = warp_all(mbar_wait_cluster(bar(kBarPeer + s), parity, a.wait_ns)))) break;
            tc_fence_after();
            const uint64_t da = desc_add(dA0, s * kStageBytes), db = desc_add(dB0, s * kStageBytes);
            mma_ss_x4_pair(tmem + acc * kWgradBN, da, desc_add(da, 2048), desc_add(da, 4096),
                           desc_add(da, 6144), db, desc_add(db, 2048), desc_add(db, 4096),
                           desc_add(db, 6144), kId, kb > c ? 1u : 0u);
            mma_commit_pair(bar(kBarEmpty + s));
            if (++s == kStages) {
              s = 0;
              parity ^= 1u;
            }
          }
          if (ok) mma_commit_pair(bar(kBarAcc + acc));
        }
      }
      mma_commit_pair(bar(kBarDrain));
      if (!warp_all(mbar_wait(bar(kBarDrain), 0, a.wait_ns)) || !ok) gave_up();
    } else if (warp == 2 && rank == 1) {
      // The odd block's operands, passed on to the issuer.  (One thread with
      // no loads or stores of its own in flight does it: an arrival that
      // releases to the cluster waits for all that its thread has begun, and
      // the converting warps always have exponent loads under way.  With
      // their own arrivals there a step took 2500 clocks.)
      if (lane == 0) {
        const int total = total_steps(a, pair, pairs);
        const uint32_t to = lead_bar(kBarPeer);
        int s = 0;
        uint32_t parity = 0;
        for (int it = 0; it < total; ++it) {
          if (!(ok = mbar_wait(bar(kBarConv + s), parity, a.wait_ns))) break;
          mbar_arrive_remote(to + 8 * s);
          if (++s == kStages) {
            s = 0;
            parity ^= 1u;
          }
        }
        if (!ok) gave_up();
      }
      __syncwarp();
    } else if (warp == 3 && rank == 1) {
      // Its accumulators read, likewise.
      if (lane == 0) {
        const uint32_t to = lead_bar(kBarPeerFree);
        int n = 0;
        for (int u = pair; u < n_units && ok; u += pairs)
          for (int chunks = unit_chunks(a, u); chunks > 0; --chunks, ++n) {
            if (!(ok = mbar_wait(bar(kBarAccFree + (n & 1)), (n >> 1) & 1, a.wait_ns))) break;
            mbar_arrive_remote(to + 8 * (n & 1));
          }
        if (!ok) gave_up();
      }
      __syncwarp();
    }
  } else if (warp < kCtrlWarps + kConvWarps) {
    // int8 -> bf16: thread (warp, lane) turns columns 8 j .. 8 j + 7, j =
    // lane % 16, of every 16th token row.  Half a warp reads one 128-byte
    // row, and eight lanes write one 128-byte row of an atom, the 16-byte
    // pieces exchanged as the swizzle wants: no bank conflicts either way.
    setmaxnreg_dec<kConvRegs>();
    const int cw = warp - kCtrlWarps, j = lane & 15, r0 = cw * 2 + (lane >> 4);
    constexpr int kRows = kWgradBK / (2 * kConvWarps);  // rows per thread and step
    constexpr int kAhead = 4;                           // steps that exponents are fetched ahead
    const int groups = a.d / kAct8Group;
    // The exponents' cursor: the step whose bytes are fetched next.
    int fu = pair, fkb = 0, fend = 0;
    const uint8_t* fat = a.e;
    auto open = [&]() {
      if (fu >= n_units) return;
      const Unit w = unit_at(a, fu);
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      // Columns past the checkpoint's last group read as zero; any exponent
      // byte that exists will do for them, as for rows past the last.
      fat = a.e + min((m0 + rank * kHalfM) / kAct8Group + (j >> 2), groups - 1);
      fkb = w.kb0;
      fend = w.kb1;
    };
    open();
    auto fetch = [&](uint32_t (&e)[kRows]) {
      if (fu >= n_units) return;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = fkb * kWgradBK + r0 + 2 * kConvWarps * i;
        e[i] = fat[static_cast<size_t>(min(row, a.rows - 1)) * groups];
      }
      if (++fkb == fend) {
        fu += pairs;
        open();
      }
    };
    uint32_t e[kAhead][kRows];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(e[i]);
    const int total = total_steps(a, pair, pairs);
    int s = 0;
    uint32_t parity = 0;
    for (int it = 0; it < total && ok; it += kAhead) {
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        if (it + h < total && ok) {
          ok = warp_all(mbar_wait(bar(kBarRaw + s), parity, a.wait_ns));
          uint2 q[kRows];
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(q[i].x), "=r"(q[i].y)
                         : "r"(sRaw(s) + (r0 + 2 * kConvWarps * i) * 128 + j * 8)
                         : "memory");
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int r = r0 + 2 * kConvWarps * i;
            Vec8 v;
            v.from_int8(q[i]);
            const uint64_t sc = f2_all(act8_scale(e[h][i]));
#pragma unroll
            for (int k = 0; k < 4; ++k) v.p[k] = f2_mul(v.p[k], sc);
            st_shared_u4(sA(s) + (j >> 3) * 8192 + r * 128 + (((j & 7) ^ (r & 7)) << 4), v.to_bf16());
          }
          fetch(e[h]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(bar(kBarConv + s));
          if (++s == kStages) {
            s = 0;
            parity ^= 1u;
          }
        }
      }
    }
    if (!ok) gave_up();
  } else {
    // Epilogue: warp w takes rows (w & 3) 32 .. + 31 of its block's half and
    // 128 of the 256 columns, in the fragment layout: a thread has two
    // neighbouring columns of four rows of every eight columns, so that a
    // store of the warp writes whole 32-byte sectors of eight rows.  (What the
    // loop needs besides the sums is formed again where it is used: registers
    // are for the sums.)
    setmaxnreg_inc<kEpiRegs>();
    const int half = (warp - kCtrlWarps - kConvWarps) >> 2;
    const uint32_t tl = tmem + half * kHalfN + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int n = 0;
    for (int u = blockIdx.x >> 1; u < unit_count(a) && ok; u += gridDim.x >> 1) {
      uint64_t sum[2][kHalfN / 16][4];  // [16 rows][16 columns][pairs]
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < kHalfN / 16; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[h][g][i] = 0;
      for (int chunks = unit_chunks(a, u); chunks > 0; --chunks, ++n) {
        const int acc = n & 1;
        if (!(ok = warp_all(mbar_wait(bar(kBarAcc + acc), (n >> 1) & 1, a.wait_ns)))) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < kHalfN / 16; ++g) {
            uint32_t v[8];
            tmem_ld_16x256b_x2_nowait(tl + (static_cast<uint32_t>(16 * h) << 16) + acc * kWgradBN + g * 16, v);
            tmem_wait_ld();
            reg_fence8(v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sum[h][g][i] =
                  f2_add(sum[h][g][i], f2_make(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarAccFree + acc));
      }
      if (!ok) {
        gave_up();
        break;
      }
      const Unit w = unit_at(a, u);
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      const bool part = w.part >= 0;
      const int r0 = static_cast<int>(cluster_ctarank()) * kHalfM + (warp & 3) * 32 + (lane >> 2);
      const int c0 = half * kHalfN + 2 * (lane & 3);
      const int left = part ? kWgradBN : a.n - n0;  // columns to write
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = r0 + 16 * h + 8 * k;
          if (!part && m0 + r >= a.d) continue;
          float* dst = part ? a.partial + (static_cast<size_t>(w.part) * kWgradBM + r) * kWgradBN + c0
                            : a.dw + static_cast<size_t>(m0 + r) * a.n + n0 + c0;
          const uint64_t scale = f2_all(part || a.row_scale == nullptr ? 1.0f : a.row_scale[m0 + r]);
#pragma unroll
          for (int g = 0; g < kHalfN / 16; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (half * kHalfN + g * 16 + 8 * i < left)
                *reinterpret_cast<uint64_t*>(dst + g * 16 + 8 * i) = f2_mul(sum[h][g][2 * i + k], scale);
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  // Neither block leaves while the other's products, copies or arrivals may
  // still reach it.
  cluster_sync();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_slot, 512);
  }
}

// The tiles that were cut along the tokens: their ranges added in ascending
// order, four columns per thread.
__global__ void __launch_bounds__(256) act8_wgrad_sum_kernel(const Act8WgradArgs a) {
  constexpr int kVecs = kWgradBM * kWgradBN / 4;
  griddep_wait();
  const int idx = blockIdx.x * 256 + threadIdx.x;
  const int rem = idx / kVecs, at = idx % kVecs;
  int m0, n0;
  tile_origin(a, a.whole_tiles + rem, &m0, &n0);
  const int r = at / (kWgradBN / 4), c = (at % (kWgradBN / 4)) * 4;
  if (m0 + r >= a.d || n0 + c >= a.n) return;
  const float4* p = reinterpret_cast<const float4*>(a.partial) +
                    static_cast<size_t>(rem) * a.splits * kVecs + at;
  float4 s = p[0];
#pragma unroll 4
  for (int z = 1; z < a.splits; ++z) {
    const float4 x = p[static_cast<size_t>(z) * kVecs];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  const float k = a.row_scale != nullptr ? a.row_scale[m0 + r] : 1.0f;
  *reinterpret_cast<float4*>(a.dw + static_cast<size_t>(m0 + r) * a.n + n0 + c) =
      make_float4(s.x * k, s.y * k, s.z * k, s.w * k);
}

}  // namespace

Act8WgradPlan act8_wgrad_plan(int rows, int d, int n) {
  Act8WgradPlan p{};
  p.tiles_m = (d + kWgradBM - 1) / kWgradBM;
  p.tiles_n = (n + kWgradBN - 1) / kWgradBN;
  const long tiles = static_cast<long>(p.tiles_m) * p.tiles_n;
  p.whole_tiles = static_cast<int>(tiles / kWgradPairs * kWgradPairs);
  const int rem = static_cast<int>(tiles - p.whole_tiles);
  // The cut that leaves the busiest pair the fewest steps, a range costing
  // about two steps of its own (writing the partial tile and adding it up).
  const int n_k = (rows + kWgradBK - 1) / kWgradBK;
  p.splits = 1;
  if (rem == 0) return p;
  double best = 0.0;
  for (int s = 1; s <= 32 && s <= n_k; ++s) {
    const int rounds = (rem * s + kWgradPairs - 1) / kWgradPairs;
    const double cost = rounds * (static_cast<double>((n_k + s - 1) / s) + (s > 1 ? 4.0 : 0.0));
    if (s == 1 || cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  return p;
}

cudaError_t launch_act8_wgrad(const CUtensorMap& mq, const CUtensorMap& mdy,
                              const Act8WgradArgs& a, cudaStream_t st) {
  static unsigned long long attr_ctx[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = current_context_id();
  if (dev >= 64 || ctx == 0 || attr_ctx[dev] != ctx) {
    e = cudaFuncSetAttribute(act8_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    // The registers at launch must cover the warpgroups' counts after
    // reallocation, or the epilogue's increase never completes: refuse to
    // launch rather than start such a kernel.
    cudaFuncAttributes fa{};
    if ((e = cudaFuncGetAttributes(&fa, act8_wgrad_kernel)) != cudaSuccess) return e;
    if (fa.numRegs * kThreads < kRegBudget) return cudaErrorInvalidConfiguration;
    if (dev < 64) attr_ctx[dev] = current_context_id();
  }
  const int rem = a.tiles_m * a.tiles_n - a.whole_tiles;
  const int units = a.whole_tiles + rem * a.splits;
  const int pairs = units < kWgradPairs ? units : kWgradPairs;
  act8_wgrad_kernel<<<2 * pairs, kThreads, kSmemBytes, st>>>(mq, mdy, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.splits == 1) return cudaSuccess;
  // A programmatic dependent: launched while the products run, it waits for
  // them before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rem * (kWgradBM * kWgradBN / 4 / 256)));
  cfg.blockDim = 256;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, act8_wgrad_sum_kernel, a);
}

cudaError_t take_wgrad_status(cudaStream_t st, unsigned* out) {
  unsigned val = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&val, g_wgrad_status, sizeof(val), 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && val)
    e = cudaMemcpyToSymbolAsync(g_wgrad_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  *out = val;
  return e;
}

}  // namespace detattn
