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
// One persistent block per SM, 128 x 256 tiles, two accumulators in TMEM so
// that a tile's epilogue runs beside the next tile's products:
//   warp 0       TMA producer: int8 and dY tiles of 64 tokens, four stages
//   warp 1       tcgen05.mma issuer (M = 128, N = 256, K = 16 per instruction)
//   warps 2-5    epilogue: TMEM -> registers -> dw (or a partial tile)
//   warps 6-13   int8 -> bf16
// Tiles left over when all blocks have taken an equal number of whole ones
// are cut along the tokens, one range per block, and a second kernel adds the
// ranges in ascending order.  Every element's sum has one fixed order.
#include <cuda_runtime.h>

#include <cstdint>

#include "act8.cuh"
#include "block_launch.h"

namespace detattn {

__device__ unsigned int g_wgrad_status;

namespace {

constexpr int kStages = 4;
constexpr int kRawBytes = kWgradBK * kWgradBM;       // 8 KB
constexpr int kABytes = kWgradBK * kWgradBM * 2;     // 16 KB: two atoms of 64 columns
constexpr int kBBytes = kWgradBK * kWgradBN * 2;     // 32 KB: four atoms
constexpr int kStageBytes = kRawBytes + kABytes + kBBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kRawBytes % 1024 == 0 && kABytes % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
constexpr int kConvWarps = 8;
constexpr int kThreads = 32 * (6 + kConvWarps);

enum : int { kBarFull = 0, kBarConv = 4, kBarEmpty = 8, kBarAcc = 12, kBarAccFree = 14, kBarDrain = 16, kNumBars = 17 };

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

// Work of one block, in order: whole tiles blockIdx.x, + gridDim.x, ..., then
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
// Tiles run down the checkpoint's columns first: the blocks at work at one
// time share few column panels of dY.
__device__ __forceinline__ void tile_origin(const Act8WgradArgs& a, int tile, int* m0, int* n0) {
  *m0 = (tile % a.tiles_m) * kWgradBM;
  *n0 = (tile / a.tiles_m) * kWgradBN;
}

__global__ void __launch_bounds__(kThreads, 1)
    act8_wgrad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdy,
                      const Act8WgradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto sRaw = [&](int s) { return s0 + s * kStageBytes; };
  auto sA = [&](int s) { return s0 + s * kStageBytes + kRawBytes; };
  auto sB = [&](int s) { return s0 + s * kStageBytes + kRawBytes + kABytes; };
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarConv + s), kConvWarps);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarAcc + i), 1);
      mbar_init(bar(kBarAccFree + i), 4);
    }
    mbar_init(bar(kBarDrain), 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mdy);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int n_units = unit_count(a);
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;  // steps so far, over all units
      for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
        const Unit w = unit_at(a, u);
        int m0, n0;
        tile_origin(a, w.tile, &m0, &n0);
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (it >= kStages &&
              !(ok = mbar_wait(bar(kBarEmpty + s), ((it / kStages) & 1) ^ 1, a.wait_ns)))
            break;
          mbar_arrive_expect_tx(bar(kBarFull + s), kRawBytes + kBBytes);
          tma_load_2d(sRaw(s), &mq, bar(kBarFull + s), m0, kb * kWgradBK);
#pragma unroll
          for (int at = 0; at < kWgradBN / 64; ++at)
            tma_load_2d(sB(s) + at * 8192, &mdy, bar(kBarFull + s), n0 + 64 * at, kb * kWgradBK);
        }
      }
      // After a wait that ran out: the copies in flight, before the block ends.
      if (!ok)
        for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
          mbar_wait(bar(kBarFull + k % kStages), (k / kStages) & 1, a.wait_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t kId = idesc_bf16(kWgradBM, kWgradBN, true, true);
    // MN-major tiles: 16 tokens are 16 rows of 128 bytes; atoms lie 8 KB apart.
    const uint64_t dA0 = sdesc_sw128(sA(0), 8192, 1024);
    const uint64_t dB0 = sdesc_sw128(sB(0), 8192, 1024);
    int it = 0, n = 0;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x, ++n) {
      const Unit w = unit_at(a, u);
      const int acc = n & 1;
      if (n >= 2 &&
          !(ok = warp_all(mbar_wait(bar(kBarAccFree + acc), ((n >> 1) & 1) ^ 1, a.wait_ns))))
        break;
      tc_fence_after();
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const int s = it % kStages;
        if (!(ok = warp_all(mbar_wait(bar(kBarFull + s), (it / kStages) & 1, a.wait_ns)))) break;
        if (!(ok = warp_all(mbar_wait(bar(kBarConv + s), (it / kStages) & 1, a.wait_ns)))) break;
        tc_fence_after();
        const uint64_t da = desc_add(dA0, s * kStageBytes), db = desc_add(dB0, s * kStageBytes);
        mma_ss_x4(tmem + acc * kWgradBN, da, desc_add(da, 2048), desc_add(da, 4096),
                  desc_add(da, 6144), db, desc_add(db, 2048), desc_add(db, 4096),
                  desc_add(db, 6144), kId, kb > w.kb0 ? 1u : 0u);
        mma_commit(bar(kBarEmpty + s));
      }
      if (ok) mma_commit(bar(kBarAcc + acc));
    }
    mma_commit(bar(kBarDrain));
    warp_all(mbar_wait(bar(kBarDrain), 0, a.wait_ns));
  } else if (warp < 6) {
    // Epilogue: warp w reads TMEM lanes 32 (w & 3) .. + 31 (rows of dw), one
    // row per thread, 32 columns at a time.
    const int quarter = warp & 3;
    int n = 0;
    for (int u = blockIdx.x; u < n_units; u += gridDim.x, ++n) {
      const Unit w = unit_at(a, u);
      const int acc = n & 1;
      if (!(ok = warp_all(mbar_wait(bar(kBarAcc + acc), (n >> 1) & 1, a.wait_ns)))) break;
      tc_fence_after();
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      const int r = quarter * 32 + lane, row = m0 + r;
      const float scale = a.row_scale != nullptr && row < a.d ? a.row_scale[row] : 1.0f;
      const uint32_t tl = tmem + acc * kWgradBN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < kWgradBN / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tl + c * 32, v);
        if (w.part >= 0) {
          float4* dst = reinterpret_cast<float4*>(
              a.partial + (static_cast<size_t>(w.part) * kWgradBM + r) * kWgradBN + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                 __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        } else if (row < a.d) {
          float4* dst =
              reinterpret_cast<float4*>(a.dw + static_cast<size_t>(row) * a.n + n0 + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + c * 32 + 4 * i < a.n)
              dst[i] = make_float4(__uint_as_float(v[4 * i]) * scale, __uint_as_float(v[4 * i + 1]) * scale,
                                   __uint_as_float(v[4 * i + 2]) * scale,
                                   __uint_as_float(v[4 * i + 3]) * scale);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarAccFree + acc));
    }
  } else {
    // int8 -> bf16: thread (warp, lane) turns columns 8 j .. 8 j + 7, j =
    // lane % 16, of every 16th token row.  Half a warp reads one 128-byte
    // row, and eight lanes write one 128-byte row of an atom, the 16-byte
    // pieces exchanged as the swizzle wants: no bank conflicts either way.
    const int cw = warp - 6, j = lane & 15, r0 = cw * 2 + (lane >> 4);
    constexpr int kRows = kWgradBK / (2 * kConvWarps);  // rows per thread and step
    const int groups = a.d / kAct8Group;
    int it = 0;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit w = unit_at(a, u);
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      // Columns past the checkpoint's last group read as zero; any exponent
      // byte that exists will do for them, as for rows past the last.
      const int g = min(m0 / kAct8Group + (j >> 2), groups - 1);
      uint32_t e[kRows];
      auto load_e = [&](int kb) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = kb * kWgradBK + r0 + 2 * kConvWarps * i;
          e[i] = row < a.rows ? a.e[static_cast<size_t>(row) * groups + g] : 127u;
        }
      };
      load_e(w.kb0);
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const int s = it % kStages;
        uint32_t sc[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) sc[i] = e[i];
        if (kb + 1 < w.kb1) load_e(kb + 1);
        if (!(ok = warp_all(mbar_wait(bar(kBarFull + s), (it / kStages) & 1, a.wait_ns)))) break;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + 2 * kConvWarps * i;
          uint2 q;
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                       : "=r"(q.x), "=r"(q.y)
                       : "r"(sRaw(s) + r * 128 + j * 8)
                       : "memory");
          float f[8];
          act8_values8(q, act8_scale(sc[i]), f);
          st_shared_u4(sA(s) + (j >> 3) * 8192 + r * 128 + (((j & 7) ^ (r & 7)) << 4),
                       float_to_bf16x8(f));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarConv + s));
      }
    }
  }
  if (!ok) atomicOr(&g_wgrad_status, 1u);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The tiles that were cut along the tokens: their ranges added in ascending
// order, four columns per thread.
__global__ void __launch_bounds__(256) act8_wgrad_sum_kernel(const Act8WgradArgs a) {
  constexpr int kVecs = kWgradBM * kWgradBN / 4;
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
  p.whole_tiles = static_cast<int>(tiles / kWgradBlocks * kWgradBlocks);
  const int rem = static_cast<int>(tiles - p.whole_tiles);
  // The cut that leaves the busiest block the fewest steps, a range costing
  // about two steps of its own (writing the partial tile and adding it up).
  const int n_k = (rows + kWgradBK - 1) / kWgradBK;
  p.splits = 1;
  if (rem == 0) return p;
  double best = 0.0;
  for (int s = 1; s <= 32 && s <= n_k; ++s) {
    const int rounds = (rem * s + kWgradBlocks - 1) / kWgradBlocks;
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
    if (dev < 64) attr_ctx[dev] = current_context_id();
  }
  const int rem = a.tiles_m * a.tiles_n - a.whole_tiles;
  const int units = a.whole_tiles + rem * a.splits;
  act8_wgrad_kernel<<<units < kWgradBlocks ? units : kWgradBlocks, kThreads, kSmemBytes, st>>>(mq, mdy, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.splits == 1) return cudaSuccess;
  act8_wgrad_sum_kernel<<<rem * (kWgradBM * kWgradBN / 4 / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
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
