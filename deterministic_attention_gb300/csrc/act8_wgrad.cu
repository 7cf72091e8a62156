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
// the dY tile, twelve warps turn the int8 tile into the swizzled bf16 operand
// next to it, and one warp issues tcgen05.mma.  Tokens are the K dimension of
// both operands, which are read MN-major as they lie in memory.
//
// Shared memory decides the tile: for a step of 64 tokens a block alone on a
// 128 x 256 tile would move 112 KB (int8 in and out 16, bf16 in and out 32, dY
// in and out 64), 896 clocks at 128 bytes a clock for 512 clocks of MMA.  A
// pair of blocks (cta_group::2) on a 256 x 256 tile shares dY: 80 KB each, 640
// clocks.  So blocks work in pairs, one persistent block per SM:
//   warp 0       TMA producer of the int8 tiles (64 tokens each)
//   warp 1       (even block) tcgen05.mma issuer, M = N = 256, K = 16
//   warp 2       TMA producer of the dY tiles
//   warps 4-15   int8 -> bf16, three groups of four taking turns
//   warps 16-23  epilogue: accumulators -> fp32 sums in registers -> dw
// Measured at 8192 x 4096 x 6144: single blocks 437 us, pairs with eight
// converting warps and arithmetic through fp32 298 us, twelve warps and bytes
// to bf16 by masks 255 us with runs of 1024 tokens, 264 to 270 with runs of 512
// on a card that took 263 with the former: 1.53 to 1.56 PFLOP/s, 79 to 81 % of
// the measured bf16 peak.  Kept busy, a card slows under its power limit: passes
// one after another take up to 306 us (a library product in bf16 alone, 220 to
// 224).  The conversion is what it pays for: 208 us of that 255 without its
// stores, 232 without its arithmetic, 238 without its loads of the bytes.
// Shared memory is nearest to its limit: copies (24 KB a step and block),
// conversion (24 KB) and operands (at least 32 KB) take 640 cycles at 128 bytes
// a cycle of the 810 that a step has, and the arithmetic holds the ALU for 330.
// The rings are deep enough (six other splits of the same shared memory were
// within 2 %).
// Two accumulators in TMEM take turns: one is added to the tile's sum in
// registers after every 512 tokens while the other fills.
// Tiles left over when all pairs have taken an equal number of whole ones
// are cut along the tokens, one range per pair, and a second kernel adds the
// ranges in ascending order.  Every element's sum has one fixed order.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "act8.cuh"
#include "block_launch.h"

namespace detattn {

__device__ unsigned int g_wgrad_status;

namespace {

constexpr int kHalfM = kWgradBM / 2, kHalfN = kWgradBN / 2;
constexpr int kRawBytes = kWgradBK * kHalfM;         // 8 KB: int8
constexpr int kABytes = kWgradBK * kHalfM * 2;       // 16 KB: two atoms of 64 columns
constexpr int kBBytes = kWgradBK * kHalfN * 2;       // 16 KB: two atoms
constexpr int kRawStages = 8, kAStages = 4, kBStages = 6;
constexpr int kSmemBytes = kRawStages * kRawBytes + kAStages * kABytes + kBStages * kBBytes + 1024;
static_assert(kSmemBytes <= 226 * 1024, "shared memory");
static_assert(kRawBytes % 1024 == 0 && kABytes % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
constexpr int kCtrlWarps = 4, kConvWarps = 12, kEpiWarps = 8;
constexpr int kConvGroups = 3, kGroupWarps = kConvWarps / kConvGroups;
static_assert(2 * kGroupWarps == 8, "a group's row step keeps the swizzle");
constexpr int kThreads = 32 * (kCtrlWarps + kConvWarps + kEpiWarps);
// Registers per thread after reallocation: an epilogue thread holds 128 sums.
constexpr int kCtrlRegs = 48, kConvRegs = 48, kEpiRegs = 144;
constexpr int kRegBudget = 32 * (kCtrlWarps * kCtrlRegs + kConvWarps * kConvRegs + kEpiWarps * kEpiRegs);

enum : int {
  kBarRaw = 0,                          // int8 tile is here (each block's own)
  kBarRawFree = kBarRaw + kRawStages,   // it has been converted (each block's own)
  kBarB = kBarRawFree + kRawStages,     // both dY halves are there (the even block's)
  kBarBFree = kBarB + kBStages,         // their products are done (each block's)
  kBarA = kBarBFree + kBStages,         // both bf16 operands are written (the even block's)
  kBarAFree = kBarA + kAStages,         // their products are done (each block's)
  kBarAcc = kBarAFree + kAStages,       // an accumulator is complete (each block's)
  kBarAccFree = kBarAcc + 2,            // it has been read by both blocks (the even block's)
  kBarDrain = kBarAccFree + 2,
  kNumBars
};

// Position in a ring: stage and parity of the phase to wait for.
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ void gave_up() { atomicOr(&g_wgrad_status, 1u); }
// Four int8 bytes times a power of two (`scale`: its bf16 bits in both halves)
// as bf16, in the order 0, 2, 1, 3: masks then leave the bytes where they are.
// With m the low seven bits and s the sign bit, a value is (128 + m) - 128 (1 +
// s): both terms are bf16 numbers that take one LOP3 from the bytes (0x4300 |
// m and 0xC300 | s << 7), and every step is exact.  (Ten ALU instructions
// for eight values; through fp32 and its packing conversion it takes
// fourteen.)
// The masks are held in registers: an instruction takes one of them as an
// immediate, and the compiler otherwise makes two of each.
struct ByteMasks {
  uint32_t low = 0x007F007Fu, m = 0x43004300u, sign = 0x00800080u, c = 0xC300C300u;
  __device__ __forceinline__ ByteMasks() {
    asm volatile("" : "+r"(low), "+r"(m), "+r"(sign), "+r"(c));
  }
};
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of_bytes(uint32_t x, uint32_t scale, const ByteMasks& k) {
  const uint32_t m = and_or(x, k.low, k.m), c = and_or(x, k.sign, k.c);
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\t"
      "add.rn.bf16x2 t, %1, %2;\n\t"
      "mul.rn.bf16x2 %0, t, %3;\n\t}"
      : "=r"(r)
      : "r"(m), "r"(c), "r"(scale));
  return r;
}
// Where the column at position p of a tile lies in the checkpoint: the order
// above, i.e. the two low bits of p exchanged.
__device__ __forceinline__ int column_of(int p) { return (p & ~3) | ((p & 1) << 1) | ((p >> 1) & 1); }

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
    w.kb0 = n_k * z / a.splits;  // (n_k is at most 2^18, splits 32)
    w.kb1 = n_k * (z + 1) / a.splits;
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
  auto sRaw = [&](int s) { return s0 + s * kRawBytes; };
  const uint32_t sA0 = s0 + kRawStages * kRawBytes, sB0 = sA0 + kAStages * kABytes;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto lead_bar = [&](int i) { return map_shared_rank(smem_u32(&bars[i]), 0); };
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(bar(kBarRaw + s), 1);
      mbar_init(bar(kBarRawFree + s), kGroupWarps);
    }
    for (int s = 0; s < kBStages; ++s) {
      mbar_init(bar(kBarB + s), 1);
      mbar_init(bar(kBarBFree + s), 1);
    }
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(bar(kBarA + s), 2 * kGroupWarps);
      mbar_init(bar(kBarAFree + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarAcc + i), 1);
      mbar_init(bar(kBarAccFree + i), 2 * kEpiWarps);
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
  int steps = 0;  // warp 1: products issued (even block), or to be issued (odd block)

  if (warp < kCtrlWarps) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      // int8 tiles.
      if (lane == 0) {
        Ring r;
        int it = 0;  // steps so far, over all units
        for (int u = pair; u < n_units && ok; u += pairs) {
          const Unit w = unit_at(a, u);
          int m0, n0;
          tile_origin(a, w.tile, &m0, &n0);
          for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
            if (it >= kRawStages && !(ok = mbar_wait_hint(bar(kBarRawFree + r.s), r.parity ^ 1u, a.wait_ns)))
              break;
            mbar_arrive_expect_tx(bar(kBarRaw + r.s), kRawBytes);
            tma_load_2d(sRaw(r.s), &mq, bar(kBarRaw + r.s), m0 + rank * kHalfM, kb * kWgradBK);
            r.next(kRawStages);
          }
        }
        // The copies in flight, before the block ends.
        bool landed = true;
        for (int k = it > kRawStages ? it - kRawStages : 0; k < it && landed; ++k)
          landed = mbar_wait_hint(bar(kBarRaw + k % kRawStages), (k / kRawStages) & 1, a.wait_ns);
        if (!ok || !landed) gave_up();
      }
      __syncwarp();
    } else if (warp == 2) {
      // dY tiles: this block's half of the columns, on the even block's barrier.
      if (lane == 0) {
        Ring r;
        int it = 0;
        for (int u = pair; u < n_units && ok; u += pairs) {
          const Unit w = unit_at(a, u);
          int m0, n0;
          tile_origin(a, w.tile, &m0, &n0);
          n0 += rank * kHalfN;
          for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
            if (it >= kBStages && !(ok = mbar_wait_hint(bar(kBarBFree + r.s), r.parity ^ 1u, a.wait_ns)))
              break;
            if (rank == 0) mbar_arrive_expect_tx(bar(kBarB + r.s), 2 * kBBytes);
            const uint32_t to = lead_bar(kBarB + r.s), dst = sB0 + r.s * kBBytes;
            tma_load_2d_pair(dst, &mdy, to, n0, kb * kWgradBK);
            tma_load_2d_pair(dst + 8192, &mdy, to, n0 + 64, kb * kWgradBK);
            r.next(kBStages);
          }
        }
        // The copies in flight.  The odd block's complete here too; it leaves
        // no earlier than this block.
        bool landed = true;
        if (rank == 0)
          for (int k = it > kBStages ? it - kBStages : 0; k < it && landed; ++k)
            landed = mbar_wait_hint(bar(kBarB + k % kBStages), (k / kBStages) & 1, a.wait_ns);
        if (!ok || !landed) gave_up();
      }
      __syncwarp();
    } else if (warp == 1 && rank == 1) {
      steps = total_steps(a, pair, pairs);
    } else if (warp == 1) {
      constexpr uint32_t kId = idesc_bf16(kWgradBM, kWgradBN, true, true);
      // MN-major tiles: 16 tokens are 16 rows of 128 bytes; atoms lie 8 KB apart.
      const uint64_t dA0 = sdesc_sw128(sA0, 8192, 1024);
      const uint64_t dB0 = sdesc_sw128(sB0, 8192, 1024);
      Ring ra, rb;
      int n = 0;  // accumulators filled
      for (int u = pair; u < n_units && ok; u += pairs) {
        const Unit w = unit_at(a, u);
        for (int c = w.kb0; c < w.kb1 && ok; c += kWgradChunk, ++n) {
          const int acc = n & 1, end = min(c + kWgradChunk, w.kb1);
          if (n >= 2 &&
              !(ok = warp_all(mbar_wait_hint<true>(bar(kBarAccFree + acc), ((n >> 1) & 1) ^ 1, a.wait_ns))))
            break;
          tc_fence_after();
          for (int kb = c; kb < end; ++kb) {
            if (!(ok = warp_all(mbar_wait_hint(bar(kBarB + rb.s), rb.parity, a.wait_ns)))) break;
            if (!(ok = warp_all(mbar_wait_hint<true>(bar(kBarA + ra.s), ra.parity, a.wait_ns)))) break;
            tc_fence_after();
            const uint64_t da = desc_add(dA0, ra.s * kABytes), db = desc_add(dB0, rb.s * kBBytes);
            mma_ss_x4_pair(tmem + acc * kWgradBN, da, desc_add(da, 2048), desc_add(da, 4096),
                           desc_add(da, 6144), db, desc_add(db, 2048), desc_add(db, 4096),
                           desc_add(db, 6144), kId, kb > c ? 1u : 0u);
            mma_commit_pair(bar(kBarAFree + ra.s));
            mma_commit_pair(bar(kBarBFree + rb.s));
            ra.next(kAStages);
            rb.next(kBStages);
            ++steps;
          }
          if (ok) mma_commit_pair(bar(kBarAcc + acc));
        }
      }
      mma_commit_pair(bar(kBarDrain));
    }
  } else if (warp < kCtrlWarps + kConvWarps) {
    // int8 -> bf16: thread (warp, lane) turns columns 8 j .. 8 j + 7, j =
    // lane % 16, of every eighth token row.  Half a warp reads one 128-byte
    // row, and eight lanes write one 128-byte row of an atom, the 16-byte
    // pieces exchanged as the swizzle wants: no bank conflicts either way.
    // The groups take steps in turn, so that one group's waits and fences run
    // beside the others' arithmetic.
    setmaxnreg_dec<kConvRegs>();
    const int cw = warp - kCtrlWarps, group = cw / kGroupWarps, j = lane & 15;
    const int r0 = (cw % kGroupWarps) * 2 + (lane >> 4);
    constexpr int kRowStep = 2 * kGroupWarps, kRows = kWgradBK / kRowStep;  // eight rows per thread
    const uint32_t groups = a.d / kAct8Group;
    // The exponents' cursor: the step whose bytes are fetched next, which is
    // the group's own next one (three steps before it is turned).
    int fu = pair, fkb = 0, fend = 0;
    const uint8_t* fat = a.e;
    auto open = [&]() {
      if (fu >= n_units) {  // past the last: what is fetched is not used
        fkb = 0;
        fend = INT_MAX;
        return;
      }
      const Unit w = unit_at(a, fu);
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      // Columns past the checkpoint's last group read as zero; any exponent
      // byte that exists will do for them, as for rows past the last.
      fat = a.e + min(static_cast<uint32_t>((m0 + rank * kHalfM) / kAct8Group + (j >> 2)), groups - 1);
      fkb = w.kb0;
      fend = w.kb1;
    };
    auto skip = [&](int n) {
      fkb += n;
      while (fkb >= fend) {
        const int over = fkb - fend;
        fu += pairs;
        open();
        fkb += over;
      }
    };
    // Volatile: the loads are issued here and waited for where the bytes are
    // used.
    auto fetch = [&](uint32_t (&e)[kRows]) {
      const int row = fkb * kWgradBK + r0;
      if (fkb * kWgradBK + kWgradBK <= a.rows) {
        const uint8_t* p = fat + static_cast<size_t>(row) * groups;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(e[i]) : "l"(p + i * kRowStep * groups));
      } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          asm volatile("ld.global.nc.u8 %0, [%1];"
                       : "=r"(e[i])
                       : "l"(fat + static_cast<size_t>(min(row + kRowStep * i, a.rows - 1)) * groups));
      }
      skip(kConvGroups);
    };
    open();
    if (group > 0) skip(group);
    uint32_t e[kRows];
    fetch(e);
    const ByteMasks masks;
    const int total = total_steps(a, pair, pairs);
    Ring rr, ra;
    for (int i = 0; i < group; ++i) {
      rr.next(kRawStages);
      ra.next(kAStages);
    }
    for (int it = group; it < total && ok; it += kConvGroups) {
      ok = warp_all(mbar_wait_hint(bar(kBarRaw + rr.s), rr.parity, a.wait_ns));
      if (ok && it >= kAStages)
        ok = warp_all(mbar_wait_hint(bar(kBarAFree + ra.s), ra.parity ^ 1u, a.wait_ns));
      const uint32_t raw = sRaw(rr.s) + r0 * 128 + j * 8;
      const uint32_t out = sA0 + ra.s * kABytes + (j >> 3) * 8192 + r0 * 128 + (((j & 7) ^ r0) << 4);
      // Eight rows down, the swizzle (row % 8) is the same.
#pragma unroll
      for (int i0 = 0; i0 < kRows; i0 += 4) {
        uint2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                       : "=r"(q[i].x), "=r"(q[i].y)
                       : "r"(raw + kRowStep * (i0 + i) * 128));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // 2^(e - 127), twice.  (Volatile: formed here, not where the byte
          // is loaded, or the load would be waited for there.)
          uint32_t sc;
          asm volatile("mul.lo.u32 %0, %1, 0x00800080;" : "=r"(sc) : "r"(e[i0 + i]));
          st_shared_u4(out + kRowStep * (i0 + i) * 128,
                       make_uint4(bf16x2_of_bytes(q[i].x, sc, masks), bf16x2_of_bytes(q[i].x >> 8, sc, masks),
                                  bf16x2_of_bytes(q[i].y, sc, masks), bf16x2_of_bytes(q[i].y >> 8, sc, masks)));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && ok) {
        mbar_arrive(bar(kBarRawFree + rr.s));
        mbar_arrive_pair(lead_bar(kBarA + ra.s));
      }
      fetch(e);
#pragma unroll
      for (int k = 0; k < kConvGroups; ++k) {
        rr.next(kRawStages);
        ra.next(kAStages);
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
        if (!(ok = warp_all(mbar_wait_hint(bar(kBarAcc + acc), (n >> 1) & 1, a.wait_ns)))) break;
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
        if (lane == 0) mbar_arrive_pair(lead_bar(kBarAccFree + acc));
      }
      if (!ok) {
        gave_up();
        break;
      }
      const Unit w = unit_at(a, u);
      int m0, n0;
      tile_origin(a, w.tile, &m0, &n0);
      const bool part = w.part >= 0;
      const int r0 = static_cast<int>(cluster_ctarank()) * kHalfM + (warp & 3) * 32 + column_of(lane >> 2);
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
  // A commit arrives in both blocks on its own time: neither a barrier of the
  // threads nor the other block's copy of it orders that arrival.  So each
  // block waits for its own copy of every commit that nobody here has waited
  // for: the last round of both rings (the converting warps and the dY producer
  // have seen all earlier ones, so the parities are not ambiguous), and the
  // last commit of all.  (The epilogue has seen the accumulators'.)
  if (warp == 1) {
    for (int k = steps > kAStages ? steps - kAStages : 0; k < steps && ok; ++k)
      ok = warp_all(mbar_wait_hint(bar(kBarAFree + k % kAStages), (k / kAStages) & 1, a.wait_ns));
    for (int k = steps > kBStages ? steps - kBStages : 0; k < steps && ok; ++k)
      ok = warp_all(mbar_wait_hint(bar(kBarBFree + k % kBStages), (k / kBStages) & 1, a.wait_ns));
    if (!warp_all(mbar_wait_hint(bar(kBarDrain), 0, a.wait_ns)) || !ok) gave_up();
    __syncwarp();
  }
  // Then neither leaves before the other: the even block's products read the
  // odd one's shared memory, and the odd one's copies and arrivals go to the
  // even one's barriers.
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

// Failure-detection self-test: this kernel's two waits on a barrier that
// nothing arrives on.
__global__ void wgrad_wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_barrier_init();
  }
  __syncwarp();
  const bool own = warp_all(mbar_wait_hint(smem_u32(&bar), 0, limit_ns));
  const bool pair = warp_all(mbar_wait_hint<true>(smem_u32(&bar), 0, limit_ns));
  if (threadIdx.x == 0 && !own && !pair) gave_up();
}

}  // namespace

cudaError_t launch_wgrad_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  wgrad_wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

Act8WgradPlan act8_wgrad_plan(int rows, int d, int n) {
  Act8WgradPlan p{};
  p.tiles_m = (d + kWgradBM - 1) / kWgradBM;
  p.tiles_n = (n + kWgradBN - 1) / kWgradBN;
  const long tiles = static_cast<long>(p.tiles_m) * p.tiles_n;
  p.whole_tiles = static_cast<int>(tiles / kWgradPairs * kWgradPairs);
  const int rem = static_cast<int>(tiles - p.whole_tiles);
  // The cut that leaves the busiest pair the fewest steps.  Cutting at all
  // costs about twelve (the partial tiles written and added up, a second
  // launch): 1000 x 768 x 1280 takes 17.5 us a call cut in five and 16.4
  // whole, 500 rows 17.0 and 12.7; 1777 x 1184 x 1000 17.1 cut in three and
  // 20.5 whole.
  const int n_k = (rows + kWgradBK - 1) / kWgradBK;
  p.splits = 1;
  if (rem == 0) return p;
  double best = 0.0;
  for (int s = 1; s <= 32 && s <= n_k; ++s) {
    const int rounds = (rem * s + kWgradPairs - 1) / kWgradPairs;
    const double cost = rounds * (static_cast<double>((n_k + s - 1) / s) + (s > 1 ? 12.0 : 0.0));
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
