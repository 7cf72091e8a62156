// Norms before and after a block, fused with the block's gate, its scale and
// the residual stream, for sm_103a (RustingBrain vs PyTorch/TensorFlow page,
// "The setup": a decoder-only model with RMSNorm; "What didn't work": folding
// the residual add into the norm).
//
// Forward, per row of width d (r, s: residual and block scale, g the gate or
// its sigmoid; every norm is x / sqrt(mean x^2 + eps)):
//   yhat = y rstd_y,  x' = r x + s g (yhat w_post),  xhat = x' rstd_x,  h = xhat w_pre
// Backward, from dx' and dh:
//   D  = dx' + rstd_x (dh w_pre - xhat mean(dh w_pre xhat)),   dx = r D
//   dz = s g D,  dg = s (yhat w_post) D  (through the sigmoid: times g (1 - g))
//   dy = rstd_y (dz w_post - yhat mean(dz w_post yhat))
//   dw_pre = sum_rows dh xhat,  dw_post = sum_rows dz yhat,  dgate = sum of dg
//            over the rows that share a gate row
// xhat and yhat come from the stored tensors or from 8-bit checkpoints that
// the forward wrote while it had them in registers.
//
// Everything is 32-bit between the loads and the one rounding at each store.
// Column sums have a fixed order and no atomics: a row team's threads own
// fixed columns and add their rows in ascending order in registers, the teams
// of a block are added in team order, and a second kernel adds the blocks in
// block order.  The deal of rows follows from the shape alone.
//
// Both move each tensor once and should be bound by memory.  The forward is:
// 32768 x 1536 with an fp32 stream and a sigmoid gate for every element, 705
// MB, takes 110 us, 6.4 TB/s or 95 % of the measured copy rate (what L2 keeps
// of the pass before included).  The backward is not quite: 32768 x 1536 in
// bf16 with 32 gate rows, 605 MB, takes 113 us (79 %); it issues 37
// instructions an element, of which a third are a row's own (its sums, waits
// and addresses), at 0.45 of the issue rate.  4096 x 768 from checkpoints, 32
// MB, takes 14 us with the second kernel, of which two to three rows per team
// and the two launches' ramps are most.  Where one team fills a block a row's
// exchange has nothing beside it: 8192 x 4096 without a gate takes 82 us, 4096 x
// 8192 76 us (59 either at the copy rate), 16384 x 2048 with three teams 72.  A
// gate of each element's own leaves eleven warps, and its values are read for
// both passes: 32768 x 1536 takes 202 us, 232 through a sigmoid (119 at the
// copy rate).  Gate rows shared by two rows each keep two of eleven teams at
// work: 32768 x 768 with 16384 of them takes 698 us, 56 without a gate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act8.cuh"
#include "block_launch.h"

namespace detattn {

// Set when a bounded wait of the backward runs out.
__device__ unsigned int g_norm_status;

namespace {

__device__ __forceinline__ void set_norm_status() { atomicOr(&g_norm_status, 1u); }

// ------------------------------------------------------------ row teams
// A row belongs to a team of W warps; thread t of the team holds the vectors
// of eight columns t, t + 32 W, ... (CH of them).  Sums over a row: shuffles,
// then, where W > 1, one word per warp in shared memory and the team's own
// barrier.  `slot` alternates between two sets of words, so one barrier per
// sum is enough.
template <bool MULTI>
__device__ __forceinline__ float team_sum(float v, float* words, int W, int team, int warp_in_team,
                                          int lane, int& slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (MULTI) {
    float* w = words + slot * 32 + team * W;
    if (lane == 0) w[warp_in_team] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(W * 32) : "memory");
    v = 0.0f;
    for (int i = 0; i < W; ++i) v += w[i];
    slot ^= 1;
  }
  return v;
}

// Eight gate values of the bf16 or fp32 gate from element `at` on.
__device__ __forceinline__ void load_gate(const void* gate, size_t at, bool fp32, Vec8& g) {
  if (fp32)
    g.from_f32(static_cast<const float*>(gate) + at);
  else
    g.from_bf16(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(gate) + at));
}

// Eight stream values (bf16 or fp32) as raw words.
template <bool F32>
struct Raw8 {
  uint4 a, b;  // b: fp32 only
  __device__ __forceinline__ void zero() {
    a = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (F32) b = a;
  }
  __device__ __forceinline__ void load(const void* p, size_t at) {
    if constexpr (F32) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      a = q[0];
      b = q[1];
    } else {
      a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
    }
  }
  __device__ __forceinline__ void get(Vec8& v) const {
    if constexpr (F32) {
      v.p[0] = f2_make(__uint_as_float(a.x), __uint_as_float(a.y));
      v.p[1] = f2_make(__uint_as_float(a.z), __uint_as_float(a.w));
      v.p[2] = f2_make(__uint_as_float(b.x), __uint_as_float(b.y));
      v.p[3] = f2_make(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
      v.from_bf16(a);
    }
  }
};
template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t at, const Vec8& v) {
  if constexpr (F32)
    v.to_f32(static_cast<float*>(p) + at);
  else
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) = v.to_bf16();
}
// Eight checkpointed values v mult; lanes past the row (`in` false) take part
// in the group's shuffles and store nothing.
__device__ __forceinline__ void keep8(const Vec8& v, float mult, bool in, size_t at, int8_t* q, uint8_t* e) {
  uint2 out;
  float f[8];
  v.to_float(f);
  const uint32_t ex = act8_quantise8(f, mult, &out);
  if (in) {
    *reinterpret_cast<uint2*>(q + at) = out;
    if ((at & 31) == 0) e[at >> 5] = static_cast<uint8_t>(ex);
  }
}

// Three sums at once.  The first two exchanges of a warp halve the sums as
// well as the lanes, so that six shuffles do, not fifteen: lanes 0 to 7 end
// with the first sum, 8 to 15 with the second, 16 to 23 with the third.
template <bool MULTI>
__device__ __forceinline__ void team_sum3(float (&v)[3], float* words, int W, int team, int warp_in_team,
                                          int lane, int& slot) {
  const bool up = (lane & 16) != 0, odd = (lane & 8) != 0;
  float k0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[2], 16);
  const float k1 = v[1] + __shfl_xor_sync(0xFFFFFFFFu, v[1], 16);
  k0 = (odd ? k1 : k0) + __shfl_xor_sync(0xFFFFFFFFu, odd ? k0 : k1, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) k0 += __shfl_xor_sync(0xFFFFFFFFu, k0, o);
  if constexpr (MULTI) {
    float* w = words + slot * 64 + team * W * 4;
    if ((lane & 7) == 0) w[warp_in_team * 4 + (lane >> 3)] = k0;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(W * 32) : "memory");
    v[0] = v[1] = v[2] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < W; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(w + i * 4);
      v[0] += x.x;
      v[1] += x.y;
      v[2] += x.z;
    }
    slot ^= 1;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, k0, 8 * k);
  }
}

// ------------------------------------------------------------ forward
constexpr int kFwdWarps = 4;  // warps per block where a row takes one warp

// Blocks of 128 threads that fit an SM with the registers they get: seven,
// but for 1024 columns in fp32, which would spill (4096 x 1024 in bf16 with
// checkpoints: 9.6 us with seven, 14.1 with six).
constexpr int fwd_blocks(int ch, bool multi, bool f32) {
  return multi ? (ch == 3 ? 4 : 3) : (ch == 4 && f32 ? 6 : 7);
}
// SIG: a gate that goes through its sigmoid (a kernel for both takes the
// registers of the sigmoid in every call: 32768 x 1536 with checkpoints and no
// sigmoid 85 us against 82).
template <int CH, bool MULTI, bool F32, bool KEEP8, bool SIG>
__global__ void __launch_bounds__(MULTI ? 256 : 128, fwd_blocks(CH, MULTI, F32))
    block_norm_fwd_kernel(const BlockNormFwdArgs a) {
  __shared__ float words[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = MULTI ? blockDim.x >> 5 : 1;
  const int team = MULTI ? 0 : warp, wt = MULTI ? warp : 0;
  const int t = wt * 32 + lane;
  const int row = MULTI ? blockIdx.x : blockIdx.x * kFwdWarps + warp;
  if (row >= a.N) return;
  const int n_vec = a.d >> 3;
  const size_t base = static_cast<size_t>(row) * a.d;
  int slot = 0;

  Raw8<F32> xr[CH];
  uint4 yr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int v = c * W * 32 + t;
    xr[c].zero();
    yr[c] = make_uint4(0u, 0u, 0u, 0u);
    if (v < n_vec) {
      if (a.y) yr[c] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.y) + base + v * 8);
      xr[c].load(a.x, base + v * 8);
    }
  }
  float rstd_y = 1.0f;
  if (a.w_post) {
    uint64_t sum = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      Vec8 f;
      f.from_bf16(yr[c]);
      f.squares(sum);
    }
    const float ss = team_sum<MULTI>(f2_sum(sum), words, W, team, wt, lane, slot);
    rstd_y = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
    if (t == 0) a.rstd_post[row] = rstd_y;
  }
  Vec8 x[CH];
  uint64_t sum = 0;
  const size_t gate_row = a.gate ? static_cast<size_t>(row / a.rows_per_gate) * a.d : 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int v = c * W * 32 + t;
    const bool in = v < n_vec;
    xr[c].get(x[c]);
    if (a.y) {
      Vec8 z;
      z.from_bf16(yr[c]);
      if constexpr (KEEP8) keep8(z, rstd_y, in, base + v * 8, a.yhat_q, a.yhat_e);
      if (in) {
        if (a.w_post) {
          Vec8 w;
          w.from_f32(a.w_post + v * 8);
          z.scale(rstd_y);
          z.mul(w);
        }
        if (a.gate) {
          Vec8 g;
          load_gate(a.gate, gate_row + v * 8, a.gate_fp32, g);
          if constexpr (SIG) g.sigmoid();
          z.mul(g);
        }
        const uint64_t r = f2_all(a.res_scale), s = f2_all(a.block_scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c].p[i] = f2_fma(s, z.p[i], f2_mul(r, x[c].p[i]));
        store8<F32>(a.x_out, base + v * 8, x[c]);
      }
    }
    x[c].squares(sum);
  }
  if (!a.w_pre) return;
  const float ss = team_sum<MULTI>(f2_sum(sum), words, W, team, wt, lane, slot);
  const float rstd_x = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
  if (t == 0) a.rstd_pre[row] = rstd_x;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int v = c * W * 32 + t;
    const bool in = v < n_vec;
    if constexpr (KEEP8) keep8(x[c], rstd_x, in, base + v * 8, a.xhat_q, a.xhat_e);
    if (in) {
      Vec8 w;
      w.from_f32(a.w_pre + v * 8);
      x[c].scale(rstd_x);
      w.mul(x[c]);
      store8<false>(a.h, base + v * 8, w);
    }
  }
}

// ------------------------------------------------------------ backward
// One persistent block per SM: row teams and one producer warp.  Every team
// has a ring of stages in shared memory; lane i of the producer fills team
// i's with bulk copies, rows ahead (each tensor's row is one contiguous
// piece), so that loads are in flight at all times while the teams' registers
// hold the column sums.  The exponent bytes of the checkpoints (rows of d / 32
// bytes, not a multiple of 16) come by plain loads a row ahead.
// Warps in row teams (one more fills the rings) by the vectors of eight
// columns that a thread holds: with three, 11 warps' registers fit; with two, 15,
// unless a gate of each row's own takes registers too.
constexpr int bwd_warps(int ch, bool multi, bool row_gate) {
  return multi && ch == 2 && !row_gate ? 15 : 11;
}
constexpr int kBwdMaxTeams = 11;
constexpr int kBwdBlocks = 152;     // one block per SM of the GB300
constexpr int kBwdMaxStages = 4;
constexpr int kBwdSmem = 225 * 1024;  // dynamic shared memory at most (2 KB are left for the static part)

// Where the pieces of a row lie in a stage, and the ring's shape.
struct BwdRing {
  int off_d, off_x, off_y, bytes;  // dh at 0
  int teams, stages;
  int W;             // warps per team
  bool w_near;       // w_pre has a copy behind the column multipliers (always, but for fp32 tensors)
};

// This team's rows, in order: rows team, team + teams, ... of each item.
struct BwdCursor {
  int item, row, end;
  __device__ __forceinline__ void open(const BlockNormBwdArgs& a, int team) {
    const int group_rows = a.N / (a.items / a.slices);
    const int per = (group_rows + a.slices - 1) / a.slices;
    const int group = item / a.slices, slice = item - group * a.slices;
    const int lo = min(slice * per, group_rows), hi = min(lo + per, group_rows);
    row = group * group_rows + lo + team;
    end = group * group_rows + hi;
  }
  // To the first row at or after `row`; false when there is none.
  __device__ __forceinline__ bool settle(const BlockNormBwdArgs& a, int team) {
    while (row >= end) {
      if (item + static_cast<int>(gridDim.x) >= a.items) return false;
      item += gridDim.x;
      open(a, team);
    }
    return true;
  }
};

// All threads of the row teams.
__device__ __forceinline__ void teams_sync(int threads) {
  asm volatile("bar.sync 15, %0;" ::"r"(threads) : "memory");
}

// Adds the teams' column sums in team order and hands each eight columns to
// `out(column, sums)`.  With `wide`, through [teams][d] words of scratch;
// without, through [d], one team after the other.
template <int CH, class Out>
__device__ __forceinline__ void block_columns(const Vec8 (&acc)[CH], float* scratch, bool wide, int d,
                                              int W, int teams, int team, int t, Out out) {
  const int n_vec = d >> 3, threads = teams * W * 32;
  if (wide) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int v = c * W * 32 + t;
      if (v < n_vec) acc[c].to_f32(scratch + team * d + v * 8);
    }
    teams_sync(threads);
    for (int v = team * W * 32 + t; v < n_vec; v += threads) {
      Vec8 f;
      f.from_f32(scratch + v * 8);
      for (int k = 1; k < teams; ++k) {
        Vec8 g;
        g.from_f32(scratch + k * d + v * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = f2_add(f.p[i], g.p[i]);
      }
      out(v * 8, f);
    }
    return;
  }
  for (int k = 0; k < teams; ++k) {
    if (team == k) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int v = c * W * 32 + t;
        if (v < n_vec) {
          Vec8 f = acc[c];
          if (k > 0) {
            Vec8 before;
            before.from_f32(scratch + v * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) f.p[i] = f2_add(before.p[i], f.p[i]);
          }
          if (k < teams - 1)
            f.to_f32(scratch + v * 8);
          else
            out(v * 8, f);
        }
      }
    }
    if (k < teams - 1) teams_sync(threads);
  }
}

// Eight gate values and their slopes by the stored value.
__device__ __forceinline__ void gate_pairs(const BlockNormBwdArgs& a, size_t at, Vec8& g, Vec8& slope) {
  load_gate(a.gate, at, a.gate_fp32, g);
  slope.fill(1.0f);
  if (a.gate_sigmoid) g.sigmoid(slope);
}

// What the compiler knows of a call: that every input is there and no row has
// a gate of its own; only the latter; that every row has one, as it is or
// through its sigmoid (32768 x 1536 with the flag read at run time took 220
// and 252 us).
enum BwdMode { kBwdFull, kBwdPlain, kBwdRowGate, kBwdRowSigmoid };
constexpr bool of_row_gate(BwdMode m) { return m == kBwdRowGate || m == kBwdRowSigmoid; }
template <int CH, bool MULTI, bool F32, bool FROM8, BwdMode MODE>
__global__ void __launch_bounds__((bwd_warps(CH, MULTI, of_row_gate(MODE)) + 1) * 32, 1)
    block_norm_bwd_kernel(const BlockNormBwdArgs a, const BwdRing ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float words[2 * 64];  // two sets of four per warp
  __shared__ __align__(8) uint64_t bars[2 * kBwdMaxTeams * kBwdMaxStages];  // full, empty
  constexpr bool FULL = MODE == kBwdFull, per_row_gate = of_row_gate(MODE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = MULTI ? ring.W : 1;
  const int teams = ring.teams, team_threads = teams * W * 32;
  const int n_vec = a.d >> 3;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool pre = FULL || a.dh != nullptr;
  const bool with_dx = FULL || a.dx_out != nullptr;
  const bool post = FULL || a.w_post != nullptr;
  const bool sum_gate = !per_row_gate && a.gate != nullptr;
  const bool with_dy = FULL || per_row_gate || a.dy != nullptr;
  const bool need_y = FULL || per_row_gate || (with_dy && (post || a.gate != nullptr));
  constexpr int kX = F32 ? 4 : 2;
  float* cols = reinterpret_cast<float*>(smem + teams * ring.stages * ring.bytes);  // [d]
  float* near_w = cols + a.d;                                                       // [d]: w_pre
  auto full = [&](int team, int s) { return smem_u32(&bars[team * kBwdMaxStages + s]); };
  auto empty = [&](int team, int s) {
    return smem_u32(&bars[(kBwdMaxTeams + team) * kBwdMaxStages + s]);
  };
  if (threadIdx.x < teams) {
    for (int s = 0; s < ring.stages; ++s) {
      mbar_init(full(threadIdx.x, s), 1);
      mbar_init(empty(threadIdx.x, s), W);
    }
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();

  if (warp == teams * W) {
    // The producer.
    const uint32_t row_tx = (pre ? 2u * a.d : 0u) + (with_dx ? kX * a.d : 0u) +
                            (pre ? (FROM8 ? 1u : kX) * a.d : 0u) + (need_y ? (FROM8 ? 1u : 2u) * a.d : 0u);
    const int team = lane;
    bool live = team < teams, gave_up = false;
    BwdCursor cur{};
    cur.item = blockIdx.x;
    if (live) {
      cur.open(a, team);
      live = cur.settle(a, team);
    }
    int n = 0, s = 0;
    uint32_t parity = 1;
    uint64_t since = globaltimer_ns();
    while (__any_sync(0xFFFFFFFFu, live)) {
      bool idle = true;
      if (live) {
        if (n < ring.stages || mbar_test_wait(empty(team, s), parity)) {
          idle = false;
          const size_t at = static_cast<size_t>(cur.row) * a.d;
          const uint32_t dst = smem_u32(smem) + (team * ring.stages + s) * ring.bytes, bar = full(team, s);
          mbar_arrive_expect_tx(bar, row_tx);
          if (pre) {
            bulk_load(dst, static_cast<const uint8_t*>(a.dh) + at * 2, 2 * a.d, bar);
            if constexpr (FROM8)
              bulk_load(dst + ring.off_x, a.xhat_q + at, a.d, bar);
            else
              bulk_load(dst + ring.off_x, static_cast<const uint8_t*>(a.x) + at * kX, kX * a.d, bar);
          }
          if (with_dx)
            bulk_load(dst + ring.off_d, static_cast<const uint8_t*>(a.dx_out) + at * kX, kX * a.d, bar);
          if (need_y) {
            if constexpr (FROM8)
              bulk_load(dst + ring.off_y, a.yhat_q + at, a.d, bar);
            else
              bulk_load(dst + ring.off_y, static_cast<const uint8_t*>(a.y) + at * 2, 2 * a.d, bar);
          }
          ++n;
          if (++s == ring.stages) {
            s = 0;
            parity ^= 1u;
          }
          cur.row += teams;
          live = cur.settle(a, team);
          since = globaltimer_ns();
        } else if (globaltimer_ns() - since > a.wait_ns) {
          live = false;
          gave_up = true;
        }
      }
      if (__all_sync(0xFFFFFFFFu, idle)) __nanosleep(40);
    }
    // The copies in flight, before the block can end.
    for (int k = n > ring.stages ? n - ring.stages : 0; k < n; ++k)
      if (!mbar_wait(full(team, k % ring.stages), (k / ring.stages) & 1, a.wait_ns)) gave_up = true;
    if (gave_up) set_norm_status();
    return;
  }

  const int team = warp / W, wt = warp - team * W;
  const int t = wt * 32 + lane;
  uint8_t* mine = smem + team * ring.stages * ring.bytes;
  int slot = 0;
  bool ok = true;
  // What plain loads bring, one row ahead.
  struct Small {
    float rx, ry;
    uint32_t e[CH];  // exponent bytes: xhat's, yhat's << 8
  };
  auto load_small = [&](int row) {
    Small m;
    m.rx = pre ? a.rstd_pre[row] : 0.0f;
    m.ry = post ? a.rstd_post[row] : 1.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      m.e[c] = 0u;
      if constexpr (FROM8) {
        const int v = c * W * 32 + t;
        const size_t at = static_cast<size_t>(row) * (a.d >> 5) + (v >> 2);
        if (v < n_vec) {
          if (pre) m.e[c] = a.xhat_e[at];
          if (need_y) m.e[c] |= static_cast<uint32_t>(a.yhat_e[at]) << 8;
        }
      }
    }
    return m;
  };

  // Column sums of this thread: of dh xhat over all rows, and of D yhat (the
  // gate left out where a whole item shares it) over the item's rows.  From
  // the second follow both dgate and dw_post: what multiplies a column is
  // applied where the item is written out.
  Vec8 acc_pre[CH], acc_y[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    acc_pre[c].fill(0.0f);
    acc_y[c].fill(0.0f);
  }

  const bool w_near = FROM8 || !F32 || ring.w_near;
  if (pre && w_near) {
    for (int v = threadIdx.x; v < n_vec; v += team_threads) {
      Vec8 w;
      w.from_f32(a.w_pre + v * 8);
      w.to_f32(near_w + v * 8);
    }
    teams_sync(team_threads);
  }

  int s = 0;           // this row's stage
  uint32_t phase = 0;  // and the parity of its barrier
  BwdCursor cur;
  for (cur.item = blockIdx.x; cur.item < a.items; cur.item += gridDim.x) {
    cur.open(a, team);
    const int group = cur.item / a.slices;
    const size_t group_gate = static_cast<size_t>(group) * a.d;
    if (need_y) {
      // What multiplies a column on the way to y: the norm's weight times the
      // gate that the item's rows share.  (The same words hold the teams'
      // sums when an item that is not the block's last is written out.)
      teams_sync(team_threads);
      for (int v = threadIdx.x; v < n_vec; v += team_threads) {
        Vec8 w, g, slope;
        w.fill(1.0f);
        if (post) w.from_f32(a.w_post + v * 8);
        if (sum_gate) {
          gate_pairs(a, group_gate + v * 8, g, slope);
#pragma unroll
          for (int i = 0; i < 4; ++i) w.p[i] = f2_mul(w.p[i], g.p[i]);
        }
        w.to_f32(cols + v * 8);
      }
      teams_sync(team_threads);
    }
    Small next{};
    if (cur.row < cur.end) next = load_small(cur.row);
    for (; cur.row < cur.end; cur.row += teams) {
      const int row = cur.row;
      const size_t base = static_cast<size_t>(row) * a.d;
      const uint8_t* st = mine + s * ring.bytes;
      const Small m = next;
      if (row + teams < cur.end) next = load_small(row + teams);
      if (ok) ok = mbar_wait(full(team, s), phase, a.wait_ns);
      // xhat = scale_x raw_x, yhat = scale_y raw_y: the row's 1 / rms and the
      // stored number, or the group's power of two and the checkpoint's.
      auto raw_x = [&](int v, Vec8& f) {
        if constexpr (FROM8)
          f.from_int8(*reinterpret_cast<const uint2*>(st + ring.off_x + v * 8));
        else if constexpr (F32)
          f.from_f32(st + ring.off_x + v * 32);
        else
          f.from_bf16(*reinterpret_cast<const uint4*>(st + ring.off_x + v * 16));
      };
      auto raw_y = [&](int v, Vec8& f) {
        if constexpr (FROM8)
          f.from_int8(*reinterpret_cast<const uint2*>(st + ring.off_y + v * 8));
        else
          f.from_bf16(*reinterpret_cast<const uint4*>(st + ring.off_y + v * 16));
      };
      auto scale_x = [&](int c) { return FROM8 ? act8_scale(m.e[c] & 255u) : m.rx; };
      auto scale_y = [&](int c) { return FROM8 ? act8_scale(m.e[c] >> 8) : m.ry; };
      // D = p - x k1, p = dx' + rstd dh w_pre, needs a sum over the row, and
      // dy one over D; but with D the second is linear in k1:
      //   sum D gw y = sum p gw y - k1 sum x gw y
      // so that all sums come from one pass and one exchange.
      Vec8 keep[CH];  // p
      float sums[3] = {0.0f, 0.0f, 0.0f};  // dh w_pre xhat; p gw yhat; xhat gw yhat
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int v = c * W * 32 + t;
        if (v < n_vec) {
          if (!with_dx)
            keep[c].fill(0.0f);
          else if constexpr (F32)
            keep[c].from_f32(st + ring.off_d + v * 32);
          else
            keep[c].from_bf16(*reinterpret_cast<const uint4*>(st + ring.off_d + v * 16));
          Vec8 x;
          if (pre) {
            Vec8 dh, w;
            dh.from_bf16(*reinterpret_cast<const uint4*>(st + v * 16));
            raw_x(v, x);
            if (w_near)
              w.from_f32(near_w + v * 8);
            else
              w.from_f32(a.w_pre + v * 8);
            const uint64_t sc = f2_all(scale_x(c)), rx = f2_all(m.rx);
            uint64_t part = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t q = f2_mul(dh.p[i], w.p[i]);
              acc_pre[c].p[i] = f2_fma(f2_mul(dh.p[i], x.p[i]), sc, acc_pre[c].p[i]);
              part = f2_fma(q, x.p[i], part);
              keep[c].p[i] = f2_fma(q, rx, keep[c].p[i]);
            }
            sums[0] = fmaf(f2_sum(part), scale_x(c), sums[0]);
          }
          if (post) {
            Vec8 gw, f;
            gw.from_f32(cols + v * 8);
            raw_y(v, f);
            gw.mul(f);
            if constexpr (per_row_gate) {
              load_gate(a.gate, base + v * 8, a.gate_fp32, f);
              if constexpr (MODE == kBwdRowSigmoid) f.sigmoid();
              gw.mul(f);
            }
            uint64_t part = 0, cross = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              part = f2_fma(keep[c].p[i], gw.p[i], part);
              if (pre) cross = f2_fma(x.p[i], gw.p[i], cross);
            }
            sums[1] = fmaf(f2_sum(part), scale_y(c), sums[1]);
            if (pre) sums[2] = fmaf(f2_sum(cross), scale_x(c) * scale_y(c), sums[2]);
          }
        }
      }
      if (pre || post) team_sum3<MULTI>(sums, words, W, team, wt, lane, slot);
      const float kx = -m.rx * sums[0] * inv_d;  // D = p + kx xhat
      const float ky = -m.ry * a.block_scale * inv_d * (pre ? fmaf(kx, sums[2], sums[1]) : sums[1]);
      const float kd = (post ? m.ry : 1.0f) * a.block_scale;  // dy = kd D gw + ky yhat
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int v = c * W * 32 + t;
        if (v < n_vec) {
          const size_t at = base + v * 8;
          if (pre) {
            Vec8 x;
            raw_x(v, x);
            const uint64_t k = f2_all(kx * scale_x(c));
#pragma unroll
            for (int i = 0; i < 4; ++i) keep[c].p[i] = f2_fma(x.p[i], k, keep[c].p[i]);
          }
          Vec8 o = keep[c];
          o.scale(a.res_scale);
          store8<F32>(a.dx, at, o);
          if (with_dy) {
            if (need_y) {
              Vec8 y, e, gw;
              raw_y(v, y);
              gw.from_f32(cols + v * 8);
              e = keep[c];
              e.mul(y);
              keep[c].scale(kd);
              keep[c].mul(gw);
              if constexpr (per_row_gate) {
                // dgate = block_scale D yhat w_post slope.  (Pair by pair: with
                // eight slopes at a time fp32 rows of 768 columns spilled.)
                Vec8 g;
                gw.mul(e);
                gw.scale(a.block_scale * scale_y(c));
                load_gate(a.gate, at, a.gate_fp32, g);
                if constexpr (MODE == kBwdRowSigmoid)
                  g.logistic([&](int i, uint64_t t) {
                    gw.p[i] = f2_mul(gw.p[i], f2_mul(f2_mul(t, g.p[i]), g.p[i]));
                  });
                e.mul(g);
                keep[c].mul(g);
                if (a.gate_fp32)
                  store8<true>(a.dgate, at, gw);
                else
                  store8<false>(a.dgate, at, gw);
              }
              const uint64_t sc = f2_all(scale_y(c));
#pragma unroll
              for (int i = 0; i < 4; ++i) acc_y[c].p[i] = f2_fma(e.p[i], sc, acc_y[c].p[i]);
              if (post) {
                const uint64_t k = f2_all(ky * scale_y(c));
#pragma unroll
                for (int i = 0; i < 4; ++i) keep[c].p[i] = f2_fma(y.p[i], k, keep[c].p[i]);
              }
            } else {
              keep[c].scale(kd);
            }
            store8<false>(a.dy, at, keep[c]);
          }
        }
      }
      // This warp is past the stage.
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(team, s));
      if (++s == ring.stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (post || sum_gate) {
      // This item's sums: its share of dgate (all of it without a part), and
      // of dw_post, which the block adds up over its items.
      // After the last item the ring is free.
      const bool last = cur.item + static_cast<int>(gridDim.x) >= a.items;
      teams_sync(team_threads);
      float* post_sums = a.part_post + static_cast<size_t>(blockIdx.x) * a.d;
      const bool first = cur.item == blockIdx.x;
      block_columns<CH>(acc_y, last ? reinterpret_cast<float*>(smem) : cols, last, a.d, W, teams, team, t, [&](int col, Vec8& f) {
        const uint64_t k = f2_all(a.block_scale);
        Vec8 g, slope;
        g.fill(1.0f);
        if (sum_gate) {
          gate_pairs(a, group_gate + col, g, slope);
          Vec8 w;
          if (post)
            w.from_f32(a.w_post + col);
          else
            w.fill(1.0f);
#pragma unroll
          for (int i = 0; i < 4; ++i) slope.p[i] = f2_mul(f2_mul(slope.p[i], w.p[i]), f2_mul(f.p[i], k));
          if (a.part_gate)
            slope.to_f32(a.part_gate + static_cast<size_t>(cur.item) * a.d + col);
          else if (a.gate_fp32)
            slope.to_f32(static_cast<float*>(a.dgate) + group_gate + col);
          else
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dgate) + group_gate + col) = slope.to_bf16();
        }
        if (post) {
          Vec8 sum;
          if (first)
            sum.fill(0.0f);
          else
            sum.from_f32(post_sums + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum.p[i] = f2_fma(f2_mul(f.p[i], k), g.p[i], sum.p[i]);
          sum.to_f32(post_sums + col);
        }
      });
#pragma unroll
      for (int c = 0; c < CH; ++c) acc_y[c].fill(0.0f);
    }
  }
  if (pre) {
    teams_sync(team_threads);
    float* out = a.part_pre + static_cast<size_t>(blockIdx.x) * a.d;
    block_columns<CH>(acc_pre, reinterpret_cast<float*>(smem), true, a.d, W, teams, team, t,
                      [&](int col, Vec8& f) { f.to_f32(out + col); });
  }
  if (!ok) set_norm_status();
}

// Adds the parts of a column sum in ascending order: 32 columns per block,
// sixteen runs of parts each, then the runs in order.
constexpr int kSumRuns = 16;
struct SumJob {
  const float* parts;  // [n][d]
  void* out;           // [d]
  int n;
  bool out_fp32;
};
struct SumJobs {
  SumJob pre, post, gate;  // gate: row z of [G][d], parts [G][n][d]
  int n_pre, n_post;       // 1 or 0
  int d;
};
__global__ void __launch_bounds__(kSumRuns * 32) sum_parts_kernel(const SumJobs j) {
  __shared__ float run[kSumRuns][32];
  const int z = blockIdx.y;
  SumJob s;
  size_t at = 0;
  if (z < j.n_pre) {
    s = j.pre;
  } else if (z < j.n_pre + j.n_post) {
    s = j.post;
  } else {
    s = j.gate;
    at = z - j.n_pre - j.n_post;
  }
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx;
  griddep_wait();
  const float* p = s.parts + at * s.n * j.d + col;
  const int per = (s.n + kSumRuns - 1) / kSumRuns, lo = min(ty * per, s.n), hi = min(lo + per, s.n);
  float acc = 0.0f;
  if (col < j.d) {
#pragma unroll 8
    for (int k = lo; k < hi; ++k) acc += p[static_cast<size_t>(k) * j.d];
  }
  run[ty][tx] = acc;
  __syncthreads();
  if (ty == 0 && col < j.d) {
    for (int k = 1; k < kSumRuns; ++k) acc += run[k][tx];
    if (s.out_fp32)
      static_cast<float*>(s.out)[at * j.d + col] = acc;
    else
      static_cast<__nv_bfloat16*>(s.out)[at * j.d + col] = __float2bfloat16(acc);
  }
}

// Failure-detection self-test: the row teams' wait on a barrier that nothing
// arrives on.
__global__ void norm_wait_selftest_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(smem_u32(&bar), 1);
  fence_barrier_init();
  if (!mbar_wait(smem_u32(&bar), 0, limit_ns)) set_norm_status();
}

template <int CH, bool MULTI>
cudaError_t fwd_of(const BlockNormFwdArgs& a, bool f32, int W, cudaStream_t st) {
  const unsigned grid = MULTI ? a.N : (a.N + kFwdWarps - 1) / kFwdWarps;
  const unsigned block = MULTI ? W * 32 : kFwdWarps * 32;
  const bool keep = a.xhat_q != nullptr || a.yhat_q != nullptr;
  const bool sig = a.gate != nullptr && a.gate_sigmoid;
  auto launch = [&](auto kernel) {
    kernel<<<grid, block, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (f32) {
    if (keep)
      return launch(sig ? block_norm_fwd_kernel<CH, MULTI, true, true, true>
                        : block_norm_fwd_kernel<CH, MULTI, true, true, false>);
    return launch(sig ? block_norm_fwd_kernel<CH, MULTI, true, false, true>
                      : block_norm_fwd_kernel<CH, MULTI, true, false, false>);
  }
  if (keep)
    return launch(sig ? block_norm_fwd_kernel<CH, MULTI, false, true, true>
                      : block_norm_fwd_kernel<CH, MULTI, false, true, false>);
  return launch(sig ? block_norm_fwd_kernel<CH, MULTI, false, false, true>
                    : block_norm_fwd_kernel<CH, MULTI, false, false, false>);
}

template <int CH, bool MULTI, bool F32, bool FROM8, BwdMode MODE>
cudaError_t bwd_mode(const BlockNormBwdArgs& a, int W, cudaStream_t st) {
  static unsigned long long attr_ctx[64] = {};
  auto kernel = block_norm_bwd_kernel<CH, MULTI, F32, FROM8, MODE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long ctx = current_context_id();
  if (dev >= 64 || ctx == 0 || attr_ctx[dev] != ctx) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_ctx[dev] = current_context_id();
  }
  const bool pre = a.dh != nullptr;
  const bool need_y = a.dy != nullptr && (a.w_post != nullptr || a.gate != nullptr);
  const int x_bytes = F32 ? 4 : 2;
  BwdRing r{};
  r.off_d = pre ? 2 * a.d : 0;
  r.off_x = r.off_d + (a.dx_out ? x_bytes * a.d : 0);
  r.off_y = r.off_x + (pre ? (FROM8 ? 1 : x_bytes) * a.d : 0);
  r.bytes = r.off_y + (need_y ? (FROM8 ? 1 : 2) * a.d : 0);
  r.W = W;
  r.teams = bwd_warps(CH, MULTI, of_row_gate(MODE)) / W;
  // The rings leave no L1 to speak of, so w_pre would come from L2 for every
  // row: it has a copy behind the column multipliers, for which only fp32 rows
  // of more than 7200 columns leave no room (32768 x 1536: 118.5 us without,
  // 117.0 with it).
  int cols = (pre ? 8 : 4) * a.d;
  while (r.teams > 1 && r.teams * 2 * r.bytes + cols > kBwdSmem) --r.teams;
  r.w_near = pre && r.teams * 2 * r.bytes + cols <= kBwdSmem;
  if (!r.w_near) cols = 4 * a.d;
  r.stages = 2;
  while (r.stages < kBwdMaxStages && r.teams * (r.stages + 1) * r.bytes + cols <= kBwdSmem) ++r.stages;
  const int smem = r.teams * r.stages * r.bytes + cols;
  kernel<<<a.blocks, (r.teams * W + 1) * 32, smem, st>>>(a, r);
  return cudaGetLastError();
}

template <int CH, bool MULTI, bool F32, bool FROM8>
cudaError_t bwd_typed(const BlockNormBwdArgs& a, int W, cudaStream_t st) {
  if (a.gate != nullptr && a.rows_per_gate == 1)
    return a.gate_sigmoid ? bwd_mode<CH, MULTI, F32, FROM8, kBwdRowSigmoid>(a, W, st)
                          : bwd_mode<CH, MULTI, F32, FROM8, kBwdRowGate>(a, W, st);
  if (a.dh != nullptr && a.dx_out != nullptr && a.dy != nullptr && a.w_post != nullptr)
    return bwd_mode<CH, MULTI, F32, FROM8, kBwdFull>(a, W, st);
  return bwd_mode<CH, MULTI, F32, FROM8, kBwdPlain>(a, W, st);
}

template <int CH, bool MULTI>
cudaError_t bwd_of(const BlockNormBwdArgs& a, bool f32, int W, cudaStream_t st) {
  const bool from8 = a.xhat_q != nullptr || a.yhat_q != nullptr;
  if (f32)
    return from8 ? bwd_typed<CH, MULTI, true, true>(a, W, st) : bwd_typed<CH, MULTI, true, false>(a, W, st);
  return from8 ? bwd_typed<CH, MULTI, false, true>(a, W, st) : bwd_typed<CH, MULTI, false, false>(a, W, st);
}

}  // namespace

cudaError_t launch_block_norm_fwd(const BlockNormFwdArgs& a, bool x_fp32, cudaStream_t st) {
  // Up to 1024 columns a row is one warp's; beyond, W warps share it.  Three
  // or four vectors per thread then: at 32768 x 1536, when three took 124 us
  // (112 now), two took 132, one 149 and six 175.
  const int W = (a.d + 1023) / 1024, ch = (a.d + 256 * W - 1) / (256 * W);
  if (W == 1) {
    if (ch == 1) return fwd_of<1, false>(a, x_fp32, W, st);
    if (ch == 2) return fwd_of<2, false>(a, x_fp32, W, st);
    if (ch == 3) return fwd_of<3, false>(a, x_fp32, W, st);
    return fwd_of<4, false>(a, x_fp32, W, st);
  }
  if (ch <= 3) return fwd_of<3, true>(a, x_fp32, W, st);
  return fwd_of<4, true>(a, x_fp32, W, st);
}

namespace {

// Warps per row and vectors per thread.  Up to 768 columns a row is one
// warp's; beyond, two vectors per thread keep more warps at work than three
// where their teams fill the block as well (32768 x 1536: five teams of three
// warps took 119 us where five of two took 124).
struct BwdShape {
  int W, ch;
};
BwdShape bwd_shape(int d, bool row_gate) {
  if (d <= 768) return {1, (d + 255) / 256};
  const int w3 = (d + 767) / 768, w2 = (d + 511) / 512;
  const int n3 = bwd_warps(3, true, row_gate), n2 = bwd_warps(2, true, row_gate);
  if (w2 <= n2 && n2 / w2 * w2 > n3 / w3 * w3) return {w2, 2};
  return {w3, 3};
}

}  // namespace

BlockNormBwdPlan block_norm_bwd_plan(int N, int d, int G) {
  BlockNormBwdPlan p{};
  const BwdShape sh = bwd_shape(d, false);
  const int teams = bwd_warps(sh.ch, sh.W > 1, false) / sh.W;
  const bool shared = G > 1 && G < N;
  if (!shared) {
    const int want = (N + teams - 1) / teams;
    p.blocks = want < 1 ? 1 : (want < kBwdBlocks ? want : kBwdBlocks);
    p.slices = p.items = p.blocks;
    p.gate_parts = G == 1 && N > 1;
    return p;
  }
  // About four items per block, so that their number divides well.  Slices of
  // `per` rows each (the last may be shorter): as many as that gives, so that
  // none is without rows.
  const int rows = N / G;
  int s = 4 * kBwdBlocks / G;
  s = s < 1 ? 1 : (s < rows ? s : rows);
  const int per = (rows + s - 1) / s;
  p.slices = (rows + per - 1) / per;
  p.items = G * p.slices;
  p.blocks = p.items < kBwdBlocks ? p.items : kBwdBlocks;
  p.gate_parts = p.slices > 1;
  return p;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool x_fp32, cudaStream_t st) {
  const auto [W, ch] = bwd_shape(a.d, a.gate != nullptr && a.rows_per_gate == 1);
  cudaError_t e;
  if (W == 1)
    e = ch == 1   ? bwd_of<1, false>(a, x_fp32, W, st)
        : ch == 2 ? bwd_of<2, false>(a, x_fp32, W, st)
                  : bwd_of<3, false>(a, x_fp32, W, st);
  else
    e = ch == 2 ? bwd_of<2, true>(a, x_fp32, W, st) : bwd_of<3, true>(a, x_fp32, W, st);
  if (e != cudaSuccess) return e;
  SumJobs j{};
  j.d = a.d;
  j.n_pre = a.dh != nullptr;
  j.n_post = a.w_post != nullptr;
  j.pre = {a.part_pre, a.dw_pre, a.blocks, true};
  j.post = {a.part_post, a.dw_post, a.blocks, true};
  j.gate = {a.part_gate, a.dgate, a.slices, a.gate_fp32};
  const int rows = j.n_pre + j.n_post + (a.part_gate ? a.items / a.slices : 0);
  if (rows == 0) return cudaSuccess;
  // A programmatic dependent: launched while the rows are at work, it waits
  // for them before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.d + 31) / 32, rows);
  cfg.blockDim = kSumRuns * 32;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sum_parts_kernel, j);
}

cudaError_t launch_norm_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  norm_wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

cudaError_t take_norm_status(cudaStream_t st, unsigned* out) {
  unsigned val = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&val, g_norm_status, sizeof(val), 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && val)
    e = cudaMemcpyToSymbolAsync(g_norm_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  *out = val;
  return e;
}

}  // namespace detattn
