// Internal interface of the training-block kernels (block_norm.cu, act8_ops.cu,
// act8_wgrad.cu): argument blocks and launch functions.  Not part of the
// public API.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace detattn {

// An 8-bit checkpoint of a [rows, d] activation: q int8 [rows, d] and one
// exponent byte for every kAct8Group consecutive columns, e [rows, d / 32];
// the value is q 2^(e - 127) (e = 255: the group held an infinity or NaN and
// reads back as NaN).
constexpr int kAct8Group = 32;

constexpr int kNormMaxD = 8192;

struct BlockNormFwdArgs {
  const void* x;          // bf16 or fp32 [N, d]
  const void* y;          // bf16 [N, d] or null (x' = x, nothing written to x_out)
  const void* gate;       // bf16 or fp32 [G, d] or null
  const float* w_post;    // fp32 [d] or null
  const float* w_pre;     // fp32 [d] or null
  void* x_out;            // x's type [N, d]
  void* h;                // bf16 [N, d]
  float* rstd_post;       // [N]
  float* rstd_pre;        // [N]
  int8_t* yhat_q;         // checkpoints (null: none kept)
  uint8_t* yhat_e;
  int8_t* xhat_q;
  uint8_t* xhat_e;
  int N, d;
  int rows_per_gate;      // N / G
  bool gate_fp32, gate_sigmoid;
  float res_scale, block_scale, eps;
};

struct BlockNormBwdArgs {
  const void* dx_out;     // x's type [N, d] or null (zero)
  const void* dh;         // bf16 [N, d] or null (no norm after)
  const void* x;          // x's type [N, d]: x' of the forward (null with xhat_q or without dh)
  const void* y;          // bf16 [N, d] (null with yhat_q, or where nothing needs it)
  const int8_t* xhat_q;
  const uint8_t* xhat_e;
  const int8_t* yhat_q;
  const uint8_t* yhat_e;
  const void* gate;
  const float* w_post;
  const float* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  void* dx;               // x's type [N, d]
  void* dy;               // bf16 [N, d] or null (no block output: plain norm)
  void* dgate;            // the gate's type [G, d]
  float* dw_post;         // [d]
  float* dw_pre;          // [d]
  int N, d;
  int rows_per_gate;
  bool gate_fp32, gate_sigmoid;
  float res_scale, block_scale;
  // Workspace: column sums of the row blocks (laid out by the host, norm_layout).
  float* part_pre;        // [parts, d]
  float* part_post;       // [parts, d]
  float* part_gate;       // [items, d] (null: nothing to add up over blocks)
  int slices;             // row slices of every gate row; items = G * slices
  int items;
  int blocks;             // grid (parts)
  unsigned long long wait_ns;
};

// How the backward deals its rows, from the shape alone.  An item is one
// slice of the rows that share a gate row (of all rows where no gate row is
// shared by some but not all of them).
struct BlockNormBwdPlan {
  int blocks, slices, items;
  bool gate_parts;        // the slices' gate sums are added up by the second kernel
};
BlockNormBwdPlan block_norm_bwd_plan(int N, int d, int G);

cudaError_t launch_block_norm_fwd(const BlockNormFwdArgs& a, bool x_fp32, cudaStream_t st);
cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool x_fp32, cudaStream_t st);

cudaError_t launch_act8_pack(const void* x, int8_t* q, uint8_t* e, long rows, int d,
                             cudaStream_t st);
cudaError_t launch_act8_unpack(const int8_t* q, const uint8_t* e, void* x, long rows, int d,
                               cudaStream_t st);
// u [rows, 2 f] = [a | b]: h = silu(a) b.  q, e (not null): the checkpoint of u.
cudaError_t launch_swiglu_fwd(const void* u, void* h, int8_t* q, uint8_t* e, long rows, int f,
                              cudaStream_t st);
// From u, or from its checkpoint (u null): du [rows, 2 f]; h (may be null) again.
cudaError_t launch_swiglu_bwd(const void* dh, const void* u, const int8_t* q, const uint8_t* e,
                              void* du, void* h, long rows, int f, cudaStream_t st);

// ------------------------------------------------------------ weight gradient from a checkpoint
// A pair of blocks works on a tile of 256 columns of the checkpoint (rows of
// dw, half of them each) by 256 columns of dy, 64 tokens a step.
constexpr int kWgradBM = 256;
constexpr int kWgradBN = 256;
constexpr int kWgradBK = 64;
// Steps that one accumulator takes before it is added to the tile's sum in
// fp32 registers: the tensor core's own additions lose about 2e-7 of a
// sum of 512 tokens, and in proportion to their number.  (Runs of 1024 tokens
// left the result a little further from 64 bits than a product in fp32, at
// 8192 x 4096 x 6144 in 263 us against 269; runs of 256 would take 287.)
constexpr int kWgradChunk = 8;
// Persistent pairs, one block per SM of the GB300.  A constant, so that the
// deal of the work, and with it every bit, follows from the shape alone (no
// pair waits for another, so any SM count is correct).
constexpr int kWgradPairs = 76;

struct Act8WgradArgs {
  const uint8_t* e;       // [rows, d / 32]
  const float* row_scale; // [d] or null
  float* dw;              // [d, n]
  float* partial;         // [tiles that are cut * splits][256][256]
  int rows, d, n;
  int tiles_m, tiles_n;
  int whole_tiles;        // tiles computed by one pair each
  int splits;             // row ranges of each of the other tiles (1: none split)
  unsigned long long wait_ns;
};
struct Act8WgradPlan {
  int tiles_m, tiles_n, whole_tiles, splits;
};
Act8WgradPlan act8_wgrad_plan(int rows, int d, int n);
// mq: uint8 map {d, rows}, box {kWgradBM / 2, 64}, no swizzle; mdy: bf16 map {n,
// rows}, box {64, 64}, 128-byte swizzle.
cudaError_t launch_act8_wgrad(const CUtensorMap& mq, const CUtensorMap& mdy,
                              const Act8WgradArgs& a, cudaStream_t st);
// Read-and-clear of the status words (bit 0: a wait ran out); synchronous on `st`.
cudaError_t take_wgrad_status(cudaStream_t st, unsigned* out);
cudaError_t take_norm_status(cudaStream_t st, unsigned* out);
// One warp whose waits run out and set the status word.
cudaError_t launch_wgrad_wait_selftest(unsigned long long limit_ns, cudaStream_t st);
cudaError_t launch_norm_wait_selftest(unsigned long long limit_ns, cudaStream_t st);

unsigned long long current_context_id();

}  // namespace detattn
