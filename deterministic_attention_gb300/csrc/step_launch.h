// Internal interface of the kernels at the ends of a training step (rope.cu,
// linear_ce.cu, muon.cu): argument blocks and launch functions.  Not part of
// the public API.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace detattn {

// ------------------------------------------------------------ rotary positions
struct TurnArgs {
  const void* q;           // [tokens, Hq, D], a token every q_ld elements
  const void* k;           // [tokens, Hkv, D] (null with Hkv = 0)
  void* q_out;
  void* k_out;
  const double* freqs;     // [rot / 2] radians per position
  const int* positions;    // [n_pos] or null: position = token % T
  long tokens, n_pos;
  long q_ld, k_ld, q_out_ld, k_out_ld;
  int T, Hq, Hkv, D, rot;
  bool interleaved, fp32;
  float mscale, sign;      // sign -1: the opposite angle
};
cudaError_t launch_turn(const TurnArgs& a, cudaStream_t st);

// ------------------------------------------------------------ products
// Work of one launch of the tensor-core product (product.cuh): C tiles of 256 x 256,
// two blocks on one tile.
constexpr int kCeTile = 256;
struct ProductPlan {
  int tiles_m, tiles_n;
  int n_k;                 // steps of 64 along K
  int band;                // tile rows that are walked together, column by column
  int whole;               // tiles computed by one team each
  int splits;              // K ranges of each of the other tiles (1: none cut)
  int units;               // whole + (tiles - whole) * splits
  int teams;               // pairs at work
  unsigned long long wait_ns;
};
// Teams of the GB300's 152 SMs.  Constants, so that the deal of the work, and
// with it every bit, follows from the shape alone.
constexpr int kProductSms = 152;
inline int product_teams(int ctas) { return kProductSms / ctas; }
// cut: whether tiles of an incomplete last round are cut along K (the caller
// has then room for partial tiles and adds them up).
ProductPlan product_plan(long M, long N, long K, bool cut);
inline size_t product_partial_bytes(const ProductPlan& p) {
  const size_t cut = static_cast<size_t>(p.tiles_m) * p.tiles_n - p.whole;
  return p.splits == 1 ? 0 : cut * p.splits * kCeTile * kCeTile * sizeof(float);
}

// ------------------------------------------------------------ cross entropy of the output projection
// Logits of a 256 x 256 tile leave two (largest, sum) pairs per row.
struct CeStatsArgs {
  const int* targets;      // [N]
  float2* part;            // [2 * column tiles][N]: (m, sum 2^(z log2e - m log2e))
  float* z_target;         // [N] the target's logit
  int N, V;
};
struct CeFinishArgs {
  const int* targets;
  const float2* part;
  const float* z_target;
  float* loss;
  float* lse;
  int N, V, parts;
};
struct CeGradArgs {
  const int* targets;      // [N]
  const float* lse;        // [N]
  const float* dloss;      // [N]
  const float* dlse;       // [N] or null
  const float* unit;       // dz is held over this (launch_ce_unit)
  void* dz;                // bf16 [N, ld]: columns v0 .. v0 + width - 1 of dz
  int N, V;
  int v0, width;
  long ld;
};
// What becomes of a tile's sum s = *unit * sum: out (bf16 or fp32) = [acc +] s, or acc = [acc +] s.
struct CeStoreArgs {
  const float* unit;
  void* out;               // [rows, cols]; null: the sum goes to acc
  float* acc;              // fp32 [rows, cols] or null
  float* partial;          // tiles cut along K
  int rows, cols;
  int add;                 // add what acc holds
  int out_fp32;
  int wide;                // rows of out begin on 32 bytes
};
// mx: x [N, d] as rows of K; mw: w [V, d] as rows of K.
cudaError_t launch_ce_stats(const CUtensorMap& mx, const CUtensorMap& mw, const ProductPlan& p,
                            const CeStatsArgs& a, cudaStream_t st);
cudaError_t launch_ce_finish(const CeFinishArgs& a, cudaStream_t st);
// *unit = the largest |dloss| of the rows that have a target, as a rule (ce_unit_kernel).
cudaError_t launch_ce_unit(const int* targets, const float* dloss, const float* dlse, float* unit, int N,
                           int V, cudaStream_t st);
cudaError_t launch_ce_dz(const CUtensorMap& mx, const CUtensorMap& mw, const ProductPlan& p,
                         const CeGradArgs& a, cudaStream_t st);
// mdz: dz as rows of K; mw: w with K along its rows.
cudaError_t launch_ce_dx(const CUtensorMap& mdz, const CUtensorMap& mw, const ProductPlan& p,
                         const CeStoreArgs& a, cudaStream_t st);
// mdz: dz with K along its rows; mx: x likewise.
cudaError_t launch_ce_dw(const CUtensorMap& mdz, const CUtensorMap& mx, const ProductPlan& p,
                         const CeStoreArgs& a, cudaStream_t st);
cudaError_t take_ce_status(cudaStream_t st, unsigned* out);  // bit 0: wait, bit 1: target >= V
cudaError_t launch_ce_wait_selftest(unsigned long long limit_ns, cudaStream_t st);

// ------------------------------------------------------------ orthogonalised update
struct MuonInArgs {
  const void* g;           // bf16 or fp32 [batch, m * n]
  float* momentum;         // fp32 [batch, m * n] or null
  double* sums;            // [batch][blocks]
  unsigned* counts;        // [n_counts] put to zero
  int n_counts;
  void* x;                 // fp16 [batch, m * n]: the update over its norm, times kMuonX
  long count;              // m * n (a multiple of 8)
  int batch, blocks;       // blocks per matrix
  bool g_fp32, nesterov;
  float beta, eps;
};
// Scales of the stored fp16 matrices (65,504 is the largest): singular values of X are
// about 1.2 at most, and 15.9 fit; X X^T holds their squares, so 128 is the most that fits
// where X does (its entries below 2^-21 have fewer bits, off by 2^-32 at most, next to
// the a of P); the polynomial is about 3, and 63.9 fit.
constexpr float kMuonX = 4096.0f, kMuonA = 128.0f, kMuonP = 1024.0f;
int muon_sum_blocks(int batch, long count);
cudaError_t launch_muon_momentum(const MuonInArgs& a, cudaStream_t st);
cudaError_t launch_muon_scale(const MuonInArgs& a, cudaStream_t st);
// Counts lie on lines of their own: many blocks look at one while others add to
// the next.
constexpr int kMuonCountStride = 32;
// All products of an update in one launch (muon.cu).
struct MuonChainArgs {
  // Of each matrix a map for operands with K contiguous and one for K along the rows.
  CUtensorMap x[2][2];     // X in either buffer
  CUtensorMap gram[2], poly[2];
  void* x_out[2];          // fp16 [batch, m, n]
  void* gram_out;          // fp16 [batch, side, ld]
  void* poly_out;
  void* o;                 // bf16 [batch, m, n]
  unsigned* counts;        // [batch][3][tiles_s], zero at the start
  int batch, m, n, side;
  long ld;
  int steps;
  int tiles_s, tiles_o;    // tiles along the shorter side and along the other
  int sym_tiles;           // tiles on and below the diagonal of a symmetric product
  int wide;                // m <= n
  int o_on32;              // rows of o begin on 32 bytes
  unsigned long long wait_ns;
  float coeffs[64][3];
};
struct MuonPlan {
  int ctas;                // blocks on one tile: of 128 x 128, or two on 256 x 256
  int tiles_s, tiles_o, sym_tiles;
  long units;              // tiles of all products of one step, all matrices
};
MuonPlan muon_plan(int batch, int m, int n);
cudaError_t launch_muon_chain(const MuonChainArgs& a, int ctas, long units, cudaStream_t st);
cudaError_t take_muon_status(cudaStream_t st, unsigned* out);
cudaError_t launch_muon_wait_selftest(unsigned long long limit_ns, cudaStream_t st);

unsigned long long current_context_id();

}  // namespace detattn
