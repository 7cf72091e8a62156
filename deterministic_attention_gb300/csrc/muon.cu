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
// A and P are symmetric: their tiles on and below the diagonal are computed and
// written twice.  Between the products the matrices are fp16, scaled by powers
// of two (kMuonX, kMuonP): the singular values stay below about 1.2, so fp16's
// eleven bits cost a step 2^-12 of a value where bf16 costs 2^-9, at the same
// rate; five steps leave 1.2e-3 of the result's norm (768 x 768 of normal
// numbers; bf16 9.8e-3).  Sums are fp32 throughout, the norm's in double.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

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
  const size_t base = static_cast<size_t>(blockIdx.y) * a.count;
  const long vecs = a.count / 8;
  double total = 0.0;
  for (long i = static_cast<long>(blockIdx.x) * kInThreads + threadIdx.x; i < vecs;
       i += static_cast<long>(a.blocks) * kInThreads) {
    const size_t at = base + static_cast<size_t>(i) * 8;
    float g[8];
    load8(a, at, g);
    if (a.momentum != nullptr) {
      float m[8];
      load_momentum(a, at, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = fmaf(a.beta, m[j], g[j]);
        g[j] = a.nesterov ? fmaf(a.beta, m[j], g[j]) : m[j];
      }
      float4* p = reinterpret_cast<float4*>(a.momentum + at);
      p[0] = make_float4(m[0], m[1], m[2], m[3]);
      p[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
    Squares sq;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq.add(g[j]);
    total += sq.total();
  }
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
  griddep_launch_dependents();
  griddep_wait();
  double total = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += kInThreads)
    total += a.sums[static_cast<size_t>(blockIdx.y) * a.blocks + i];
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = total;
  __syncthreads();
  total = 0.0;
  for (int i = 0; i < kInThreads / 32; ++i) total += sh[i];
  // In two factors: neither the norm's inverse nor the values overflow.
  const double norm = sqrt(total) + static_cast<double>(a.eps);
  int e = 0;
  const double part = frexp(norm, &e);  // norm = part 2^e
  const float f0 = static_cast<float>(static_cast<double>(kMuonX) / part);
  const int e0 = -e / 2, e1 = -e - e0;
  const float s0 = exp2f(static_cast<float>(e0)), s1 = exp2f(static_cast<float>(e1)) * f0;
  const size_t base = static_cast<size_t>(blockIdx.y) * a.count;
  const long vecs = a.count / 8;
  for (long i = static_cast<long>(blockIdx.x) * kInThreads + threadIdx.x; i < vecs;
       i += static_cast<long>(a.blocks) * kInThreads) {
    const size_t at = base + static_cast<size_t>(i) * 8;
    float g[8];
    if (a.momentum != nullptr && !a.nesterov) {
      load_momentum(a, at, g);
    } else {
      load8(a, at, g);
      if (a.momentum != nullptr) {
        float m[8];
        load_momentum(a, at, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = fmaf(a.beta, m[j], g[j]);
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(g[2 * j] * s0 * s1, g[2 * j + 1] * s0 * s1);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__half*>(a.x) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------ products
template <int CTAS>
struct MuonEpi {
  static constexpr int kCols = 64 * CTAS;
  using Args = MuonStoreArgs;
  const Args& a;
  int row, col;
  bool mirror;
  size_t base, at;
  uint4 add[kCols / 8];
  __device__ __forceinline__ MuonEpi(const Args& args, const product::Unit& w, int r, int c, int)
      : a(args), row(r), col(c), mirror(w.mt != w.nt) {
    base = static_cast<size_t>(w.batch) * args.batch_stride;
    at = base + static_cast<size_t>(row) * a.ld + col;
    // What is added is under way while the tile is computed.
    if (a.add != nullptr) {
      const __half* p = static_cast<const __half*>(a.add) + at;
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i)
        add[i] = row < a.rows && col + 8 * i < a.cols ? *reinterpret_cast<const uint4*>(p + 8 * i)
                                                      : make_uint4(0, 0, 0, 0);
    }
  }
  template <bool LOWER>
  __device__ __forceinline__ void take_as(uint32_t taddr) {
    each32<kCols>(taddr, [&](int c, uint32_t (&v)[32]) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = a.alpha * __uint_as_float(v[2 * i]), y = a.alpha * __uint_as_float(v[2 * i + 1]);
        if (a.add != nullptr) {
          const uint4 q = add[c / 8 + i / 4];
          const uint32_t s = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s));
          x = fmaf(a.beta, f.x, x);
          y = fmaf(a.beta, f.y, y);
          if (row == col + c + 2 * i) x += a.diag;
          if (row == col + c + 2 * i + 1) y += a.diag;
        }
        if (a.bf16) {
          w[i] = pack_bf16x2(x, y);
        } else {
          const __half2 h = __floats2half2_rn(x, y);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      const bool mine = row < a.rows;
      __half* dst = static_cast<__half*>(a.out) + at + c;
      if (mine) {
        if (a.wide && col + c + 32 <= a.cols) {
          store32(dst, w);
          store32(dst + 16, w + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + c + 8 * i < a.cols)
              *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      if (LOWER && mirror) {
        // The tile's transpose: lanes 2 k and 2 k + 1 exchange, so that each has
        // two neighbouring rows of one column (rows of the result are whole
        // vectors: a row past the last is never read).
        const int odd = row & 1;
        __half* to = static_cast<__half*>(a.out) + base + (row & ~1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, w[i], 1);
          const uint32_t two = odd ? __byte_perm(other, w[i], 0x7632) : __byte_perm(w[i], other, 0x5410);
          const int k = col + c + 2 * i + odd;
          if (k < a.rows && (row & ~1) < a.rows)
            *reinterpret_cast<uint32_t*>(to + static_cast<size_t>(k) * a.ld) = two;
        }
      }
    });
  }
};
// All tiles of a result, and those of a symmetric one on and below the
// diagonal, written twice.
template <int CTAS>
struct FullEpi : MuonEpi<CTAS> {
  using MuonEpi<CTAS>::MuonEpi;
  __device__ __forceinline__ void take(uint32_t t) { this->template take_as<false>(t); }
};
template <int CTAS>
struct LowerEpi : MuonEpi<CTAS> {
  using MuonEpi<CTAS>::MuonEpi;
  __device__ __forceinline__ void take(uint32_t t) { this->template take_as<true>(t); }
};

template <int CTAS>
cudaError_t launch_product_t(const CUtensorMap& ma, const CUtensorMap& mb, bool mn_a, bool mn_b,
                             const ProductPlan& p, const MuonStoreArgs& a, cudaStream_t st) {
  using product::launch;
  if (p.lower)
    return mn_a ? launch<CTAS, true, true, true, LowerEpi<CTAS>>(ma, mb, p, a, true, st)
                : launch<CTAS, false, false, true, LowerEpi<CTAS>>(ma, mb, p, a, true, st);
  if (mn_a) return launch<CTAS, true, true, true, FullEpi<CTAS>>(ma, mb, p, a, true, st);
  return mn_b ? launch<CTAS, false, true, true, FullEpi<CTAS>>(ma, mb, p, a, true, st)
              : launch<CTAS, false, false, true, FullEpi<CTAS>>(ma, mb, p, a, true, st);
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
ProductPlan muon_plan(long M, long N, long K, int batch, bool symmetric) {
  ProductPlan best{};
  double least = 0.0;
  for (int form = 0; form < 4; ++form) {
    const int ctas = 1 + (form & 1);
    const bool lower = form >= 2;
    if (lower && !symmetric) continue;
    const ProductPlan p = product_plan(ctas, M, N, K, batch, lower, false);
    // Clocks: rounds of tiles, 512 a step of K for a pair, 256 for a block and a
    // quarter more for its loads, then the last tile's epilogue.
    const long rounds = (p.units + product_teams(ctas) - 1) / product_teams(ctas);
    const double cost = static_cast<double>(rounds) * p.n_k * (ctas == 2 ? 512.0 : 320.0) +
                        ctas * (lower ? 2200.0 : 1600.0);
    if (form == 0 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}
cudaError_t launch_muon_product(const CUtensorMap& ma, const CUtensorMap& mb, bool mn_a, bool mn_b,
                                const ProductPlan& p, const MuonStoreArgs& a, cudaStream_t st) {
  return p.ctas == 2 ? launch_product_t<2>(ma, mb, mn_a, mn_b, p, a, st)
                     : launch_product_t<1>(ma, mb, mn_a, mn_b, p, a, st);
}
cudaError_t take_muon_status(cudaStream_t st, unsigned* out) { return product::take_status(st, out); }
cudaError_t launch_muon_wait_selftest(unsigned long long limit_ns, cudaStream_t st) {
  product::wait_selftest_kernel<<<1, 32, 0, st>>>(limit_ns);
  return cudaGetLastError();
}

}  // namespace detattn
