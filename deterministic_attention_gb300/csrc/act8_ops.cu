// Activation checkpoints in 8 bits (made and read back) and the gated unit
// h = silu(a) b with its checkpoint, for sm_103a.
//
// RustingBrain vs PyTorch/TensorFlow page, "The setup": the model's
// feed-forward layer is SwiGLU.  Its input u = [a | b] is the largest
// activation a layer keeps for the backward; in 8 bits it takes 2.06 bytes an
// element pair instead of 4, and the backward returns h again, so that the
// next projection's weight gradient needs nothing else.
//
// All four kernels stream: each value is read once with 16-byte loads (8-byte
// ones for checkpoints) and written once, and memory bounds them.  A thread
// holds eight consecutive columns and an aligned quad of lanes one group of
// 32, so a group's largest magnitude takes two shuffles.  Measured: a round
// trip of 8192 x 4096 (203 MB) in 32 us, the gated unit's backward at 32768 x
// 4096 from 8 bits (1.35 GB) in 193 us, 7.0 TB/s (part of what the pass before
// left is still in L2).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act8.cuh"
#include "block_launch.h"

namespace detattn {

namespace {

constexpr int kThreads = 256;

// Pack: kPackVecs vectors of eight values per thread, all loaded before the
// first is used.
constexpr int kPackVecs = 2;
__global__ void __launch_bounds__(kThreads)
    act8_pack_kernel(const uint4* __restrict__ x, uint2* __restrict__ q, uint8_t* __restrict__ e,
                     long n_vec) {
  const long v0 = static_cast<long>(blockIdx.x) * (kThreads * kPackVecs) + threadIdx.x;
  uint4 raw[kPackVecs];
#pragma unroll
  for (int j = 0; j < kPackVecs; ++j)
    raw[j] = v0 + j * kThreads < n_vec ? x[v0 + j * kThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int j = 0; j < kPackVecs; ++j) {
    const long v = v0 + j * kThreads;
    float f[8];
    uint2 out;
    bf16x8_to_float(raw[j], f);
    const uint32_t ex = act8_quantise8(f, 1.0f, &out);
    if (v < n_vec) {
      q[v] = out;
      if ((v & 3) == 0) e[v >> 2] = static_cast<uint8_t>(ex);
    }
  }
}

// Unpack: likewise, kUnpackVecs vectors of eight per thread.  (Sixteen values
// per thread, loaded as one 16-byte word, leave a warp's stores 32 bytes
// apart: 8192 x 4096 took 18.1 us against 13.2.)
constexpr int kUnpackVecs = 4;
__global__ void __launch_bounds__(kThreads)
    act8_unpack_kernel(const uint2* __restrict__ q, const uint8_t* __restrict__ e,
                       uint4* __restrict__ x, long n_vec) {
  const long v0 = static_cast<long>(blockIdx.x) * (kThreads * kUnpackVecs) + threadIdx.x;
  uint2 raw[kUnpackVecs];
  uint32_t ex[kUnpackVecs];
#pragma unroll
  for (int j = 0; j < kUnpackVecs; ++j) {
    const long v = v0 + j * kThreads;
    if (v < n_vec) {
      raw[j] = q[v];
      ex[j] = e[v >> 2];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnpackVecs; ++j) {
    const long v = v0 + j * kThreads;
    if (v < n_vec) {
      Vec8 f;
      f.from_int8(raw[j]);
      f.scale(act8_scale(ex[j]));
      x[v] = f.to_bf16();
    }
  }
}

// sigma(a) = f^2 r and 1 - sigma(a), by w = exp(-|a| / 2) and r = 1 / (1 + w^2):
// f is 1 for a >= 0 and w below.  sigma is applied as two factors f, one to
// each factor of a product: a sigma(a) b with a at -90 or -150 and a large b is
// an ordinary number, though sigma(a) alone is below 2^-126.  (w is zero from
// a = -174 on, where h is below 2^-115 for every bf16 b.)  Powers and quotients
// are the special-function unit's, within 2^-22 and 2^-23, and the exponent's
// rounding is left in, |a| 2^-24: all far below half a step of the bf16 stores.
struct Logistic {
  float f, r, rest;  // rest: 1 - sigma
  __device__ __forceinline__ explicit Logistic(float a) {
    const float w = ex2_approx(-0.72134752f * fabsf(a));
    r = rcp_approx(fmaf(w, w, 1.0f));
    f = a < 0.0f ? w : 1.0f;
    rest = a < 0.0f ? r : w * w * r;
  }
};

template <bool KEEP8>
__global__ void __launch_bounds__(kThreads)
    swiglu_fwd_kernel(const uint4* __restrict__ u, uint4* __restrict__ h, uint2* __restrict__ q,
                      uint8_t* __restrict__ e, unsigned n_vec, unsigned f8) {
  const unsigned v = blockIdx.x * kThreads + threadIdx.x;
  const bool in = v < n_vec;
  const unsigned row = (in ? v : 0u) / f8, col = (in ? v : 0u) - row * f8;
  const size_t ia = static_cast<size_t>(row) * (2 * f8) + col, ib = ia + f8;
  const uint4 ra = u[ia], rb = u[ib];
  float a[8], b[8], o[8];
  bf16x8_to_float(ra, a);
  bf16x8_to_float(rb, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Logistic s(a[i]);
    o[i] = (a[i] * s.f) * (b[i] * s.f) * s.r;
  }
  if (in) h[v] = float_to_bf16x8(o);
  if constexpr (KEEP8) {
    uint2 qa, qb;
    const uint32_t ea = act8_quantise8(a, 1.0f, &qa), eb = act8_quantise8(b, 1.0f, &qb);
    if (in) {
      q[ia] = qa;
      q[ib] = qb;
      if ((v & 3) == 0) {
        e[ia >> 2] = static_cast<uint8_t>(ea);
        e[ib >> 2] = static_cast<uint8_t>(eb);
      }
    }
  }
}

// da = dh b s (1 + a (1 - s)), db = dh a s with s = sigma(a).
template <bool FROM8, bool WITH_H>
__global__ void __launch_bounds__(kThreads, 8)
    swiglu_bwd_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ u,
                      const uint2* __restrict__ q, const uint8_t* __restrict__ e,
                      uint4* __restrict__ du, uint4* __restrict__ h, unsigned n_vec, unsigned f8) {
  const unsigned v = blockIdx.x * kThreads + threadIdx.x;
  if (v >= n_vec) return;
  const unsigned row = v / f8, col = v - row * f8;
  const size_t ia = static_cast<size_t>(row) * (2 * f8) + col, ib = ia + f8;
  Vec8 va, vb;
  float g[8], a[8], b[8], da[8], db[8], o[8];
  const uint4 rg = dh[v];
  if constexpr (FROM8) {
    const uint2 qa = q[ia], qb = q[ib];
    const float sa = act8_scale(e[ia >> 2]), sb = act8_scale(e[ib >> 2]);
    va.from_int8(qa);
    vb.from_int8(qb);
    va.scale(sa);
    vb.scale(sb);
    va.to_float(a);
    vb.to_float(b);
  } else {
    const uint4 ra = u[ia], rb = u[ib];
    bf16x8_to_float(ra, a);
    bf16x8_to_float(rb, b);
  }
  bf16x8_to_float(rg, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Logistic s(a[i]);
    const float as = a[i] * s.f * s.r, bs = b[i] * s.f, gs = g[i] * s.f;
    da[i] = gs * (bs * s.r) * fmaf(a[i], s.rest, 1.0f);
    db[i] = gs * as;
    o[i] = as * bs;
  }
  du[ia] = float_to_bf16x8(da);
  du[ib] = float_to_bf16x8(db);
  if constexpr (WITH_H) h[v] = float_to_bf16x8(o);
}

unsigned blocks_of(long n, long per_block) { return static_cast<unsigned>((n + per_block - 1) / per_block); }

}  // namespace

cudaError_t launch_act8_pack(const void* x, int8_t* q, uint8_t* e, long rows, int d,
                             cudaStream_t st) {
  const long n_vec = rows * (d / 8);
  act8_pack_kernel<<<blocks_of(n_vec, kThreads * kPackVecs), kThreads, 0, st>>>(
      static_cast<const uint4*>(x), reinterpret_cast<uint2*>(q), e, n_vec);
  return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const int8_t* q, const uint8_t* e, void* x, long rows, int d,
                               cudaStream_t st) {
  const long n_vec = rows * (d / 8);
  act8_unpack_kernel<<<blocks_of(n_vec, kThreads * kUnpackVecs), kThreads, 0, st>>>(
      reinterpret_cast<const uint2*>(q), e, static_cast<uint4*>(x), n_vec);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_fwd(const void* u, void* h, int8_t* q, uint8_t* e, long rows, int f,
                              cudaStream_t st) {
  const unsigned f8 = static_cast<unsigned>(f / 8), n_vec = static_cast<unsigned>(rows * f8);
  const unsigned grid = blocks_of(n_vec, kThreads);
  if (q != nullptr)
    swiglu_fwd_kernel<true><<<grid, kThreads, 0, st>>>(static_cast<const uint4*>(u),
                                                       static_cast<uint4*>(h),
                                                       reinterpret_cast<uint2*>(q), e, n_vec, f8);
  else
    swiglu_fwd_kernel<false><<<grid, kThreads, 0, st>>>(
        static_cast<const uint4*>(u), static_cast<uint4*>(h), nullptr, nullptr, n_vec, f8);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const void* dh, const void* u, const int8_t* q, const uint8_t* e,
                              void* du, void* h, long rows, int f, cudaStream_t st) {
  const unsigned f8 = static_cast<unsigned>(f / 8), n_vec = static_cast<unsigned>(rows * f8);
  const unsigned grid = blocks_of(n_vec, kThreads);
  const auto* g = static_cast<const uint4*>(dh);
  const auto* uu = static_cast<const uint4*>(u);
  const auto* qq = reinterpret_cast<const uint2*>(q);
  auto* o = static_cast<uint4*>(du);
  auto* hh = static_cast<uint4*>(h);
  if (u == nullptr) {
    if (h != nullptr)
      swiglu_bwd_kernel<true, true><<<grid, kThreads, 0, st>>>(g, uu, qq, e, o, hh, n_vec, f8);
    else
      swiglu_bwd_kernel<true, false><<<grid, kThreads, 0, st>>>(g, uu, qq, e, o, hh, n_vec, f8);
  } else {
    if (h != nullptr)
      swiglu_bwd_kernel<false, true><<<grid, kThreads, 0, st>>>(g, uu, qq, e, o, hh, n_vec, f8);
    else
      swiglu_bwd_kernel<false, false><<<grid, kThreads, 0, st>>>(g, uu, qq, e, o, hh, n_vec, f8);
  }
  return cudaGetLastError();
}

}  // namespace detattn
