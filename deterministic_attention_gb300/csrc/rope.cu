// Rotary positions for sm_103a (RustingBrain vs PyTorch/TensorFlow page, "The
// setup": rotary positions on the queries and keys):
//
//   (a, b) -> m (a cos t theta_i - b sin t theta_i,  b cos t theta_i + a sin t theta_i)
//
// for the pairs i < rot / 2 of every head, (a, b) components (2 i, 2 i + 1) or
// (i, i + rot / 2); components from rot on pass.  sign = -1 turns back.
//
// Angles: theta_i / 2 pi, a double, becomes a 64-bit fixed-point fraction of a
// turn F_i; t F_i in 64-bit integers, which drop whole turns by themselves, is
// the phase to within t 2^-54 turns at any position, and its upper 32 bits go
// to sincospif.  (In fp32 the angle t theta of t = 131072 is off by 2^-8.)
//
// Memory bounds it: every element is read and written once.  A block takes a
// few tokens, forms their cosines and sines once in shared memory for all heads
// of q and k, and then moves 16-byte vectors, kBatch of them loaded before the
// first is stored.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103_ptx.cuh"
#include "step_launch.h"

namespace detattn {
namespace {

constexpr int kThreads = 256, kBatch = 4;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// 16 bytes as floats and back.
template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void get(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void get(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};

// One token's one head: where it is read and written.
template <class T>
struct Head {
  const T* src;
  T* dst;
};
template <class T>
__device__ __forceinline__ Head<T> head_at(const TurnArgs& a, long token, int h) {
  if (h < a.Hq)
    return {static_cast<const T*>(a.q) + token * a.q_ld + static_cast<long>(h) * a.D,
            static_cast<T*>(a.q_out) + token * a.q_out_ld + static_cast<long>(h) * a.D};
  h -= a.Hq;
  return {static_cast<const T*>(a.k) + token * a.k_ld + static_cast<long>(h) * a.D,
          static_cast<T*>(a.k_out) + token * a.k_out_ld + static_cast<long>(h) * a.D};
}

// VEC: rows, heads and halves begin on 16 bytes; else element by element.
template <class T, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kThreads) turn_kernel(const TurnArgs a, int tokens_per_block) {
  extern __shared__ __align__(16) float2 cs[];  // [tokens][rot / 2]: m cos, m sin
  const int half = a.rot / 2;
  const long first = static_cast<long>(blockIdx.x) * tokens_per_block;
  const int here = static_cast<int>(min(static_cast<long>(tokens_per_block), a.tokens - first));
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = a.freqs[i] * 0.15915494309189535;  // 1 / (2 pi)
    // The fraction of a turn in units of 2^-64 (formed in units of 2^-62, which
    // holds every double in [0, 1) and 1 itself).
    const unsigned long long f =
        static_cast<unsigned long long>(__double2ll_rn((turns - floor(turns)) * 4611686018427387904.0)) << 2;
    for (int k = 0; k < here; ++k) {
      const long token = first + k;
      const int t = a.positions != nullptr ? a.positions[token % a.n_pos] : static_cast<int>(token % a.T);
      const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(t)) * f;
      float s, c;
      sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
      cs[k * half + i] = make_float2(c * a.mscale, s * a.mscale * a.sign);
    }
  }
  __syncthreads();
  const int H = a.Hq + a.Hkv;
  if constexpr (VEC) {
    constexpr int n = Vec<T>::n;
    // Items of one head: pieces that turn (halves: two vectors each), then
    // vectors that pass.
    const int turning = INTERLEAVED ? a.rot / n : half / n, per = turning + (a.D - a.rot) / n;
    const int items = here * H * per;
    for (int i0 = threadIdx.x; i0 < items; i0 += kThreads * kBatch) {
      uint4 x[kBatch], y[kBatch];
      Head<T> at[kBatch];
      int piece[kBatch], k[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * kThreads;
        if (i >= items) continue;
        piece[b] = i % per;
        const int th = i / per;
        k[b] = th / H;
        at[b] = head_at<T>(a, first + k[b], th - k[b] * H);
        if (piece[b] < turning) {
          x[b] = *reinterpret_cast<const uint4*>(at[b].src + piece[b] * n);
          if constexpr (!INTERLEAVED) y[b] = *reinterpret_cast<const uint4*>(at[b].src + half + piece[b] * n);
        } else {
          x[b] = *reinterpret_cast<const uint4*>(at[b].src + a.rot + (piece[b] - turning) * n);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (i0 + b * kThreads >= items) continue;
        if (piece[b] >= turning) {
          *reinterpret_cast<uint4*>(at[b].dst + a.rot + (piece[b] - turning) * n) = x[b];
        } else if constexpr (INTERLEAVED) {
          float f[n];
          Vec<T>::get(x[b], f);
          const float2* w = cs + k[b] * half + piece[b] * (n / 2);
#pragma unroll
          for (int j = 0; j < n; j += 2) {
            const float2 t = w[j / 2];
            const float u = f[j], v = f[j + 1];
            f[j] = u * t.x - v * t.y;
            f[j + 1] = v * t.x + u * t.y;
          }
          *reinterpret_cast<uint4*>(at[b].dst + piece[b] * n) = Vec<T>::put(f);
        } else {
          float f[n], g[n];
          Vec<T>::get(x[b], f);
          Vec<T>::get(y[b], g);
          const float2* w = cs + k[b] * half + piece[b] * n;
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const float2 t = w[j];
            const float u = f[j], v = g[j];
            f[j] = u * t.x - v * t.y;
            g[j] = v * t.x + u * t.y;
          }
          *reinterpret_cast<uint4*>(at[b].dst + piece[b] * n) = Vec<T>::put(f);
          *reinterpret_cast<uint4*>(at[b].dst + half + piece[b] * n) = Vec<T>::put(g);
        }
      }
    }
  } else {
    // Items of one head: its pairs, then the components that pass.
    const int per = half + a.D - a.rot;
    const int items = here * H * per;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int piece = i % per, th = i / per, k = th / H;
      const Head<T> at = head_at<T>(a, first + k, th - k * H);
      if (piece < half) {
        const int p0 = INTERLEAVED ? 2 * piece : piece, p1 = INTERLEAVED ? p0 + 1 : piece + half;
        const float2 t = cs[k * half + piece];
        const float u = to_f(at.src[p0]), v = to_f(at.src[p1]);
        from_f(at.dst[p0], u * t.x - v * t.y);
        from_f(at.dst[p1], v * t.x + u * t.y);
      } else {
        const int p = a.rot + piece - half;
        at.dst[p] = at.src[p];
      }
    }
  }
}

template <class T, bool INTERLEAVED>
cudaError_t launch_turn_t(const TurnArgs& a, cudaStream_t st) {
  const int n = 16 / static_cast<int>(sizeof(T)), half = a.rot / 2;
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool vec = on16(a.q) && on16(a.k) && on16(a.q_out) && on16(a.k_out) && a.q_ld % n == 0 &&
                   a.k_ld % n == 0 && a.q_out_ld % n == 0 && a.k_out_ld % n == 0 && a.D % n == 0 &&
                   (INTERLEAVED ? a.rot : half) % n == 0;
  // Tokens of a block: about four vectors a thread, at most 32 KB of cosines
  // and sines, and no fewer than about 600 blocks as long as there are tokens.
  const long per_token = static_cast<long>(a.Hq + a.Hkv) * a.D / n;
  long tb = 4l * kThreads / (per_token > 0 ? per_token : 1);
  const long most = 32768 / (static_cast<long>(half) * sizeof(float2));
  if (tb > a.tokens / 608) tb = a.tokens / 608;
  if (tb > most) tb = most;
  if (tb < 1) tb = 1;
  const long blocks = (a.tokens + tb - 1) / tb;
  const size_t smem = static_cast<size_t>(tb) * half * sizeof(float2);
  if (vec)
    turn_kernel<T, INTERLEAVED, true><<<static_cast<unsigned>(blocks), kThreads, smem, st>>>(a, static_cast<int>(tb));
  else
    turn_kernel<T, INTERLEAVED, false><<<static_cast<unsigned>(blocks), kThreads, smem, st>>>(a, static_cast<int>(tb));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_turn(const TurnArgs& a, cudaStream_t st) {
  if (a.fp32) return a.interleaved ? launch_turn_t<float, true>(a, st) : launch_turn_t<float, false>(a, st);
  return a.interleaved ? launch_turn_t<__nv_bfloat16, true>(a, st) : launch_turn_t<__nv_bfloat16, false>(a, st);
}

}  // namespace detattn
