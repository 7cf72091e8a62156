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
// of q and k while its first vectors are under way, and then moves 16-byte
// vectors, the next loaded before the last is stored.  32 + 8 heads of 128 over
// 65,536 positions: 209 us, 6.4 TB/s, 94 % of the copy rate (two vectors a thread at
// once 232 us, four 261: fewer blocks fit an SM; one round of vectors a block 239).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103_ptx.cuh"
#include "step_launch.h"

namespace detattn {
namespace {

constexpr int kThreads = 256, kMaxPairs = 512;
// Items of a thread in a block, about.
constexpr int kRounds = 4;

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
  __shared__ unsigned long long turn[kMaxPairs];
  const int half = a.rot / 2;
  const long first = static_cast<long>(blockIdx.x) * tokens_per_block;
  const int here = static_cast<int>(min(static_cast<long>(tokens_per_block), a.tokens - first));
  const int H = a.Hq + a.Hkv;
  // The fraction of a turn per position in units of 2^-64 (formed in units of
  // 2^-62, which hold every double in [0, 1) and 1 itself).
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = a.freqs[i] * 0.15915494309189535;  // 1 / (2 pi)
    turn[i] = static_cast<unsigned long long>(__double2ll_rn((turns - floor(turns)) * 4611686018427387904.0)) << 2;
  }
  auto table = [&]() {
    __syncthreads();
    for (int idx = threadIdx.x; idx < here * half; idx += kThreads) {
      const int k = idx / half;
      const long token = first + k;
      const int t = a.positions != nullptr ? a.positions[token % a.n_pos] : static_cast<int>(token % a.T);
      const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(t)) * turn[idx - k * half];
      float s, c;
      sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
      cs[idx] = make_float2(c * a.mscale, s * a.mscale * a.sign);
    }
    __syncthreads();
  };
  if constexpr (VEC) {
    constexpr int n = Vec<T>::n;
    // Items of one head: pieces that turn (halves: two vectors each), then
    // vectors that pass.
    const int turning = INTERLEAVED ? a.rot / n : half / n, per = turning + (a.D - a.rot) / n;
    const int items = here * H * per;
    uint4 x = {}, y = {};
    T* dst = nullptr;
    int cs_at = 0;  // -1: the vector passes
    auto load = [&](int i) {
      if (i >= items) return;
      const int piece = i % per, th = i / per, k = th / H;
      const Head<T> at = head_at<T>(a, first + k, th - k * H);
      const bool turns = piece < turning;
      const int from = turns ? piece * n : a.rot + (piece - turning) * n;
      dst = at.dst + from;
      cs_at = turns ? k * half + piece * (INTERLEAVED ? n / 2 : n) : -1;
      x = __ldcs(reinterpret_cast<const uint4*>(at.src + from));
      if constexpr (!INTERLEAVED)
        if (turns) y = __ldcs(reinterpret_cast<const uint4*>(at.src + half + from));
    };
    // The first vectors are under way while the table is formed.
    load(threadIdx.x);
    table();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      T* const to = dst;
      const int at = cs_at;
      const uint4 px = x, py = y;
      load(i + kThreads);
      if (at < 0) {
        __stcs(reinterpret_cast<uint4*>(to), px);
        continue;
      }
      const float4* w = reinterpret_cast<const float4*>(cs + at);
      float f[n];
      Vec<T>::get(px, f);
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < n; j += 4) {
          const float4 t = w[j / 4];
          const float u0 = f[j], v0 = f[j + 1], u1 = f[j + 2], v1 = f[j + 3];
          f[j] = u0 * t.x - v0 * t.y;
          f[j + 1] = v0 * t.x + u0 * t.y;
          f[j + 2] = u1 * t.z - v1 * t.w;
          f[j + 3] = v1 * t.z + u1 * t.w;
        }
      } else {
        float g[n];
        Vec<T>::get(py, g);
#pragma unroll
        for (int j = 0; j < n; j += 2) {
          const float4 t = w[j / 2];
          const float u0 = f[j], v0 = g[j], u1 = f[j + 1], v1 = g[j + 1];
          f[j] = u0 * t.x - v0 * t.y;
          g[j] = v0 * t.x + u0 * t.y;
          f[j + 1] = u1 * t.z - v1 * t.w;
          g[j + 1] = v1 * t.z + u1 * t.w;
        }
        __stcs(reinterpret_cast<uint4*>(to + half), Vec<T>::put(g));
      }
      __stcs(reinterpret_cast<uint4*>(to), Vec<T>::put(f));
    }
  } else {
    // Items of one head: its pairs, then the components that pass.
    const int per = half + a.D - a.rot;
    const int items = here * H * per;
    table();
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
  // Tokens of a block: about kRounds items a thread, at most 32 KB of cosines and
  // sines, and no fewer than about 600 blocks as long as there are tokens.
  const long per_token = static_cast<long>(a.Hq + a.Hkv) * a.D / (INTERLEAVED ? n : 2 * n);
  const long most = 32768 / (static_cast<long>(half) * sizeof(float2));
  long tb = kRounds * kThreads / (per_token > 0 ? per_token : 1);
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
