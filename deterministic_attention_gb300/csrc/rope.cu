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
// the phase to within t 2^-54 turns at any position (theta_i up to 1; two roundings
// of theta_i / 2 pi), and its upper 32 bits go to sincospif.  (In fp32 the angle t theta of t = 131072 is off by 2^-8.)
//
// Memory bounds it: every element is read and written once.  A block takes a
// few tokens, forms their cosines and sines once in shared memory for all heads
// of q and k while its first vectors are under way, and then moves 16-byte
// vectors, the next loaded before the last is stored.  32 + 8 heads of 128 over
// 65,536 positions: 196 us, 6.8 TB/s, the copy rate.  (Four rounds of vectors a
// block 200 us, two 231; without that order of loads 209; two vectors a thread at
// once 232, four 261: fewer blocks fit an SM; the table before the first load 363.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103_ptx.cuh"
#include "step_launch.h"

namespace detattn {
namespace {

constexpr int kThreads = 256, kMaxPairs = 512;
// Items of a thread in a block, about.
constexpr int kRounds = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// N elements (16, 8 or 4 bytes) as floats and back.
template <int BYTES>
struct Words;
template <>
struct Words<16> {
  using type = uint4;
};
template <>
struct Words<8> {
  using type = uint2;
};
template <>
struct Words<4> {
  using type = unsigned int;
};
template <class T, int N>
struct Vec {
  using Raw = typename Words<N * static_cast<int>(sizeof(T))>::type;
  static constexpr int kWords = static_cast<int>(sizeof(Raw)) / 4;
  static __device__ __forceinline__ void get(const Raw& v, float (&f)[N]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
  }
  static __device__ __forceinline__ Raw put(const float (&f)[N]) {
    Raw v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(f[i]);
      else
        w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
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

// Vectors of N elements, with which rows, heads and halves begin; N = 1: element
// by element.
template <class T, bool INTERLEAVED, int N>
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
      // (Tokens are at most 2^30.)
      const unsigned at = static_cast<unsigned>(token);
      const int t = a.positions != nullptr ? a.positions[at % static_cast<unsigned>(a.n_pos)]
                                           : static_cast<int>(at % static_cast<unsigned>(a.T));
      const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(t)) * turn[idx - k * half];
      float s, c;
      sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
      cs[idx] = make_float2(c * a.mscale, s * a.mscale * a.sign);
    }
    __syncthreads();
  };
  if constexpr (N > 1) {
    using V = Vec<T, N>;
    using Raw = typename V::Raw;
    // Items of one head: pieces that turn (halves: two vectors each), then
    // vectors that pass.
    const int turning = INTERLEAVED ? a.rot / N : half / N, per = turning + (a.D - a.rot) / N;
    const int items = here * H * per;
    Raw x = {}, y = {};
    T* dst = nullptr;
    int cs_at = 0;  // -1: the vector passes
    auto load = [&](int i) {
      if (i >= items) return;
      const int piece = i % per, th = i / per, k = th / H;
      const Head<T> at = head_at<T>(a, first + k, th - k * H);
      const bool turns = piece < turning;
      const int from = turns ? piece * N : a.rot + (piece - turning) * N;
      dst = at.dst + from;
      cs_at = turns ? k * half + piece * (INTERLEAVED ? N / 2 : N) : -1;
      x = __ldcs(reinterpret_cast<const Raw*>(at.src + from));
      if constexpr (!INTERLEAVED)
        if (turns) y = __ldcs(reinterpret_cast<const Raw*>(at.src + half + from));
    };
    // The first vectors are under way while the table is formed.
    load(threadIdx.x);
    table();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      T* const to = dst;
      const int at = cs_at;
      const Raw px = x, py = y;
      load(i + kThreads);
      if (at < 0) {
        __stcs(reinterpret_cast<Raw*>(to), px);
        continue;
      }
      // The table's entries: two at a time where a vector has an even number.
      constexpr int kPairs = INTERLEAVED ? N / 2 : N;
      float2 w[kPairs];
      if constexpr (kPairs % 2 == 0) {
#pragma unroll
        for (int j = 0; j < kPairs; j += 2) {
          const float4 t = reinterpret_cast<const float4*>(cs + at)[j / 2];
          w[j] = make_float2(t.x, t.y);
          w[j + 1] = make_float2(t.z, t.w);
        }
      } else {
        w[0] = cs[at];
      }
      float f[N];
      V::get(px, f);
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float u = f[2 * j], v = f[2 * j + 1];
          f[2 * j] = u * w[j].x - v * w[j].y;
          f[2 * j + 1] = v * w[j].x + u * w[j].y;
        }
      } else {
        float g[N];
        V::get(py, g);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float u = f[j], v = g[j];
          f[j] = u * w[j].x - v * w[j].y;
          g[j] = v * w[j].x + u * w[j].y;
        }
        __stcs(reinterpret_cast<Raw*>(to + half), V::put(g));
      }
      __stcs(reinterpret_cast<Raw*>(to), V::put(f));
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

template <class T, bool INTERLEAVED, int N>
cudaError_t launch_turn_n(const TurnArgs& a, cudaStream_t st) {
  const int half = a.rot / 2;
  // Tokens of a block: about kRounds items a thread, at most 32 KB of cosines and
  // sines, and no fewer than about 600 blocks as long as there are tokens.
  const long per_token = static_cast<long>(a.Hq + a.Hkv) * a.D / (INTERLEAVED ? N : 2 * N);
  const long most = 32768 / (static_cast<long>(half) * sizeof(float2));
  long tb = kRounds * kThreads / (per_token > 0 ? per_token : 1);
  if (tb > a.tokens / 608) tb = a.tokens / 608;
  if (tb > most) tb = most;
  if (tb < 1) tb = 1;
  const long blocks = (a.tokens + tb - 1) / tb;
  const size_t smem = static_cast<size_t>(tb) * half * sizeof(float2);
  turn_kernel<T, INTERLEAVED, N><<<static_cast<unsigned>(blocks), kThreads, smem, st>>>(a, static_cast<int>(tb));
  return cudaGetLastError();
}

// The widest vectors that everything begins with: 16 bytes as a rule; 8 or 4 for
// halves or heads that are no multiples of them (20 fp32 heads of 80 with 20
// components turned, 16,384 tokens: 64 us a call with 8 bytes, 103 element by element).
template <class T, bool INTERLEAVED>
cudaError_t launch_turn_t(const TurnArgs& a, cudaStream_t st) {
  const long unit = INTERLEAVED ? a.rot : a.rot / 2;
  auto fits = [&](int n) {
    const uintptr_t bytes = n * sizeof(T);
    for (const void* p : {a.q, a.k, static_cast<const void*>(a.q_out), static_cast<const void*>(a.k_out)})
      if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
    for (long v : {a.q_ld, a.k_ld, a.q_out_ld, a.k_out_ld, static_cast<long>(a.D), unit})
      if (v % n != 0) return false;
    return true;
  };
  constexpr int kMost = 16 / static_cast<int>(sizeof(T));
  if (fits(kMost)) return launch_turn_n<T, INTERLEAVED, kMost>(a, st);
  if (fits(kMost / 2)) return launch_turn_n<T, INTERLEAVED, kMost / 2>(a, st);
  if constexpr (kMost == 8)
    if (fits(2)) return launch_turn_n<T, INTERLEAVED, 2>(a, st);
  return launch_turn_n<T, INTERLEAVED, 1>(a, st);
}

}  // namespace

cudaError_t launch_turn(const TurnArgs& a, cudaStream_t st) {
  if (a.fp32) return a.interleaved ? launch_turn_t<float, true>(a, st) : launch_turn_t<float, false>(a, st);
  return a.interleaved ? launch_turn_t<__nv_bfloat16, true>(a, st) : launch_turn_t<__nv_bfloat16, false>(a, st);
}

}  // namespace detattn
