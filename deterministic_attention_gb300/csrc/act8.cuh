// The 8-bit checkpoint format on the device: int8 values with one power-of-two
// exponent for every 32 consecutive columns of a row.
//
// For a group whose largest magnitude is m, the exponent is the smallest k
// with m <= 127 2^k, and a value x is stored as q = x 2^-k rounded to the
// nearest whole number (ties to even).  A power of two makes both directions
// exact but for that one rounding: x 2^-k is exact in fp32, and q 2^k has at
// most 7 significant bits, so it is a bf16 number and a tensor core can take
// it as it is.  The rounding is off by at most 2^(k-1), m / 127 at worst.
// (int8 with a shared exponent rather than e4m3: for the near-normal values
// of a norm its error is about a third of e4m3's 2^-4 steps.)
#pragma once
#include <cstdint>

#include "exp2_poly.cuh"
#include "block_ptx.cuh"

namespace detattn {

// Bits of |x|: ordered like the magnitudes, with infinity and every NaN on top
// (a floating-point maximum would drop a NaN).
__device__ __forceinline__ uint32_t act8_abs_bits(float x) {
  return __float_as_uint(x) & 0x7FFFFFFFu;
}

// Exponent byte of a group with largest magnitude bits m.  With m = f 2^E, f
// in [1, 2): m <= 127 2^k needs k = E - 6 when f <= 127 / 64, else E - 5.
// Kept at 1 (k = -126) from below: what is smaller rounds to multiples of
// 2^-126.
__device__ __forceinline__ uint32_t act8_exponent(uint32_t m) {
  if (m >= 0x7F800000u) return 255u;
  const int e = static_cast<int>(m >> 23) - 6 + ((m & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return static_cast<uint32_t>(e > 1 ? e : 1);
}

// Eight values v times `mult` >= 0 of one lane; the four lanes of an aligned
// quad hold one group.  Returns the exponent byte and writes the eight int8
// values.  Every lane of the warp takes part.  (v mult 2^-k is rounded once,
// to a whole number: 2^-k mult is exact.)
__device__ __forceinline__ uint32_t act8_quantise8(const float (&v)[8], float mult, uint2* q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, act8_abs_bits(v[i]));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t e = act8_exponent(act8_abs_bits(__uint_as_float(m) * mult));
  if (e == 255u) {
    *q = make_uint2(0u, 0u);
    return e;
  }
  // x 2^-k + 1.5 2^23: the sum's low byte is the rounded value in two's
  // complement.
  const float inv = __uint_as_float((254u - e) << 23);
  float r[8];
  uint32_t b[8];
  if (e >= 64u && mult < 0x1p60f) {
    const float k = inv * mult;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fmaf(v[i], k, 12582912.0f);
  } else {
    // Groups of (near) zeros, where 2^-k mult may pass the largest float.
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fmaf(v[i] * mult, inv, 12582912.0f);
  }
  // k = 122: 64 2^122 would be infinity, so what rounds there stays at 63.
  if (e == 249u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fminf(fmaxf(r[i], 12582912.0f - 63.0f), 12582912.0f + 63.0f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(r[i]);
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  *q = make_uint2(lo, hi);
  return e;
}

// 2^(e - 127); infinity for e = 255, whose group holds zeros: 0 * inf is NaN.
__device__ __forceinline__ float act8_scale(uint32_t e) { return __uint_as_float(e << 23); }

// ------------------------------------------------------------ eight values as four pairs
// The norms' arithmetic runs on f32x2 instructions: two results an issue slot.
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_all(float x) { return f2_make(x, x); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {  // a NaN stays one
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n\tmin.NaN.f32 %0, %0, %3;" : "=&f"(d) : "f"(x), "f"(lo), "f"(hi));
  return d;
}
struct Vec8 {
  uint64_t p[4];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2_all(x);
  }
  __device__ __forceinline__ void from_bf16(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = f2_make(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void from_f32(const void* at) {
    const ulonglong2* q = static_cast<const ulonglong2*>(at);
    const ulonglong2 a = q[0], b = q[1];
    p[0] = a.x;
    p[1] = a.y;
    p[2] = b.x;
    p[3] = b.y;
  }
  // The whole numbers of eight int8 bytes: byte + 128 in the low bits of 2^23's
  // mantissa, less 2^23 + 128.
  __device__ __forceinline__ void from_int8(uint2 q) {
    const uint32_t u[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
    const uint64_t off = f2_all(-8388736.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = f2_add(f2_make(__uint_as_float(__byte_perm(u[i >> 1], 0x4B000000u, i & 1 ? 0x7442 : 0x7440)),
                            __uint_as_float(__byte_perm(u[i >> 1], 0x4B000000u, i & 1 ? 0x7443 : 0x7441))),
                    off);
  }
  __device__ __forceinline__ void to_float(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(p[i], f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void mul(const Vec8& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2_mul(p[i], b.p[i]);
  }
  __device__ __forceinline__ void scale(float x) {
    const uint64_t k = f2_all(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2_mul(p[i], k);
  }
  // Adds the squares to a pair of sums.
  __device__ __forceinline__ void squares(uint64_t& sum) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = f2_fma(p[i], p[i], sum);
  }
  // Logistic function 1 / (1 + t), t = 2^(-x log2 e).  What rounding -x log2 e
  // to p loses, |x| 2^-24 of t, is put back with the product's remainder d:
  // t = 2^p (1 - d ln 2).  With the power (2^-22) and the quotient (two units
  // in the last place) sigma is within 11 2^-24 of its value at any x.  x is
  // kept in [-88, 128]: t stays finite, and a quotient below 2^-126 is given
  // as 0.  `more` of every pair: its t.
  template <class More>
  __device__ __forceinline__ void logistic(More more) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2_split(p[i], a, b);
      const uint64_t x = f2_make(clamp_nan(a, -88.0f, 128.0f), clamp_nan(b, -88.0f, 128.0f));
      const uint64_t e = f2_mul(x, f2_all(-1.44269502f));
      // log2 e = 1.44269502 (as rounded) + 1.92596303e-8
      const uint64_t d = f2_fma(x, f2_all(1.92596303e-8f), f2_fma(x, f2_all(1.44269502f), e));
      f2_split(e, a, b);
      const uint64_t t0 = f2_make(ex2_approx(a), ex2_approx(b));
      const uint64_t t = f2_fma(f2_mul(t0, f2_all(-0.693147181f)), d, t0);
      f2_split(f2_add(t, f2_all(1.0f)), a, b);
      p[i] = f2_make(__fdividef(1.0f, a), __fdividef(1.0f, b));
      more(i, t);
    }
  }
  __device__ __forceinline__ void sigmoid() {
    logistic([](int, uint64_t) {});
  }
  // And its slope, t sigma^2: 1 - sigma = t sigma keeps its digits however
  // large x is, where sigma - sigma^2 from a sigma rounded next to 1 has lost
  // them all at x = 17.
  __device__ __forceinline__ void sigmoid(Vec8& slope) {
    logistic([&](int i, uint64_t t) { slope.p[i] = f2_mul(f2_mul(t, p[i]), p[i]); });
  }
  __device__ __forceinline__ uint4 to_bf16() const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      f2_split(p[i], lo, hi);
      w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void to_f32(void* at) const {
    ulonglong2* q = static_cast<ulonglong2*>(at);
    q[0] = make_ulonglong2(p[0], p[1]);
    q[1] = make_ulonglong2(p[2], p[3]);
  }
};

// Eight separate values.
__device__ __forceinline__ void bf16x8_to_float(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 float_to_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

}  // namespace detattn
