// RoPE angles shared by the rotation kernels: inv_freq_i in fp64 from the host
// (theta^(-2i/D), or a caller's table such as a context-extension one) and the same
// frequencies as 64-bit fractions of a turn, from which the angle phi = p * inv_freq_i
// is reduced exactly in integer arithmetic before sin and cos are taken in fp32 (at
// p ~ 1.3e5 an fp32 product would already be off by ~1e-2 rad; fp64 arithmetic runs at
// a small fraction of the fp32 rate on this GPU).
#pragma once

#include <math.h>

namespace decattn {

struct InvFreq {
  double v[64];  // i = 0 .. D/2 - 1
};

// 2*pi split into a double head and the double nearest the remainder.
constexpr double kTwoPiHi = 6.283185307179586;
constexpr double kTwoPiLo = 2.4492935982947064e-16;
constexpr double kInvTwoPi = 0.15915494309189535;

// A rotated K element again, in fp64, for the rare element whose fp32 result cancels:
// own and other are the exact pre-rotation values of this element and its pair partner
// (the raw bf16 value, or its product with a bf16 norm weight, which fp32 holds
// exactly), rstd the head's QK-norm scale (1 without it). The first element of a pair
// becomes own cos - other sin, the second own cos + other sin. The fp32 path's error is a
// few 2^-24 of |own| + |other|; when the result is smaller than about 2^-12 of that,
// the error would exceed half a bf16 ulp of the result, and this path keeps the stored
// bf16 within one ulp of the exact rotation. (fp64 runs at a small fraction of the fp32
// rate here, so only those elements take it.)
__device__ __noinline__ inline float rope_exact(int p, double inv_freq, float own, float other,
                                                float rstd, bool second) {
  const double phi = (double)p * inv_freq;
  const double k = rint(phi * kInvTwoPi);
  double r = fma(-k, kTwoPiHi, phi);
  r = fma(-k, kTwoPiLo, r);
  double s, c;
  sincos(r, &s, &c);
  const double o = second ? (double)other : -(double)other;
  return (float)(fma((double)own, c, o * s) * (double)rstd);
}

// The same from the pair's frequency as a fraction of a turn (RopeTurns below): p * turns
// modulo 2^64 is the angle's fractional turn, its nearest quarter turn goes off exactly in
// integers, and the Taylor series of sine and cosine run to x^15 and x^16 at |x| <= pi / 4 (the
// next terms are below 5e-17). About 25 fp64 operations where a general sincos takes hundreds.
__device__ __noinline__ inline float rope_exact_turns(int p, unsigned long long turns, float own,
                                                      float other, float rstd, bool second) {
  const unsigned long long t = (unsigned long long)(unsigned)p * turns;
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);
  const double x = (double)(long long)(t - ((unsigned long long)quarter << 62)) *
                   (kTwoPiHi * 0x1p-64);
  const double z = x * x;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = fma(s, z, 1.0 / 6227020800.0);
  c = fma(c, z, -1.0 / 87178291200.0);
  s = fma(s, z, -1.0 / 39916800.0);
  c = fma(c, z, 1.0 / 479001600.0);
  s = fma(s, z, 1.0 / 362880.0);
  c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, -1.0 / 5040.0);
  c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 120.0);
  c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, -1.0 / 6.0);
  c = fma(c, z, 1.0 / 24.0);
  c = fma(c, z, -0.5);
  s = fma(s * z, x, x);
  c = fma(c, z, 1.0);
  double cs = quarter & 1 ? -s : c, sn = quarter & 1 ? c : s;
  if (quarter & 2) cs = -cs, sn = -sn;
  const double o = second ? (double)other : -(double)other;
  return (float)(fma((double)own, cs, o * sn) * (double)rstd);
}

// A rotated pair in fp32 with its roundings spelled out. Left to the compiler, which product of a
// sum is fused with it differs from kernel to kernel, and with it the last bit of one result in
// some 1e5. The rotating kernels that promise each other's bits form the pair here.
__device__ __forceinline__ float rope_first(float a, float b, float c, float s) {  // a c - b s
  return fmaf(a, c, -__fmul_rn(b, s));
}
// a s + b c. The interleaved layout at D = 64 rounds a s first, the others b c.
template <bool kRoundsA>
__device__ __forceinline__ float rope_second(float a, float b, float c, float s) {
  return kRoundsA ? fmaf(b, c, __fmul_rn(a, s)) : fmaf(a, s, __fmul_rn(b, c));
}

// Whether a fp32 rotation result y of a pair whose normalised values have magnitudes
// a and b cancels enough to be formed again by rope_exact.
__device__ __forceinline__ bool rope_cancels(float y, float a, float b) {
  return fabsf(y) < 0x1p-11f * (fabsf(a) + fabsf(b));
}

// Host: the plain table theta^(-2i/D) for head_dim D.
InvFreq make_inv_freq(int D, double theta);

// The angles without fp64 arithmetic on the device. turns_i = inv_freq_i / (2 pi) as a
// 64-bit binary fraction (units of 2^-64 of a turn), rounded on the host; then p * turns_i computed
// modulo 2^64 is the angle's fractional turn exactly (the whole turns fall off the top),
// and its top 32 bits, read as a signed integer, give radians in [-pi, pi) after the
// rounding to fp32 (the angle is within 2^-32 of a turn plus that rounding).
struct RopeTurns {
  unsigned long long v[64];
};
// Any finite inv_freq_i >= 0: whole turns per position fall off like the others.
RopeTurns make_rope_turns(int D, const InvFreq &inv);

__device__ __forceinline__ void rope_sincos_turns(int p, unsigned long long turns, float &s,
                                                  float &c) {
  const unsigned long long t = (unsigned long long)(unsigned)p * turns;
  const int hi = (int)(t >> 32);
  const float r = (float)hi * 1.4629180792671596e-09f;  // 2 pi / 2^32
  sincosf(r, &s, &c);
}

}  // namespace decattn
