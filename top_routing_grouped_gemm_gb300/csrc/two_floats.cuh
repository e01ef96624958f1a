// Numbers as unevaluated sums of two floats, hi + lo with |lo| at most half a step of hi (T. J. Dekker,
// "A Floating-Point Technique for Extending the Available Precision", 1971), for the order of nearly
// equal routing scores.  Its operations are plain fp32 ones; 64-bit floating point runs at a
// sixty-fourth of their rate on this GPU.  (The intrinsics are never contracted into fused products.)
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {

struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
// |a| >= |b| (or a = 0)
__device__ __forceinline__ Two quick_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Two u = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
  return quick_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p)));
  return quick_sum(p, e);
}
__device__ __forceinline__ Two operator/(Two a, Two b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const float r = __fadd_rn(__fmaf_rn(-q, b.hi, a.hi), __fmaf_rn(-q, b.lo, a.lo));
  return quick_sum(q, __fdiv_rn(r, b.hi));
}

// 2^(j / 32), from its definition in 60 digits.
__device__ const Two kPowers[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f},
    {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f},
    {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b550p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f},
    {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f},
    {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246eb0p-26f},
};

// exp(x), x <= 0, to about 2^-45 of it (0 below -87): a table of 2^(j/32) and a short polynomial of
// the rest, as P. T. P. Tang, "Table-Driven Implementation of the Exponential Function in IEEE
// Floating-Point Arithmetic", 1989, does it in 64 bits.  With n = x 32 / ln 2 rounded and
// r = x - n ln 2 / 32, |r| < 0.011: r + r^2 / 2 as two floats, and r^3 / 6 + ... < 2^-22 as one.
__device__ __forceinline__ Two two_exp(Two x) {
  if (!(x.hi >= -87.f)) return {0.f, 0.f};
  const float n = rintf(__fmul_rn(x.hi, 46.16624f));
  // ln 2 / 32 in three parts; the first has 11 bits, so n times it is exact
  const float r0 = __fmaf_rn(-n, 0x1.63p-6f, x.hi);
  const float p = __fmul_rn(n, -0x1.bd0106p-18f);
  const float p_lo = __fmaf_rn(n, -0x1.bd0106p-18f, -p);
  Two r = two_sum(r0, -p);
  r = quick_sum(r.hi, __fadd_rn(__fsub_rn(r.lo, p_lo), __fmaf_rn(-n, 0x1.cf79acp-45f, x.lo)));
  const Two half_square = Two{0.5f * r.hi, 0.5f * r.lo} * r;
  const float h = r.hi;
  const float rest = h * h * h * fmaf(h, fmaf(h, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
  Two e = quick_sum(r.hi, half_square.hi);
  e = quick_sum(e.hi, __fadd_rn(e.lo, __fadd_rn(__fadd_rn(r.lo, half_square.lo), rest)));
  const Two one = quick_sum(1.f, e.hi);
  e = quick_sum(one.hi, __fadd_rn(one.lo, e.lo));
  const int i = static_cast<int>(n);
  e = e * kPowers[i & 31];
  const float scale = __int_as_float(((i >> 5) + 127) << 23);  // i >> 5 >= -126
  return {e.hi * scale, e.lo * scale};
}

// A 64-bit key in the numbers' order.  What is not a number comes with -inf.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint64_t two_key(Two v) {
  if (v.hi != v.hi) v.hi = -INFINITY;
  if (isinf(v.hi)) v.lo = 0.f;
  return static_cast<uint64_t>(ordered_bits(v.hi)) << 32 | ordered_bits(v.lo);
}

}  // namespace moe
