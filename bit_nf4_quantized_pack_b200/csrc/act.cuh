// Device arithmetic shared by the gated block's kernels and the 8-bit
// activation checkpoints: the activation functions, and the 8-bit codec.
#pragma once

#include <float.h>
#include <stdint.h>

#include "common.cuh"

namespace qnf4 {

// ---------------------------------------------------------------------------
// act(g) = g * s with s = 1 / (1 + exp(-z)):
//   silu         z = g                               act' = s + g s (1 - s)
//   gelu (tanh)  z = 2 sqrt(2/pi) (g + 0.044715 g^3)  act' = s + g s (1 - s) z'
// (0.5 (1 + tanh(y)) = 1 / (1 + exp(-2 y)), which keeps its relative precision
// where the sum 1 + tanh cancels).  The exponential is the hardware's base-2
// one: a relative error below 2^-21 over the range that matters, against the
// 2^-9 of the bf16 result.
// ---------------------------------------------------------------------------
constexpr float kGelu2K = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float kGelu2KC = 0.07135481282679626f;  // 2 sqrt(2/pi) * 0.044715
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x within a unit in the last place (0 for infinity)
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 values an instruction
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float f32x2_lo(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float f32x2_hi(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 1 / (1 + exp(-z))
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + ex2(-z * kLog2E)); }

// act(g) u of two pairs as two bf16, with packed arithmetic: half the
// instructions (the fused epilogue holds up the products while it runs)
__device__ __forceinline__ uint32_t act_mul2(int act, float g0, float g1, float u0, float u1) {
  const uint64_t g = f32x2(g0, g1);
  uint64_t z = mul_f32x2(g, f32x2(-kLog2E, -kLog2E));
  if (act != QLORA_ACT_SILU)
    z = mul_f32x2(z, fma_f32x2(mul_f32x2(g, f32x2(kGelu2KC, kGelu2KC)), g, f32x2(kGelu2K, kGelu2K)));
  const uint64_t d = add_f32x2(f32x2(ex2(f32x2_lo(z)), ex2(f32x2_hi(z))), f32x2(1.0f, 1.0f));
  const uint64_t h = mul_f32x2(mul_f32x2(g, f32x2(rcp(f32x2_lo(d)), rcp(f32x2_hi(d)))), f32x2(u0, u1));
  return pack_bf16x2(f32x2_lo(h), f32x2_hi(h));
}

// act(g), and its derivative in `d`
__device__ __forceinline__ float act_value_grad(int act, float g, float& d) {
  const float g2 = g * g;
  const bool silu = act == QLORA_ACT_SILU;
  const float z = silu ? g : g * fmaf(kGelu2KC, g2, kGelu2K);
  const float dz = silu ? 1.0f : fmaf(3.0f * kGelu2KC, g2, kGelu2K);
  const float s = logistic(z);
  const float a = g * s;
  // 1 - s = 1 / (1 + exp(z)): where it has underflowed a * 0 must stay 0
  // although dz may have overflowed
  const float t = a * (1.0f - s);
  d = t == 0.0f ? s : fmaf(t, dz, s);
  return a;
}

// ---------------------------------------------------------------------------
// 8-bit activation checkpoint: a row is cut into blocks of 64; scale
// s = fl32(amax / 127), or 1 where that is below the normal fp32 range (an
// all-zero block among them); code q = rint(fl32(x / s)), ties to even;
// value = bf16(fl32(q * s)).
// ---------------------------------------------------------------------------
// fl32(amax / 127) for a bf16 amax: the product with the rounded reciprocal and
// one exact remainder (equal to the division for every finite bf16 magnitude
// whose quotient is normal, by enumeration; smaller ones give 1 either way).
__device__ __forceinline__ float act8_scale(float amax) {
  constexpr float r = 1.0f / 127.0f;
  const float q = __fmul_rn(amax, r);
  const float s = __fmaf_rn(__fmaf_rn(-127.0f, q, amax), r, q);
  return s >= FLT_MIN ? s : 1.0f;
}
// a factor for act8_round: 1 / s within two units in the last place (2^-22)
__device__ __forceinline__ float act8_inverse(float s) { return __fdividef(1.0f, s); }

// rint(fl32(x / s)): the product with the inverse, t, and one step with its exact
// remainder, t + (x - t s) / s, give fl32(x / s), and the addition of 1.5 *
// 2^23 rounds that to an integer in the low byte.  (By enumeration of the bf16
// magnitudes of x and of the block's largest, for every inverse within four units
// in the last place of 1 / s.  Below kAct8Tiny the remainder can be subnormal and
// inexact: there the divisions are carried out.)  A test for values near a tie
// with a division for those few was slower: an x and a largest magnitude of 8 bits
// each often meet a tie, 1.4 values in a thousand.  The arithmetic is packed, two
// values an instruction: the codec is bound by the instructions it issues.
constexpr float kAct8Magic = 12582912.0f;
constexpr float kAct8Tiny = 1.0f / (1ull << 50) / (1ull << 50);   // 2^-100
__device__ __forceinline__ uint32_t act8_exact(float x, float s) {
  return __float_as_uint(__fadd_rn(rintf(__fdiv_rn(x, s)), kAct8Magic));
}
// the low bytes of four words
__device__ __forceinline__ uint32_t act8_pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// the codes of 2 n bf16 values, each in the low byte of a word (inv = act8_inverse(s))
template <int n>
__device__ __forceinline__ void act8_round(const uint32_t (&w)[n], float s, float inv, uint32_t (&r)[2 * n]) {
  const uint64_t inv2 = f32x2(inv, inv), minus_s = f32x2(-s, -s), magic2 = f32x2(kAct8Magic, kAct8Magic);
#pragma unroll
  for (int k = 0; k < n; ++k) {
    const uint64_t x = f32x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
    const uint64_t t = mul_f32x2(x, inv2);
    const uint64_t q = add_f32x2(fma_f32x2(fma_f32x2(t, minus_s, x), inv2, t), magic2);
    r[2 * k] = static_cast<uint32_t>(q);
    r[2 * k + 1] = static_cast<uint32_t>(q >> 32);
  }
  if (s < kAct8Tiny) {
#pragma unroll
    for (int k = 0; k < n; ++k) {
      r[2 * k] = act8_exact(__uint_as_float(w[k] << 16), s);
      r[2 * k + 1] = act8_exact(__uint_as_float(w[k] & 0xFFFF0000u), s);
    }
  }
}
// sixteen values' codes
__device__ __forceinline__ uint4 act8_codes16(const uint32_t (&w)[8], float s, float inv) {
  uint32_t r[16];
  act8_round(w, s, inv, r);
  return make_uint4(act8_pack(r[0], r[1], r[2], r[3]), act8_pack(r[4], r[5], r[6], r[7]),
                    act8_pack(r[8], r[9], r[10], r[11]), act8_pack(r[12], r[13], r[14], r[15]));
}

// The values of four codes before their rounding to bf16, fl32(code * s).  A code
// becomes a float through the mantissa (2^23 + 128 + code, less 2^23 + 128: both
// exact), since the conversion instruction runs at a quarter of the rate.
__device__ __forceinline__ void act8_values4(uint32_t codes, float s, float (&v)[4]) {
  const uint32_t u = codes ^ 0x80808080u;
  const uint64_t off = f32x2(-8388736.0f, -8388736.0f), s2 = f32x2(s, s);
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint64_t m = f32x2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540 + 2 * i)),
                             __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541 + 2 * i)));
    const uint64_t x = mul_f32x2(add_f32x2(m, off), s2);
    v[2 * i] = __uint_as_float(static_cast<uint32_t>(x));
    v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(x >> 32));
  }
}

}  // namespace qnf4
