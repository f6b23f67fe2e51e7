// 8-bit codes of the paged cache: rounding on the way in, exact conversions on
// the way out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "paged_ptx.cuh"

namespace tsa {

// Code kinds of a cache as template arguments.
constexpr int kPlain = 0, kI8 = 1, kE4M3 = 2;

template <int CODE>
__device__ __forceinline__ constexpr float code_max() {
  return CODE == kI8 ? 127.f : 448.f;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// |x| M / a for a row whose largest magnitude is a > 0, rounded so that rounding
// it once more to the code's grid gives what the exact quotient would.  r: 1 / a,
// off by a few units in the last place at most.
//
// The quotient is the product with r and one correction by its remainder
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  The product is off by some 2^-22 of the quotient, the
// remainder is exact, and its product with r off by 2^-22 again: a quotient that
// fp32 holds, so every tie of a grid of at most 8 bits, comes out exact, and any
// other within fp32's rounding.  With 8-bit significands (bf16 rows) no other
// quotient lies within 2^-16 of a border between two codes, so this decides
// every case.  fp32 rows can come closer: next to a border b the sign of
// x M - b a decides.  Both products are known exactly there: x M as its rounded
// value and the remainder of the rounding, and x M - b a because b has at most
// 8 bits and the two agree in at least 12.
// x, a: scaled by the row's power of two so that no product over- or underflows.
template <int CODE, bool WIDE>
__device__ __forceinline__ float code_quotient(float x, float a, float r) {
  constexpr float M = code_max<CODE>();
  const float p = x * M;
  const float t0 = p * r;
  float t = fmaf(fmaf(-t0, a, p), r, t0);
  if (WIDE) {
    float b;
    bool close;
    if (CODE == kI8) {
      b = floorf(t) + 0.5f;
      close = fabsf(t - b) < 1e-4f;
    } else if (t < 0.015625f) {  // below 2^-6 the grid is 2^-9
      b = (floorf(t * 512.f) + 0.5f) * 0.001953125f;
      close = fabsf(t - b) < 1e-7f;
    } else {
      const uint32_t u = __float_as_uint(t);
      b = __uint_as_float((u & 0xFFF00000u) | 0x00080000u);
      close = (u & 0xFFFFFu) - 0x7FFF0u <= 0x20u;
    }
    if (close) {
      const float s = fmaf(-b, a, p) + fmaf(x, M, -p);
      const uint32_t ub = __float_as_uint(b);
      t = s > 0.f ? __uint_as_float(ub + 1) : s < 0.f ? __uint_as_float(ub - 1) : b;
    }
  }
  return t;
}

// (a & b) | c in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// The same for two elements at once, signs included (a zero keeps its own).
template <int CODE>
__device__ __forceinline__ void code_quotients(float& x, float& y, float a, float r) {
  using namespace tc;
  const uint64_t nr = f2_pack(-r, -r);
  const uint64_t np = f2_mul(f2_pack(x, y), f2_pack(-code_max<CODE>(), -code_max<CODE>()));
  const uint64_t t0 = f2_mul(np, nr);
  f2_unpack(f2_fma(f2_fma(t0, f2_pack(a, a), np), nr, t0), x, y);
}

// Two bytes of `w` (at bits 0-7 and 16-23; the rest is ignored) as int8 -> bf16x2.
// With the low seven bits in the mantissa of 128 .. 255, code + 128 (or + 256
// where the sign is set) is a bf16 number, and the difference is exact.
__device__ __forceinline__ uint32_t i8_pair(uint32_t w) {
  const uint32_t a = and_or(w, 0x007f007fu, 0x43004300u);  // 128 + low bits
  const uint32_t b = and_or(w, 0x00800080u, 0xC300C300u);  // -128, or -256 for a negative code
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0x3F803F80u), "r"(b));
  return r;
}
// Two bytes at bits 8-15 and 24-31 as e4m3 -> bf16x2: the fields shifted into
// place give the value times 2^-120 (bias 127 against 7), subnormals included.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
  const uint32_t r = and_or(w, 0x80008000u, (w >> 4) & 0x07f007f0u);
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(r), "r"(0x7B807B80u), "r"(0x80008000u));  // times 2^120
  return y;
}

// bf16x2 of the codes in bytes 0 and 2, and in bytes 1 and 3.
template <int CODE>
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  return CODE == kI8 ? i8_pair(w) : e4m3_pair(w << 8);
}
template <int CODE>
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  return CODE == kI8 ? i8_pair(w >> 8) : e4m3_pair(w);
}
// bf16x2 of the codes in bytes i and i + 1 of w (i = 0 or 2).
template <int CODE, int I>
__device__ __forceinline__ uint32_t codes_next(uint32_t w) {
  if (CODE == kI8) return i8_pair(__byte_perm(w, 0, I == 0 ? 0x4140 : 0x4342));
  return e4m3_pair(__byte_perm(w, 0, I == 0 ? 0x1404 : 0x3424));
}
// f16x2 of byte B of w0 and byte B of w1 in units of 2^code_f16_unit, exact for both kinds.  int8 words have been through
// codes_unsigned: with the offset code u = code + 128 in the mantissa of 1024 .. 2047, u + 1024 is an
// f16 number, and the difference to 1152 exact.  e4m3: the fields shifted into place give the value in units of
// 2^8 (bias 15 against 7), subnormals included.  The conversion instruction is shorter but makes a NaN of the codes
// 0x7f and 0xff, which count as +-480 here as everywhere else.
template <int CODE>
__device__ __forceinline__ constexpr float code_f16_unit() {
  return CODE == kI8 ? 0.f : 8.f;
}
template <int CODE>
__device__ __forceinline__ uint32_t codes_unsigned(uint32_t w) {
  return CODE == kI8 ? w ^ 0x80808080u : w;
}
template <int CODE, int B>
__device__ __forceinline__ uint32_t codes_across_f16(uint32_t w0, uint32_t w1) {
  uint32_t r;
  if (CODE == kI8) {
    const uint32_t w = and_or(__byte_perm(w0, w1, (uint32_t)B | ((uint32_t)(B + 4) << 8)), 0x00ff00ffu, 0x64006400u);
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xE480E480u));
  } else {
    constexpr uint32_t sel = (uint32_t)B | ((uint32_t)B << 4) | ((uint32_t)(B + 4) << 8) | ((uint32_t)(B + 4) << 12);
    const uint32_t w = __byte_perm(w0, w1, sel);
    r = and_or(w, 0x80008000u, (w << 7) & 0x3f803f80u);
  }
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace tsa
