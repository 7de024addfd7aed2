// int8 codes of a row of fp32 values.
//
// The quotient: 127 / m is held as a rounded value and its remainder, so that
// p hi + p lo, rounded once, is the quotient's own rounding to fp32.  Adding
// 1.5 * 2^23 then rounds it to a whole number, ties to even.
//   - p and m with significands of 16 bits (bf16 rows, times a bf16 weight or
//     none): a quotient q that is not halfway is at least q / (254 * 65535) from
//     it, more than the 2^-24 q that a rounding moves it, and a tie is an fp32
//     value itself, so the codes are right as they are.
//   - fp32 rows or weights: a value within 2^-16 of a half is settled by the
//     sign of 127 |p| - h m, h the half.  Both products are taken as a rounded
//     value and its exact remainder, the values' difference is exact (they are
//     within a factor of 2), and so is the remainders' (at most 508 units of
//     the smaller operand's last place), so the sign is the exact one.
#pragma once

#include "q4_api_internal.h"
#include "q4_common.cuh"

namespace q4 {

// What a row's reduction gives every thread of it.
struct RowScale {
  float rstd;   // 1 without a norm
  float scale;  // the row's scale
  float up;     // a power of two that brings m near 1 where 127 / m or 127 m could leave fp32's range
  float m;      // max |p| * up
  float inv;    // 127 / m rounded, 0 for a row of zeros
  float low;    // what its rounding left
  bool bad;     // a value is not finite, or the squares' sum is not
};

__device__ __forceinline__ RowScale row_scale(float m, float sum, bool norm, int H, float eps) {
  RowScale s;
  s.bad = !(m < INFINITY) || (norm && !(sum < INFINITY));
  s.rstd = norm ? rsqrtf(sum / (float)H + eps) : 1.0f;
  s.scale = norm ? m * s.rstd / 127.0f : m / 127.0f;
  s.up = m < 0x1p-60f && m > 0.0f ? 0x1p100f : (m > 0x1p60f ? 0x1p-100f : 1.0f);
  s.m = m * s.up;
  s.inv = s.m > 0.0f ? 127.0f / s.m : 0.0f;
  s.low = s.m > 0.0f ? fmaf(-s.inv, s.m, 127.0f) / s.m : 0.0f;
  if (s.bad) {
    s.rstd = __uint_as_float(0x7fc00000u);
    s.scale = s.rstd;
    s.inv = s.low = 0.0f;
  }
  return s;
}

// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
  return d;
}

// Two fp32 operations an instruction (each rounded as the single one is).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d.v) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void split(F2 d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d.v));
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

// The rounding of 127 p / m where r, the quotient rounded to fp32, is within
// 2^-16 of a half (see above).
__device__ __forceinline__ float near_half(float p, float r, float m) {
  const float a = fabsf(p), lo = floorf(fabsf(r)), h = lo + 0.5f;
  const float pa = 127.0f * a, pb = h * m;
  const float d = (pa - pb) + (fmaf(127.0f, a, -pa) - fmaf(h, m, -pb));
  const float odd = lo - 2.0f * floorf(0.5f * lo);
  return copysignf(lo + (d > 0.0f ? 1.0f : (d < 0.0f ? 0.0f : odd)), p);
}

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even

// The codes of p as the low bytes of c.
template <int VEC>
__device__ __forceinline__ void codes(const float p[VEC], const RowScale& s, bool exact, uint32_t c[VEC]) {
  float r[VEC], t[VEC];
  if constexpr (VEC == 8) {
    const F2 inv = f2(s.inv, s.inv), low = f2(s.low, s.low), up = f2(kRound, kRound);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const F2 pp = f2(p[i], p[i + 1]), rr = fma(pp, inv, mul(pp, low));
      split(rr, r[i], r[i + 1]);
      split(add(rr, up), t[i], t[i + 1]);
    }
  } else {
    r[0] = fmaf(p[0], s.inv, p[0] * s.low);
    t[0] = r[0] + kRound;
  }
  if (!exact) {
    constexpr float kFar = 0.5f - 0x1p-16f;
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) far = fmaxf(far, fabsf(r[i] - (t[i] - kRound)));
    if (far > kFar) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (fabsf(r[i] - (t[i] - kRound)) > kFar) t[i] = near_half(p[i], r[i], s.m) + kRound;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) c[i] = __float_as_uint(t[i]);
}

// p as it stands in registers, brought near 1 (rarely) or to zeros (a bad row).
template <int VEC>
__device__ __forceinline__ void ready(float p[VEC], const RowScale& s) {
  if (s.bad || s.up != 1.0f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = s.bad ? 0.0f : p[i] * s.up;
  }
}

// Eight codes as two words.
__device__ __forceinline__ uint2 pack_codes(const uint32_t c[8]) {
  return make_uint2(prmt(prmt(c[0], c[1], 0x0040), prmt(c[2], c[3], 0x0040), 0x5410),
                    prmt(prmt(c[4], c[5], 0x0040), prmt(c[6], c[7], 0x0040), 0x5410));
}

__device__ __forceinline__ float warp_max(float m) {
  // magnitudes compare as their bits do, a NaN above infinity
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

// 8 bf16 values.
__device__ __forceinline__ void unpack(uint4 a, float v[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

}  // namespace q4
