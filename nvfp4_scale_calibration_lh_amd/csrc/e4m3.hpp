// E4M3 codes of quotients, decided as on the exact quotient: two roundings of an approximate quotient that
// bracket it, and one exact fma where they differ.
#pragma once

#include <hip/hip_runtime.h>

namespace lh {

// The reciprocal and its neighbours that bracket an exact quotient: through the 1-ulp hardware
// reciprocal (and the rounding of 6 g) a quotient is within 2^-21 of the exact one, so what it rounds
// to when pushed up and down by 2^-19 differs only where the exact decision has to be taken.
constexpr float kUp = 1.0000019073486328125f, kDown = 0.9999980926513671875f;

// E4M3 code of a / (6 s) between codes lo and lo + 1: the sign of 6 m s - a (m their midpoint, so 6 m
// has at most 7 significant bits) is exact in one fma; a tie goes to the even code.
__device__ inline unsigned e4m3_resolve6(float a, float s, unsigned lo) {
  const float x = __builtin_amdgcn_cvt_f32_fp8((int)lo, 0), y = __builtin_amdgcn_cvt_f32_fp8((int)lo + 1, 0);
  const float d = fmaf(3.0f * (x + y), s, -a);
  return d < 0.0f ? lo + 1 : (d > 0.0f ? lo : lo + (lo & 1));
}

// Four signed E4M3 bytes of x / s, saturating; s in [2^-100, 2^100], `is` its hardware reciprocal.
__device__ inline unsigned e4m3_word(const float* x, float s, float is) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float iu = is * kUp, id = is * kDown;
  auto pack = [&](float f) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __builtin_amdgcn_fmed3f(x[k] * f, -448.0f, 448.0f);
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
  };
  const unsigned up = pack(iu), dn = pack(id);
  unsigned out = up;
  if (up != dn) {
    // The sign of m s - |x|, m the midpoint of the two codes, is exact in one fma; where they are one code either
    // choice is that.  At a tie the even code: d < 2^-149 is d <= 0 (d is a multiple of it).  Without branches and
    // byte by byte, so that the code stays short: one row of the norm 3.1 us, 3.4 with a branch for each element.
    const v2f u[2] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)up, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)up, true)};
    const v2f n[2] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)dn, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)dn, true)};
    out = dn;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = fmaf(fabsf(u[k / 2][k % 2] + n[k / 2][k % 2]), 0.5f * s, -fabsf(x[k]));
      const float least = __uint_as_float((~up >> (8 * k)) & 1u);
      const unsigned byte = 255u << (8 * k);
      out = d < least ? (out & ~byte) | (up & byte) : out;
    }
  }
  return out;
}

}  // namespace lh
