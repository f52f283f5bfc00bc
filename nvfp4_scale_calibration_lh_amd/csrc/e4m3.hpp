// E4M3 codes of quotients, decided as on the exact quotient: two roundings of an approximate quotient that
// bracket it, and one exact fma where they differ.
#pragma once

#include <hip/hip_runtime.h>

namespace lh {

// The reciprocal and its neighbours that bracket an exact quotient: through the 1-ulp hardware
// reciprocal (and the rounding of 6 g) a quotient is within 2^-21 of the exact one, so what it rounds
// to when pushed up and down by 2^-19 differs only where the exact decision has to be taken.
constexpr float kUp = 1.0000019073486328125f, kDown = 0.9999980926513671875f;

// E4M3 code of a / (f s) between codes lo and lo + 1: the sign of f m s - a (m their midpoint, so f m
// has at most 7 significant bits for f = 1 or 6) is exact in one fma; a tie goes to the even code.
template <int F>
__device__ inline unsigned e4m3_resolve(float a, float s, unsigned lo) {
  const float x = __builtin_amdgcn_cvt_f32_fp8((int)lo, 0), y = __builtin_amdgcn_cvt_f32_fp8((int)lo + 1, 0);
  const float d = fmaf(0.5f * F * (x + y), s, -a);
  return d < 0.0f ? lo + 1 : (d > 0.0f ? lo : lo + (lo & 1));
}

// Four signed E4M3 bytes of x / s, saturating; s in [2^-100, 2^100], `is` its hardware reciprocal.
__device__ inline unsigned e4m3_word(const float* x, float s, float is) {
  const float iu = is * kUp, id = is * kDown;
  auto pack = [&](float f) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = fminf(fmaxf(x[k] * f, -448.0f), 448.0f);
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
  };
  unsigned up = pack(iu);
  const unsigned dn = pack(id);
  if (up != dn) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned cu = (up >> (8 * k)) & 127u, cd = (dn >> (8 * k)) & 127u;
      if (cu != cd) up = (up & ~(127u << (8 * k))) | (e4m3_resolve<1>(fabsf(x[k]), s, cd) << (8 * k));
    }
  }
  return up;
}

}  // namespace lh
