// NVFP4 weights as operands of matrix instructions: the layout in which a wave reads them, their values in bf16 or
// fp16, and the rows they are multiplied with.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace lh {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v4u_a8 __attribute__((ext_vector_type(4), aligned(8)));   // rows are 8-byte aligned
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v2u_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned v4u_a1 __attribute__((ext_vector_type(4), aligned(1)));

enum { kXBf16 = 0, kXF32 = 1, kXE4m3 = 2 };

constexpr int kChunk = 128;                  // elements of k a wave takes at a time

template <int X>
struct Frag {
  using type = b8;
  static constexpr int pieces = 1;
};
template <>
struct Frag<kXF32> {
  using type = b8;
  static constexpr int pieces = 3;
};
template <>
struct Frag<kXE4m3> {
  using type = h8;
  static constexpr int pieces = 1;
};

template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// Eight weights: the nibbles of word w times the E4M3 scale in byte B (0 or 2) of `code`.
template <int X, int B>
__device__ inline typename Frag<X>::type weights(unsigned w, unsigned code) {
  typename Frag<X>::type out;
  if constexpr (X == kXE4m3) {
    const h2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)code, 1.0f, B == 2);
    const h2 s = {s2[0], s2[0]};
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, P) * s;
      out[2 * P] = v[0];
      out[2 * P + 1] = v[1];
    });
  } else {
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)code, B);
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, P);
      const b2 r = __builtin_convertvector((v2f){v[0] * s, v[1] * s}, b2);   // exact
      out[2 * P] = r[0];
      out[2 * P + 1] = r[1];
    });
  }
  return out;
}

// Which elements of a chunk a lane multiplies at step S (8 of the 32 that an instruction takes).  A
// lane loads 32 neighbouring weights, element 8 * (4 * quarter + word).  Their words are exchanged
// between the quarters of the wave so that a load of x covers whole runs of a row, 64 bytes over the
// four quarters, where it would otherwise touch four runs (16 rows of bf16 took 4 times the cycles
// of the vector memory path, 10 us of 20 at 12288x4096):
//   bf16, fp32: both bits of the quarter against both of the word; element 8 * (4 * S + quarter)
//   E4M3: the quarter's high bit against the word's high bit, so a lane's 16 bytes of x are two words:
//         element 64 * (S / 2) + 32 * (quarter % 2) + 16 * (quarter / 2) + 8 * (S % 2)
template <int X>
__device__ inline v4u exchange(v4u w) {
  auto swap32 = [](unsigned& a, unsigned& b) {       // a's upper half of the wave against b's lower half
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  auto swap16 = [](unsigned& a, unsigned& b) {       // a's odd quarters against b's even quarters
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  unsigned n0 = w[0], n1 = w[1], n2 = w[2], n3 = w[3];
  swap32(n0, n2);
  swap32(n1, n3);
  if constexpr (X != kXE4m3) {
    swap16(n0, n1);
    swap16(n2, n3);
  }
  return v4u{n0, n1, n2, n3};
}
// The scale bytes of a lane's words 0, 1 (in bytes 0 and 2 of the first) and 2, 3, from a chunk's 8.
template <int X>
__device__ inline v2u lane_codes(v2u c, int quarter) {
  if constexpr (X == kXE4m3) {                       // words 0, 1 are one block of the first four, 2, 3 of the others
    const int by = 8 * (2 * (quarter & 1) + (quarter >> 1));
    return v2u{c[0] >> by, c[1] >> by};
  } else {                                           // word S is block 2 * S + quarter / 2
    const int by = 8 * (quarter >> 1);
    return v2u{c[0] >> by, c[1] >> by};
  }
}

__device__ inline v4f mfma(b8 a, b8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline v4f mfma(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

}  // namespace
}  // namespace lh
