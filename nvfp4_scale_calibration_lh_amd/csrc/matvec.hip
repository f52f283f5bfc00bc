// Products of a few rows with NVFP4 weights as the scale sweep leaves them, dense or per expert:
//   Y[t, c] = g * sum_k E2M1(nibble[c, k]) * E4M3(code[c, k / 16]) * x[t, k],
//   g = fp32(amax / (6 * norm)), for the rows t of each group against that group's matrix;
//   x is bf16, fp32, or E4M3 bytes times a scale per row or per 128 channels of a row.
//
// Bound by reading the weights once (0.5625 bytes each), so the layout is the one they are stored
// in: a lane reads 16 bytes (32 elements, two blocks) of one output channel, 16 channels by 128
// elements a wave, as the A operand of 16x16x32 matrix instructions whose columns are the rows of x
// (in the same order of k, which a dot product does not mind).  The waves of a workgroup take 128
// elements of k in turn and add their sums in LDS in a fixed order.
//
// E2M1 * E4M3 has at most 6 significant bits, so it is exact in bf16 (bf16 and fp32 x) and, its
// range being [2^-10, 2688], in fp16 (E4M3 x, also exact in fp16).  fp32 x is split exactly into
// three bf16 pieces.  Every product is exact; sums are fp32.
#include "lh_internal.hpp"

#include <algorithm>

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

constexpr int kChunk = 128;                  // elements of k a wave takes at a time
constexpr int kMaxWaves = 16;

enum { kXBf16 = 0, kXF32 = 1, kXE4m3 = 2 };

struct Args {
  const void* x;
  const float* x_scale;
  const uint8_t* code;
  const uint8_t* fp4;
  const float* amax;
  const int64_t* offsets;
  void* y;
  int64_t rows, n_groups;
  int cout, cin, x_scales;                   // x_scales: scales of one row (1, or cin / 128 rounded up)
  float gdiv;
};

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
__device__ inline void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// Eight weights: the nibbles of word w times the E4M3 scale in byte B of `code`.
template <int X, int B>
__device__ inline typename Frag<X>::type weights(unsigned w, unsigned code) {
  typename Frag<X>::type out;
  if constexpr (X == kXE4m3) {
    const h2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)code, 1.0f, false);
    const h2 s = {s2[B], s2[B]};
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

// The 32 elements of x a lane holds of one chunk, as loaded.
template <int X>
struct Raw {
  v4u v[X == kXF32 ? 8 : (X == kXBf16 ? 4 : 2)];
};
template <int X>
__device__ inline void load_x(Raw<X>& r, const void* row, int k, int n) {   // n of the 32 exist (0, 16 or 32)
  constexpr int per = X == kXF32 ? 4 : (X == kXBf16 ? 8 : 16);              // elements of 16 bytes
  const v4u* p = (const v4u*)((const uint8_t*)row + (int64_t)k * (16 / per));
#pragma unroll
  for (int j = 0; j < 32 / per; ++j) r.v[j] = j * per < n ? p[j] : v4u{0, 0, 0, 0};
}
// Step S (8 elements) of it as matrix operands.
template <int X, int S>
__device__ inline void frag_x(const Raw<X>& r, typename Frag<X>::type* f) {
  if constexpr (X == kXBf16) {
    f[0] = __builtin_bit_cast(b8, r.v[S]);
  } else if constexpr (X == kXE4m3) {
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.v[S / 2][2 * (S % 2) + P / 2], 1.0f, P % 2 == 1);
      f[0][2 * P] = v[0];
      f[0][2 * P + 1] = v[1];
    });
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {                    // truncated pieces: 8 + 8 + 8 bits
      const float x = __uint_as_float(r.v[2 * S + e / 4][e % 4]);
      const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
      const float r1 = x - hi;
      const float mid = __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
      f[0][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(hi) >> 16));
      f[1][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(mid) >> 16));
      f[2][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(r1 - mid) >> 16));
    }
  }
}

__device__ inline v4f mfma(b8 a, b8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline v4f mfma(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// The piece-th run of at most `tile` rows of one group, over all groups in order: its group and
// rows, or group -1 past the last.  Every thread of the workgroup calls it.
struct Piece {
  int64_t group, row, rows;
};
__device__ inline Piece find_piece(const Args& a, int64_t piece, int tile) {
  if (a.n_groups == 1) {
    const int64_t row = piece * tile;
    return {row < a.rows ? 0 : -1, row, min((int64_t)tile, a.rows - row)};
  }
  __shared__ int64_t sums[kMaxWaves];
  __shared__ Piece found;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if (threadIdx.x == 0) found = {-1, 0, 0};
  int64_t before = 0;                                // pieces of the groups before this round's
  for (int64_t g0 = 0; g0 < a.n_groups; g0 += blockDim.x) {
    const int64_t g = g0 + threadIdx.x;
    int64_t lo = 0, n = 0;
    if (g < a.n_groups) {
      lo = min(max(a.offsets[g], (int64_t)0), a.rows);
      n = min(a.offsets[g + 1], a.rows) - lo;
    }
    const int64_t mine = n > 0 ? (n + tile - 1) / tile : 0;
    int64_t upto = mine;                             // inclusive scan over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    __syncthreads();                                 // the last round's sums have been read
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int64_t first = before + upto - mine;
    for (int w = 0; w < waves; ++w) {
      if (w < wave) first += sums[w];
      before += sums[w];
    }
    if (piece >= first && piece < first + mine) {
      const int64_t at = (piece - first) * tile;
      found = {g, lo + at, min((int64_t)tile, n - at)};
    }
    if (before > piece) break;                       // the same for every thread
  }
  __syncthreads();
  return found;
}

// X: type of x.  MT: 16-row tiles of x a workgroup takes.  NT: 16-channel tiles of the output a
// workgroup takes.  Workgroups count the channel tiles of one piece of rows, then the next piece's.
template <int X, int MT, int NT>
__global__ __launch_bounds__(1024) void k_matvec(const Args a) {
  constexpr int kPieces = Frag<X>::pieces;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = lane & 15, quarter = lane >> 4;
  const unsigned tiles = (unsigned)(a.cout + 16 * NT - 1) / (16 * NT);
  const Piece pc = find_piece(a, blockIdx.x / tiles, 16 * MT);
  if (pc.group < 0) return;
  const int c0 = (int)(blockIdx.x % tiles) * (16 * NT);

  const uint8_t* w[NT];
  const uint8_t* codes[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {                     // channels past the last repeat it; not stored
    const int64_t c = pc.group * a.cout + min(c0 + 16 * n + i, a.cout - 1);
    w[n] = a.fp4 + c * (a.cin / 2) + quarter * 16;
    codes[n] = a.code + c * (a.cin / 16) + quarter * 2;
  }
  constexpr int kSize = X == kXF32 ? 4 : (X == kXBf16 ? 2 : 1);
  const uint8_t* x[MT];
  const float* xs[MT];
  bool has[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    has[m] = 16 * m + i < pc.rows;
    const int64_t r = pc.row + (has[m] ? 16 * m + i : 0);
    x[m] = (const uint8_t*)a.x + r * a.cin * kSize;
    xs[m] = X == kXE4m3 ? a.x_scale + r * a.x_scales : nullptr;
  }
  v4f acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0, 0, 0, 0};

  for (int kb = wave * kChunk; kb < a.cin; kb += waves * kChunk) {
    const int k = kb + quarter * 32;
    const int left = a.cin - k;                      // a multiple of 16
    v4u nib[NT];
    unsigned cd[NT];
    if (left >= 32) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        nib[n] = *(const v4u_a8*)(w[n] + kb / 2);
        const uint8_t* p = codes[n] + kb / 16;
        cd[n] = p[0] | (unsigned)p[1] << 8;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        nib[n] = v4u{0, 0, 0, 0};
        cd[n] = 0;
        if (left == 16) {
          const v2u v = *(const v2u*)(w[n] + kb / 2);
          nib[n][0] = v[0], nib[n][1] = v[1];
          cd[n] = codes[n][kb / 16];
        }
      }
    }
    Raw<X> raw[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) load_x<X>(raw[m], x[m], k, has[m] ? max(min(left, 32), 0) : 0);
    v4f part[NT][MT];
    if constexpr (X == kXE4m3) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[n][m] = v4f{0, 0, 0, 0};
    }
    auto& sum = *(X == kXE4m3 ? &part : &acc);
    each<4>([&](auto st) {
      constexpr int S = decltype(st)::value;
      typename Frag<X>::type fx[MT][kPieces];
#pragma unroll
      for (int m = 0; m < MT; ++m) frag_x<X, S>(raw[m], fx[m]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const auto fw = weights<X, S / 2>(nib[n][S], cd[n]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < kPieces; ++p) sum[n][m] = mfma(fw, fx[m][p], sum[n][m]);
      }
    });
    if constexpr (X == kXE4m3) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float s = has[m] ? xs[m][a.x_scales > 1 ? kb / kChunk : 0] : 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][m] += s * part[n][m];
      }
    }
  }

  // the waves' sums, in their order: lane holds channels 4*quarter + r of row i
  extern __shared__ float red[];
  float* mine = red + wave * (NT * MT * 256) + lane;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) mine[((n * MT + m) * 4 + r) * 64] = acc[n][m][r];
  __syncthreads();
  const float g = a.amax[pc.group] / a.gdiv;
  for (int e = threadIdx.x; e < NT * MT * 256; e += blockDim.x) {
    const int n = e / (MT * 256), m = e / 256 % MT, row = 16 * m + (e / 16) % 16, c = e % 16;
    const int at = (n * MT + m) * 256 + (c % 4) * 64 + (c / 4) * 16 + row % 16;
    float s = 0.0f;
    for (int v = 0; v < waves; ++v) s += red[v * (NT * MT * 256) + at];
    const int channel = c0 + 16 * n + c;
    if (row >= pc.rows || channel >= a.cout) continue;
    const int64_t to = (pc.row + row) * a.cout + channel;
    if constexpr (X == kXF32)
      ((float*)a.y)[to] = s * g;
    else
      ((__bf16*)a.y)[to] = (__bf16)(s * g);
  }
}

template <int X, int MT, int NT>
void launch_tile(const Args& a, int waves, hipStream_t stream) {
  const int tile = 16 * MT;
  const int64_t pieces = a.n_groups == 1 ? (a.rows + tile - 1) / tile : a.rows / tile + std::min(a.n_groups, a.rows);
  const dim3 grid((unsigned)(pieces * ((a.cout + 16 * NT - 1) / (16 * NT))));
  hipLaunchKernelGGL((k_matvec<X, MT, NT>), grid, dim3(64 * waves), (size_t)waves * NT * MT * 1024, stream, a);
}

template <int X>
void launch_x(const Args& a, hipStream_t stream) {
  const int chunks = (a.cin + kChunk - 1) / kChunk;
  const int waves = chunks >= 8 ? 8 : (chunks >= 4 ? 4 : (chunks >= 2 ? 2 : 1));
  if (a.n_groups > 1 || a.rows <= 16) launch_tile<X, 1, 1>(a, waves, stream);
  else if (a.rows <= 32) launch_tile<X, 2, 1>(a, waves, stream);
  else launch_tile<X, 4, 1>(a, std::min(waves, 8), stream);
}

}  // namespace

hipError_t launch_matvec(const void* x, int x_type, const float* x_scale, int64_t x_scales, int64_t rows, int64_t cin,
                         int64_t cout, const int64_t* offsets, int64_t n_groups, const uint8_t* code, const uint8_t* fp4,
                         const float* amax, float gdiv, void* y, hipStream_t stream) {
  Args a{};
  a.x = x;
  a.x_scale = x_scale;
  a.code = code;
  a.fp4 = fp4;
  a.amax = amax;
  a.offsets = offsets;
  a.y = y;
  a.rows = rows;
  a.n_groups = n_groups;
  a.cout = (int)cout;
  a.cin = (int)cin;
  a.x_scales = (int)x_scales;
  a.gdiv = gdiv;
  if (x_type == kXBf16) launch_x<kXBf16>(a, stream);
  else if (x_type == kXF32) launch_x<kXF32>(a, stream);
  else launch_x<kXE4m3>(a, stream);
  return hipGetLastError();
}

}  // namespace lh
