// Root-mean-square norm of a residual stream, with the residual's addition and an E4M3 output:
//   h = round(x + r) in the input type (h = x without r),  y = h / sqrt(mean h^2 + eps) * gamma,
//   per row or per 128 channels of it: s = max|y| * fp32(1/448), q = E4M3 nearest to the exact y / s, ties to
//   the even code.
//
// HBM-bound: a row is read once and kept in registers between its two reductions (the sum of
// squares, then the largest |y|), so the kernel moves the input, h, q and the scales once.  A row
// belongs to TPR threads; unit j * TPR + t (16 bytes) belongs to thread t, so loads and stores are
// contiguous over a wave and the 128 channels of a scale are 16 (bf16) or 32 (fp32) neighbouring
// lanes.  A row of up to 128 units takes one wave and no barrier: 8192 rows of 512 bf16 8.3 us against
// 13.3 for a workgroup a row, of 128 5.0 against 10.8.  8192 x 4096 bf16 with the residual: 39.3 us, 6.0 TB/s
// (a 2 GiB copy runs at 4.9 TB/s; part of this working set stays in the memory-side cache), without it 23 us, fp32
// with it 76; one row of 4096 3.1 us, the floor of a launch and 0.2 for exact codes.  Sums are fp32.  The only roundings to fewer bits are h (the carried residual has the
// input's type, and the norm is of what is carried) and q.
#include "e4m3.hpp"
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kThreads = 256;
constexpr float kInv448 = 1.0f / 448.0f;
constexpr int kGroup = 128;           // channels of one scale where a row has several
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

struct Args {
  const v4u* x;
  const v4u* r;
  const v4u* gamma;
  v4u* h;
  uint8_t* q;
  float* s;
  int64_t rows;
  int units;                          // 16-byte units of one row
  int scales;                         // scales of one row
  float eps;
  float inv_cin;
};

template <bool BF16>
__device__ inline void unpack(const v4u v, float* f) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (BF16) {
      f[2 * p] = __uint_as_float(v[p] << 16);
      f[2 * p + 1] = __uint_as_float(v[p] & 0xFFFF0000u);
    } else {
      f[p] = __uint_as_float(v[p]);
    }
  }
}

// h of one unit (rounded to the input type) from x and r.
template <bool BF16>
__device__ inline v4u add_unit(const v4u x, const v4u r) {
  float a[8], b[8];
  unpack<BF16>(x, a);
  unpack<BF16>(r, b);
  v4u o;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (BF16) {
      const v2bf v = __builtin_convertvector((v2f){a[2 * p] + b[2 * p], a[2 * p + 1] + b[2 * p + 1]}, v2bf);
      o[p] = __builtin_bit_cast(unsigned, v);
    } else {
      o[p] = __float_as_uint(a[p] + b[p]);
    }
  }
  return o;
}

// E4M3 bytes nearest to y / s (ties to the even code), at most 448: a subnormal s may lie far below max|y| / 448
// (the quotient reaches 671).  A scale out of the range of e4m3_word is brought there with y by a power of
// two, which changes no decision: a y that loses bits by it is 2^-60 of s at most.  A scale that is 0, infinite
// or NaN gives 0.
template <int N>
__device__ inline void quantise(const float* y, float s, unsigned* out) {
  const bool live = s > 0.0f && s < INFINITY;
  const float by = s < 0x1p-100f ? 0x1p60f : (s > 0x1p100f ? 0x1p-60f : 1.0f);
  const float sb = live ? s * by : 1.0f, is = __builtin_amdgcn_rcpf(sb);
#pragma unroll
  for (int w = 0; w < N / 4; ++w) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = y[4 * w + k] * by;
    const unsigned v = e4m3_word(t, sb, is);
    out[w] = live ? v : 0u;
  }
}

// 1 / sqrt(v); 0 for a row of zeros without eps, whose y is 0 and not 0 times infinity; NaN for a row that
// holds one.
__device__ inline float inv_rms(float v) { return v == 0.0f ? 0.0f : 1.0f / sqrtf(v); }

// The larger of the two, NaN if either is: a scale over a NaN is NaN, and so is what is read through it.
__device__ inline float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = larger(v, __shfl_xor(v, o, 64));
  return v;
}

// One row per TPR threads (a wave, or the workgroup); every row fits in U units a thread.
template <bool BF16, bool RES, int TPR, int U>
__global__ __launch_bounds__(kThreads) void k_rms_norm(const Args a) {
  constexpr int N = BF16 ? 8 : 4;
  constexpr int kWaves = TPR / 64;
  __shared__ float red[2][kWaves > 1 ? kWaves : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (TPR != kThreads && row >= a.rows) return;  // a whole wave; rows of one wave need no barrier
  const int64_t base = row * a.units;
  v4u v[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = j * TPR + t;
    v[j] = u < a.units ? __builtin_nontemporal_load(a.x + base + u) : v4u{0, 0, 0, 0};
  }
  if constexpr (RES) {
    v4u w[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = j * TPR + t;
      w[j] = u < a.units ? __builtin_nontemporal_load(a.r + base + u) : v4u{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = j * TPR + t;
      v[j] = add_unit<BF16>(v[j], w[j]);
      if (u < a.units) a.h[base + u] = v[j];
    }
  }
  float y[U][N];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    unpack<BF16>(v[j], y[j]);
#pragma unroll
    for (int k = 0; k < N; ++k) ss = fmaf(y[j][k], y[j][k], ss);
  }
  ss = wave_sum(ss);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = red[0][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) ss += red[0][w];
  }
  const float rstd = inv_rms(ss * a.inv_cin + a.eps);
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = j * TPR + t;
    float g[N], m = 0.0f;
    unpack<BF16>(u < a.units ? a.gamma[u] : v4u{0, 0, 0, 0}, g);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      y[j][k] = y[j][k] * rstd * g[k];
      m = larger(m, fabsf(y[j][k]));
    }
    if (a.scales == 1) {
      top = larger(top, m);
    } else {                           // this unit's 128 channels
#pragma unroll
      for (int o = kGroup / N / 2; o >= 1; o >>= 1) m = larger(m, __shfl_xor(m, o, 64));
      const float s = m * kInv448;
      if (u < a.units) {
        unsigned out[N / 4];
        quantise<N>(y[j], s, out);
        if constexpr (BF16)
          ((v2u*)a.q)[base + u] = v2u{out[0], out[1]};
        else
          ((unsigned*)a.q)[base + u] = out[0];
        if (u % (kGroup / N) == 0) a.s[row * a.scales + u / (kGroup / N)] = s;
      }
    }
  }
  if (a.scales != 1) return;
  top = wave_max(top);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = top;
    __syncthreads();
    top = red[1][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = larger(top, red[1][w]);
  }
  const float s = top * kInv448;
  if (t == 0) a.s[row] = s;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = j * TPR + t;
    if (u >= a.units) continue;
    unsigned out[N / 4];
    quantise<N>(y[j], s, out);
    if constexpr (BF16)
      ((v2u*)a.q)[base + u] = v2u{out[0], out[1]};
    else
      ((unsigned*)a.q)[base + u] = out[0];
  }
}

// Rows longer than the registers hold: the row is read three times (sum of squares, largest |y|,
// output).  h is written in the last pass, by the thread that reads its unit, after the barriers
// that end the other passes, so h may be x or r.
template <bool BF16, bool RES>
__global__ __launch_bounds__(1024) void k_rms_norm_long(const Args a) {
  constexpr int N = BF16 ? 8 : 4;
  constexpr int T = 1024;
  __shared__ float red[2][T / 64];
  const int64_t base = (int64_t)blockIdx.x * a.units;
  auto load = [&](int u) {
    v4u v = u < a.units ? a.x[base + u] : v4u{0, 0, 0, 0};
    if (RES) v = add_unit<BF16>(v, u < a.units ? a.r[base + u] : v4u{0, 0, 0, 0});
    return v;
  };
  float ss = 0.0f;
  for (int u = threadIdx.x; u < a.units; u += T) {
    float f[8];
    unpack<BF16>(load(u), f);
    for (int k = 0; k < N; ++k) ss = fmaf(f[k], f[k], ss);
  }
  ss = wave_sum(ss);
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = ss;
  __syncthreads();
  ss = 0.0f;
  for (int w = 0; w < T / 64; ++w) ss += red[0][w];
  const float rstd = inv_rms(ss * a.inv_cin + a.eps);
  auto normed = [&](const v4u v, int u, float* y) {
    float g[8];
    unpack<BF16>(v, y);
    unpack<BF16>(u < a.units ? a.gamma[u] : v4u{0, 0, 0, 0}, g);
    float m = 0.0f;
    for (int k = 0; k < N; ++k) {
      y[k] = y[k] * rstd * g[k];
      m = larger(m, fabsf(y[k]));
    }
    return m;
  };
  float s = 0.0f, y[8];
  if (a.scales == 1) {
    float top = 0.0f;
    for (int u = threadIdx.x; u < a.units; u += T) top = larger(top, normed(load(u), u, y));
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < T / 64; ++w) s = larger(s, red[1][w]);
    s = s * kInv448;
    if (threadIdx.x == 0) a.s[blockIdx.x] = s;
  }
  for (int u0 = 0; u0 < a.units; u0 += T) {        // every thread takes part in the group's shuffles
    const int u = u0 + threadIdx.x;
    const v4u v = load(u);
    float m = normed(v, u, y);
    if (a.scales != 1) {
      for (int o = kGroup / N / 2; o >= 1; o >>= 1) m = larger(m, __shfl_xor(m, o, 64));
      s = m * kInv448;
      if (u < a.units && u % (kGroup / N) == 0) a.s[(int64_t)blockIdx.x * a.scales + u / (kGroup / N)] = s;
    }
    if (u >= a.units) continue;
    if (RES) a.h[base + u] = v;
    unsigned out[N / 4];
    quantise<N>(y, s, out);
    if constexpr (BF16)
      ((v2u*)a.q)[base + u] = v2u{out[0], out[1]};
    else
      ((unsigned*)a.q)[base + u] = out[0];
  }
}

template <bool BF16, bool RES>
hipError_t launch_typed(const Args& a, hipStream_t stream) {
  const int per = (a.units + kThreads - 1) / kThreads;
  auto go = [&](auto kernel, int rows, int threads) {
    return launch_kernel(kernel, dim3((unsigned)((a.rows + rows - 1) / rows)), dim3(threads), 0, stream, a);
  };
  if (a.units <= 64) return go(k_rms_norm<BF16, RES, 64, 1>, kThreads / 64, kThreads);
  if (a.units <= 128) return go(k_rms_norm<BF16, RES, 64, 2>, kThreads / 64, kThreads);
  if (per <= 1) return go(k_rms_norm<BF16, RES, kThreads, 1>, 1, kThreads);
  if (per <= 2) return go(k_rms_norm<BF16, RES, kThreads, 2>, 1, kThreads);
  if (per <= 4) return go(k_rms_norm<BF16, RES, kThreads, 4>, 1, kThreads);
  if (per <= 8) return go(k_rms_norm<BF16, RES, kThreads, 8>, 1, kThreads);
  return go(k_rms_norm_long<BF16, RES>, 1, 1024);
}

}  // namespace

hipError_t launch_rms_norm(const void* x, const void* r, bool bf16, int64_t rows, int64_t cin, const void* gamma,
                           float eps, bool grouped, void* h, uint8_t* q, float* s, hipStream_t stream) {
  Args a{};
  a.x = (const v4u*)x;
  a.r = (const v4u*)r;
  a.gamma = (const v4u*)gamma;
  a.h = (v4u*)h;
  a.q = q;
  a.s = s;
  a.rows = rows;
  a.units = (int)(cin / (bf16 ? 8 : 4));
  a.scales = grouped ? (int)((cin + kGroup - 1) / kGroup) : 1;
  a.eps = eps;
  a.inv_cin = 1.0f / (float)cin;
  if (bf16) return r ? launch_typed<true, true>(a, stream) : launch_typed<true, false>(a, stream);
  return r ? launch_typed<false, true>(a, stream) : launch_typed<false, false>(a, stream);
}

}  // namespace lh
