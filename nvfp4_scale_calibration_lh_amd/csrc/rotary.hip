// Rotary positions of queries and keys:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos) for the pairs of the first `rot` elements of every head, pair j turned
//   by the token's position times frequency j; pairs are elements (j, j + rot / 2), or (2j, 2j + 1) interleaved.
//
// Bound by memory: every element is read and written once.  A thread makes the sine and cosine of its pairs of one
// token once and takes them through several heads.  One token of 40 heads of 128 bf16 3.1 us, a launch; 8191 tokens 34.8 us (168 MB at
// 4.8 TB/s, as a copy); 3001 tokens of 10 heads of 256 fp32, 64 turned, 12.5 us (61 MB, as a copy).
//
// The angle: position * frequency is a product of 31 and 24 bits; it is taken in turns, as a sum of two 64-bit
// numbers, and reduced to an eighth of a turn there, so that positions up to 2^31 lose nothing (at frequencies up to 2^16: the second number
// stays under 2^-7 turns and their sum right to 2^-60; over 2^20 it could pass that eighth).  What is left
// goes through the power series of sine and cosine in fp32 (|x| <= pi/4: the terms left out are under
// 7e-12 and 2e-10).  Results are fp32, rounded once to the output's type.
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void *q, *k;
  void *qo, *ko;
  const int* positions;
  const float* frequencies;
  int64_t q_stride, k_stride, qo_stride, ko_stride;
  unsigned tokens, heads, q_heads, dim, rot;
  unsigned pieces, groups;                   // threads of one head; runs of heads of one token
  unsigned turning;                          // pieces that hold pairs; the others are copied
  float scale;
  bool inverse, in_place;                    // in place: what is not turned is there already
};

__device__ inline void turn(int position, float frequency, float& c, float& s) {
  // 1 / (2 pi) as the sum of two 64-bit numbers
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;
  const double f = frequency, n = position;
  const double hi = f * kHigh, lo = __builtin_fma(f, kHigh, -hi) + f * kLow;
  const double t = n * hi, rest = __builtin_fma(n, hi, -t) + n * lo;
  const double quarter = __builtin_rint(4.0 * t);
  const double r = __builtin_fma(quarter, -0.25, t) + rest;         // in [-1/8, 1/8] turns, or hardly more
  const float x = (float)(r * 6.283185307179586), y = x * x;
  float sn = fmaf(y, -1.0f / 39916800.0f, 1.0f / 362880.0f);
  sn = fmaf(sn, y, -1.0f / 5040.0f);
  sn = fmaf(sn, y, 1.0f / 120.0f);
  sn = fmaf(sn, y, -1.0f / 6.0f);
  sn = fmaf(sn * y, x, x);
  float cs = fmaf(y, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  cs = fmaf(cs, y, -1.0f / 720.0f);
  cs = fmaf(cs, y, 1.0f / 24.0f);
  cs = fmaf(cs, y, -0.5f);
  cs = fmaf(cs, y, 1.0f);
  // quarter turns: 4 t is under 2^47 in magnitude, its two lowest bits are those of the number mod 4
  const int turns = (int)(quarter - 4.0 * __builtin_floor(quarter * 0.25));
  const bool swap = turns & 1;
  const float a = swap ? sn : cs, b = swap ? cs : sn;
  c = (turns == 1 || turns == 2) ? -a : a;
  s = turns >= 2 ? -b : b;
}

template <class T>
__device__ inline float widen(T v) { return (float)v; }

// N neighbouring elements, aligned to all of them.
template <class T, int N>
struct Run {
  typedef T all_t __attribute__((ext_vector_type(N)));
  T v[N];
  __device__ inline void load(const T* p) {
    const all_t u = *(const all_t*)p;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = u[j];
  }
  __device__ inline void store(T* p) const {
    all_t u;
#pragma unroll
    for (int j = 0; j < N; ++j) u[j] = v[j];
    *(all_t*)p = u;
  }
};
template <class T>
struct Run<T, 1> {
  T v[1];
  __device__ inline void load(const T* p) { v[0] = *p; }
  __device__ inline void store(T* p) const { *p = v[0]; }
};

// V pairs a thread (with 8, lanes lie apart: the fp32 heads 16.9 us instead of 12.5, interleaved bf16 prompts 38 instead of 34.8): 4 where the halves of what is turned
// are whole units of 4 elements, otherwise 1 (20 turned of each of 40 heads of 128 bf16, 8191 tokens: 61.9 us in halves, 56.8 interleaved).
template <class T, int V, bool PAIRED>
__global__ __launch_bounds__(kThreads) void k_rotary(const Args a) {
  const unsigned item = blockIdx.x * kThreads + threadIdx.x, each = a.groups * a.pieces;
  const unsigned token = item / each, left = item - token * each;
  if (token >= a.tokens) return;
  const unsigned group = left / a.pieces, piece = left - group * a.pieces;
  const int position = a.positions[token];
  const bool turned = piece < a.turning && position >= 0;
  if (!turned && a.in_place) return;
  float c[V], s[V];
  if (turned) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      turn(position, a.frequencies[piece * V + j], c[j], s[j]);
      c[j] *= a.scale;
      s[j] *= a.inverse ? -a.scale : a.scale;
    }
  }
  const unsigned at = PAIRED || piece >= a.turning ? 2 * V * piece : V * piece;
  const unsigned apart = PAIRED || piece >= a.turning ? V : a.rot / 2;
  for (unsigned h = group; h < a.heads; h += a.groups) {
    const bool is_q = h < a.q_heads;
    const T* from = is_q ? (const T*)a.q + token * a.q_stride + h * a.dim : (const T*)a.k + token * a.k_stride + (h - a.q_heads) * a.dim;
    T* to = is_q ? (T*)a.qo + token * a.qo_stride + h * a.dim : (T*)a.ko + token * a.ko_stride + (h - a.q_heads) * a.dim;
    Run<T, V> x, y;
    x.load(from + at);
    y.load(from + at + apart);
    if (turned) {
      if constexpr (PAIRED) {
        T all[2 * V];
#pragma unroll
        for (int j = 0; j < V; ++j) all[j] = x.v[j], all[V + j] = y.v[j];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float p = widen(all[2 * j]), q = widen(all[2 * j + 1]);
          all[2 * j] = (T)fmaf(p, c[j], -(q * s[j]));
          all[2 * j + 1] = (T)fmaf(p, s[j], q * c[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) x.v[j] = all[j], y.v[j] = all[V + j];
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float p = widen(x.v[j]), q = widen(y.v[j]);
          x.v[j] = (T)fmaf(p, c[j], -(q * s[j]));
          y.v[j] = (T)fmaf(p, s[j], q * c[j]);
        }
      }
    }
    x.store(to + at);
    y.store(to + at + apart);
  }
}

template <class T, int V>
hipError_t go(Args a, bool paired, hipStream_t stream) {
  a.turning = a.rot / (2 * V);
  a.pieces = a.in_place ? a.turning : a.dim / (2 * V);
  // A run of heads for each of enough threads to fill the chip, at most 4 heads a thread.  40 heads of 128 bf16, 2048 tokens 9.6 us, 10.2
  // with twice the threads and 13 with four times; 8191 tokens 34.8 (12000 tokens of 10 heads of 256 28.4, 35 with one head a thread).
  // fp32 asks for more: 10 heads of 256, 6000 tokens 26.5 us, 29 with half the threads.
  constexpr uint64_t kFill = 2048 * (sizeof(T) == 2 ? 128 : 512);
  a.groups = a.heads;
  while (a.groups > 1 && (uint64_t)a.tokens * ((a.groups + 1) / 2) * a.pieces >= kFill && a.heads <= 2 * a.groups) a.groups = (a.groups + 1) / 2;
  const uint64_t items = (uint64_t)a.tokens * a.groups * a.pieces;
  if (items >= (uint64_t(1) << 32) - kThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)((items + kThreads - 1) / kThreads));
  return paired ? launch_kernel(k_rotary<T, V, true>, grid, dim3(kThreads), 0, stream, a)
                : launch_kernel(k_rotary<T, V, false>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_rotary(const RotaryView& v, bool bf16, hipStream_t stream) {
  Args a{};
  a.q = v.q;
  a.k = v.k;
  a.qo = v.qo;
  a.ko = v.ko;
  a.positions = v.positions;
  a.frequencies = v.frequencies;
  a.q_stride = v.q_stride;
  a.k_stride = v.k_stride;
  a.qo_stride = v.qo_stride;
  a.ko_stride = v.ko_stride;
  a.tokens = (unsigned)v.tokens;
  a.q_heads = (unsigned)v.q_heads;
  a.heads = (unsigned)(v.q_heads + v.k_heads);
  a.dim = (unsigned)v.dim;
  a.rot = (unsigned)v.rot;
  a.scale = v.scale;
  a.inverse = v.inverse;
  a.in_place = v.q == v.qo && v.k == v.ko;
  const bool wide = v.rot % 8 == 0;
  if (bf16) return wide ? go<__bf16, 4>(a, v.interleaved, stream) : go<__bf16, 1>(a, v.interleaved, stream);
  return wide ? go<float, 4>(a, v.interleaved, stream) : go<float, 1>(a, v.interleaved, stream);
}

}  // namespace lh
