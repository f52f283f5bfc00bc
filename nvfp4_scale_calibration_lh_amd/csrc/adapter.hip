// Low-rank adapters of many requests beside a projection:
//   y[t] = base[t] + s_a B_a (A_a x[t]),  a = index[t];  rows without an adapter keep base
//
// Bound by reading the adapters that are asked for once.  Two kernels, both over the adapters that (up to 64) rows ask for:
//   in   u = A_a x: k is cut over workgroups and waves, whose sums go to the workspace in parts
//   out  y = base + B_a (s u): the channels of all adapters are shared out evenly over the workgroups; one adds the parts of its adapter's rows
//        once, and a wave takes 16 channels at a time
// The rows of an adapter are the columns of 16x16 matrix instructions.  bf16 weights meet rows in bf16 pieces (E4M3 values in
// one, their scale multiplying the sum of each 128; fp32 in three, u in two or, where y is fp32, three); fp32 weights meet fp32
// rows.  Products of bf16 weights are exact, sums fp32 in a fixed order; u is held to 2^-16 (2^-24) of itself.
//
// One row, rank 16, 4096 to 12288 channels: 7.7 us, two launches.  96 rows over 64 adapters of ranks up to 64: 29.6 us; the 61 MB that are
// asked for come as 107, because lines of 128 bytes hold the padding of smaller ranks and the two 64 rows read shared adapters twice.  (128
// rows at a time: 28.3 us here, but 21 instead of 17.9 where 128 rows share four adapters, and 0.25 us more for one row.)
#include "grouping.hpp"
#include "lh_internal.hpp"
#include "nvfp4_weights.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxParts = 8;                 // workgroups that share k (96 rows: four 3.6 us more, 16 0.7; one row: 0.4 and 0.4)
constexpr int kRanks = 64;                   // of one workgroup of the first kernel
constexpr int kCopy = 2048;                  // channels that a wave copies of a row without adapter

struct Args {
  const void* x;
  const float* x_scale;
  const void *a, *b;
  const int* index;
  const float* scaling;
  const int* ranks;
  const void* base;
  void* y;
  int* hits;                                 // adapters that each 64 rows ask for
  int* plan;
  float* u;
  int64_t rows;
  int cin, cout, adapters, rank, wide, x_scales, slots, parts, groups;    // wide: rank rounded up to 32
  bool in_place;
};

__device__ inline v4f mfma_f32(float a, float b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

__device__ inline int rank_of(const Args& a, int adapter) {
  return a.ranks ? min(max(a.ranks[adapter], 0), a.rank) : a.rank;
}

// Where W is fp32: elements 16 * S + 4 * quarter + 0..3 of a row's chunk at step S.  Otherwise 32 * S + 8 * quarter + 0..7, in bf16 pieces.
template <int X>
__device__ inline v4f four(const void* x, int64_t at, float scale) {
  if constexpr (X == kXF32) return *(const v4f*)((const float*)x + at);
  if constexpr (X == kXBf16) {
    const v2u v = *(const v2u*)((const __bf16*)x + at);
    return v4f{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16), __uint_as_float(v[1] & 0xFFFF0000u)};
  }
  if constexpr (X == kXE4m3) {
    const unsigned v = *(const unsigned*)((const uint8_t*)x + at);
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
    return v4f{lo[0] * scale, lo[1] * scale, hi[0] * scale, hi[1] * scale};
  }
}
template <int X>
__device__ inline void eight(const void* x, int64_t at, b8* out) {
  if constexpr (X == kXBf16) out[0] = __builtin_bit_cast(b8, *(const v4u*)((const __bf16*)x + at));
  if constexpr (X == kXE4m3) {
    const v2u v = *(const v2u*)((const uint8_t*)x + at);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const v2f f = p % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)v[p / 2], true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)v[p / 2], false);
      out[0][2 * p] = (__bf16)f[0], out[0][2 * p + 1] = (__bf16)f[1];    // exact
    }
  }
  if constexpr (X == kXF32) {
    const v4f f[2] = {*(const v4f*)((const float*)x + at), *(const v4f*)((const float*)x + at + 4)};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __bf16 three[3];
      split<3>(f[e / 4][e % 4], three);
      out[0][e] = three[0], out[1][e] = three[1], out[2][e] = three[2];
    }
  }
}

// RT: 16-row tiles of A a wave takes.
template <int X, bool WF32, int RT>
__global__ __launch_bounds__(kThreads) void k_adapter_in(const Args a) {
  constexpr int P = WF32 ? 1 : Frag<X>::pieces;
  constexpr bool SCALED = X == kXE4m3 && !WF32;
  __shared__ uint64_t bits[64];
  __shared__ int rows[kTokens];
  __shared__ int found;
  __shared__ v4f red[kWaves][RT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, quarter = lane >> 4;
  const int rgroups = (a.rank + kRanks - 1) / kRanks;
  const int part = blockIdx.x % (unsigned)a.parts, rest = blockIdx.x / (unsigned)a.parts;
  const int first = rest % rgroups * kRanks, slot = rest / rgroups;
  const bool leads = part == 0 && first == 0;
  int* plan = a.plan + ((int64_t)blockIdx.y * a.slots + slot) * kPlan;
  const int64_t t = (int64_t)blockIdx.y * kTokens + lane;
  const int wanted = t < a.rows ? a.index[t] : -1;
  if (threadIdx.x < 64) bits[threadIdx.x] = 0;
  __syncthreads();
  if (wave == 0 && wanted >= 0 && wanted < a.adapters) atomicOr((unsigned long long*)&bits[wanted >> 6], 1ull << (wanted & 63));
  __syncthreads();
  if (leads && slot == 0 && wave == 0) {
    int hits = __popcll(bits[lane]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) hits += __shfl_xor(hits, o, 64);
    if (lane == 0) a.hits[blockIdx.y] = hits;
  }
  const int adapter = find_expert(bits, slot);
  if (adapter < 0) return;
  const int ranks = rank_of(a, adapter);
  const int chunks = (a.cin + kChunk - 1) / kChunk;
  constexpr int kUnits = WF32 ? 8 : 4, kEach = WF32 ? 4 : 8;         // loads of a chunk, elements of one
  v4u w[RT][kUnits];
  auto load_w = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < RT; ++j) {           // rows past the adapter's rank repeat its last: the second kernel leaves them out
      const int64_t at = ((int64_t)adapter * a.rank + min(first + 16 * j + i, max(ranks - 1, 0))) * a.cin;
#pragma unroll
      for (int s = 0; s < kUnits; ++s) {
        const int k = min(c * kChunk + (4 * s + quarter) * kEach, a.cin - kEach);
        w[j][s] = WF32 ? *(const v4u*)((const float*)a.a + at + k) : *(const v4u*)((const __bf16*)a.a + at + k);
      }
    }
  };
  const int own = part * kWaves + wave;
  if (own < chunks) load_w(own);
  if (wave == 0) {
    const uint64_t hit = __ballot(wanted == adapter);
    const int at = __popcll(hit & ((1ull << lane) - 1));
    if (wanted == adapter) rows[at] = (int)t;
    if (leads) {
      if (lane == 0) plan[0] = adapter, plan[1] = __popcll(hit), plan[2] = ranks;
      if (wanted == adapter) plan[4 + at] = (int)t;
    }
    if (lane == 0) found = __popcll(hit);
  }
  __syncthreads();
  const int n = found;
  if (first >= ranks) return;
  const int tiles = min(RT, (ranks - first + 15) / 16);
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int row = rows[min(r0 + i, n - 1)];
    const int64_t x_at = (int64_t)row * a.cin;
    v4f acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = v4f{0, 0, 0, 0};
    for (int c = own; c < chunks; c += a.parts * kWaves) {
      if (c > own || r0 > 0) load_w(c);
      float scale = 1.0f;
      if constexpr (X == kXE4m3) scale = a.x_scale[(int64_t)row * a.x_scales + (a.x_scales > 1 ? c : 0)];
      if constexpr (WF32) {
        v4f x[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) x[s] = four<X>(a.x, x_at + min(c * kChunk + 16 * s + 4 * quarter, a.cin - 4), scale);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          if (j >= tiles) break;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if (c * kChunk + 16 * s >= a.cin) break;                 // rows are multiples of 16
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j] = mfma_f32(__uint_as_float(w[j][s][e]), x[s][e], acc[j]);
          }
        }
      } else {
        b8 x[4][P];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = c * kChunk + 32 * s + 8 * quarter;
          eight<X>(a.x, x_at + min(k, a.cin - 8), x[s]);
          if (k >= a.cin)
#pragma unroll
            for (int p = 0; p < P; ++p) x[s][p] = __builtin_bit_cast(b8, v4u{0, 0, 0, 0});
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          if (j >= tiles) break;
          v4f sum = SCALED ? v4f{0, 0, 0, 0} : acc[j];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const v4u held = c * kChunk + 32 * s + 8 * quarter < a.cin ? w[j][s] : v4u{0, 0, 0, 0};
#pragma unroll
            for (int p = 0; p < P; ++p) sum = mfma(__builtin_bit_cast(b8, held), x[s][p], sum);
          }
          acc[j] = SCALED ? acc[j] + scale * sum : sum;
        }
      }
    }
    __syncthreads();                         // what was in red has been read
#pragma unroll
    for (int j = 0; j < RT; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < tiles; j += kWaves) {
      v4f sum = red[0][j][lane];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) sum += red[v][j][lane];
      if (r0 + i < n) *(v4f*)(a.u + ((int64_t)part * a.rows + row) * a.wide + first + 16 * j + 4 * quarter) = sum;
    }
  }
}

// Workgroups of the second kernel on a compute unit, all resident, as the registers for rk steps of 32 ranks and u's LDS (28 KB for three pieces of
// rank 64, so five) allow.  96 rows over 64 adapters of rank 64: 29.6 us with six; 35 with three, 31.1 with four, 29.9 with five, 29.1 with seven and
// 35.4 with eight, whose weights spill; 128 rows over four: 17.5, 17.6, 17.9, 18.5 and 20.6 against 17.9.  With fp32 rows, whose sixth would
// wait for another to end, 31.9 us with five and 38.5 with six, and 20.4 and 22.5.
template <bool YF32, bool WF32>
constexpr int resident(int rk) { return rk <= (WF32 ? 1 : 2) ? (YF32 && !WF32 && rk == 2 ? 5 : 6) : (rk <= 2 ? 4 : (rk == 4 ? 3 : 2)); }

// RK: steps of 32 ranks; P: bf16 pieces of u.  A workgroup makes its adapter's u once and takes several steps of channels, 16 a wave, the
// weights and the base of the next on their way (32 channels a wave: 1.8 us more for 96 rows over 64 adapters).
template <bool YF32, bool WF32, int RK>
__global__ __launch_bounds__(kThreads, (resident<YF32, WF32>(RK))) void k_adapter_out(const Args a) {
  constexpr int P = WF32 ? 1 : (YF32 ? 3 : 2);
  constexpr int kWide = 32 * RK + 8;         // a row of u in LDS, so that 16 rows lie in different banks
  constexpr int kRows = RK <= 2 ? 64 : (RK == 4 ? 32 : 16);          // rows whose u is held
  using T = std::conditional_t<YF32, float, __bf16>;
  using U = std::conditional_t<WF32, float, __bf16>;
  using four_t = T __attribute__((ext_vector_type(4)));
  __shared__ int rows[kTokens];
  __shared__ __attribute__((aligned(16))) U us[P][kRows][kWide];
  static_assert(resident<YF32, WF32>(RK) * (sizeof(us) + sizeof(rows)) <= 160 * 1024, "LDS of the workgroups of a compute unit");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, quarter = lane >> 4;
  const T* base = (const T*)a.base;
  T* y = (T*)a.y;
  // a workgroup serves up to 64 chunks of 64 rows
  const int chunk0 = (int)blockIdx.y * 64, chunks = (int)min((int64_t)64, (a.rows + kTokens - 1) / kTokens - chunk0);
  if (blockIdx.x >= (unsigned)a.groups) {                            // rows without an adapter, one a wave
    const int place = blockIdx.x - a.groups, parts = (a.cout + kCopy - 1) / kCopy;
    const int64_t row = (int64_t)chunk0 * kTokens + (int64_t)(place / parts) * kWaves + wave;
    if (row >= a.rows) return;
    const int id = a.index[row];
    if (id >= 0 && id < a.adapters) return;
    constexpr int kUnit = 16 / sizeof(T);
    const int c0 = place % parts * kCopy, c1 = min(c0 + kCopy, a.cout);
    const T* from = base + row * a.cout;
    T* to = y + row * a.cout;
    if (a.cout % kUnit == 0) {
#pragma unroll
      for (int k = 0; k < kCopy; k += 64 * kUnit) {
        const int c = c0 + k + lane * kUnit;
        if (c < c1) *(v4u*)(to + c) = *(const v4u*)(from + c);
      }
    } else {
      for (int c = c0 + lane; c < c1; c += 64) to[c] = from[c];
    }
    return;
  }
  // the steps of all adapters of these chunks, shared out evenly
  constexpr int kStep = 16 * kWaves;    // channels of a step
  int upto = lane < chunks ? a.hits[chunk0 + lane] : 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  const unsigned steps = (a.cout + kStep - 1) / kStep, all = __builtin_amdgcn_readlane(upto, 63) * steps, per = all / a.groups, over = all - per * a.groups;
  unsigned place = per * blockIdx.x + min(blockIdx.x, over);
  const unsigned end = place + per + (blockIdx.x < over);
  const bool whole = a.cout % 4 == 0;        // four neighbouring channels are one load
  constexpr int kUnits = WF32 ? 2 * RK : RK, kEach = WF32 ? 4 : 8;
  while (place < end) {                       // the share's part of one adapter
    const int hit = place / steps, s0 = place - hit * steps, s1 = min(steps, s0 + (end - place));
    place += s1 - s0;
    const int chunk = __ffsll((unsigned long long)__ballot(upto > hit)) - 1, slot = hit - (chunk > 0 ? __builtin_amdgcn_readlane(upto, chunk - 1) : 0);
    const int* plan = a.plan + ((int64_t)(chunk0 + chunk) * a.slots + slot) * kPlan;
    const int adapter = __builtin_amdgcn_readfirstlane(plan[0]), n = __builtin_amdgcn_readfirstlane(plan[1]), ranks = __builtin_amdgcn_readfirstlane(plan[2]);
    v4u next[kUnits];
    auto load_w = [&](int step) __attribute__((always_inline)) {
      const int64_t at = ((int64_t)adapter * a.cout + min(step * kStep + wave * 16 + i, a.cout - 1)) * a.rank;
#pragma unroll
      for (int s = 0; s < kUnits; ++s) {
        if (s > 0 && s * 4 * kEach >= ranks) break;
        const int k = min((s * 4 + quarter) * kEach, a.rank - kEach);
        next[s] = WF32 ? *(const v4u*)((const float*)a.b + at + k) : *(const v4u*)((const __bf16*)a.b + at + k);
      }
    };
    load_w(s0);
    __syncthreads();                            // the rows before have been used
    if (threadIdx.x < kTokens) rows[threadIdx.x] = plan[4 + threadIdx.x];
    const float scaling = a.scaling ? a.scaling[adapter] : 1.0f;
    for (int r0 = 0; r0 < n; r0 += kRows) {
      const int live = min(kRows, n - r0);
      __syncthreads();
      for (int at = threadIdx.x; at < live * 32 * RK; at += kThreads) {
        const int r = at / (32 * RK), k = at % (32 * RK);
        float v = 0.0f;
        if (k < ranks) {
          const float* from = a.u + (int64_t)rows[r0 + r] * a.wide + k;
          float got[kMaxParts];
#pragma unroll
          for (int p = 0; p < kMaxParts; ++p) got[p] = from[(int64_t)min(p, a.parts - 1) * a.rows * a.wide];
#pragma unroll
          for (int p = 0; p < kMaxParts; ++p) v += p < a.parts ? got[p] : 0.0f;
          v *= scaling;
        }
        if constexpr (WF32) {
          us[0][r][k] = v;
        } else {
          __bf16 pieces[P];
          split<P>(v, pieces);
#pragma unroll
          for (int p = 0; p < P; ++p) us[p][r][k] = pieces[p];
        }
      }
      __syncthreads();
      if (r0 > 0) load_w(s0);
      four_t soon;                              // base of the first 16 rows, with the weights
      auto load_base = [&](four_t& to, int t, int step) __attribute__((always_inline)) {
        const int64_t row = rows[r0 + min(t + i, live - 1)];
        to = *(const four_t*)(base + row * a.cout + min(step * kStep + wave * 16 + 4 * quarter, a.cout - 4));
      };
      if (whole) load_base(soon, 0, s0);
      for (int step = s0; step < s1; ++step) {
        const int c = step * kStep + wave * 16 + 4 * quarter;
        four_t old = soon;
        asm volatile("" : "+v"(old));           // waits for these loads here, before the next are issued, not behind those
        v4u w[kUnits];                          // what is past the adapter's rank counts as 0
#pragma unroll
        for (int s = 0; s < kUnits; ++s) {
          const int left = ranks - (s * 4 + quarter) * kEach;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (WF32)
              w[s][e] = e < left ? next[s][e] : 0u;
            else
              w[s][e] = 2 * e + 1 < left ? next[s][e] : (2 * e < left ? next[s][e] & 0xFFFFu : 0u);
          }
          asm volatile("" : "+v"(w[s]));
        }
        if (step + 1 < s1) {
          load_w(step + 1);
          if (whole) load_base(soon, 0, step + 1);
        }
        for (int t = 0; t < live; t += 16) {
          if (t > 0 && whole) load_base(old, t, step);
          v4f acc = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < kUnits; ++s)
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const v4u u = *(const v4u*)&us[p][min(t + i, live - 1)][(s * 4 + quarter) * kEach];
              if constexpr (WF32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = mfma_f32(__uint_as_float(w[s][e]), __uint_as_float(u[e]), acc);
              } else {
                acc = mfma(__builtin_bit_cast(b8, w[s]), __builtin_bit_cast(b8, u), acc);
              }
            }
          if (t + i >= live || c >= a.cout) continue;
          const int64_t at = (int64_t)rows[r0 + t + i] * a.cout + c;
          if (whole) {
            four_t v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = (T)((float)old[r] + acc[r]);
            *(four_t*)(y + at) = v;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (c + r < a.cout) y[at + r] = (T)((float)base[at + r] + acc[r]);
          }
        }
      }
    }
  }
}

struct Layout {
  int64_t slots, chunks, parts, wide, hits, plan, all;                 // chunks of rows; bytes
};
Layout layout(const AdapterView& v) {
  Layout l{};
  l.slots = std::min<int64_t>(v.adapters, std::min<int64_t>(v.rows, kTokens));
  l.chunks = (v.rows + kTokens - 1) / kTokens;
  l.parts = std::clamp<int64_t>(((v.cin + kChunk - 1) / kChunk + kWaves - 1) / kWaves, 1, kMaxParts);
  l.wide = (v.rank + 31) / 32 * 32;
  l.plan = (l.slots * l.chunks * kPlan * 4 + 255) / 256 * 256;
  l.hits = (l.chunks * 4 + 255) / 256 * 256;
  l.all = l.hits + l.plan + l.parts * v.rows * l.wide * 4;
  return l;
}

template <int X, bool WF32>
hipError_t go_in(const Args& a, const Layout& l, hipStream_t stream) {
  const dim3 grid((unsigned)(l.slots * l.parts * ((a.rank + kRanks - 1) / kRanks)), (unsigned)l.chunks);
  if (a.rank <= 16) return launch_kernel(k_adapter_in<X, WF32, 1>, grid, dim3(kThreads), 0, stream, a);
  if (a.rank <= 32) return launch_kernel(k_adapter_in<X, WF32, 2>, grid, dim3(kThreads), 0, stream, a);
  return launch_kernel(k_adapter_in<X, WF32, 4>, grid, dim3(kThreads), 0, stream, a);
}

template <bool YF32, bool WF32, int RK>
hipError_t go_out(Args a, const Layout& l, hipStream_t stream) {
  const int64_t steps = (a.cout + 16 * kWaves - 1) / (16 * kWaves), chunks = std::min<int64_t>(l.chunks, 64);
  if (l.slots * chunks * steps >= int64_t(1) << 31) return hipErrorInvalidConfiguration;
  a.groups = (int)std::min<int64_t>(l.slots * chunks * steps, 256 * resident<YF32, WF32>(RK));
  const int64_t n = a.groups + (a.in_place ? 0 : (a.cout + kCopy - 1) / kCopy * ((std::min<int64_t>(chunks * kTokens, a.rows) + kWaves - 1) / kWaves));
  if (n >= int64_t(1) << 24) return hipErrorInvalidConfiguration;
  return launch_kernel(k_adapter_out<YF32, WF32, RK>, dim3((unsigned)n, (unsigned)((l.chunks + 63) / 64)), dim3(kThreads), 0, stream, a);
}

template <bool YF32, bool WF32>
hipError_t go_rank(const Args& a, const Layout& l, hipStream_t stream) {
  if (a.rank <= 32) return go_out<YF32, WF32, 1>(a, l, stream);
  if (a.rank <= 64) return go_out<YF32, WF32, 2>(a, l, stream);
  if (a.rank <= 128) return go_out<YF32, WF32, 4>(a, l, stream);
  return go_out<YF32, WF32, 8>(a, l, stream);
}

}  // namespace

int64_t adapter_workspace(const AdapterView& v) { return layout(v).all; }

hipError_t launch_adapter(const AdapterView& v, void* work, hipStream_t stream) {
  const Layout l = layout(v);
  Args a{};
  a.x = v.x;
  a.x_scale = v.x_scale;
  a.a = v.a;
  a.b = v.b;
  a.index = v.index;
  a.scaling = v.scaling;
  a.ranks = v.ranks;
  a.base = v.base;
  a.y = v.y;
  a.hits = (int*)work;
  a.plan = (int*)((char*)work + l.hits);
  a.u = (float*)((char*)work + l.hits + l.plan);
  a.rows = v.rows;
  a.cin = (int)v.cin;
  a.cout = (int)v.cout;
  a.adapters = (int)v.adapters;
  a.rank = (int)v.rank;
  a.wide = (int)l.wide;
  a.x_scales = (int)v.x_scales;
  a.slots = (int)l.slots;
  a.parts = (int)l.parts;
  a.in_place = v.base == v.y;
  hipError_t e;
  if (v.x_type == kXBf16)
    e = v.w_f32 ? go_in<kXBf16, true>(a, l, stream) : go_in<kXBf16, false>(a, l, stream);
  else if (v.x_type == kXF32)
    e = v.w_f32 ? go_in<kXF32, true>(a, l, stream) : go_in<kXF32, false>(a, l, stream);
  else
    e = v.w_f32 ? go_in<kXE4m3, true>(a, l, stream) : go_in<kXE4m3, false>(a, l, stream);
  if (e != hipSuccess) return e;
  if (v.x_type == kXF32) return v.w_f32 ? go_rank<true, true>(a, l, stream) : go_rank<true, false>(a, l, stream);
  return v.w_f32 ? go_rank<false, true>(a, l, stream) : go_rank<false, false>(a, l, stream);
}

}  // namespace lh
